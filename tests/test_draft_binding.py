"""The binding's checks of the rotation, draft trees and compaction, on the
CPU: a recorder stands in for the library, so a call that passes the checks
shows what would have reached the kernels, and nothing runs."""
import types

import pytest
import torch


class Recorder:
    """libpa's device calls: each records its arguments and succeeds.  (An
    allocator of another test may be collected meanwhile: not recorded.)"""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            if not name.startswith(("pa_alloc", "pa_seq")):
                self.calls.append((name, a))
            return 0
        call.__name__ = name
        return call

    def pa_decode_tree_workspace_bytes(self, *a):
        return 4096


@pytest.fixture
def pa(monkeypatch):
    from paged_kv_cache_blocks_gb300 import binding

    def here(*ts):
        if not all(t.is_contiguous() for t in ts):
            raise ValueError("not contiguous")

    rec = Recorder()
    monkeypatch.setattr(binding, "lib", lambda: rec)
    monkeypatch.setattr(binding, "_need_here", here)
    monkeypatch.setattr(binding, "_stream", lambda stream: None)
    return types.SimpleNamespace(binding=binding, calls=rec.calls)


def rope_args(T=6, hq=4, hkv=2, D=128, dtype=torch.float16):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    return dict(q=z(T, hq, D), k=z(T, hkv, D), v=z(T, hkv, D), positions=torch.zeros(T, dtype=torch.int32),
                slot_mapping=torch.zeros(T, dtype=torch.int64), inv_freq=torch.zeros(D // 2, dtype=torch.float64),
                k_cache=z(3, hkv, 16, D), v_cache=z(3, hkv, 16, D))


def e4m3_args(T=6, hq=4, hkv=2):
    a = rope_args(T, hq, hkv)
    a.pop("k_cache"), a.pop("v_cache")
    return a | dict(k_scale=torch.ones(hkv), v_scale=torch.ones(hkv),
                    k_cache8=torch.zeros(3, hkv, 16, 128, dtype=torch.uint8),
                    v_cache8=torch.zeros(3, hkv, 128, 16, dtype=torch.uint8))


def test_rope_calls_pass(pa):
    pa.binding.pa_rope_cache_write(**rope_args())
    pa.binding.pa_rope_cache_write_fp8(**e4m3_args())
    assert [c[0] for c in pa.calls] == ["pa_rope_cache_write", "pa_rope_cache_write_fp8"]


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_rope_refuses_one_row_repeated_over_the_tokens(pa, name):
    """Token stride 0 means "packed" to the library: it would read T rows of a tensor that holds one."""
    for call, a in ((pa.binding.pa_rope_cache_write, rope_args()), (pa.binding.pa_rope_cache_write_fp8, e4m3_args())):
        a[name] = a[name][:1].expand(6, -1, -1)
        assert a[name].stride(0) == 0
        with pytest.raises(ValueError):
            call(**a)
    assert not pa.calls
    a = rope_args(T=1)
    a[name] = a[name].as_strided(a[name].shape, (0, 128, 1))      # one token: its stride means nothing
    pa.binding.pa_rope_cache_write(**a)
    assert len(pa.calls) == 1


def test_rope_refuses_caches_of_another_layout(pa):
    """As many elements, but rows and dimensions the other way round."""
    for name in ("k_cache", "v_cache"):
        a = rope_args()
        a[name] = torch.zeros(3, 2, 128, 16, dtype=torch.float16)
        with pytest.raises(TypeError):
            pa.binding.pa_rope_cache_write(**a)
    for name, shape in (("k_cache8", (3, 2, 128, 16)), ("v_cache8", (3, 2, 16, 128)), ("v_cache8", (2, 3, 128, 16))):
        a = e4m3_args()
        a[name] = torch.zeros(*shape, dtype=torch.uint8)
        with pytest.raises(TypeError):
            pa.binding.pa_rope_cache_write_fp8(**a)
    assert not pa.calls


def tree_args(T=6, hq=4, hkv=2, D=128, dtype=torch.float16):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(q=z(T, hq, D), k_cache=z(3, hkv, 16, D), v_cache=z(3, hkv, 16, D), block_tables=i(2, 4),
                seq_lens=i(2), q_offsets=i(3), masks=torch.zeros(T, 1, dtype=torch.int64), scale=0.1)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float32, torch.float64])
def test_q_that_is_not_16_bit_is_refused(pa, dtype):
    """Beside bit-pattern caches q's element type was not looked at: a one-byte q is half as long as what is read."""
    bits = dict(k_cache=torch.zeros(3, 2, 16, 128, dtype=torch.int16), v_cache=torch.zeros(3, 2, 16, 128, dtype=torch.int16))
    with pytest.raises(TypeError):
        pa.binding.pa_decode_tree(**(tree_args() | bits | dict(q=torch.zeros(6, 4, 128, dtype=dtype))), dtype="f16")
    with pytest.raises(TypeError):
        pa.binding.pa_rope_cache_write(**(rope_args(dtype=dtype) | bits), dtype="f16")
    a = {k: v.to(dtype) if k in ("q", "k", "v") else v for k, v in e4m3_args().items()}
    with pytest.raises(TypeError):
        pa.binding.pa_rope_cache_write_fp8(**a, dtype="f16")
    assert not pa.calls
    pa.binding.pa_decode_tree(**(tree_args() | bits), dtype="f16")
    pa.binding.pa_decode_tree(**(tree_args(dtype=torch.int16)), dtype="bf16")
    assert len(pa.calls) == 2
