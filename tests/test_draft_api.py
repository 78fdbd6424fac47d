"""Host side of the rotation, draft trees and compaction: refusals (no kernel
runs here), frequencies, truncation in the allocator."""
import ctypes
import math

import numpy as np
import pytest

from oracle.allocator import AllocatorModel


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_blocks_gb300 import build, binding
    build.build()
    binding.lib()
    return binding


P = ctypes.c_void_p
A = 1 << 20     # an aligned address that nothing reads


def rope_rc(pa, fp8=False, opts=True, **kw):
    a = dict(q=A, k=A, v=A, pos=A, slots=A, T=4, hq=8, hkv=2, D=128, ks=A, vs=A, out=A, kc=A, vc=A, nb=10, dtype=1,
             rotary=128, inter=0, factor=1.0, eps=1e-6, freq=A, qn=0, kn=0, qst=0, kst=0, vst=0) | kw
    o = pa.PaRopeOpts(a["rotary"], a["inter"], a["factor"], a["eps"], a["freq"], a["qn"], a["kn"], a["qst"], a["kst"],
                      a["vst"])
    scales = [P(a["ks"]), P(a["vs"])] if fp8 else []
    f = pa.lib().pa_rope_cache_write_fp8 if fp8 else pa.lib().pa_rope_cache_write
    return f(P(a["q"]), P(a["k"]), P(a["v"]), P(a["pos"]), P(a["slots"]), a["T"], a["hq"], a["hkv"], a["D"], *scales,
             P(a["out"]), P(a["kc"]), P(a["vc"]), a["nb"], a["dtype"], None, ctypes.byref(o) if opts else None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(D=96), 3), (dict(dtype=2), 3), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(nb=0), 1),
    (dict(rotary=8), 3), (dict(rotary=144), 3), (dict(rotary=-16), 3), (dict(inter=2), 1),
    (dict(factor=float("nan")), 1), (dict(qn=A, eps=-1.0), 1), (dict(kn=A, eps=float("inf")), 1), (dict(kst=4), 1),
    (dict(qst=1), 1), (dict(vst=-3), 1), (dict(q=0), 1), (dict(pos=0), 1), (dict(slots=0), 1), (dict(freq=0), 1),
    (dict(out=0), 1), (dict(kc=A + 8), 1), (dict(qn=A + 2), 1), (dict(v=A + 4), 1), (dict(slots=A + 4), 1),
    (dict(opts=False), 1), (dict(hq=1 << 30), 3),
])
def test_rope_rejects_bad_arguments(pa, bad, code):
    assert rope_rc(pa, **bad) == code, pa.lib().pa_last_error_string()
    assert b"pa_rope_cache_write" in pa.lib().pa_last_error_string()


def test_rope_fp8_rejects_and_no_tokens_is_a_noop(pa):
    assert rope_rc(pa, True, D=64, rotary=64) == 3
    assert rope_rc(pa, True, ks=0) == 1 and rope_rc(pa, True, vs=A + 2) == 1
    assert rope_rc(pa, T=0) == 0 and rope_rc(pa, True, T=0) == 0


def tree_rc(pa, **kw):
    a = dict(q=A, k=A, v=A, nb=100, tab=A, mb=8, lens=A, off=A, masks=A, words=1, B=4, Tq=40, msl=0, hq=8, hkv=2, D=128,
             scale=0.1, dtype=1, out=A, ws=A, wsb=1 << 40, opts=None) | kw
    return pa.lib().pa_decode_tree(P(a["q"]), P(a["k"]), P(a["v"]), a["nb"], P(a["tab"]), a["mb"], P(a["lens"]),
                                   P(a["off"]), P(a["masks"]), a["words"], a["B"], a["Tq"], a["msl"], a["hq"], a["hkv"],
                                   a["D"], a["scale"], a["dtype"], P(a["out"]), P(a["ws"]), a["wsb"], None,
                                   ctypes.byref(a["opts"]) if a["opts"] else None)


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), 3), (dict(dtype=7), 3), (dict(hq=6, hkv=4), 1), (dict(hq=32, hkv=2), 3), (dict(words=0), 3),
    (dict(words=5), 3), (dict(nb=0), 1), (dict(mb=0), 1), (dict(msl=129), 1), (dict(scale=float("nan")), 1),
    (dict(scale=0.0), 1), (dict(scale=-0.1), 1), (dict(masks=0), 1), (dict(masks=A + 4), 1), (dict(off=0), 1),
    (dict(ws=A | 8), 1), (dict(wsb=512), 1), (dict(B=-1), 1), (dict(Tq=-1), 1), (dict(nb=1 << 27, hkv=2, hq=2), 3),
    (dict(Tq=1 << 29), 3), (dict(mb=1 << 28), 1),
])
def test_tree_rejects_bad_arguments(pa, bad, code):
    assert tree_rc(pa, **bad) == code, pa.lib().pa_last_error_string()
    assert b"pa_decode_tree" in pa.lib().pa_last_error_string()


def test_tree_empty_is_a_noop_and_options(pa):
    assert tree_rc(pa, B=0) == 0 and tree_rc(pa, Tq=0) == 0
    for o in (pa.PaDecodeOpts(variant=2), pa.PaDecodeOpts(flags=1), pa.PaDecodeOpts(partition_tokens=512)):
        assert tree_rc(pa, opts=o) == 1


def test_tree_workspace_sizes(pa):
    f = pa.lib().pa_decode_tree_workspace_bytes
    assert 0 < f(4, 40, 8, 2, 128, 128) < f(4, 40, 8, 2, 128, 4096) <= f(4, 40, 8, 2, 128, 1 << 20)
    # the state of at most 1824 items of 128 rows: it does not grow with the context or the batch
    most = 1824 * 128 * (128 + 2) * 4
    assert most <= f(256, 2048, 64, 8, 128, 1 << 20) <= most + 256 * 1024
    assert f(4, 40, 6, 4, 128, 128) == f(4, 40, 8, 2, 96, 128) == f(-1, 40, 8, 2, 128, 128) == f(1, 1, 48, 2, 64, 9) == 0


def plan_rc(pa, **kw):
    a = dict(par=A, off=A, lens=A, B=2, Tq=9, words=1, masks=A, pos=A, err=0) | kw
    return pa.lib().pa_tree_plan(P(a["par"]), P(a["off"]), P(a["lens"]), a["B"], a["Tq"], a["words"], P(a["masks"]),
                                 P(a["pos"]), P(a["err"]), None)


def test_plan_rejects_bad_arguments(pa):
    for bad, code in ((dict(B=-1), 1), (dict(Tq=-1), 1), (dict(words=0), 3), (dict(words=5), 3), (dict(par=0), 1),
                      (dict(masks=A + 4), 1), (dict(pos=0), 1), (dict(err=A + 2), 1)):
        assert plan_rc(pa, **bad) == code
    assert plan_rc(pa, B=0) == 0 and plan_rc(pa, Tq=0) == 0


def compact_rc(pa, **kw):
    a = dict(ks=[A, A], vs=[A, A], n=2, nb=10, hkv=2, D=64, tab=A, mb=4, lens=A, off=A, acc=A, num=A, most=3, B=2, new=0,
             err=0) | kw
    arr = lambda x: (P * max(len(x), 1))(*x) if x is not None else None
    return pa.lib().pa_cache_compact(arr(a["ks"]), arr(a["vs"]), a["n"], a["nb"], a["hkv"], a["D"], P(a["tab"]), a["mb"],
                                     P(a["lens"]), P(a["off"]), P(a["acc"]), P(a["num"]), a["most"], a["B"], P(a["new"]),
                                     P(a["err"]), None)


def test_compact_rejects_bad_arguments(pa):
    for bad, code in ((dict(B=-1), 1), (dict(most=-1), 1), (dict(D=80), 3), (dict(n=0), 1), (dict(hkv=0), 1),
                      (dict(nb=0), 1), (dict(mb=0), 1), (dict(mb=1 << 28), 1), (dict(ks=None), 1), (dict(ks=[A, 0]), 1),
                      (dict(vs=[A, A + 8]), 1), (dict(acc=0), 1), (dict(num=0), 1), (dict(new=A), 1), (dict(err=A + 1), 1)):
        assert compact_rc(pa, **bad) == code, bad
    assert compact_rc(pa, B=0) == 0


# ------------------------------------------------------------------------------ frequencies

def test_frequencies(pa):
    f, a = pa.pa_rope_frequencies(64, 10000.0, device="cpu")
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.allclose(f.numpy(), want, rtol=1e-14) and a == 1.0
    lin, a = pa.pa_rope_frequencies(64, 10000.0, "linear", factor=8.0, device="cpu")
    assert np.allclose(lin.numpy(), want / 8, rtol=1e-14) and a == 1.0
    b, a = pa.pa_rope_frequencies(64, 10000.0, "base", factor=8.0, device="cpu")
    assert b[0] == 1.0 and np.isclose(b[-1].item(), want[-1] / 8, rtol=1e-12) and a == 1.0
    assert (np.diff(b.numpy() / want) < 0).all()
    y, a = pa.pa_rope_frequencies(128, 500000.0, "ramp", factor=8.0, trained_tokens=8192, device="cpu")
    f = 500000.0 ** (-np.arange(0, 128, 2) / 128)
    turns = 8192 * f / (2 * math.pi)
    ratio = y.numpy() / f
    assert np.allclose(ratio[turns >= 32], 1, rtol=1e-14) and np.allclose(ratio[turns <= 1], 1 / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.allclose(ratio[mid], 1 / 8 + 7 / 8 * (turns[mid] - 1) / 31, rtol=1e-12)
    assert np.isclose(a, 0.1 * math.log(8.0) + 1, rtol=1e-7)


def test_frequencies_reject_bad_arguments(pa):
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("inf")),
               dict(rotary_dim=64, scaling="linear", factor=0.5), dict(rotary_dim=2, scaling="base", factor=2.0),
               dict(rotary_dim=64, scaling="ramp", factor=2.0), dict(rotary_dim=64, scaling="ramp", factor=2.0,
                                                                     trained_tokens=64, beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(pa.PaError):
            pa.pa_rope_frequencies(**kw, device="cpu")
    with pytest.raises(ValueError):
        pa.pa_rope_frequencies(64, scaling="none", device="cpu")


# ------------------------------------------------------------------------------ truncation

def model_truncate(m, sid, tokens):
    s = m._get(sid)
    keep = -(-tokens // m.block_size)
    for blk in s["table"][keep:]:
        m.ref[blk] -= 1
        if m.ref[blk] == 0:
            m.free.append(blk)
    s["table"], s["len"] = s["table"][:keep], tokens


def same(a, m, live):
    assert a.block_table(live, 32) == tuple(m.block_table(live, 32))
    st, ms = a.stats(), m.stats()
    assert all(st[k] == ms[k] for k in ms)


def test_truncate_matches_model(pa):
    r = np.random.default_rng(2)
    order = r.permutation(60)
    a, m = pa.Allocator(60, order), AllocatorModel(60, 16, order)
    live = [a.seq_create() for _ in range(4)]
    assert live == [m.seq_create() for _ in range(4)]
    for _ in range(400):
        s = int(r.choice(live))
        length = m.seqs[s]["len"]
        what = r.integers(4)
        if what == 0:
            n = int(r.integers(0, length + 1))
            a.seq_truncate(s, n)
            model_truncate(m, s, n)
        elif what == 1 and len(live) < 6:
            n = int(r.integers(0, length + 1))
            live.append(a.seq_fork(s, n))
            assert live[-1] == m.seq_fork(s, n)
        elif what == 2 and len(live) > 2:
            live.remove(s)
            a.seq_free(s)
            m.seq_free(s)
        else:
            n = int(r.integers(1, 40))
            try:
                want = m.append_slots([s], n)
            except Exception as e:
                with pytest.raises(pa.PaError) as got:
                    a.append_slots([s], n)
                assert got.value.code == e.code
            else:
                assert a.append_slots([s], n) == tuple(want)
        same(a, m, live)


def test_truncate_refuses(pa):
    a = pa.Allocator(4)
    s = a.seq_create()
    a.append_slots([s], 20)
    for sid, n in ((s, 21), (s, -1), (s + 1, 0)):
        with pytest.raises(pa.PaError) as e:
            a.seq_truncate(sid, n)
        assert e.value.code == pa.PA_ERR_INVALID
    a.seq_truncate(s, 20)
    assert a.block_table([s], 4)[1] == [20] and a.stats()["free"] == 2
    a.seq_truncate(s, 0)
    assert a.block_table([s], 4)[1] == [0] and a.stats()["free"] == 4
    assert pa.lib().pa_seq_truncate(None, 0, 0) == pa.PA_ERR_INVALID


# ------------------------------------------------------------------------------ memory that calls may not share

def test_compact_refuses_layers_that_share_memory(pa):
    """A layer named twice would have its rows moved twice."""
    size = 10 * 2 * 16 * 64 * 2                                # bytes of a cache of compact_rc's shape
    ks, vs = [A, A + size], [A + 2 * size, A + 3 * size]
    for bad in (dict(ks=[A, A]), dict(ks=[A, A + size - 16]), dict(vs=[A + size, A + 4 * size]), dict(ks=vs),
                dict(ks=[A + 2 * size + 16, A]), dict(n=1, ks=[A], vs=[A])):
        assert compact_rc(pa, **(dict(ks=ks, vs=vs) | bad)) == pa.PA_ERR_INVALID, bad
        assert b"share memory" in pa.lib().pa_last_error_string()


def test_compact_refuses_new_lengths_over_its_inputs(pa):
    """They are written by one thread of a sequence while others still read its inputs."""
    size = 10 * 2 * 16 * 64 * 2
    ok = dict(ks=[A, A + size], vs=[A + 2 * size, A + 3 * size], lens=A + 256, off=A + 512, acc=A + 1024, num=A + 2048)
    for new in (ok["lens"] + 4, ok["lens"] - 4, ok["off"] + 8, ok["acc"] + 20, ok["num"], ok["num"] - 4):
        assert compact_rc(pa, **(ok | dict(new=new))) == pa.PA_ERR_INVALID, new
        assert b"new_seq_lens" in pa.lib().pa_last_error_string()


def test_rope_refuses_an_output_over_its_inputs(pa):
    """q_out is q itself, packed, or apart from q, k and v: other threads still read what it would write."""
    S = 4 * 8 * 128 * 2                                        # bytes of packed q
    ok = dict(q=A, k=A + 2 * S, v=A + 3 * S, out=A + 4 * S)
    row = (8 + 2 + 2) * 128                                    # elements of a projection's row
    for bad in (dict(out=A + 16), dict(out=A + 2 * S), dict(out=A + 3 * S - 16), dict(out=A + S // 2),
                dict(out=A, qst=row),                          # q in place, but not packed
                dict(out=A + 16, q=A + 3 * row * 2 + 32, qst=-row)):
        for fp8 in (False, True):
            assert rope_rc(pa, fp8, **(ok | bad)) == pa.PA_ERR_INVALID, bad
            assert b"q_out" in pa.lib().pa_last_error_string()


def test_tree_refuses_lengths_that_round_up_past_32_bits(pa):
    """The kernels count keys in 32 bits, in chunks of 128: the last length that rounds up within them is 2^31 - 128."""
    most = (1 << 31) - 128
    for bad in (dict(msl=most + 1), dict(msl=most + 112), dict(msl=0)):
        assert tree_rc(pa, mb=(1 << 27) - 1, wsb=0, **bad) == pa.PA_ERR_UNSUPPORTED
        assert b"max_seq_len" in pa.lib().pa_last_error_string()
    assert tree_rc(pa, mb=(1 << 27) - 1, wsb=0, msl=most) == pa.PA_ERR_INVALID           # past that check, to the workspace's
    assert b"workspace" in pa.lib().pa_last_error_string()


def test_frequencies_ramped_over_the_pairs(pa):
    """The ramp that checkpoints of the YaRN scaling are served with: linear in the pair's index, between the indexes
    (rounded outward) where a pair turns beta_fast and beta_slow times within the trained length."""
    for r, base, factor, trained, fast, slow in ((128, 1e6, 4.0, 32768, 32, 1), (64, 1e4, 40.0, 4096, 32, 1),
                                                 (128, 5e5, 8.0, 8192, 32, 1), (16, 1e4, 2.0, 64, 1.2, 1.1),
                                                 (32, 1e4, 16.0, 10 ** 9, 32, 1), (32, 1e4, 4.0, 10 ** 15, 32, 1), (32, 1e4, 4.0, 2, 32, 1)):
        y, a = pa.pa_rope_frequencies(r, base, "ramp_index", factor=factor, trained_tokens=trained, beta_fast=fast,
                                      beta_slow=slow, device="cpu")
        at = lambda turns: r / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
        low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), r - 1)
        if high <= low:
            high = low + 0.001
        for i in range(r // 2):
            f = base ** (-2 * i / r)
            along = min(max((i - low) / (high - low), 0), 1)
            assert math.isclose(y[i].item(), f * (1 - along) + f / factor * along, rel_tol=1e-12), (r, i)
        assert math.isclose(a, 0.1 * math.log(factor) + 1, rel_tol=1e-7)
    # by hand: base 1e4, 64 values, trained 4096: indexes 10.47 and 22.51, so pairs 0-10 are kept and from 23 on divided
    y, _ = pa.pa_rope_frequencies(64, 1e4, "ramp_index", factor=40.0, trained_tokens=4096, device="cpu")
    ratio = y.numpy() * 1e4 ** (np.arange(0, 64, 2) / 64)
    assert np.allclose(ratio[:11], 1, rtol=1e-12) and np.allclose(ratio[23:], 1 / 40, rtol=1e-12)
    assert np.allclose(np.diff(ratio[10:24]), -(1 - 1 / 40) / 13, rtol=1e-9)
    for kw in (dict(), dict(trained_tokens=64, beta_fast=1.0, beta_slow=1.0), dict(trained_tokens=64, factor=0.5)):
        with pytest.raises(pa.PaError):
            pa.pa_rope_frequencies(64, scaling="ramp_index", device="cpu", **({"factor": 2.0} | kw))
