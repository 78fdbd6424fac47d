"""pa_rope_cache_write and its E4M3 form against the definition in fp64."""
import numpy as np
import pytest
import torch

import draft_reference as ref
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return require_gpu()


def make(T, hq, hkv, D, dt, seed, strided, far=5000, pool=None, rotary=None):
    g = torch.Generator().manual_seed(seed)
    pool = pool or T // 8 + 3
    qkv = torch.randn(T, hq + 2 * hkv + 1, D, generator=g).to(TORCH_DT[dt]).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(pool * 16, generator=g)[:T].cuda()
    kc = torch.randn(pool, hkv, 16, D, generator=g).to(TORCH_DT[dt]).cuda()
    vc = torch.randn(pool, hkv, 16, D, generator=g).to(TORCH_DT[dt]).cuda()
    r = D if rotary is None else rotary
    f = torch.tensor([500000.0 ** (-2 * i / max(r, 1)) for i in range(r // 2)], dtype=torch.float64).cuda()
    return q, k, v, pos, slots, f, kc, vc


def n64(t):
    return t.double().cpu().numpy()


def bound(z, size, dt):
    """One rounding of the value (half a step; of a subnormal fp16, 2^-25) and fp32 arithmetic: the norm's sum of D
    squares is off by at most D 2^-24 relative, half of that after the root; cos and sin by 2^-23; the products and
    sums by 2^-24 each: under 2^-16 of |y_a| + |y_b|."""
    u = torch.finfo(TORCH_DT[dt]).eps / 2
    return u * np.abs(z) * (1 + 2.0 ** -8) + 2.0 ** -16 * size + 2.0 ** -24


SHAPES = [(1, 4, 2, 64, "f16"), (3, 1, 1, 128, "bf16"), (17, 8, 1, 64, "bf16"), (33, 5, 3, 128, "f16"),
          (70, 64, 8, 128, "bf16"), (257, 32, 8, 128, "f16")]


@pytest.mark.parametrize("T,hq,hkv,D,dt", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,strided,part", [(False, False, 1.0), (True, True, 1.0), (True, False, 0.25),
                                               (False, True, 0.0)])
def test_matches_definition(pa, T, hq, hkv, D, dt, interleaved, norm, strided, part):
    q, k, v, pos, slots, f, kc, vc = make(T, hq, hkv, D, dt, 3 * T + hq, strided, rotary=int(D * part))
    w = [(1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(9 + i))).to(q.dtype).cuda()
         for i in range(2)] if norm else [None, None]
    wn = [None if x is None else n64(x) for x in w]
    if T > 2:
        slots[1] = -1                       # padding
        slots[2] = kc.shape[0] * 16         # outside the pool
    kc0, vc0, q0 = kc.clone(), vc.clone(), q.clone()
    out = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc, q_norm=w[0], k_norm=w[1], eps=1e-5,
                                 interleaved=interleaved, attn_factor=1.25)
    p, fr = pos.cpu().numpy(), f.cpu().numpy()
    z, size = ref.rope(n64(q), p, fr, interleaved, 1.25, wn[0], 1e-5)
    assert (np.abs(n64(out) - z) <= bound(z, size, dt)).all()
    assert torch.equal(q, q0)
    z, size = ref.rope(n64(k), p, fr, interleaved, 1.25, wn[1], 1e-5)
    want_k, want_v, tol = n64(kc0), vc0.clone(), np.zeros(kc.shape)
    s = slots.cpu().numpy()
    for t in range(T):
        if 0 <= s[t] < kc.shape[0] * 16:
            want_k[s[t] // 16, :, s[t] % 16] = z[t]
            tol[s[t] // 16, :, s[t] % 16] = bound(z[t], size[t], dt)
            want_v[s[t] // 16, :, s[t] % 16] = v[t]
    assert (np.abs(n64(kc) - want_k) <= tol).all()                       # rows not written: exactly as before
    assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))   # v: a bit copy


def test_one_norm_weight_alone(pa):
    q, k, v, pos, slots, f, kc, vc = make(20, 8, 2, 128, "bf16", 5, False)
    w = torch.full((128,), 1.5, dtype=q.dtype).cuda()
    for a, b in ((w, None), (None, w)):
        out = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc, q_norm=a, k_norm=b)
        for x, y, m in ((out, q, a), (torch.stack([kc[s // 16, :, s % 16] for s in slots.tolist()]), k, b)):
            z, size = ref.rope(n64(y), pos.cpu().numpy(), f.cpu().numpy(), False, 1.0, None if m is None else n64(m), 1e-6)
            assert (np.abs(n64(x) - z) <= bound(z, size, "bf16")).all()


def test_v_keeps_nan_payloads_and_q_may_be_written_in_place(pa):
    q, k, v, pos, slots, f, kc, vc = make(9, 4, 2, 128, "bf16", 6, False)
    v.view(torch.int16)[:, :, ::3] = 0x7FA5
    want = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    got = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc, out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(vc[s // 16, :, s % 16].view(torch.int16), v[t].view(torch.int16))


@pytest.mark.parametrize("position", [0, 1, 1000003, 2 ** 31 - 1, -7])
def test_far_positions(pa, position):
    q, k, v, pos, slots, f, kc, vc = make(2, 2, 1, 128, "f16", 8, False)
    pos.fill_(position)
    out = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    # the reference's own angle in fp64 is off by up to position * 2^-53 relative: reduce it exactly first
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768, 10 ** 36)
    turns = [Fraction(float(x)) * position / two_pi for x in f.cpu().numpy()]
    ang = np.array([float((t - round(t)) * two_pi) for t in turns])
    z, size = ref.rope(n64(q), np.ones(2), ang, False, 1.0)
    # the frequency is rounded to 2^-54 of a turn: 2^31 tokens away that is 2 pi 2^-23
    far = abs(position) * 2 * np.pi * 2.0 ** -53
    assert (np.abs(n64(out) - z) <= bound(z, size, "f16") + far * size).all()


@pytest.mark.parametrize("T,hq,hkv,dt,interleaved,run", [(1, 8, 1, "bf16", False, False), (40, 16, 2, "f16", True, False),
                                                         (100, 8, 3, "bf16", False, True)])
def test_e4m3_cache(pa, T, hq, hkv, dt, interleaved, run):
    q, k, v, pos, slots, f, _, _ = make(T, hq, hkv, 128, dt, 77 + T, True, rotary=96)
    pool = T // 8 + 3
    if run:                                   # a prompt: consecutive rows from within a page on
        slots = torch.arange(5, 5 + T).cuda()
    if T > 2:
        slots[1] = -1
    g = torch.Generator().manual_seed(4)
    kc = torch.randint(0, 0x7F, (pool, hkv, 16, 128), generator=g, dtype=torch.uint8).cuda()
    vc = torch.randint(0, 0x7F, (pool, hkv, 128, 16), generator=g, dtype=torch.uint8).cuda()
    ks, vs = (0.002 + 0.02 * torch.rand(hkv, generator=g)).cuda(), (0.002 + 0.02 * torch.rand(hkv, generator=g)).cuda()
    kc0, vc0 = kc.clone(), vc.clone()
    out = pa.pa_rope_cache_write_fp8(q, k, v, pos, slots, f, ks, vs, kc, vc, interleaved=interleaved)
    p, fr = pos.cpu().numpy(), f.cpu().numpy()
    z, size = ref.rope(n64(q), p, fr, interleaved, 1.0)
    assert (np.abs(n64(out) - z) <= bound(z, size, dt)).all()
    zk, sk = ref.rope(n64(k), p, fr, interleaved, 1.0)
    f8 = lambda t: t.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    touched_k, touched_v = np.zeros(kc.shape, bool), np.zeros(vc.shape, bool)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        for got, want, size, scale in ((f8(kc)[s // 16, :, s % 16], zk[t], sk[t], n64(ks)[:, None]),
                                       (f8(vc)[s // 16, :, :, s % 16], n64(v)[t], np.abs(n64(v)[t]), n64(vs)[:, None])):
            x = np.clip(want / scale, -448, 448)
            # half a step of e4m3 (subnormal: 2^-10), and the fp32 value and 1 / scale before it
            assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 + 2.0 ** -15 * size / scale).all()
        touched_k[s // 16, :, s % 16] = touched_v[s // 16, :, :, s % 16] = True
    assert np.array_equal(kc.cpu().numpy()[~touched_k], kc0.cpu().numpy()[~touched_k])
    assert np.array_equal(vc.cpu().numpy()[~touched_v], vc0.cpu().numpy()[~touched_v])
    # v and the unrotated part of k: the codes of pa_cache_write_fp8, bit for bit
    k8, v8 = kc0.clone(), vc0.clone()
    pa.pa_cache_write_fp8(k.contiguous(), v.contiguous(), slots, ks, vs, k8, v8)
    assert torch.equal(v8, vc) and torch.equal(k8[..., 96:], kc[..., 96:])


def test_captured_and_on_another_stream(pa):
    q, k, v, pos, slots, f, kc, vc = make(30, 8, 2, 128, "bf16", 12, True)
    want = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    kw, vw = kc.clone(), vc.clone()
    out = torch.empty_like(want)
    kc.zero_(), vc.zero_(), kw.masked_fill_(torch.ones_like(kw, dtype=torch.bool), 0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc, out=out)
    for shift in (0, 3):
        pos.add_(shift)
        want = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kw, vw.zero_())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kc, kw) and torch.equal(vc, vw)


def test_binding_refuses(pa):
    q, k, v, pos, slots, f, kc, vc = make(6, 4, 2, 128, "f16", 1, False)
    for kw in (dict(positions=pos.long()), dict(slot_mapping=slots.int()), dict(inv_freq=f.float()),
               dict(q_norm=torch.ones(64, dtype=q.dtype).cuda()), dict(k=k.bfloat16()), dict(positions=pos[:3]),
               dict(out=torch.empty(6, 4, 64, dtype=q.dtype).cuda())):
        a = dict(q=q, k=k, v=v, positions=pos, slot_mapping=slots, inv_freq=f, k_cache=kc, v_cache=vc) | kw
        with pytest.raises((TypeError, ValueError)):
            pa.pa_rope_cache_write(**a)
    with pytest.raises(TypeError):
        pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc.bfloat16(), vc.bfloat16())
    with pytest.raises(ValueError):
        pa.pa_rope_cache_write(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, pos, slots, f, kc, vc)
    with pytest.raises(pa.PaError):
        pa.pa_rope_cache_write(q, k, v, pos, slots, f[:3], kc, vc)           # rotary_dim 6


def test_bit_pattern_tensors(pa):
    """int16 tensors with dtype=: the same bits as the typed call."""
    q, k, v, pos, slots, f, kc, vc = make(12, 4, 2, 64, "bf16", 21, True)
    k2, v2 = kc.clone(), vc.clone()
    want = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    i16 = lambda t: t.view(torch.int16)
    got = pa.pa_rope_cache_write(i16(q), i16(k), i16(v), pos, slots, f, i16(k2), i16(v2), dtype="bf16")
    assert got.dtype == torch.int16 and torch.equal(got, i16(want))
    assert torch.equal(i16(k2), i16(kc)) and torch.equal(i16(v2), i16(vc))


def test_no_tokens_and_all_padding(pa):
    q, k, v, pos, slots, f, kc, vc = make(5, 4, 2, 128, "f16", 22, False)
    k0, v0 = kc.clone(), vc.clone()
    assert pa.pa_rope_cache_write(q[:0], k[:0], v[:0], pos[:0], slots[:0], f, kc, vc).shape == (0, 4, 128)
    slots.fill_(-1)
    out = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    z, size = ref.rope(n64(q), pos.cpu().numpy(), f.cpu().numpy(), False, 1.0)
    assert (np.abs(n64(out) - z) <= bound(z, size, "f16")).all()
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


@pytest.mark.parametrize("T", [128, 129, 300, 1000])
@pytest.mark.parametrize("dt,interleaved,norm", [("bf16", False, True), ("f16", True, True), ("bf16", True, False),
                                                 ("f16", False, False)])
def test_e4m3_cache_of_a_long_piece(pa, T, dt, interleaved, norm):
    """A prompt's piece from within a page on, in pages of any order, with padding inside and at both ends: runs of V
    rows go over the edges of the groups of tokens that are written together.  Bounds as in test_e4m3_cache."""
    hq, hkv, D, rotary = 4, 3, 128, 64
    q, k, v, pos, _, f, _, _ = make(T, hq, hkv, D, dt, 5 * T, True, rotary=rotary)
    g = torch.Generator().manual_seed(T)
    pool = T // 16 + 4
    at = torch.arange(5, 5 + T)
    slots = torch.randperm(pool, generator=g)[at // 16] * 16 + at % 16
    gone = torch.tensor([0, 40, 127, T // 2, T - 1])
    slots[gone] = -1
    slots[41] = pool * 16                     # outside the pool
    slots = slots.cuda()
    kc = torch.randint(0, 0x7F, (pool, hkv, 16, D), generator=g, dtype=torch.uint8).cuda()
    vc = torch.randint(0, 0x7F, (pool, hkv, D, 16), generator=g, dtype=torch.uint8).cuda()
    ks, vs = (0.002 + 0.02 * torch.rand(hkv, generator=g)).cuda(), (0.002 + 0.02 * torch.rand(hkv, generator=g)).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(q.dtype).cuda() for _ in range(2)] if norm else [None, None]
    wn = [None if x is None else n64(x) for x in w]
    kc0, k8, v8 = kc.clone(), kc.clone(), vc.clone()
    out = pa.pa_rope_cache_write_fp8(q, k, v, pos, slots, f, ks, vs, kc, vc, q_norm=w[0], k_norm=w[1], eps=1e-5,
                                     interleaved=interleaved, attn_factor=1.25)
    p, fr = pos.cpu().numpy(), f.cpu().numpy()
    z, size = ref.rope(n64(q), p, fr, interleaved, 1.25, wn[0], 1e-5)
    assert (np.abs(n64(out) - z) <= bound(z, size, dt)).all()
    z, size = ref.rope(n64(k), p, fr, interleaved, 1.25, wn[1], 1e-5)
    s = slots.cpu().numpy()
    live = (s >= 0) & (s < pool * 16)
    got = kc.view(torch.float8_e4m3fn).float().double().cpu().numpy()[s[live] // 16, :, s[live] % 16]
    scale = n64(ks)[:, None]
    x = np.clip(z[live] / scale, -448, 448)
    assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 + 2.0 ** -15 * size[live] / scale).all()
    same = np.ones((pool, 16), bool)
    same[s[live] // 16, s[live] % 16] = False
    assert torch.equal(kc.transpose(1, 2)[torch.from_numpy(same).cuda()], kc0.transpose(1, 2)[torch.from_numpy(same).cuda()])
    # v, and k where nothing turns or norms it: the codes of pa_cache_write_fp8, the rows around them as they were
    pa.pa_cache_write_fp8(k.contiguous(), v.contiguous(), slots, ks, vs, k8, v8)
    assert torch.equal(v8, vc) and (norm or torch.equal(k8[..., rotary:], kc[..., rotary:]))


@pytest.mark.parametrize("position", [12345, 1000003, 2 ** 31 - 1, -(2 ** 31) + 5])
def test_far_angles_near_the_zeros_of_sine_and_cosine(pa, position):
    """q = (1, 0) turns into (cos t, sin t); the frequencies put t close to a zero of one of them, where fp16 resolves
    2^-24.  The frequency is held as a 64-bit fraction of a turn, off by 2 units at most; the angle is cut to 32 bits
    of a turn, and then rounded to fp32, which moves it by pi 2^-25 near a quarter turn and not at all near 0."""
    from fractions import Fraction
    r = np.random.default_rng(abs(position))
    two_pi = Fraction(6283185307179586476925286766559005768, 10 ** 36)
    quarter = np.arange(64) % 2               # odd pairs: a quarter of a turn further
    near = r.uniform(1e-5, 1e-4, 64) * r.choice([-1, 1], 64)
    turns = (r.uniform(0.001, 0.25, 64) * abs(position)).astype(np.int64) + quarter * 0.25
    f = torch.tensor((turns * 2 * np.pi + near) / abs(position), dtype=torch.float64)
    q = torch.cat([torch.ones(64), torch.zeros(64)]).half().view(1, 1, 128).cuda()
    kc = torch.zeros(1, 1, 16, 128, dtype=torch.float16, device="cuda")
    out = pa.pa_rope_cache_write(q, q, q, torch.tensor([position], dtype=torch.int32).cuda(),
                                 torch.tensor([3]).cuda(), f.cuda(), kc, kc.clone())
    got = n64(out)[0, 0]
    for i in range(64):
        t = Fraction(f[i].item()) * position / two_pi
        t = float((t - round(t)) * two_pi)
        exact = np.sin(t) if not quarter[i] else np.cos(t)
        assert abs(exact) < 2e-4, t
        tol = 2.0 ** -25 + 2 * np.pi * (2.0 ** -32 + abs(position) * 2.0 ** -63) + 2.0 ** -21 * abs(exact)
        assert abs(got[64 + i if not quarter[i] else i] - exact) <= tol + quarter[i] * np.pi * 2.0 ** -25, i
    assert torch.equal(kc[0, 0, 3], out[0, 0])


def test_pages_past_4_gib(pa):
    """The last pages of pools of 5 GiB: the same rows as in a small pool, and nothing at their offsets modulo 2^32."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    T, hq, hkv = 40, 8, 8
    q, k, v, pos, slots, f, kc, vc = make(T, hq, hkv, 128, "bf16", 31, True, pool=12)
    page = hkv * 16 * 128 * 2
    far = (5 << 30) // page
    big = [torch.zeros(far + 12, hkv, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kc.zero_(), vc.zero_()
    want = pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc, vc)
    got = pa.pa_rope_cache_write(q, k, v, pos, slots + far * 16, f, *big)
    assert torch.equal(got, want)
    for x, y in zip(big, (kc, vc)):
        assert torch.equal(x[far:], y)
        assert not x[:far].view(torch.int16).any()
    del big, x
    ks, vs = (torch.full((hkv,), 0.02, device="cuda") for _ in range(2))
    k8, v8 = torch.zeros(12, hkv, 16, 128, dtype=torch.uint8, device="cuda"), torch.zeros(12, hkv, 128, 16, dtype=torch.uint8, device="cuda")
    far *= 2
    b8 = [torch.zeros(far + 12, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in (k8, v8)]
    pa.pa_rope_cache_write_fp8(q, k, v, pos, slots, f, ks, vs, k8, v8)
    pa.pa_rope_cache_write_fp8(q, k, v, pos, slots + far * 16, f, ks, vs, *b8)
    for x, y in zip(b8, (k8, v8)):
        assert torch.equal(x[far:], y) and not x[:far].any()
