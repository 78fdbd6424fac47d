"""pa_tree_plan and pa_decode_tree against their definitions in fp64."""
import numpy as np
import pytest
import torch

import draft_reference as ref
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return require_gpu()


def dev(a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a if dt is None else a.astype(dt))).cuda()


def trees(r, sizes, deep=False):
    return np.concatenate([[j - 1 if deep else int(r.integers(-1, j)) for j in range(n)] for n in sizes]
                          + [[]]).astype(np.int32)


# ------------------------------------------------------------------------------ plan

@pytest.mark.parametrize("words,sizes,deep", [(1, [1], False), (1, [64, 1, 0, 33], False), (1, [64], True),
                                              (2, [65, 128, 7], False), (3, [192, 129], True), (4, [256, 255, 2], False),
                                              (4, [256], True), (4, [3] * 300, False)])
def test_plan(pa, words, sizes, deep):
    r = np.random.default_rng(len(sizes) + words)
    parents = trees(r, sizes, deep)
    before = r.integers(0, 1000, len(sizes))
    off = np.concatenate([[0], np.cumsum(sizes)])
    err = torch.zeros(1, dtype=torch.int32).cuda()
    masks, pos = pa.pa_tree_plan(dev(parents), dev(off, np.int32), dev(before + sizes, np.int32), mask_words=words,
                                 error_bits=err)
    want, depth = ref.tree_masks(parents, sizes, words)
    assert np.array_equal(masks.cpu().numpy().view(np.uint64), want)
    assert np.array_equal(pos.cpu().numpy(), np.repeat(before, sizes) + depth)
    assert err.item() == 0 and pa.pa_decode_check(err) == 0


def test_plan_flags_bad_trees_and_leaves_other_rows(pa):
    err = torch.zeros(1, dtype=torch.int32).cuda()
    masks, pos = torch.full((9, 1), 77).cuda(), torch.full((9,), 55, dtype=torch.int32).cuda()
    off, lens = dev(np.array([0, 3, 6]), np.int32), dev(np.array([10, 20]), np.int32)
    pa.pa_tree_plan(dev(np.array([-1, 1, 0, -1, 5, -2, 0, 0, 0]), np.int32), off, lens, masks=masks, positions=pos,
                    error_bits=err)
    assert err.item() == pa.PA_DEVERR_TREE and pa.pa_decode_check(err) == pa.PA_DEVERR_TREE
    assert masks[:, 0].tolist() == [1, 2, 5, 1, 2, 4, 77, 77, 77]
    assert pos.tolist() == [7, 7, 8, 17, 17, 17, 55, 55, 55]
    for o, l in (([0, 3, 70], [10, 80]), ([0, 5, 3], [10, 20]), ([0, 3, 6], [2, 20])):   # too long, backwards, L < n
        err.zero_()
        pa.pa_tree_plan(dev(np.full(70, -1), np.int32), dev(np.array(o), np.int32), dev(np.array(l), np.int32),
                        error_bits=err)
        assert err.item() & pa.PA_DEVERR_SEQ_LEN


# ------------------------------------------------------------------------------ attention

def make(r, befores, sizes, hq, hkv, D, dt, words=None, poison=True, spare=2, bits=None):
    """q, caches, tables, lens, offsets, masks (device) of sequences; unused rows of the pool NaN."""
    lens = np.array(befores) + np.array(sizes)
    pages = -(-lens // 16)
    pool = int(pages.sum()) + 3
    ids = r.permutation(pool)
    table = np.full((len(lens), max(1, pages.max()) + spare), ids[-1], np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    g = torch.Generator().manual_seed(int(r.integers(1 << 30)))
    kc, vc = (torch.randn(pool, hkv, 16, D, generator=g).to(TORCH_DT[dt]) for _ in range(2))
    if poison:
        used = torch.zeros(pool, 16, dtype=torch.bool)
        for b, L in enumerate(lens):
            for p in range(L):
                used[table[b, p // 16], p % 16] = True
        for c in (kc, vc):
            c.masked_fill_(~used[:, None, :, None], float("nan"))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    words = words or max(1, (max(sizes) + 63) // 64)
    masks = ref.tree_masks(trees(r, sizes), sizes, words)[0] if bits is None else bits
    q = torch.randn(int(off[-1]), hq, D, generator=g).to(TORCH_DT[dt])
    return dict(q=q.cuda(), k_cache=kc.cuda(), v_cache=vc.cuda(), block_tables=dev(table),
                seq_lens=dev(lens.astype(np.int32)), q_offsets=dev(off), masks=dev(masks.view(np.int64)),
                scale=1.0 / np.sqrt(D))


def check(a, out, dt, rows=None):
    """Against fp64.  With u half a step of the type and A the softmax-weighted |V|: the result is rounded once
    (u |out|), each softmax weight once for the product (u A); scores are fp32 dots of D products, off by at most
    (D + 4) 2^-24 sum |q k| scale = e each, which moves numerator and denominator by e (2 e A); 2^x is good to
    2^-21; sums of L terms in fp32 (tensor cores may truncate: 2^-23 a step) and their rescalings."""
    n = lambda t: t.double().cpu().numpy()
    want, size, dots = ref.tree_attention(n(a["q"]), n(a["k_cache"]), n(a["v_cache"]), a["block_tables"].cpu().numpy(),
                                          a["seq_lens"].cpu().numpy(), a["q_offsets"].cpu().numpy(),
                                          a["masks"].cpu().numpy().view(np.uint64), a["scale"])
    u = torch.finfo(TORCH_DT[dt]).eps / 2
    D, L = a["q"].shape[2], int(a["seq_lens"].max())
    e = (D + 4) * 2.0 ** -24 * dots[..., None]
    tol = u * np.abs(want) + (u + 2 * e + 2.0 ** -20 + (L + 64) * 2.0 ** -22) * size * (1 + 2 * u) + 2.0 ** -24
    got = n(out)
    inside = slice(0, int(a["q_offsets"][-1]))
    assert np.isfinite(got[inside]).all()
    worst = (np.abs(got - want)[inside] / tol[inside]).max(initial=0)
    assert worst <= 1, worst
    return want


def ws(pa, a, msl):
    B, (Tq, Hq, D) = a["seq_lens"].numel(), a["q"].shape
    return torch.empty(pa.pa_decode_tree_workspace_bytes(B, Tq, Hq, a["k_cache"].shape[1], D, msl), dtype=torch.uint8,
                       device="cuda")


CASES = [  # tokens before the trees, sizes of the trees
    ([0], [1]), ([0], [5]), ([1], [1]), ([15, 16, 17], [1, 1, 1]), ([127, 128, 129, 63], [1, 2, 7, 1]),
    ([0, 3, 100, 640], [0, 64, 13, 0]), ([250], [64]), ([61, 190], [65, 130]), ([1000, 7, 333], [33, 256, 1]),
    ([2500], [3]),
]


@pytest.mark.parametrize("befores,sizes", CASES)
@pytest.mark.parametrize("hq,hkv,D,dt", [(4, 2, 64, "f16"), (8, 1, 128, "bf16"), (3, 3, 128, "f16"), (8, 2, 64, "bf16")])
def test_tree(pa, befores, sizes, hq, hkv, D, dt):
    a = make(np.random.default_rng(sum(befores) + len(sizes)), befores, sizes, hq, hkv, D, dt)
    w = ws(pa, a, a["block_tables"].shape[1] * 16)
    out = pa.pa_decode_tree(**a, workspace=w)
    assert pa.pa_decode_check(w) == 0
    check(a, out, dt)
    assert torch.equal(out, pa.pa_decode_tree(**a))          # split or not by the same rule: the same bits


def test_many_sequences(pa):
    r = np.random.default_rng(3)
    n = 1100                                                  # more than the plan holds at a time
    a = make(r, r.integers(0, 200, n).tolist(), r.integers(0, 4, n).tolist(), 2, 2, 64, "bf16")
    check(a, pa.pa_decode_tree(**a), "bf16")


def test_long_contexts_split_and_mixed(pa):
    r = np.random.default_rng(4)
    a = make(r, [9000, 40, 5000, 300] + [20] * 8, [20, 3, 1, 40] + [2] * 8, 8, 1, 128, "bf16", poison=False)
    check(a, pa.pa_decode_tree(**a), "bf16")


def test_any_masks_and_empty_rows(pa):
    """Masks are any bits: rows that see nothing give zeros, bits past the tree do not count."""
    r = np.random.default_rng(5)
    sizes, befores = [40, 70, 3], [0, 0, 200]
    bits = r.integers(0, 1 << 63, (sum(sizes), 2), dtype=np.int64).view(np.uint64)
    bits[3] = bits[50] = 0
    bits[4] = np.array([1 << 60, 3], np.uint64)               # only past this tree of 40
    a = make(r, befores, sizes, 8, 2, 128, "bf16", words=2, bits=bits)
    out = pa.pa_decode_tree(**a)
    check(a, out, "bf16")
    assert (out[[3, 50, 4]] == 0).all()


def test_chain_is_the_prefill_and_one_token_the_decode(pa):
    r = np.random.default_rng(6)
    befores, sizes = [300, 0, 1500], [48, 17, 64]
    bits = np.array([[(1 << (j + 1)) - 1] for n in sizes for j in range(n)], np.uint64)
    a = make(r, befores, sizes, 16, 2, 128, "bf16", bits=bits)
    out = pa.pa_decode_tree(**a)
    want = check(a, out, "bf16")
    b = {k: v for k, v in a.items() if k != "masks"}
    other = pa.pa_prefill(**b).double().cpu().numpy()
    assert np.abs(other - want).max() <= 2e-2
    a = make(r, [5, 700, 2100], [1, 1, 1], 16, 2, 128, "f16")
    out = pa.pa_decode_tree(**a)
    want = check(a, out, "f16")
    d = pa.pa_decode(a["q"], a["k_cache"], a["v_cache"], a["block_tables"], a["seq_lens"], a["scale"])
    assert np.abs(d.double().cpu().numpy() - want).max() <= 1e-2


def test_padded_batch_leaves_rows_as_they_were(pa):
    a = make(np.random.default_rng(7), [100, 30], [6, 9], 8, 2, 128, "bf16")
    tail = 10
    a["q"] = torch.cat([a["q"], torch.full((tail, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    a["masks"] = torch.cat([a["masks"], torch.full((tail, 1), -1, device="cuda")])
    out = torch.full_like(a["q"], 3.0)
    pa.pa_decode_tree(**a, out=out)
    check(a, out, "bf16")
    assert (out[15:] == 3.0).all()


def test_large_scores_and_lowest_values(pa):
    """Scores of hundreds (the running maximum moves), keys of the type's lowest value in places nobody sees."""
    r = np.random.default_rng(8)
    a = make(r, [400], [12], 8, 1, 128, "bf16")
    a["q"] *= 8
    a["k_cache"] *= 4
    bits = a["masks"].clone()
    bits &= ~(1 << 5)                                          # nobody sees token 5, itself neither
    a["masks"] = bits
    p = 405
    page = int(a["block_tables"][0, p // 16])
    a["k_cache"][page, :, p % 16] = torch.finfo(torch.bfloat16).min
    b = dict(a, k_cache=a["k_cache"].clone())
    out = pa.pa_decode_tree(**a)
    b["k_cache"][page, :, p % 16] = 0
    check(b, out, "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("before", [0, 50, 125, 700])
def test_nan_and_infinity_reach_only_who_sees_them(pa, D, before):
    r = np.random.default_rng(9 + before)
    n = 70
    a = make(r, [before, 90], [n, 4], 8, 2, D, "bf16")
    clean = dict(a, v_cache=a["v_cache"].clone(), k_cache=a["k_cache"].clone())
    inf, nan = float("inf"), float("nan")
    bad = {3: (nan, None), 10: (None, inf), 11: (-inf, None), 40: (nan, nan), 69: (None, nan)}   # token: (K, V)
    table = a["block_tables"].cpu().numpy()
    hit = np.zeros(n, bool)
    masks = a["masks"].cpu().numpy().view(np.uint64)
    for i, (k, v) in bad.items():
        page, row = int(table[0, (before + i) // 16]), (before + i) % 16
        if k is not None:
            a["k_cache"][page, 1, row, 5] = k
        if v is not None:
            a["v_cache"][page, 1, row, 7] = v
    for t in range(n):
        hit[t] = any((int(masks[t, i >> 6]) >> (i & 63)) & 1 for i in bad)
    out, good = pa.pa_decode_tree(**a), pa.pa_decode_tree(**clean)
    assert torch.equal(out[:n, :4], good[:n, :4]) and torch.equal(out[n:], good[n:])   # the other KV head, sequence
    keep = torch.from_numpy(~hit).cuda()
    assert keep.any() and (~keep).any()
    assert torch.equal(out[:n, 4:][keep], good[:n, 4:][keep])
    sees_v = torch.tensor([any(v is not None and (int(masks[t, i >> 6]) >> (i & 63)) & 1 for i, (k, v) in bad.items())
                           for t in range(n)]).cuda()
    assert not torch.isfinite(out[:n, 4:, 7][sees_v]).any()


def test_bad_device_data_is_flagged(pa):
    a = make(np.random.default_rng(10), [100, 30, 64], [6, 9, 2], 8, 2, 128, "bf16")
    good = pa.pa_decode_tree(**a)
    msl = a["block_tables"].shape[1] * 16
    w = ws(pa, a, msl)
    b = dict(a, block_tables=a["block_tables"].clone())
    b["block_tables"][1, 0] = b["k_cache"].shape[0]
    b["block_tables"][2, 0] = -5
    out = pa.pa_decode_tree(**b, workspace=w)
    assert pa.pa_decode_check(w) == pa.PA_DEVERR_BLOCK_ID
    check(b, out, "bf16")                                     # those pages read as zeros
    assert torch.equal(out[:6], good[:6])
    for lens in ([106, msl + 1, 66], [106, 39, -3], [106, 39, 1]):
        b = dict(a, seq_lens=dev(np.array(lens), np.int32))
        out = pa.pa_decode_tree(**b, workspace=w)
        assert pa.pa_decode_check(w) & pa.PA_DEVERR_SEQ_LEN
        assert torch.equal(out[:6], good[:6])
    for off in ([0, 6, 5, 17], [0, 6, 15, 40], [2, 6, 15, 17]):
        pa.pa_decode_tree(**dict(a, q_offsets=dev(np.array(off), np.int32)), workspace=w)
        assert pa.pa_decode_check(w) & pa.PA_DEVERR_SEQ_LEN
    assert torch.equal(pa.pa_decode_tree(**a, workspace=w), good) and pa.pa_decode_check(w) == 0
    # a tree longer than its masks reach: its first tokens as ever, the rest left alone
    a = make(np.random.default_rng(11), [20, 30], [70, 5], 8, 2, 128, "bf16")
    out = torch.full_like(a["q"], 9.0)
    w = ws(pa, a, 160)
    pa.pa_decode_tree(**dict(a, masks=a["masks"][:, :1].contiguous()), out=out, workspace=w)
    assert pa.pa_decode_check(w) == pa.PA_DEVERR_SEQ_LEN
    assert torch.equal(out[:64], pa.pa_decode_tree(**a)[:64]) and (out[64:70] == 9.0).all()


def test_captured_replayed_and_on_another_stream(pa):
    r = np.random.default_rng(12)
    a = make(r, [3000, 10], [16, 8], 8, 1, 128, "bf16", poison=False)
    w, out = ws(pa, a, a["block_tables"].shape[1] * 16), torch.empty_like(a["q"])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    pa.pa_decode_tree(**a, workspace=w)
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        pa.pa_decode_tree(**a, workspace=w, out=out)
    for lens in ([3016, 18], [2900, 18], [40, 8]):
        a["seq_lens"].copy_(dev(np.array(lens), np.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(a, out, "bf16")
    # two at once, each with a workspace of its own
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(pa.pa_decode_tree(**a))
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_binding_refuses(pa):
    a = make(np.random.default_rng(13), [10], [4], 8, 2, 128, "bf16")
    for kw in (dict(masks=a["masks"].int()), dict(masks=a["masks"][:2]), dict(q_offsets=a["q_offsets"][:1]),
               dict(seq_lens=a["seq_lens"].long()), dict(out=a["q"].float()), dict(v_cache=a["v_cache"].half()),
               dict(k_cache=a["k_cache"].half(), v_cache=a["v_cache"].half())):
        with pytest.raises((TypeError, ValueError)):
            pa.pa_decode_tree(**(a | kw))
    with pytest.raises(pa.PaError):
        pa.pa_decode_tree(**a, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PaError):
        pa.pa_decode_tree(**(a | dict(scale=0.0)))


# ------------------------------------------------------------------------------ larger shapes, fp64 on the GPU

def gpu_case(r, befores, sizes, hq, hkv, D, dt, far=0):
    """Like make(), built on the GPU; with ``far`` the pool starts with that many unused pages."""
    lens = np.array(befores) + np.array(sizes)
    pages = -(-lens // 16)
    pool = far + int(pages.sum()) + 1
    ids = far + r.permutation(int(pages.sum()))
    table = np.full((len(lens), max(1, pages.max())), pool - 1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    g = torch.Generator(device="cuda").manual_seed(int(r.integers(1 << 30)))
    kc, vc = (torch.empty(pool, hkv, 16, D, dtype=TORCH_DT[dt], device="cuda") for _ in range(2))
    for c in (kc, vc):
        c[far:].normal_(generator=g)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    masks = ref.tree_masks(trees(r, sizes), sizes, max(1, (max(sizes) + 63) // 64))[0]
    q = torch.empty(int(off[-1]), hq, D, dtype=TORCH_DT[dt], device="cuda").normal_(generator=g)
    return dict(q=q, k_cache=kc, v_cache=vc, block_tables=dev(table), seq_lens=dev(lens.astype(np.int32)),
                q_offsets=dev(off), masks=dev(masks.view(np.int64)), scale=1.0 / np.sqrt(D))


def gpu_check(a, out, dt):
    """check() with the reference as matrix products in fp64 on the GPU, per sequence and KV head."""
    u, D, G = torch.finfo(TORCH_DT[dt]).eps / 2, a["q"].shape[2], a["q"].shape[1] // a["k_cache"].shape[1]
    off, lens = a["q_offsets"].tolist(), a["seq_lens"].tolist()
    worst = 0.0
    for b, L in enumerate(lens):
        lo, hi = off[b], off[b + 1]
        if lo == hi:
            continue
        n = hi - lo
        words = a["masks"][lo:hi].cpu().numpy().view(np.uint8)
        bits = torch.from_numpy(np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)).cuda()
        hide = torch.cat([torch.zeros(n, L - n, dtype=torch.bool, device="cuda"), ~bits], 1).repeat_interleave(G, 0)
        pages = a["block_tables"][b, :-(-L // 16)].long()
        for h in range(a["k_cache"].shape[1]):
            K, V = (a[c][pages, h].reshape(-1, D)[:L].double() for c in ("k_cache", "v_cache"))
            q = a["q"][lo:hi, h * G:(h + 1) * G].double().reshape(-1, D)
            p = torch.softmax((q @ K.T * a["scale"]).masked_fill(hide, -torch.inf), -1)
            want, size = p @ V, p @ V.abs()
            e = (D + 4) * 2.0 ** -24 * a["scale"] * (q.abs() @ K.abs().T).amax(-1, keepdim=True)
            tol = u * want.abs() + (u + 2 * e + 2.0 ** -20 + (L + 64) * 2.0 ** -22) * size * (1 + 2 * u) + 2.0 ** -24
            got = out[lo:hi, h * G:(h + 1) * G].double().reshape(-1, D)
            worst = max(worst, ((got - want).abs() / tol).max().item())
    assert worst <= 1, worst


@pytest.mark.parametrize("befores,sizes,hq,hkv,D,dt", [
    ([5000, 0, 30000], [256, 200, 1], 16, 2, 128, "bf16"),        # sixteen tiles of rows
    ([4000] * 4, [64] * 4, 32, 4, 128, "f16"),                    # shares cut along the sequences
    ([2000, 5000, 1], [256, 3, 256], 3, 3, 64, "bf16"),           # two tiles without grouped heads
    ([10] * 1500 + [5000] * 3, [2] * 1500 + [40] * 3, 4, 1, 64, "f16"),
    ([20000], [5], 8, 8, 64, "f16"), ([70000], [61], 8, 1, 128, "bf16"),
])
def test_larger_shapes(pa, befores, sizes, hq, hkv, D, dt):
    a = gpu_case(np.random.default_rng(len(sizes)), befores, sizes, hq, hkv, D, dt)
    w = ws(pa, a, a["block_tables"].shape[1] * 16)
    out = pa.pa_decode_tree(**a, workspace=w)
    assert pa.pa_decode_check(w) == 0
    gpu_check(a, out, dt)
    for _ in range(3):
        assert torch.equal(out, pa.pa_decode_tree(**a, workspace=w))


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(pa, seed):
    r = np.random.default_rng(100 + seed)
    n = int(np.exp(r.uniform(0, np.log(150))))
    top = int(np.exp(r.uniform(np.log(4), np.log(40000 / n + 5))))
    befores, sizes = r.integers(0, top + 1, n).tolist(), r.integers(0, r.integers(2, 140), n).tolist()
    if not sum(sizes):
        sizes[0] = 1
    hkv, G, D = int(r.choice([1, 2, 3, 5, 8])), int(r.choice([1, 2, 4, 8])), int(r.choice([64, 128]))
    dt = str(r.choice(["f16", "bf16"]))
    a = gpu_case(r, befores, sizes, hkv * G, hkv, D, dt)
    gpu_check(a, pa.pa_decode_tree(**a), dt)


def test_pages_past_4_gib(pa):
    """Pages whose bytes, and whose elements, lie past 2^32 in both caches; rotation and compaction there too."""
    far = (1 << 33) // (8 * 16 * 128 * 2)
    a = gpu_case(np.random.default_rng(31), [700, 90], [20, 64], 16, 8, 128, "bf16", far=far)
    out = pa.pa_decode_tree(**a)
    gpu_check(a, out, "bf16")
    near = {k: a[k][far:].contiguous() for k in ("k_cache", "v_cache")}
    b = dict(a, **near, block_tables=a["block_tables"] - far)
    assert torch.equal(out, pa.pa_decode_tree(**b))
    acc, num = dev(np.array([[1, 5, 19], [0, 62, 63]], np.int32)), dev(np.array([3, 2], np.int32))
    args = (a["seq_lens"], a["q_offsets"], acc, num)
    pa.pa_cache_compact([a["k_cache"]], [a["v_cache"]], a["block_tables"], *args)
    pa.pa_cache_compact([near["k_cache"]], [near["v_cache"]], b["block_tables"], *args)
    slots = a["block_tables"][:, 0].long() * 16 + 5
    q, k = a["q"][:2], a["q"][:2, :8].contiguous()
    f = torch.ones(64, dtype=torch.float64, device="cuda")
    for c, s in ((a, slots), (near, slots - far * 16)):
        pa.pa_rope_cache_write(q, k, k, acc[:, 0].contiguous(), s, f, c["k_cache"], c["v_cache"])
    for c in ("k_cache", "v_cache"):
        assert torch.equal(a[c][far:].view(torch.int16), near[c].view(torch.int16))


def test_calls_on_a_given_stream(pa):
    """``stream=``: outputs and the workspace belong to that stream, whatever the current one does meanwhile."""
    a = gpu_case(np.random.default_rng(32), [9000, 60], [30, 9], 8, 1, 128, "bf16")
    want = pa.pa_decode_tree(**a)
    parents = dev(trees(np.random.default_rng(1), [30, 9]))
    plan = pa.pa_tree_plan(parents, a["q_offsets"], a["seq_lens"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = pa.pa_decode_tree(**a, stream=side)
        got_plan = pa.pa_tree_plan(parents, a["q_offsets"], a["seq_lens"], stream=side)
        junk = [torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda") for _ in range(40)]   # freed blocks, rewritten
        side.synchronize()
        assert torch.equal(got, want) and all(torch.equal(x, y) for x, y in zip(got_plan, plan))
        del junk


def test_no_trees(pa):
    """No sequences, no tokens, and only empty trees: nothing is written."""
    a = make(np.random.default_rng(41), [40, 9], [3, 2], 8, 2, 128, "bf16")
    none = dict(a, q=a["q"][:0], masks=a["masks"][:0], q_offsets=dev(np.zeros(3, np.int32)))
    assert pa.pa_decode_tree(**none).shape == (0, 8, 128)
    assert pa.pa_decode_tree(**dict(none, q_offsets=dev(np.zeros(1, np.int32)), seq_lens=a["seq_lens"][:0],
                                    block_tables=a["block_tables"][:0])).shape == (0, 8, 128)
    out = torch.full_like(a["q"], 5.0)
    w = ws(pa, a, 80)
    pa.pa_decode_tree(**dict(a, q_offsets=dev(np.zeros(3, np.int32))), out=out, workspace=w)
    assert (out == 5.0).all() and pa.pa_decode_check(w) == 0


def test_threads_call_at_once(pa):
    """Host threads, each with a stream and a workspace of its own."""
    import threading
    cases = [gpu_case(np.random.default_rng(50 + i), [3000 * i, 70], [9 + i, 33], 8, 2, (64, 128)[i % 2], "bf16")
             for i in range(4)]
    want = [pa.pa_decode_tree(**c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = pa.pa_decode_tree(**cases[i])
                s.synchronize()
                if not torch.equal(got, want[i]):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("gap", [20.7, 24.4, 26.3])
@pytest.mark.parametrize("hq,hkv,D,dt", [(4, 2, 64, "f16"), (8, 1, 128, "f16"), (8, 1, 128, "bf16")])
def test_weights_far_below_the_largest(pa, gap, hq, hkv, D, dt):
    """Keys whose weight is 2^-gap of the largest and that alone have values: fp16 weights of theirs would be
    subnormal, or nothing.  Two keys of every 1024 have the largest weight, one in either half of a chunk, and the
    value 0.  Beside check()'s terms: a stored fp16 weight, 2^7 times its share of the largest, may be off by half a
    subnormal step, 2^-25, so all of them by keys 2^-32 against a sum of at least the largest weights' number."""
    r = np.random.default_rng(14)
    L, n = 8192, 5
    a = make(r, [L - n], [n], hq, hkv, D, dt, poison=False)
    k, v = torch.zeros(L, dtype=a["q"].dtype), torch.full((L,), 64, dtype=a["q"].dtype)
    top = [p for p in range(L - n) if p % 1024 in (0, 64)]
    k[top], v[top] = gap / (16 * a["scale"] * np.log2(np.e)), 0
    table = a["block_tables"][0, :L // 16].long()
    a["q"].zero_()[..., 0] = 16
    a["k_cache"].zero_()[table, :, :, 0] = k.cuda().view(-1, 1, 16)
    a["v_cache"][table] = v.cuda().view(-1, 1, 16, 1)
    out = pa.pa_decode_tree(**a)
    m = lambda t: t.double().cpu().numpy()
    want, size, dots = ref.tree_attention(m(a["q"]), m(a["k_cache"]), m(a["v_cache"]), a["block_tables"].cpu().numpy(),
                                          a["seq_lens"].cpu().numpy(), a["q_offsets"].cpu().numpy(),
                                          a["masks"].cpu().numpy().view(np.uint64), a["scale"])
    u, e = torch.finfo(TORCH_DT[dt]).eps / 2, (D + 4) * 2.0 ** -24 * dots[..., None]
    tol = u * np.abs(want) + (u + 2 * e + 2.0 ** -20 + (L + 64) * 2.0 ** -22) * size * (1 + 2 * u) + 2.0 ** -24
    tol += 64 * L / len(top) * 2.0 ** -32
    assert (np.abs(m(out) - want) <= tol).all(), (np.abs(m(out) - want) / tol).max()


def test_many_sequences_some_of_them_split(pa):
    """More than the plan holds at a time, long ones among the first and among the others."""
    r = np.random.default_rng(15)
    befores, sizes = r.integers(0, 150, 1100), r.integers(0, 3, 1100)
    befores[[3, 1050]], sizes[[3, 1050]] = [30000, 17000], [3, 2]
    a = make(r, befores.tolist(), sizes.tolist(), 4, 4, 64, "bf16", poison=False)
    a["block_tables"] = a["block_tables"].contiguous()
    w = ws(pa, a, a["block_tables"].shape[1] * 16)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    out = pa.pa_decode_tree(**a, workspace=w, events=events)
    assert pa.pa_decode_check(w) == 0 and events[0].elapsed_time(events[1]) > 0
    check(a, out, "bf16")


def test_fp16_scores_of_tens_of_millions_stay_finite(pa):
    """The maximum of such scores is rounded by whole units, so a weight may exceed what the reference allows for by
    some powers of two.  All values are 1: so is the result, but for a rounding each of the weights and the output."""
    a = make(np.random.default_rng(16), [380], [4], 8, 1, 128, "f16", poison=False)
    table = a["block_tables"][0, :24].long()
    for first in (7880, 7096, 4000):
        for second in (48, 64, 80):
            k = torch.zeros(24 * 16, 128, dtype=torch.float16)
            k[:, 0] = first
            k[128:256, 1], k[256:, 1] = second, 2 * second
            a["q"].zero_()[..., :2] = torch.tensor([60000.0, 1.0])
            a["k_cache"][table] = k.cuda().view(24, 1, 16, 128)
            a["v_cache"].fill_(1)
            out = pa.pa_decode_tree(**a)
            assert (out.double() - 1).abs().max() <= 2.0 ** -10 + 2.0 ** -20, (first, second)


def test_rows_of_no_tree(pa):
    """A captured batch whose sequences have no drafts this time: nothing is written, nothing flagged."""
    a = make(np.random.default_rng(17), [100, 30, 0], [3, 2, 1], 8, 2, 128, "bf16")
    a["q_offsets"].zero_()
    w = ws(pa, a, a["block_tables"].shape[1] * 16)
    out = torch.full_like(a["q"], 5.0)
    pa.pa_decode_tree(**a, workspace=w, out=out)
    assert pa.pa_decode_check(w) == 0 and (out == 5.0).all()
    err = torch.zeros(1, dtype=torch.int32).cuda()
    masks, pos = torch.full((6, 1), 7).cuda(), torch.full((6,), 8, dtype=torch.int32).cuda()
    pa.pa_tree_plan(torch.full((6,), -1, dtype=torch.int32).cuda(), a["q_offsets"], a["seq_lens"], masks=masks,
                    positions=pos, error_bits=err)
    assert (masks == 7).all() and (pos == 8).all() and err.item() == 0


def test_two_graphs_at_once(pa):
    """Replayed on two streams together, each with a workspace of its own."""
    r = np.random.default_rng(18)
    cases = [make(r, [3000, 10, 700], [16, 8, 40], 8, 1, 128, "bf16", poison=False) for _ in range(2)]
    graphs, outs, want = [], [], []
    for a in cases:
        w, out, g = ws(pa, a, a["block_tables"].shape[1] * 16), torch.empty_like(a["q"]), torch.cuda.CUDAGraph()
        want.append(pa.pa_decode_tree(**a, workspace=w))
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(5):
                pa.pa_decode_tree(**a, workspace=w, out=out)
        graphs.append(g), outs.append((out, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (out, w), x in zip(outs, want):
        assert torch.equal(out, x) and pa.pa_decode_check(w) == 0
