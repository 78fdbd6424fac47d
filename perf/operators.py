"""Cases of the speculative-decoding operators over the paged KV cache.

Four operators that run together when a model verifies drafted tokens:

  rope     per-head norm of q and k, position rotation, K/V into the pages
  plan     parents of the drafted tokens -> ancestor masks and positions
  tree     attention of each draft tree over its sequence's pages
  compact  accepted tokens' K/V rows moved to consecutive positions

``own`` false: elementary torch operations in 32 bits (angles in 64).
``own`` true: the library's calls.
"""
import functools
import math

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a handful of chats, one new token each: launch latency is all there is
        dict(name="rope_tiny_step", op="rope", tokens=4, hq=4, hkv=2, d=64, dtype="f16", rotary=64,
             interleaved=False, norm=False, yarn=1.0, fp8=False, fused=False, padded=0, far=2048),
        # the decode step of a full batch at the 70B shape, padded as for a captured graph, normed heads
        dict(name="rope_step_70b", op="rope", tokens=256, hq=64, hkv=8, d=128, dtype="bf16", rotary=128,
             interleaved=False, norm=True, yarn=1.0, fp8=False, fused=True, padded=11, far=34000),
        # one piece of a long prompt with 20 decode tokens, rotation scaled for a long context
        dict(name="rope_piece_70b", op="rope", tokens=3770, hq=64, hkv=8, d=128, dtype="bf16", rotary=128,
             interleaved=True, norm=False, yarn=8.0, fp8=False, fused=True, padded=0, far=30000),
        # a whole 30,000-token prompt into an E4M3 cache, half of each head rotated
        dict(name="rope_prompt_fp8", op="rope", tokens=30000, hq=64, hkv=8, d=128, dtype="bf16", rotary=64,
             interleaved=False, norm=True, yarn=1.0, fp8=True, fused=False, padded=0, far=30000),
        # a few chats with small trees
        dict(name="plan_few", op="plan", seqs=4, nodes=8, words=1, far=2048),
        # a full batch with the largest trees
        dict(name="plan_full", op="plan", seqs=256, nodes=256, words=4, far=34000),
        # the smallest verification: four short chats, five drafted tokens each
        dict(name="tree_tiny", op="tree", seqs=4, lo=1, hi=100, long=0, far=0, nodes=5, ragged=False, hq=4,
             hkv=2, d=64, dtype="f16"),
        # a batch of chats at the 8B shape, trees of up to 32 nodes
        dict(name="tree_batch_8b", op="tree", seqs=64, lo=128, hi=2048, long=0, far=0, nodes=32, ragged=True,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # the mixed batch at the 70B shape: most chats short, a tenth with documents, trees of up to 8
        dict(name="tree_mix_70b", op="tree", seqs=256, lo=301, hi=400, long=26, far=34000, nodes=8, ragged=True,
             hq=64, hkv=8, d=128, dtype="bf16"),
        # long contexts with full 64-node trees: the products bound it, not the pages
        dict(name="tree_long_8b", op="tree", seqs=8, lo=32768, hi=32768, long=0, far=0, nodes=64, ragged=False,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # one layer of a few chats
        dict(name="compact_few", op="compact", seqs=4, lo=1, hi=100, nodes=8, most=5, layers=1, hkv=2, d=64,
             dtype="f16"),
        # every layer of the 8B shape after one verification of a batch
        dict(name="compact_8b", op="compact", seqs=64, lo=16, hi=256, nodes=64, most=8, layers=32, hkv=8, d=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    op = rng.choice(["rope", "plan", "tree", "tree", "compact"])
    if op == "plan":
        words = rng.randint(1, 4)
        return dict(op=op, seqs=_log(rng, 1, 256), nodes=rng.randint(1, 64 * words), words=words,
                    far=_log(rng, 16, 34000))
    dtype, d = rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op == "rope":
        fp8 = d == 128 and rng.random() < 0.4
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hq, hkv=hkv, d=d, dtype=dtype,
                    rotary=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5, norm=rng.random() < 0.5,
                    yarn=rng.choice([1.0, 4.0, 8.0]), fp8=fp8, fused=rng.random() < 0.5, padded=rng.randint(0, 5),
                    far=_log(rng, 16, 1000000))
    if op == "tree":
        seqs = _log(rng, 1, 96)
        hi = _log(rng, 16, max(16, 65536 // seqs))
        return dict(op=op, seqs=seqs, lo=rng.randint(0, hi // 2), hi=hi, long=0, far=0,
                    nodes=rng.choice([1, 3, 8, 17, 32, 61, 64, 100]), ragged=rng.random() < 0.7, hq=hq, hkv=hkv, d=d,
                    dtype=dtype)
    return dict(op=op, seqs=_log(rng, 1, 128), lo=0, hi=_log(rng, 16, 256), nodes=rng.randint(2, 100),
                most=rng.randint(1, 12), layers=_log(rng, 1, 32), hkv=hkv, d=d, dtype=dtype)


# --------------------------------------------------------------------------- inputs

def _seeds(case, seed):
    """A numpy generator for what the host lays out and a CUDA one for values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return np.random.default_rng([int(seed), 7]), g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[dtype])


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _trees(r, sizes, words):
    """Parents of random draft trees, and each node's ancestor mask and depth."""
    total = int(sizes.sum())
    parents = np.full(total, -1, np.int32)
    masks = np.zeros((total, words), np.uint64)
    depth = np.zeros(total, np.int32)
    pick = r.random(total)
    at = 0
    for n in sizes:
        for j in range(n):
            p = -1 if j == 0 else int(pick[at + j] ** 0.5 * (j + 1)) - 1   # later nodes are likelier parents
            parents[at + j] = p
            if p >= 0:
                masks[at + j] = masks[at + p]
                depth[at + j] = depth[at + p] + 1
            masks[at + j, j >> 6] |= np.uint64(1) << np.uint64(j & 63)
        at += int(n)
    return parents, masks.view(np.int64), depth


def _tables(r, lens, pool=None):
    """Shuffled pages for sequences of these lengths: [seqs, most pages] ids and the pool's size."""
    pages = (lens + BLOCK - 1) // BLOCK
    pool = int(math.ceil(1.25 * pages.sum())) + 1 if pool is None else pool
    ids = r.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(1, int(pages.max()))), ids[-1], np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool


def _nodes_of(case):
    """Nodes of the draft trees: up to ``nodes``, evenly spread where they are ragged."""
    seqs, most = case["seqs"], case["nodes"]
    return 1 + np.arange(seqs) * most // seqs if case.get("ragged", True) else np.full(seqs, most)


def _sizes(r, case):
    """Nodes of each sequence's tree and its length with them."""
    n = r.permutation(_nodes_of(case))
    lens = r.integers(case["lo"], case["hi"] + 1, case["seqs"])
    if case.get("long"):
        lens[r.permutation(case["seqs"])[:case["long"]]] = case["far"] - r.integers(0, 4000, case["long"])
    return n.astype(np.int64), (lens + n).astype(np.int64)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def prepare(case, seed):
    r, g = _seeds(case, seed)
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        t, hq, hkv, d, dt = (case[k] for k in ("tokens", "hq", "hkv", "d", "dtype"))
        qkv = _normal(g, (t, hq + 2 * hkv, d), dt)
        # fused: views of the projection's rows, as it wrote them; else tensors of their own
        s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], dim=1)
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
        s["positions"] = _dev(r.integers(0, case["far"], t).astype(np.int32))
        pool = (t + BLOCK - 1) // BLOCK * 5 // 4 + 1
        slots = r.permutation(pool * BLOCK)[:t].astype(np.int64)
        if case["padded"]:
            slots[-min(t, case["padded"]):] = -1
        s["slots"] = _dev(slots)
        # frequencies by the ramp that leaves fast pairs alone and stretches slow ones over a longer context
        rot, base, trained = case["rotary"], 500000.0, 8192
        f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
        turns = trained * f / (2 * math.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        s["inv_freq"] = _dev(f * keep + f / case["yarn"] * (1 - keep))
        s["factor"] = 0.1 * math.log(case["yarn"]) + 1.0
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.1 * _normal(g, (d,), dt) for _ in range(2))
        if case["fp8"]:
            s["k_scale"], s["v_scale"] = (0.01 + 0.02 * torch.rand(hkv, generator=g, device="cuda") for _ in range(2))
            s["kc"], s["vc"] = (torch.randint(0, 0x7f, (pool, hkv) + x, generator=g, device="cuda", dtype=torch.uint8)
                                for x in ((BLOCK, d), (d, BLOCK)))
        else:
            s["kc"], s["vc"] = (_normal(g, (pool, hkv, BLOCK, d), dt) for _ in range(2))
        return s
    if op == "plan":
        n = r.permutation(_nodes_of(case))
        s["parents"] = _dev(_trees(r, n, case["words"])[0])
        s["offsets"], s["lens"] = _dev(_offsets(n)), _dev((n + r.integers(0, case["far"], len(n))).astype(np.int32))
        return s
    n, lens = _sizes(r, case)
    # every layer's pool has room for the longest sequences: its size does not go by the lengths drawn
    room = case["seqs"] * ((case["hi"] + case["nodes"]) // BLOCK + 1) + 1 if op == "compact" else None
    table, pool = _tables(r, lens, room)
    s["offsets"], s["lens"], s["tables"] = _dev(_offsets(n)), _dev(lens.astype(np.int32)), _dev(table)
    s["most"], s["most_nodes"] = int(lens.max()), int(n.max())
    hkv, d, dt = case["hkv"], case["d"], case["dtype"]
    if op == "tree":
        s["masks"] = _dev(_trees(r, n, (case["nodes"] + 63) // 64)[1])
        s["q"] = _normal(g, (int(n.sum()), case["hq"], d), dt)
        s["kc"], s["vc"] = (_normal(g, (pool, hkv, BLOCK, d), dt) for _ in range(2))
        s["scale"] = 1 / math.sqrt(d)
        return s
    took = np.minimum(r.integers(0, case["most"] + 1, len(n)), n)
    acc = np.full((len(n), case["most"]), -1, np.int32)
    for b, k in enumerate(took):
        acc[b, :k] = np.sort(r.permutation(n[b])[:k])
    s["accepted"], s["took"] = _dev(acc), _dev(took.astype(np.int32))
    s["kc"], s["vc"] = (_normal(g, (case["layers"], pool, hkv, BLOCK, d), dt) for _ in range(2))
    return s


# --------------------------------------------------------------------------- plain forms

def _normed(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _e4m3(x, scale):
    """Codes of x / scale, [tokens, heads, d]."""
    return (x * (1 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_rope(s):
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    turn = functools.partial(_rotated, cos=cos, sin=sin, interleaved=s["case"]["interleaved"])
    q, k = turn(_normed(s["q"], s["q_norm"], 1e-6)), turn(_normed(s["k"], s["k_norm"], 1e-6))
    live = s["slots"] >= 0
    at = s["slots"][live]
    page, row = at // BLOCK, at % BLOCK
    k, v = k[live], s["v"][live]
    if s["case"]["fp8"]:
        s["kc"][page, :, row] = _e4m3(k, s["k_scale"])
        s["vc"][page, :, :, row] = _e4m3(v.float(), s["v_scale"])
    else:
        s["kc"][page, :, row] = k.to(s["kc"].dtype)
        s["vc"][page, :, row] = v
    return q.to(s["q"].dtype)


def _nodes(s):
    """Which sequence each drafted token belongs to, and its index in the tree."""
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    return n, b, torch.arange(len(b), device="cuda") - s["offsets"][b]


def _plain_plan(s):
    n, b, j = _nodes(s)
    words = s["case"]["words"]
    size = 64 * words
    reach = torch.eye(size, device="cuda").repeat(len(n), 1, 1)
    has = s["parents"] >= 0
    reach[b[has], j[has], s["parents"][has].long()] = 1
    # paths of up to 2^k steps, k = 1 .. 8
    reach = functools.reduce(lambda m, _: (m @ m).clamp(max=1), range(8), reach)[b, j] > 0
    bits = reach.view(-1, words, 64).long() << torch.arange(64, device="cuda")
    return bits.sum(-1), ((s["lens"].long() - n)[b] + reach.sum(-1) - 1).int()


def _plain_tree(s):
    """Split over parts of 512 keys, their maxima and sums joined by sequence."""
    part, c = 512, s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    n, b, j = _nodes(s)
    seqs, most = len(n), s["most_nodes"]
    q = torch.zeros(seqs, most, hq, d, device="cuda")
    q[b, j] = s["q"].float()
    q = q.view(seqs, most, hkv, hq // hkv, d).transpose(1, 2).reshape(seqs, hkv, -1, d)
    masks = torch.zeros(seqs, most, s["masks"].shape[1], dtype=torch.int64, device="cuda")
    masks[b, j] = s["masks"]
    lens = s["lens"].long()
    parts = (lens + part - 1) // part
    of = torch.repeat_interleave(torch.arange(seqs, device="cuda"), parts)
    first = (torch.arange(len(of), device="cuda") - (parts.cumsum(0) - parts)[of]) * part
    key = first[:, None] + torch.arange(part, device="cuda")
    there = key < lens[of][:, None]
    pages = s["tables"][of[:, None], (key[:, ::BLOCK] // BLOCK).clamp(max=s["tables"].shape[1] - 1)].long()
    k, v = (x[pages].transpose(1, 2).reshape(len(of), hkv, part, d).float() for x in (s["kc"], s["vc"]))
    v = torch.where(there[:, None, :, None], v, 0.0)
    node = key - (lens - n)[of][:, None]
    word = (node.clamp(min=0) >> 6).clamp(max=masks.shape[2] - 1)
    bit = torch.gather(masks[of], 2, word[:, None].expand(-1, most, -1)) >> (node & 63)[:, None]
    sees = there[:, None] & ((node < 0)[:, None] | ((bit & 1) == 1))
    sees = sees[:, None, :, None].expand(-1, hkv, -1, hq // hkv, -1).reshape(len(of), hkv, -1, part)
    x = (q[of] @ k.transpose(2, 3)) * s["scale"]
    x = torch.where(sees, x, -math.inf)
    top = torch.full(q.shape[:3], -math.inf, device="cuda").index_reduce_(0, of, x.amax(-1), "amax")
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top)[of][..., None])
    total = torch.zeros(q.shape[:3], device="cuda").index_add_(0, of, p.sum(-1))
    out = torch.zeros(q.shape, device="cuda").index_add_(0, of, p @ v)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    out = out.view(seqs, hkv, most, hq // hkv, d).transpose(1, 2).reshape(seqs, most, hq, d)
    return out[b, j].to(s["q"].dtype)


def _plain_compact(s):
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    lens, acc = s["lens"].long(), s["accepted"].long()
    j = torch.arange(acc.shape[1], device="cuda")
    b, j = torch.nonzero(j < s["took"][:, None], as_tuple=True)
    src, dst = (lens - n)[b] + acc[b, j], (lens - n)[b] + j
    sp, dp = s["tables"][b, src // BLOCK].long(), s["tables"][b, dst // BLOCK].long()
    for c in (s["kc"], s["vc"]):
        c[:, dp, :, dst % BLOCK] = c[:, sp, :, src % BLOCK]
    return (lens - n + s["took"]).int()


# --------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "rope":
        return _rope_outputs(s, _plain_rope(s))
    if op == "plan":
        return _plain_plan(s)
    if op == "tree":
        return _plain_tree(s)
    return _bits(s["kc"]), _bits(s["vc"]), _plain_compact(s)


def _bits(c):
    """A cache whose rows are only ever copied: its bits."""
    return c.view(torch.int16)


def _rope_outputs(s, q):
    if s["case"]["fp8"]:
        return q, s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn)
    return q, s["kc"], _bits(s["vc"])


def _own(s, op):
    from paged_kv_cache_blocks_gb300 import binding as pa
    if op == "rope":
        c = s["case"]
        kw = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, interleaved=c["interleaved"],
                  attn_factor=s["factor"])
        if c["fp8"]:
            q = pa.pa_rope_cache_write_fp8(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                                           s["k_scale"], s["v_scale"], s["kc"], s["vc"], **kw)
        else:
            q = pa.pa_rope_cache_write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                                       s["kc"], s["vc"], **kw)
        return _rope_outputs(s, q)
    if op == "plan":
        return pa.pa_tree_plan(s["parents"], s["offsets"], s["lens"], mask_words=s["case"]["words"])
    if op == "tree":
        if "workspace" not in s:   # kept between steps, as a serving loop does
            c = s["case"]
            need = pa.pa_decode_tree_workspace_bytes(c["seqs"], s["q"].shape[0], c["hq"], c["hkv"], c["d"], s["most"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return pa.pa_decode_tree(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["offsets"], s["masks"],
                                 s["scale"], max_seq_len=s["most"], workspace=s["workspace"])
    lens = pa.pa_cache_compact(s["kc"], s["vc"], s["tables"], s["lens"], s["offsets"], s["accepted"], s["took"])
    return _bits(s["kc"]), _bits(s["vc"]), lens


# --------------------------------------------------------------------------- what a pass cannot do without

def _expected(case):
    """Expected context tokens and drafted tokens of all sequences."""
    seqs = case["seqs"]
    nodes = int(_nodes_of(case).sum())
    long = case.get("long", 0)
    return (seqs - long) * (case["lo"] + case["hi"]) / 2 + long * (case.get("far", 0) - 2000), nodes


def work(case):
    op = case["op"]
    if op == "plan":
        nodes = int(_nodes_of(case).sum())
        return {"bytes": nodes * (4 + 8 * case["words"] + 4) + 8 * case["seqs"], "flops": 0}
    row = case["d"] * 2
    if op == "rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        live = t - min(t, case["padded"])
        cached = 2 * hkv * (case["d"] if case["fp8"] else row)
        # q, k and v in, q out, cached rows out, position and slot of each token
        return {"bytes": t * (2 * hq * row + 12) + live * (2 * hkv * row + cached) + 4 * case["rotary"],
                "flops": t * (hq + hkv) * (3 * case["rotary"] + (4 * case["d"] if case["norm"] else 0))}
    ctx, nodes = _expected(case)
    if op == "tree":
        words = (case["nodes"] + 63) // 64
        per = nodes / case["seqs"]
        long = case["long"] * (case["far"] - 2000) * per
        pairs = (ctx - case["long"] * (case["far"] - 2000)) * per + long + nodes * math.log2(per + 1)
        return {"bytes": (ctx + nodes) * (2 * case["hkv"] * row + 4 / BLOCK) + nodes * (2 * case["hq"] * row + 8 * words),
                "flops": 4 * case["d"] * case["hq"] * pairs}
    # about half of the accepted tokens that can move do, read once and written once in K and in V
    took = min(case["most"] / 2, nodes / case["seqs"])
    return {"bytes": case["seqs"] * (took * (4 * case["layers"] * case["hkv"] * row + 4) + 12), "flops": 0}


# --------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_tree(s) if case["op"] == "tree" else None


def _exact_rope(s):
    c = s["case"]
    rot, pos = c["rotary"], s["positions"].double()

    def place(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6) * w.double()
        z = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            ang = (pos * s["inv_freq"][i])[:, None]
            z[..., a] = s["factor"] * (y[..., a] * torch.cos(ang) - y[..., b] * torch.sin(ang))
            z[..., b] = s["factor"] * (y[..., b] * torch.cos(ang) + y[..., a] * torch.sin(ang))
        return z

    q, k = place(s["q"], s["q_norm"]), place(s["k"], s["k_norm"])
    ok = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, row = s["slots"][ok] // BLOCK, s["slots"][ok] % BLOCK
    if not c["fp8"]:
        kc = s["kc"].double()
        kc[page, :, row] = k[ok]
        return q, kc, None

    def code(x, scale):
        # the nearest E4M3 value: 3 bits after the leading one, exponents from -6, at most 448
        x = (x / scale.double()[:, None])[ok]
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-448, 448)

    kc, vc = s["kc"].view(torch.float8_e4m3fn).double(), s["vc"].view(torch.float8_e4m3fn).double()
    kc[page, :, row] = code(k, s["k_scale"])
    vc[page, :, :, row] = code(s["v"].double(), s["v_scale"])
    return q, kc, vc


def _exact_tree(s):
    c = s["case"]
    offsets, lens, tables = (s[k].cpu().numpy() for k in ("offsets", "lens", "tables"))
    g, out = c["hq"] // c["hkv"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        lo, hi, size = int(offsets[b]), int(offsets[b + 1]), int(lens[b])
        page = torch.from_numpy(tables[b, :(size + BLOCK - 1) // BLOCK].astype(np.int64)).cuda()
        words = s["masks"][lo:hi].cpu().numpy().view(np.uint8)
        drafted = np.unpackbits(words, axis=1, bitorder="little")[:, :hi - lo].astype(bool)
        sees = torch.ones(hi - lo, size, dtype=torch.bool)
        sees[:, size - (hi - lo):] = torch.from_numpy(drafted)
        hidden = ~sees.cuda()[:, None]
        for h in range(c["hkv"]):
            k, v = (x[page, h].reshape(-1, c["d"])[:size].double() for x in (s["kc"], s["vc"]))
            q = s["q"][lo:hi, h * g:(h + 1) * g].double()
            x = (q @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
            out[lo:hi, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
    return out
