"""pa_cache_compact against its definition, byte for byte, and a whole
speculative step: plan, rotate and write, tree attention, compaction,
truncation, against the same tokens decoded without drafts."""
import numpy as np
import pytest
import torch

import draft_reference as ref
from gpu_util import TORCH_DT, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    return require_gpu()


def dev(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(dt))).cuda()


def make(seed, befores, sizes, took, layers, hkv, D, dt, most=None):
    r = np.random.default_rng(seed)
    lens = np.array(befores) + np.array(sizes)
    pages = -(-lens // 16)
    pool = int(pages.sum()) + 2
    ids = r.permutation(pool)
    table = np.full((len(lens), int(pages.max()) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    most = most or max(max(took), 1)
    acc = np.full((len(lens), most), -1, np.int32)
    for b, k in enumerate(took):
        acc[b, :k] = np.sort(r.permutation(sizes[b])[:k])
    c = [r.integers(-2 ** 15, 2 ** 15, (layers, pool, hkv, 16, D)).astype(np.int16) for _ in range(2)]
    off = np.concatenate([[0], np.cumsum(sizes)])
    return c, table, lens, off, acc, np.array(took)


def on_device(c, dt):
    return [torch.from_numpy(x.copy()).cuda().view(TORCH_DT[dt]) for x in c]


@pytest.mark.parametrize("layers,hkv,D,dt", [(1, 2, 64, "f16"), (3, 8, 128, "bf16"), (5, 3, 64, "bf16"), (130, 1, 64, "f16")])
@pytest.mark.parametrize("befores,sizes,took", [([0], [1], [1]), ([0, 5, 31], [8, 3, 17], [0, 3, 9]),
                                                ([14, 15, 16, 100], [40, 2, 1, 0], [40, 1, 1, 0]),
                                                ([7, 250], [100, 256], [31, 200])])
def test_matches_definition(pa, layers, hkv, D, dt, befores, sizes, took):
    c, table, lens, off, acc, num = make(layers + len(took), befores, sizes, took, layers, hkv, D, dt)
    k, v = on_device(c, dt)
    err = torch.zeros(1, dtype=torch.int32).cuda()
    new = pa.pa_cache_compact(k, v, dev(table), dev(lens), dev(off), dev(acc), dev(num), error_bits=err)
    want, want_lens = ref.compact(c, table, lens, off, acc, num)
    assert np.array_equal(k.view(torch.int16).cpu().numpy(), want[0])
    assert np.array_equal(v.view(torch.int16).cpu().numpy(), want[1])
    assert np.array_equal(new.cpu().numpy(), want_lens) and err.item() == 0
    k2, v2 = on_device(c, dt)                                  # the layers as tensors of their own
    pa.pa_cache_compact(list(k2), list(v2), dev(table), dev(lens), dev(off), dev(acc), dev(num))
    assert torch.equal(k2.view(torch.int16), k.view(torch.int16)) and torch.equal(v2.view(torch.int16), v.view(torch.int16))


def test_bad_lists_are_cut_and_flagged(pa):
    c, table, lens, off, acc, num = make(1, [20, 33, 4, 50], [9, 9, 9, 9], [5, 5, 5, 5], 2, 2, 64, "f16")
    acc[0] = [1, 4, 4, 6, 7]       # twice the same: ends after two
    acc[1] = [0, 3, 9, 1, 2]       # past the tree: ends after two
    acc[2] = [-1, 1, 2, 3, 4]      # negative: nothing
    num[3] = 6                     # more than the array holds: five
    k, v = on_device(c, "f16")
    err = torch.zeros(1, dtype=torch.int32).cuda()
    new = pa.pa_cache_compact(k, v, dev(table), dev(lens), dev(off), dev(acc), dev(num), error_bits=err)
    want, want_lens = ref.compact(c, table, lens, off, acc, np.array([2, 2, 0, 5]))
    assert np.array_equal(k.view(torch.int16).cpu().numpy(), want[0])
    assert np.array_equal(v.view(torch.int16).cpu().numpy(), want[1])
    assert np.array_equal(new.cpu().numpy(), want_lens) and err.item() == pa.PA_DEVERR_TREE
    # lengths and offsets that do not fit: nothing of those sequences moves
    c, table, lens, off, acc, num = make(2, [20, 33], [9, 9], [5, 5], 1, 2, 64, "f16")
    for bad_len, bad_off in (([10 ** 6, lens[1]], off), ([-4, lens[1]], off), ([3, lens[1]], off), (lens, [9, 0, 9]),
                             (lens, [-3, 9, 18])):
        k, v = on_device(c, "f16")
        err.zero_()
        new = pa.pa_cache_compact(k, v, dev(table), dev(bad_len), dev(bad_off), dev(acc), dev(num), error_bits=err)
        assert err.item() & pa.PA_DEVERR_SEQ_LEN
        pages = table[0][table[0] >= 0]                        # the first sequence's
        assert np.array_equal(k.view(torch.int16).cpu().numpy()[:, pages], c[0][:, pages])
        assert new[0].item() == max(0, bad_len[0])
    # pages outside the pool: those rows stay
    c, table, lens, off, acc, num = make(3, [20], [20], [5], 1, 2, 64, "f16")
    table[0, 1] = c[0].shape[1]
    k, v = on_device(c, "f16")
    err.zero_()
    pa.pa_cache_compact(k, v, dev(table), dev(lens), dev(off), dev(acc), dev(num), error_bits=err)
    assert err.item() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(k.view(torch.int16).cpu().numpy(), c[0])


def test_captured(pa):
    c, table, lens, off, acc, num = make(5, [20, 33], [9, 9], [5, 4], 2, 2, 128, "bf16")
    k, v = on_device(c, "bf16")
    a = [dev(x) for x in (table, lens, off, acc, num)]
    new, graph = torch.empty_like(a[1]), torch.cuda.CUDAGraph()
    k0, v0 = k.clone(), v.clone()
    with torch.cuda.graph(graph):
        pa.pa_cache_compact(k, v, *a, new_seq_lens=new)
    for took in ([5, 4], [2, 0]):
        k.copy_(k0), v.copy_(v0), a[4].copy_(dev(took))
        graph.replay()
        torch.cuda.synchronize()
        want, want_lens = ref.compact(c, table, lens, off, acc, took)
        assert np.array_equal(k.view(torch.int16).cpu().numpy(), want[0])
        assert np.array_equal(new.cpu().numpy(), want_lens)


def test_binding_refuses(pa):
    c, table, lens, off, acc, num = make(6, [20], [9], [5], 2, 2, 64, "f16")
    k, v = on_device(c, "f16")
    a = dict(k_caches=k, v_caches=v, block_tables=dev(table), seq_lens=dev(lens), q_offsets=dev(off), accepted=dev(acc),
             num_accepted=dev(num))
    for kw in (dict(accepted=dev(acc, np.int64)), dict(v_caches=v[:1]), dict(k_caches=[]), dict(k_caches=k.float()),
               dict(num_accepted=dev([1, 2]))):
        with pytest.raises((TypeError, ValueError)):
            pa.pa_cache_compact(**(a | kw))
    with pytest.raises(pa.PaError):
        pa.pa_cache_compact(**a, new_seq_lens=a["seq_lens"])


@pytest.mark.parametrize("hq,hkv,D,dt", [(8, 2, 64, "f16"), (16, 2, 128, "bf16")])
def test_speculative_steps_as_they_would_be_used(pa, hq, hkv, D, dt):
    """Three steps of drafting over two layers.  After each, the caches hold what writing the accepted tokens one by
    one would have left, bit for bit, and the allocator's tables agree."""
    r = np.random.default_rng(hq)
    g = torch.Generator().manual_seed(hq)
    layers, seqs, pool = 2, 3, 64
    alloc = pa.Allocator(pool, r.permutation(pool))
    ids = [alloc.seq_create() for _ in range(seqs)]
    shape = (layers, pool, hkv, 16, D)
    kc, vc = (torch.zeros(shape, dtype=TORCH_DT[dt], device="cuda") for _ in range(2))
    f, factor = pa.pa_rope_frequencies(D, 10000.0, "ramp", factor=4.0, trained_tokens=64)
    lens = [3, 40, 17]
    said = [[] for _ in range(seqs)]                           # (k, v) rows per layer of each kept token
    rows = lambda n: [torch.randn(n, hkv, D, generator=g).to(TORCH_DT[dt]).cuda() for _ in range(2)]

    def write(layer, q, k, v, pos, slots):
        return pa.pa_rope_cache_write(q, k, v, pos, slots, f, kc[layer], vc[layer], attn_factor=factor)

    for b, n in enumerate(lens):                               # the prompts
        slots, _ = alloc.append_slots([ids[b]], n)
        kv = [rows(n) for _ in range(layers)]
        for l in range(layers):
            write(l, torch.zeros(n, hq, D, dtype=TORCH_DT[dt], device="cuda"), *kv[l],
                  torch.arange(n, dtype=torch.int32).cuda(), torch.tensor(slots).cuda())
        said[b] = [[(k[t], v[t]) for k, v in kv] for t in range(n)]
    for step in range(3):
        size = [5, 19, 1]
        parents = np.concatenate([[int(r.integers(-1, j)) for j in range(n)] for n in size])
        slots = []
        for b in range(seqs):
            slots += alloc.append_slots([ids[b]], size[b])[0]
        tab, ln = alloc.block_table(ids, 8)
        off = np.concatenate([[0], np.cumsum(size)])
        dt_, dl, do = dev(tab), dev(ln), dev(off)
        masks, pos = pa.pa_tree_plan(dev(parents), do, dl)
        kv = [rows(sum(size)) for _ in range(layers)]
        q = torch.randn(sum(size), hq, D, generator=g).to(TORCH_DT[dt]).cuda()
        for l in range(layers):
            qr = write(l, q, *kv[l], pos, torch.tensor(slots).cuda())
            out = pa.pa_decode_tree(qr, kc[l], vc[l], dt_, dl, do, masks, 1 / np.sqrt(D))
            n64 = lambda t: t.double().cpu().numpy()
            want, _, _ = ref.tree_attention(n64(qr), n64(kc[l]), n64(vc[l]), np.array(tab), np.array(ln), off,
                                            ref.tree_masks(parents, size, 1)[0], 1 / np.sqrt(D))
            assert np.abs(n64(out) - want).max() <= 2e-2       # outputs to |out| of about 4; the tight bound has its own test
        took, acc = [], np.full((seqs, 20), -1)
        for b in range(seqs):                                  # a path from a root down to some token
            path, j = [], int(r.integers(-1, size[b]))
            while j >= 0:
                path, j = [j] + path, parents[off[b] + j]
            acc[b, :len(path)] = path
            took.append(len(path))
            said[b] += [[(kv[l][0][off[b] + j], kv[l][1][off[b] + j]) for l in range(layers)] for j in path]
        new = pa.pa_cache_compact(kc, vc, dt_, dl, do, dev(acc), dev(took))
        for b in range(seqs):
            lens[b] += took[b]
            alloc.seq_truncate(ids[b], lens[b])
        assert new.tolist() == lens == alloc.block_table(ids, 8)[1]
    plain_k, plain_v = torch.zeros_like(kc), torch.zeros_like(vc)
    tab, _ = alloc.block_table(ids, 8)
    for b in range(seqs):
        n = lens[b]
        slots = torch.tensor([tab[b][t // 16] * 16 + t % 16 for t in range(n)]).cuda()
        for l in range(layers):
            k, v = (torch.stack([said[b][t][l][i] for t in range(n)]) for i in range(2))
            pa.pa_rope_cache_write(torch.zeros(n, hq, D, dtype=TORCH_DT[dt], device="cuda"), k, v,
                                   torch.arange(n, dtype=torch.int32).cuda(), slots, f, plain_k[l], plain_v[l],
                                   attn_factor=factor)
        for t in range(n):
            at = (slice(None), tab[b][t // 16], slice(None), t % 16)
            assert torch.equal(kc[at], plain_k[at]) and torch.equal(vc[at], plain_v[at])


def test_layers_in_any_order_and_interleaved(pa):
    """K and V of a layer beside each other in one buffer, and the layers named last to first."""
    c, table, lens, off, acc, num = make(8, [20, 33], [9, 9], [5, 4], 3, 2, 64, "f16")
    both = torch.from_numpy(np.stack(c, 1)).cuda().view(torch.float16)      # [layers, K / V, ...]
    want, _ = ref.compact(c, table, lens, off, acc, num)
    a = [dev(x) for x in (table, lens, off, acc, num)]
    for order in ([0, 1, 2], [2, 0, 1]):
        x = both.clone()
        pa.pa_cache_compact([x[i, 0] for i in order], [x[i, 1] for i in order], *a)
        assert np.array_equal(x.view(torch.int16).cpu().numpy(), np.stack(want, 1))
    with pytest.raises(pa.PaError):
        pa.pa_cache_compact([both[0, 0], both[0, 0]], [both[0, 1], both[1, 1]], *a)


def test_pages_past_4_gib(pa):
    """The moved rows in the last pages of pools of 5 GiB."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of device memory")
    c, table, lens, off, acc, num = make(9, [20, 33], [9, 30], [5, 12], 1, 8, 128, "bf16")
    want, want_lens = ref.compact(c, table, lens, off, acc, num)
    far = (5 << 30) // (8 * 16 * 128 * 2)
    pool = c[0].shape[1]
    big = [torch.zeros(1, far + pool, 8, 16, 128, dtype=torch.int16, device="cuda") for _ in range(2)]
    for x, y in zip(big, c):
        x[:, far:] = torch.from_numpy(y).cuda()
    new = pa.pa_cache_compact(*big, dev(np.where(table < 0, table, table + far)), dev(lens), dev(off), dev(acc), dev(num))
    assert np.array_equal(new.cpu().numpy(), want_lens)
    for x, y in zip(big, want):
        assert np.array_equal(x[:, far:].cpu().numpy(), y) and not x[:, :far].any()
