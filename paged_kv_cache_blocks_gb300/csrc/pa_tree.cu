// Draft trees over paged K/V for sm_103a: the plan of a tree (ancestor masks
// and positions), attention of its tokens, and the merge of split sequences.
//
// A sequence of L tokens holds a tree of n drafted tokens as its last n; tree
// token j attends to the L - n tokens before the tree and to the tree tokens
// of its mask (its ancestors and itself):
//   out[j, i] = sum_t softmax_t(scale * q[j, i] . K[t, i / G]) V[t, i / G],
//   t < L - n, or bit t - (L - n) of mask_j set.
//
// Three kernels per attention call, on the caller's stream:
//   1. tree_prep  (1 CTA)  validates the sequences, chooses how many chunks of
//                          128 keys a work item covers, and lists the items of
//                          every (sequence, key range, tile of 128 query
//                          rows), largest first;
//   2. rows_tc             the tcgen05 attention kernel (pa_rows_tc.cuh), one
//                          persistent CTA per SM, items from an atomic counter;
//   3. tree_merge          joins the key ranges of split sequences, four output
//                          rows a warp.
// Trees of a few dozen rows read each page once and the pages bound them; from
// two tiles on (more than 128 rows a KV head) the products do, and the tiles of
// a key range run together so that the second reads it from L2.  Measured on
// one GB300 (us a call, graph replay; MB of pages; share of the measured copy
// rate or of the burst bf16 rate):
//   4 short chats, trees of 5, head_dim 64                     10.8
//   64 sequences of 128-2048 tokens, trees of 1-32, 32/8 heads 64    307 MB  0.71
//   256 sequences, a tenth of 34,000 tokens, trees of 1-8      548   3781 MB 1.02
//   8 x 32,768 tokens, trees of 64 (256 rows)                  228   1084 MB, 275 GFLOP 0.63
// The second spends 4 us in the plan, 4 before its first scores, 47 streaming
// pages (7 TB/s) and up to 6 in CTAs whose last items are short; the last's
// pace is that of the kernel's softmax (0.9 us per 128 x 128 scores an SM).
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows_tc.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// The plan of a tree.

// One CTA per sequence, one thread per tree token.  The mask of a token is its
// own bit and its parent's mask; with anc_k(j) the token 2^k steps above j,
//   M_{k+1}(j) = M_k(j) | M_k(anc_k(j)),  depth likewise,
// so 8 rounds reach every ancestor of a tree of 256, however deep, and the
// rounds end when every token is past its root.  Latency bounds it: offsets
// and length, then the parents, then the rounds in shared memory.
template <int W>
__global__ void __launch_bounds__(64 * W)
    tree_plan_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ q_off,
                     const int32_t* __restrict__ seq_lens, int num_q_tokens, int64_t* __restrict__ masks,
                     int32_t* __restrict__ positions, int32_t* __restrict__ error_bits) {
  __shared__ uint64_t s_mask[2][64 * W][W];
  __shared__ int s_anc[2][64 * W], s_depth[2][64 * W];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, j = threadIdx.x;
  const int a0 = q_off[b], e0 = q_off[b + 1], L = seq_lens[b];
  const int a = min(max(a0, 0), num_q_tokens), e = min(max(e0, a), num_q_tokens), n = e - a;
  int bad = 0;
  if (a != a0 || e != e0 || n > 64 * W || n > L) bad = kErrSeqLen;
  const int before = max(L - n, 0);
  int anc = -1, depth = 0;
  uint64_t m[W];
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = (j >> 6) == w ? 1ull << (j & 63) : 0ull;
  if (j < n) {
    anc = parents[a + j];
    if (anc < -1 || anc >= j) {   // not a token before this one: taken as a root
      bad |= kErrTree;
      anc = -1;
    }
    depth = anc >= 0 ? 1 : 0;
  }
  if (bad && error_bits) atomicOr(error_bits, bad);
  int buf = 0;
  while (true) {
#pragma unroll
    for (int w = 0; w < W; ++w) s_mask[buf][j][w] = m[w];
    s_anc[buf][j] = anc;
    s_depth[buf][j] = depth;
    if (!__syncthreads_or(anc >= 0)) break;
    if (anc >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) m[w] |= s_mask[buf][anc][w];
      depth += s_depth[buf][anc];
      anc = s_anc[buf][anc];
    }
    buf ^= 1;   // the next round's values go beside the ones still being read
  }
  if (j < n) {
#pragma unroll
    for (int w = 0; w < W; ++w) masks[(static_cast<int64_t>(a) + j) * W + w] = static_cast<int64_t>(m[w]);
    positions[a + j] = before + depth;
  }
  for (int t = 64 * W + j; t < n; t += 64 * W) {   // past the masks' reach (flagged): sees no tree token
#pragma unroll
    for (int w = 0; w < W; ++w) masks[(static_cast<int64_t>(a) + t) * W + w] = 0;
    positions[a + t] = before;
  }
}

int tree_plan_launch(const int32_t* parents, const int32_t* q_offsets, const int32_t* seq_lens,
                     int32_t num_seqs, int32_t num_q_tokens, int32_t mask_words, int64_t* masks,
                     int32_t* positions, int32_t* error_bits, void* stream, std::string* why) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(num_seqs)), block(64 * mask_words);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, block, 0, s, parents, q_offsets, seq_lens, static_cast<int>(num_q_tokens),
                      masks, positions, error_bits);
  };
  cudaError_t e = mask_words == 1   ? go(tree_plan_kernel<1>)
                  : mask_words == 2 ? go(tree_plan_kernel<2>)
                  : mask_words == 3 ? go(tree_plan_kernel<3>)
                                    : go(tree_plan_kernel<4>);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("tree plan launch: ") + cudaGetErrorString(e);
    return 5;
  }
  return 0;
}

// ---------------------------------------------------------------------------
// Work items of the attention.

namespace {

constexpr int kChunkKeys = 128;
constexpr int kPlanSeqs = 1024;      // sequences planned at a time, one per thread
constexpr int kTreeBins = 32;        // sizes of items, for the largest-first order; a lane each
// An item covers at least 1 / kMaxShares of the work, so that at most
// kMaxShares of them come from dividing it and as many again from rounding up.
constexpr int kMaxShares = 912;      // 6 x 152 SMs
constexpr int kMaxSlots = 2 * kMaxShares;

// Header words of the merge (in PrefillHeader::pad): split sequences, their
// (tile, KV head) pairs, most parts of one.
constexpr int kPadUnits = 0, kPadPairs = 1, kPadParts = 2;

struct TreeLayout {
  size_t off_entries, off_units, off_ml, off_acc, total;
  int64_t max_entries, max_units, max_slots;
};

TreeLayout tree_layout(int64_t num_seqs, int64_t num_q_tokens, int64_t hq, int64_t hkv, int64_t D,
                       int64_t max_seq_len) {
  const int64_t tile_tokens = 128 / (hq / hkv);
  const int64_t tiles = num_q_tokens / tile_tokens + num_seqs;
  const int64_t chunks = (max_seq_len + kChunkKeys - 1) / kChunkKeys;
  TreeLayout L;
  L.max_units = num_seqs < kMaxShares ? num_seqs : kMaxShares;
  // one slot per item of a split sequence: bounded by the shares, and by
  // every chunk of every tile being an item of its own
  L.max_slots = chunks <= 1 ? 0 : kMaxSlots;
  if (chunks * tiles * hkv < L.max_slots) L.max_slots = chunks * tiles * hkv;
  L.max_entries = tiles + L.max_slots;
  size_t o = sizeof(PrefillHeader);
  L.off_entries = o;  o = align_up(o + 2 * sizeof(int4) * L.max_entries, 256);
  L.off_units = o;    o = align_up(o + sizeof(int4) * L.max_units, 256);
  L.off_ml = o;       o = align_up(o + sizeof(float2) * 128 * L.max_slots, 256);
  L.off_acc = o;      o = align_up(o + sizeof(float) * 128 * D * L.max_slots, 256);
  L.total = o;
  return L;
}

}  // namespace

// A split sequence: the slot of (part p, tile t, KV head h) is
// slot0 + (p * tiles + t) * hkv + h.  first: (tile, head) pairs of the units
// before it; q0, rows: its query tokens.  Packed, so that the merge fetches
// all of them beside its header: first, tiles and parts in 10, 5 and 11 bits,
// slot0 and rows in 11 and 9.
struct TreeUnit {
  int first, tiles, parts, slot0, rows, q0;
  __device__ __forceinline__ int4 pack() const {
    return make_int4(first | tiles << 10 | parts << 15, slot0 | max(rows, 0) << 11, q0, 0);
  }
  __device__ __forceinline__ static TreeUnit unpack(int4 x) {
    return TreeUnit{x.x & 1023, x.x >> 10 & 31, x.x >> 15 & 2047, x.y & 2047, x.y >> 11, x.z};
  }
};
static_assert(kMaxSlots < 2048 && kMaxShares < 1024, "bits of a unit's record");

struct TreePrepArgs {
  TreeParams P;
  int max_units, max_slots, sms, grid;   // grid: CTAs of the attention
  float page_cost;                       // of a chunk of one head's pages, all SMs loading
};

// What the plan needs of a sequence: its query tokens (those within the masks'
// reach), tokens, tiles of query rows and chunks of keys.
struct TreeSeq {
  int q0, n, rows, L, tiles, chunks;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& P, int b, bool flag) {
  const PieceView v = piece_view(P, b, flag);
  if (flag && v.n > 64 * P.mask_words) atomicOr(&P.ws->error_bits, kErrSeqLen);
  const int rows = min(v.n, 64 * P.mask_words);
  return TreeSeq{v.q0, v.n, rows, v.L, (rows + P.tile_tokens - 1) / P.tile_tokens, (v.L + kChunkKeys - 1) / kChunkKeys};
}

// ceil(a / b) for -b < a <= 2^24 and b > 0: the quotient in fp32, put right by
// its remainder (a step at most below 2^22).
__device__ __forceinline__ int cdiv(int a, int b) {
  const int n = a + b - 1;
  int q = static_cast<int>(__fdividef(static_cast<float>(n), static_cast<float>(b)));
  int r = n - q * b;
  for (; r < 0; r += b) --q;
  for (; r >= b; r -= b) ++q;
  return q;
}

__device__ __forceinline__ unsigned long long cdiv64(unsigned long long a, unsigned b) {
  const unsigned long long n = a + b - 1;   // 64-bit division takes about half a microsecond
  return n >> 32 ? n / b : static_cast<unsigned>(n) / b;
}

// Work items of the call: how many chunks of keys each covers, and the list.
//
// Cost of a size, in the time an SM's products and softmax of a chunk take (0.9
// us): the work, mu a chunk where the pages' bytes bound it (the share of the
// SMs that keep them flowing: mu = 1.55 for one tile of rows at head_dim 128,
// down to 1), an item's own time (its Q, its rows written out: 3, half of it
// hidden behind the pages), one per slot (a state is written and read back,
// mostly in L2), spread over the SMs; or the waves of its large items where
// these do not fill the SMs evenly (a last wave on few SMs has the pages'
// bandwidth to itself); 5.5 for a merge at all.  Candidates, a warp each:
//   0     unsplit;
//   1     each SM's share of the work, cut along all sequences' chunks laid end
//         to end: a sequence's last part and the next one's first make up a
//         share together, so the items taken largest first fill the SMs with
//         the fewest of them;
//   2..7  equal parts of at most 1 to 1/6 of an SM's share.
// us a call with the choice forced, and the rule's (one GB300):
//                                              0     1    2, 3, 7          rule
//   1 x 8,000 tokens, 256 rows of 32 / 8 heads 65.4  25.7  25.8  29.2  36.5  26.2
//   8 x 8,000, 512 rows of 64 / 8              127   125   127   146   149   125
//   64 x 128-2,048, up to 128 rows             63.7  67.1  63.5  63.7  84.1  64.1
//   256 x (400 or 34,000), up to 64 rows       574   575   574   547   559   548
//   8 x 32,768, 256 rows                       246   228   255   262   251   229
constexpr int kItemCost = 3;
constexpr int kCands = 8;

__global__ void __launch_bounds__(kPlanSeqs) tree_prep_kernel(const TreePrepArgs A) {
  const TreeParams& P = A.P;
  __shared__ int sw[32];
  __shared__ int s_hist[kTreeBins], s_next[kTreeBins];   // records of a size, and those placed
  __shared__ int2 s_seq[kPlanSeqs];   // tiles, chunks of the first sequences
  __shared__ unsigned long long s_work;
  __shared__ int s_most, s_sizes[kCands], s_parts;
  __shared__ float s_cost[kCands];
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_work = 0;
    s_most = 0;
    s_parts = 1;
  }
  if (tid < kTreeBins) s_hist[tid] = s_next[tid] = 0;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) P.ws->error_bits = 0;
  __syncthreads();
  // one sequence per thread is kept in registers; past them they are read again
  TreeSeq mine = {};
  unsigned long long work = 0;
  int most = 0;
  for (int b = tid; b < P.num_seqs; b += nthr) {
    const TreeSeq z = tree_seq(P, b, true);
    if (b == tid) mine = z;
    if (b < kPlanSeqs) s_seq[b] = make_int2(z.tiles, z.chunks);
    work += static_cast<unsigned long long>(z.tiles) * z.chunks * P.hkv;
    if (z.tiles > 0) most = max(most, z.chunks);
  }
  auto seq = [&](int b) { return b == tid ? mine : tree_seq(P, b, false); };
  // A warp that has not come together again after a branch or a loop takes
  // shuffles one by one, at about 250 cycles each: every group of them is
  // preceded by a __syncwarp().
  __syncwarp();
#pragma unroll
  for (int o = 16; o; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    atomicAdd(&s_work, work);
    atomicMax(&s_most, most);
  }
  __syncthreads();
  if (warp < kCands) {
    const unsigned long long least = cdiv64(s_work, kMaxShares);
    const unsigned long long c = warp == 0 ? s_most : cdiv64(s_work, static_cast<unsigned>(A.sms) * max(1, warp - 1));
    // a share may be longer than any sequence (their chunks are at most 2^24)
    const unsigned long long longest = warp == 1 ? 1ull << 24 : static_cast<unsigned long long>(s_most);
    const int size = static_cast<int>(max(1ull, max(least, min(c, longest))));
    // sums in fp32: they only weigh the candidates
    const float inv = 1.f / size, half = 0.5f * min(size, s_most);
    float pairs = 0.f, pages = 0.f;   // (tile, head) pairs; chunks of a head's pages
    float items = 0.f, slots = 0.f, large = 0.f, chunks = 0.f;
    for (int b = lane; b < P.num_seqs; b += 32) {
      int2 z;
      if (b < kPlanSeqs) {
        z = s_seq[b];
      } else {
        const TreeSeq t = tree_seq(P, b, false);
        z = make_int2(t.tiles, t.chunks);
      }
      const float np = static_cast<float>(z.x) * P.hkv, parts = fmaxf(1.f, ceilf(z.y * inv)), n = np * parts;
      pairs += np;
      pages += z.x > 0 ? static_cast<float>(z.y) * P.hkv : 0.f;
      items += n;
      if (parts > 1.f) slots += n;
      if (z.y >= parts * half) {   // items of half the size at least, as a split sequence's are
        large += n;
        chunks += np * z.y;
      }
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
      pages += __shfl_xor_sync(0xffffffffu, pages, o);
      items += __shfl_xor_sync(0xffffffffu, items, o);
      slots += __shfl_xor_sync(0xffffffffu, slots, o);
      large += __shfl_xor_sync(0xffffffffu, large, o);
      chunks += __shfl_xor_sync(0xffffffffu, chunks, o);
    }
    const float work_f = static_cast<float>(s_work), sms = A.sms;
    const float mu = fmaxf(1.f, A.page_cost * pages / fmaxf(work_f, 1.f));
    const float item = fmaxf(0.5f * kItemCost, kItemCost - 2.7f * (mu - 1.f));
    float cost;
    if (warp == 1) {
      const float cuts = work_f * inv;
      const float even = (mu * work_f + item * (pairs + cuts) + fminf(2.f * cuts, cuts + pairs)) / sms;
      cost = fmaxf(even, mu * size + 2.f * item) + 5.5f;
      // its cuts fall where they may: only where the slots hold any of them, and
      // the chunks of all sequences, which it counts through, fit 32 bits
      if (cuts + 3.f * pairs > kMaxSlots - 1 || P.num_seqs > nthr || s_work > 1ull << 30) cost = 3e38f;
    } else {
      const float each = chunks / fmaxf(large, 1.f), full = fmaxf(ceilf(large / sms) - 1.f, 0.f);
      const float waves = full * mu * each + each * fmaxf(1.f, mu * (large / sms - full)) + (full + 1.f) * item;
      cost = fmaxf((mu * work_f + item * items + slots) / sms, waves) + (slots > 0.f ? 5.5f : 0.f);
    }
    if (lane == 0) {
      s_sizes[warp] = size;
      s_cost[warp] = cost;
    }
  }
  __syncthreads();
  int best = 0;
#pragma unroll
  for (int k = 1; k < kCands; ++k)
    if (s_cost[k] < s_cost[best]) best = k;
  const int size = s_sizes[best];
  const bool run = best == 1;
  int my_offset = 0;   // chunks of the sequences before this thread's
  if (run) {
    int total = 0;
    __syncwarp();
    my_offset = block_exclusive_scan(mine.tiles > 0 ? mine.chunks : 0, sw, &total);
  }
  // A sequence's parts: the first, parts - 2 of `each` chunks, the last.
  struct Split {
    int parts, first, each;
  };
  auto split_of = [&](const TreeSeq& z) {
    if (run) {   // cuts at multiples of the share, but for ends worth less than an item's own cost
      const int edge = min(size / 8, kItemCost), first = (my_offset + edge) / size * size + size - my_offset;
      if (first >= z.chunks - edge) return Split{1, max(1, z.chunks), size};
      return Split{2 + (z.chunks - edge - 1 - first) / size, first, size};
    }
    const int p = max(1, cdiv(z.chunks, size)), each = max(1, cdiv(z.chunks, p));
    return Split{max(1, cdiv(z.chunks, each)), each, each};
  };
  auto last_of = [&](const TreeSeq& z, const Split& x) {
    return x.parts == 1 ? z.chunks : z.chunks - x.first - (x.parts - 2) * x.each;
  };
  auto bin = [&](int chunks) {   // 0: the largest
    return kTreeBins - 1 - min(kTreeBins - 1, static_cast<int>(static_cast<float>(chunks) * kTreeBins / (size + 1)));
  };
  // records per size
  int longest = 1;
  for (int b = tid; b < P.num_seqs; b += nthr) {
    const TreeSeq z = seq(b);
    if (z.tiles == 0) continue;
    const Split x = split_of(z);
    longest = max(longest, x.parts);
    if (x.parts > 1) atomicAdd(&s_hist[bin(x.first)], z.tiles);
    if (x.parts > 2) atomicAdd(&s_hist[bin(x.each)], (x.parts - 2) * z.tiles);
    atomicAdd(&s_hist[bin(last_of(z, x))], z.tiles);
  }
  __syncwarp();
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) atomicMax(&s_parts, longest);
  // Slots (11 bits), split sequences and their (tile, head) pairs (10 bits
  // each) before this sequence, in one scan; their bounds follow from size >=
  // work / kMaxShares, or were checked: slots <= 2 kMaxShares, pairs <= kMaxShares.
  int carry = 0, first = 0;   // first: of the records of size `lane`
  for (int base = 0; base < P.num_seqs; base += nthr) {
    const int b = base + tid;
    TreeSeq z = {};
    Split x = {1, 1, 1};
    if (b < P.num_seqs) {
      z = seq(b);
      x = split_of(z);
    }
    const int parts = x.parts;
    const int pairs = parts > 1 ? z.tiles * P.hkv : 0;
    const int add = pairs * parts + (pairs ? 1 << 11 : 0) + (pairs << 21);
    int total = 0;
    __syncwarp();
    const int at = carry + block_exclusive_scan(add, sw, &total);   // (its barriers are the counts' too)
    carry += total;
    if (base == 0) {
      const int c = s_hist[lane];
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      first = x - c;
      if (tid == 31) P.ws->n_entries = min(x, P.max_entries);
      if (tid == 0) P.ws->next_item = A.grid;   // a CTA's first item is its own number
    }
    const int slot0 = at & 2047, unit = at >> 11 & 1023;
    // overlapping trees (flagged) can want more slots than the workspace was
    // sized for: their records are left empty
    if (pairs && (unit >= A.max_units || slot0 + pairs * parts > A.max_slots)) z.rows = -1;
    if (pairs && unit < A.max_units)
      P.units[unit] =
          TreeUnit{static_cast<int>(static_cast<unsigned>(at) >> 21), z.tiles, parts, slot0, z.rows, z.q0}.pack();
    const int bin_first = bin(x.first), bin_each = bin(x.each), bin_last = bin(last_of(z, x));
    __syncwarp();
    int to_first = __shfl_sync(0xffffffffu, first, bin_first);   // their records
    int to_each = __shfl_sync(0xffffffffu, first, bin_each), to_last = __shfl_sync(0xffffffffu, first, bin_last);
    if (z.tiles > 0) {
      if (parts > 1) to_first += atomicAdd(&s_next[bin_first], z.tiles);
      if (parts > 2) to_each += atomicAdd(&s_next[bin_each], (parts - 2) * z.tiles);
      to_last += atomicAdd(&s_next[bin_last], z.tiles);
    }
    auto put = [&](int i, const TreeSeq& s, int b, const Split& x, int to_first, int to_each, int to_last, int slot0) {
      const int p = i / s.tiles, t = i - p * s.tiles;
      const int to = p == x.parts - 1 ? to_last + t : p == 0 ? to_first + t : to_each + i - s.tiles;
      if (to >= P.max_entries) return;   // overlapping trees again: no room, not run
      if (s.rows < 0) {
        P.entries[2 * to] = make_int4(b, 0, 1, -1);
        P.entries[2 * to + 1] = make_int4(0, 0, 0, 0);
        return;
      }
      constexpr int kPer = kChunkKeys / kBlock;
      const int from = p == 0 ? 0 : x.first + (p - 1) * x.each, end = p == x.parts - 1 ? s.chunks : x.first + p * x.each;
      const int blocks = max(1, min(end * kPer, (s.L + kBlock - 1) / kBlock) - from * kPer);
      P.entries[2 * to] = make_int4(b, t | from << kTileBits, blocks, x.parts > 1 ? slot0 + (p * s.tiles + t) * P.hkv : -1);
      P.entries[2 * to + 1] = make_int4(s.q0, s.rows, s.L - s.n, s.L);
    };
    const int count = z.tiles * parts;
    const bool many = count > 8;   // a long list is written by the whole warp
    if (!many)
      for (int i = 0; i < count; ++i) put(i, z, b, x, to_first, to_each, to_last, slot0);
    __syncwarp();
    for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
      __syncwarp();
      const int who = __ffs(left) - 1;
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, who); };
      const TreeSeq s = {of(z.q0), of(z.n), of(z.rows), of(z.L), of(z.tiles), of(z.chunks)};
      const Split sx = {of(x.parts), of(x.first), of(x.each)};
      const int sb = of(b), s1 = of(to_first), s2 = of(to_each), s3 = of(to_last), ss = of(slot0);
      for (int i = lane; i < s.tiles * sx.parts; i += 32) put(i, s, sb, sx, s1, s2, s3, ss);
    }
  }
  if (tid == 0) {
    P.ws->pad[kPadUnits] = min(carry >> 11 & 1023, A.max_units);
    P.ws->pad[kPadPairs] = static_cast<int>(static_cast<unsigned>(carry) >> 21);
    P.ws->pad[kPadParts] = s_parts;
  }
}

// ---------------------------------------------------------------------------
// Merge: out = sum_p 2^(m_p - m) acc_p / sum_p 2^(m_p - m) l_p, m = max_p m_p.
// A warp takes four output rows: the parts' (m, l) a lane each, then the rows
// of D floats, coalesced; from 16 parts on four warps share the rows' parts and
// join through shared memory.  The states are read back from L2; rounds of
// loads that wait for one another bound it, so all units come beside the
// header, and a part's first rows beside the (m, l), in two rounds.
template <typename T, int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams P, int max_units) {
  constexpr int V = D / 32;   // a lane's values of a row
  constexpr int R = 4;        // rows of a warp
  constexpr int kAhead = 2;   // parts whose rows are fetched before their weights are known
  __shared__ int4 s_units[kMaxShares];
  __shared__ float s_acc[8][R][D];
  __shared__ float s_sum[8][R];
  pdl_wait();
  pdl_launch_dependents();
  const int units = P.ws->pad[kPadUnits], pairs = P.ws->pad[kPadPairs], most = P.ws->pad[kPadParts];
  for (int i = threadIdx.x; i < min(max_units, static_cast<int>(blockDim.x)); i += blockDim.x) s_units[i] = P.units[i];
  if (units == 0) return;
  for (int i = threadIdx.x + blockDim.x; i < units; i += blockDim.x) s_units[i] = P.units[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = most >= 16 ? 4 : 1, per = 8 * R / share;   // warps of a row, rows of a CTA
  const int groups = 128 / per, mine = warp % share;
  for (int w = blockIdx.x; w < pairs * groups; w += gridDim.x) {
    const int pair = w / groups, r = (w - pair * groups) * per + warp / share * R;
    int lo = 0, hi = units - 1;   // the last unit whose pairs start at or before this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((s_units[mid].x & 1023) <= pair) lo = mid;
      else hi = mid - 1;
    }
    const TreeUnit u = TreeUnit::unpack(s_units[lo]);
    const int th = pair - u.first, tile = th / P.hkv, h = th - tile * P.hkv;
    const int tok0 = tile * P.tile_tokens;
    const bool valid = tok0 + r / P.G < u.rows;   // of the first row; the same for every warp of these rows
    float acc[R][V] = {}, sum[R] = {};
    if (valid) {
      const int64_t first = (static_cast<int64_t>(u.slot0) + th) * 128 + r;
      const int64_t step = static_cast<int64_t>(u.tiles) * P.hkv * 128;
      const int n = cdiv(u.parts - mine, share);   // this warp's parts: mine, mine + share, ...
      // (m, l) of four rows of a part: 32 bytes
      auto load = [&](int p, float (&m)[R], float (&l)[R]) {
        const float4* at = reinterpret_cast<const float4*>(P.ml + first + p * step);
        const float4 x = at[0], y = at[1];
        m[0] = x.x, l[0] = x.y, m[1] = x.z, l[1] = x.w;
        m[2] = y.x, l[2] = y.y, m[3] = y.z, l[3] = y.w;
      };
      // this lane's values of row k of this warp's part j
      auto values = [&](int j, int k, float (&x)[V]) {
        const float* a = P.acc + (first + (mine + j * share) * step + k) * D + lane * V;
        if constexpr (D == 128) {
          const float4 v = *reinterpret_cast<const float4*>(a);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(a);
          x[0] = v.x, x[1] = v.y;
        }
      };
      float m0[R] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, l0[R] = {};   // part `lane`
      if (lane < u.parts) load(lane, m0, l0);
      float ahead[kAhead][R][V];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int k = 0; k < R; ++k)
          if (j < n) values(j, k, ahead[j][k]);
      float top[R];
#pragma unroll
      for (int k = 0; k < R; ++k) top[k] = m0[k];
      for (int p = lane + 32; p < u.parts; p += 32) {
        float m[R], l[R];
        load(p, m, l);
#pragma unroll
        for (int k = 0; k < R; ++k) top[k] = fmaxf(top[k], m[k]);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < R; ++k) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
        if (top[k] == -INFINITY) top[k] = 0.f;
      }
      for (int base = 0; base < n; base += 32) {
        float wt[R] = {};
        if (base + lane < n) {
          float m[R], l[R];
          if (share > 1 || base > 0) {
            load(mine + (base + lane) * share, m, l);
          } else {
#pragma unroll
            for (int k = 0; k < R; ++k) m[k] = m0[k], l[k] = l0[k];
          }
#pragma unroll
          for (int k = 0; k < R; ++k) {
            wt[k] = exp2f(m[k] - top[k]);
            sum[k] += wt[k] * l[k];
          }
        }
        __syncwarp();
        const int here = min(32, n - base);
        auto add = [&](int j, int k, const float (&x)[V]) {
          const float wj = __shfl_sync(0xffffffffu, wt[k], j);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[k][e] = fmaf(wj, x[e], acc[k][e]);
        };
        if (base == 0) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (j < here) {
#pragma unroll
              for (int k = 0; k < R; ++k) add(j, k, ahead[j][k]);
            }
        }
#pragma unroll 2
        for (int j = base == 0 ? kAhead : 0; j < here; ++j) {
          float x[R][V];
#pragma unroll
          for (int k = 0; k < R; ++k) values(base + j, k, x[k]);
#pragma unroll
          for (int k = 0; k < R; ++k) add(j, k, x[k]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < R; ++k) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
      }
    }
    if (share > 1) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) s_acc[warp][k][lane * V + e] = acc[k][e];
        if (lane == 0) s_sum[warp][k] = sum[k];
      }
      __syncthreads();
      if (mine == 0) {
        for (int x = 1; x < share; ++x) {
#pragma unroll
          for (int k = 0; k < R; ++k) {
            sum[k] += s_sum[warp + x][k];
#pragma unroll
            for (int e = 0; e < V; ++e) acc[k][e] += s_acc[warp + x][k][lane * V + e];
          }
        }
      }
      __syncthreads();
    }
    if (!valid || mine != 0) continue;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int tok = tok0 + (r + k) / P.G;
      if (tok >= u.rows) break;
      const float inv = sum[k] > 0.f ? 1.0f / sum[k] : 0.f;
      T* dst = static_cast<T*>(P.out) +
               ((static_cast<int64_t>(u.q0) + tok) * P.hq + h * P.G + (r + k) % P.G) * D + lane * V;
      const uint32_t x0 = pack2<T>(acc[k][0] * inv, acc[k][1] * inv);
      if constexpr (D == 128)
        *reinterpret_cast<uint2*>(dst) = make_uint2(x0, pack2<T>(acc[k][2] * inv, acc[k][3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = x0;
    }
  }
}

// ---------------------------------------------------------------------------

namespace {

template <typename T, int D>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const TreePrepArgs& A, const TreeArgs& a, cudaStream_t s) {
  auto kern = rows_tc_kernel<T, D, TreeParams>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(TcCfg<D>::kBytes));
  if (e != cudaSuccess) return e;
  // a sequence per thread, as the loads of a second one would wait for the first's, and a warp per candidate
  const int per_warp = (a.num_seqs + 31) / 32 * 32;
  const int plan = per_warp < 32 * kCands ? 32 * kCands : per_warp < kPlanSeqs ? per_warp : kPlanSeqs;
  e = launch_pdl(tree_prep_kernel, dim3(1), dim3(plan), 0, s, A);
  if (e != cudaSuccess) return e;
  if (a.ev_before) cudaEventRecord(static_cast<cudaEvent_t>(a.ev_before), s);
  e = launch_pdl(kern, dim3(static_cast<unsigned>(A.grid)), dim3(TcCfg<D>::kThreads), TcCfg<D>::kBytes, s, tq, tk,
                 tv, A.P);
  if (e != cudaSuccess) return e;
  if (a.ev_after) cudaEventRecord(static_cast<cudaEvent_t>(a.ev_after), s);
  if (A.max_slots == 0) return cudaSuccess;   // no sequence has two chunks
  // four rows per warp or four warps; what the SMs hold at once at most
  int64_t ctas = (static_cast<int64_t>(a.num_q_tokens) * a.num_q_heads + 7) / 8;
  if (ctas > 4 * A.sms) ctas = 4 * A.sms;
  return launch_pdl(tree_merge_kernel<T, D>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, A.P,
                    A.max_units);
}

}  // namespace

size_t tree_workspace_bytes(int64_t num_seqs, int64_t num_q_tokens, int64_t num_q_heads, int64_t num_kv_heads,
                            int64_t head_dim, int64_t max_seq_len) {
  return tree_layout(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_seq_len).total;
}

int tree_launch(const TreeArgs& a, std::string* why) {
  const TreeLayout L =
      tree_layout(a.num_seqs, a.num_q_tokens, a.num_q_heads, a.num_kv_heads, a.head_dim, a.max_seq_len);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  TreePrepArgs A;
  TreeParams& P = A.P;
  P.q = a.q;
  P.out = a.out;
  P.tables = a.block_tables;
  P.seq_lens = a.seq_lens;
  P.q_off = a.q_offsets;
  P.ws = reinterpret_cast<PrefillHeader*>(ws);
  P.entries = reinterpret_cast<int4*>(ws + L.off_entries);
  P.num_blocks = a.num_blocks;
  P.max_blocks = a.max_blocks_per_seq;
  P.num_seqs = a.num_seqs;
  P.num_q_tokens = a.num_q_tokens;
  P.max_seq_len = a.max_seq_len;
  P.hq = a.num_q_heads;
  P.hkv = a.num_kv_heads;
  P.G = a.num_q_heads / a.num_kv_heads;
  P.tile_tokens = 128 / P.G;
  P.max_entries = static_cast<int>(L.max_entries);
  P.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  P.v_cache = a.v_cache;
  P.masks = a.masks;
  P.mask_words = a.mask_words;
  P.acc = reinterpret_cast<float*>(ws + L.off_acc);
  P.ml = reinterpret_cast<float2*>(ws + L.off_ml);
  P.units = reinterpret_cast<int4*>(ws + L.off_units);
  A.max_units = static_cast<int>(L.max_units);
  A.max_slots = static_cast<int>(L.max_slots);
  A.page_cost = 1.55f * a.head_dim / 128;
  int dev = 0;
  A.sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&A.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    *why = std::string("decode tree: ") + cudaGetErrorString(e);
    return 5;
  }
  CUtensorMap tq, tk, tv;
  if (!encode_cache_map(&tk, a.k_cache, a.num_blocks, a.num_kv_heads, a.head_dim, why) ||
      !encode_cache_map(&tv, a.v_cache, a.num_blocks, a.num_kv_heads, a.head_dim, why) ||
      !encode_q_map(&tq, a.q, a.num_q_tokens, a.num_q_heads, P.G, a.head_dim, why))
    return 5;
  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  const int64_t max_work = L.max_entries * a.num_kv_heads;
  A.grid = static_cast<int>(max_work < A.sms ? max_work : A.sms);
  e = a.dtype == 1 ? (a.head_dim == 128 ? launch_tree<__nv_bfloat16, 128>(tq, tk, tv, A, a, s)
                                        : launch_tree<__nv_bfloat16, 64>(tq, tk, tv, A, a, s))
                   : (a.head_dim == 128 ? launch_tree<__half, 128>(tq, tk, tv, A, a, s)
                                        : launch_tree<__half, 64>(tq, tk, tv, A, a, s));
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("decode tree launch: ") + cudaGetErrorString(e);
    return 5;
  }
  return 0;
}

}  // namespace pa
