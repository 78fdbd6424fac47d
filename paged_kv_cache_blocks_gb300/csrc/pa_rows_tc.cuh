// tcgen05 attention of query rows over paged K/V, shared by the chunked
// prefill (causal pieces) and the draft-tree decode (masked trees).
#pragma once

#include <cuda.h>

#include <string>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

struct PrefillHeader {
  int32_t error_bits;
  int32_t n_entries;   // tiles of all pieces
  int32_t next_item;   // dynamic work counter
  int32_t pad[61];
};
static_assert(sizeof(PrefillHeader) == 256, "header is one 256-byte line");

struct PrefillParams {
  const void* q;        // [num_q_tokens][hq][D]
  void* out;            // same shape
  const int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* q_off;  // [num_seqs + 1]
  PrefillHeader* ws;
  int4* entries;         // (sequence, tile, key blocks, 0), longest first
  int64_t num_blocks;
  int max_blocks, num_seqs, num_q_tokens, max_seq_len, hq, hkv, G;
  int tile_tokens;       // query tokens per tile = 16 * NW / G
  int max_entries;       // capacity of `entries`
  float scale_log2;
};

// Validated view of sequence b: clamped length, first query token, piece
// length.  Bad input is flagged and clamped so no access leaves its buffer.
struct PieceView {
  int L, q0, n;
};

__device__ __forceinline__ PieceView piece_view(const PrefillParams& P, int b, bool flag) {
  int L = P.seq_lens[b];
  int a = P.q_off[b], e = P.q_off[b + 1];
  bool bad = false;
  if (L < 0 || L > P.max_seq_len) {
    bad = true;
    L = L < 0 ? 0 : P.max_seq_len;
  }
  if (a < 0 || a > P.num_q_tokens || e < a || e > P.num_q_tokens || (b == 0 && a != 0)) bad = true;
  a = min(max(a, 0), P.num_q_tokens);
  e = min(max(e, a), P.num_q_tokens);
  if (e - a > L) bad = true;  // a piece longer than its sequence
  if (bad && flag) atomicOr(&P.ws->error_bits, kErrSeqLen);
  return PieceView{L, a, e - a};
}

// Draft-tree decode: query t of a sequence's tree of n tokens sees every key
// before the tree and the tree's key i where bit i of its mask is set.  A
// work item covers a range of the keys; items of a tile whose keys are split
// leave their state in a slot of 128 rows for the merge.
struct TreeParams : PrefillParams {
  const void* v_cache;
  const int64_t* masks;  // [num_q_tokens][mask_words], bit i of word i / 64: tree token i
  int mask_words;
  float* acc;            // [slots][128][D] unnormalised outputs
  float2* ml;            // [slots][128] (maximum in units of log2, sum)
  int4* units;           // split sequences, for the merge
};

// One work item of the tcgen05 kernel.  Prefill: the record is (sequence,
// tile, key blocks, 0), all heads of record 0 last (KV-head-major).  Tree:
// two words, (sequence, tile | first key chunk << kTileBits, key blocks from
// there (at least one), slot of head 0 or -1) and (first query token, query tokens, tokens
// before the tree, tokens), everything the kernel needs of the sequence in one
// round trip; the heads of a record are neighbours, so the tiles of one key
// range run at about the same time and share its K/V in L2.
constexpr int kTileBits = 5;

struct TcItem {
  int h, b, tile, c0, nkb, slot;
  int q0, rows, before, L;
};

template <typename Params>
__device__ __forceinline__ TcItem tc_item(const Params& P, int wi, int n_entries) {
  if constexpr (std::is_same<Params, TreeParams>::value) {
    const int e = wi / P.hkv, h = wi - e * P.hkv;
    const int4 x = P.entries[2 * e], y = P.entries[2 * e + 1];
    return TcItem{h, x.x, x.y & ((1 << kTileBits) - 1), x.y >> kTileBits, x.z, x.w < 0 ? -1 : x.w + h,
                  y.x, y.y, y.z, y.w};
  } else {
    const int h = wi / n_entries;
    const int4 ent = P.entries[wi - h * n_entries];
    const PieceView v = piece_view(P, ent.x, false);
    return TcItem{h, ent.x, ent.y, 0, ent.z, -1, v.q0, v.n, v.L - v.n, v.L};
  }
}

// The item's key blocks alone.
template <typename Params>
__device__ __forceinline__ int tc_blocks(const Params& P, int wi, int n_entries) {
  return std::is_same<Params, TreeParams>::value ? P.entries[2 * (wi / P.hkv)].z
                                                 : P.entries[wi % n_entries].z;
}

// Which of the 64 keys from tree index `first` (key position minus the tokens
// before the tree; negative before it) a tree token sees, as bits: every key
// before the tree, then its mask.
__device__ __forceinline__ uint64_t tree_window(const int64_t* mask, int words, int first) {
  if (first <= -64) return ~0ull;
  if (first < 0) return ((1ull << -first) - 1) | (static_cast<uint64_t>(mask[0]) << -first);
  const int w = first >> 6, sh = first & 63;
  const uint64_t lo = w < words ? static_cast<uint64_t>(mask[w]) : 0ull;
  if (sh == 0) return lo;
  const uint64_t hi = w + 1 < words ? static_cast<uint64_t>(mask[w + 1]) : 0ull;
  return (lo >> sh) | (hi << (64 - sh));
}

// Whether each 16-bit half of a word is NaN or infinite, as a mask of its bits.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  constexpr uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return ((x & e) == e ? 0x0000ffffu : 0u) | ((x >> 16 & e) == e ? 0xffff0000u : 0u);
}

// ---------------------------------------------------------------------------
// The tcgen05 kernel.  One work item = (KV head, tile of 128 query rows: a row
// = one query token x one of the G heads of the KV head), for a draft tree
// over a range of the keys.  Described for head_dim 128; at 64 a tile has one
// 64-dim half, O0 and O1 64 columns each, and the rings twice the stages.
// Per CTA (one per SM, 14 warps):
//   warps 8-11  producers: warp 8 takes items from the atomic counter,
//               publishes them in a two-slot item ring and TMA-loads the
//               tile's Q (128 rows x 128 dims, one 3-D box of tokens x heads
//               x dims) into shared memory; all four load the key blocks in
//               chunks of 8 blocks = 128 keys (K one chunk ahead of V) into
//               three-stage K and V rings, each warp issuing the copies of
//               two blocks (K and V of a chunk are 128 swizzled rows per
//               64-dim half, so one descriptor spans the chunk).  TMA issue
//               from one warp is too slow for a chunk;
//   warp 12     allocates the tensor memory (S | P | O0 | O1 | Q); one thread
//               issues S = Q K^T (M 128, N 128 keys, K 128 dims) for chunk
//               c+1 as soon as the softmax of chunk c has read S;
//   warp 13     one thread issues, per key half hk, O_hk += P[:, 64 hk ..]
//               V[64 hk .., :] (M 128, N 128 dims, K 64 keys) once that
//               half's softmax warps have written P.  Issuing a product
//               blocks the thread about as long as the product runs, hence
//               two issuers.  Both products take their A operand (Q, P) from
//               tensor memory, which runs them at the full rate where an A
//               operand in shared memory halves it; tcgen05.commit signals
//               each result on an mbarrier;
//   warps 0-7   two threads per query row (its tensor-memory lane): warp w
//               takes keys 0-63 of every chunk, warp w + 4 keys 64-127.  At
//               the start of an item each moves its 64 dims of the Q row from
//               shared to tensor memory; per chunk it reads its 64 scores,
//               applies the scale and the causal mask, runs an online softmax
//               in fp32 with its own running maximum (moved only when it
//               grows by more than 2^8, fp16 trees 2^4: the exact result
//               either way, fewer rescales of its O), scale-and-subtract and
//               row sums on the packed two-lane fp32 FMA / add, and writes its
//               P as 16-bit values, two per column.  The halves never wait for each other
//               inside an item; at its end they exchange (maximum, sum) and
//               each writes 64 dims of (O0 2^(m0-m) + O1 2^(m1-m)) / l.
// The softmax warpgroups take registers the producer warpgroup gives back
// (setmaxnreg), so that nothing spills (in the trees' kernels three words).
// For trees an item is short (its epilogue 1.2 to 2.3 us against 0.9 to 1.4 us a
// chunk), so its end overlaps the next one's start: the softmax warps fetch the
// next record and move the next Q before they wait for the last product, and
// its first S runs beside the epilogue (64 sequences of 128-2048 tokens 69 ->
// 65 us); warps without a query row only keep the barriers' phases.  The
// prefill's items are long, and its order of the same steps is faster there
// (1341 against 1329 TFLOP/s in one session).
// Every wait is bounded; a timeout flags PA_DEVERR_TIMEOUT and the CTA
// drains its copies and tensor-core work before freeing tensor memory.

// Eight consecutive floats (32-byte aligned): one whole sector per thread.
__device__ __forceinline__ void st_global_v8(float* addr, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(addr), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// One 32-bit tensor-memory column of this thread's lane, stored / loaded
// and waited for in the same statement.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr), "r"(__float_as_uint(v))
      : "memory");
}
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(taddr)
      : "memory");
  return __uint_as_float(r);
}

template <int D>
struct TcCfg {
  static constexpr int kHalf = 128 * 128;           // 128 rows x 64 16-bit values
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = kHalves * kHalf;    // Q tile
  static constexpr int kChunkBytes = kHalves * kHalf;  // K (or V) of one chunk of 128 keys
  static constexpr int kChunkBlocks = 8;
  static constexpr int kKStages = 6 / kHalves;
  static constexpr int kVStages = 6 / kHalves;
  static constexpr size_t kOffQ = 0;
  static constexpr size_t kOffK = kOffQ + kQBytes;
  static constexpr size_t kOffV = kOffK + static_cast<size_t>(kKStages) * kChunkBytes;
  static constexpr size_t kOffBar = kOffV + static_cast<size_t>(kVStages) * kChunkBytes;
  static constexpr size_t kBytes = kOffBar + 512 + 1024;
  static constexpr int kSoftmaxWarps = 8;            // warpgroups 0 and 1: key halves 0 and 1
  static constexpr int kProducerWarp0 = 8;           // warpgroup 2
  static constexpr int kProducerWarps = 4;           // one per SM sub-partition: TMA issue
                                                     // from one warp is too slow for a chunk
  static constexpr int kMmaWarp = 12;                // warps 12 (S) and 13 (PV)
  static constexpr int kMmaWarps = 2;
  static constexpr int kThreads = 32 * (kMmaWarp + kMmaWarps);
  // registers per thread: 128 at launch (four warps on one sub-partition);
  // the producers drop to 64 and the softmax threads rise to 160:
  // 256 x 160 + 128 x 64 + 64 x 128 = 57344 <= 448 x 128 = 57344
  static constexpr int kRegsLaunch = 128, kRegsProducer = 64, kRegsSoftmax = 160;
  // tensor memory: S (128 fp32 columns) | P (128 16-bit values per row in 64
  // columns, keys 0-63 then 64-127) | O0 | O1 (128 fp32 columns each: the
  // products over keys 0-63 and 64-127 of every chunk, each half with its own
  // running maximum) | Q (128 16-bit values per row in 64 columns)
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColP = 128, kColO = 192, kColQ = 448;
};
static_assert(TcCfg<128>::kBytes <= 232448 && TcCfg<64>::kBytes <= 232448, "shared memory of one CTA");
static_assert(TcCfg<128>::kColQ + 64 <= TcCfg<128>::kTmemCols, "tensor-memory columns");
static_assert(TcCfg<128>::kColO + 256 <= TcCfg<128>::kColQ, "tensor-memory columns of O0 and O1");
static_assert(32 * (TcCfg<128>::kSoftmaxWarps * TcCfg<128>::kRegsSoftmax +
                    TcCfg<128>::kProducerWarps * TcCfg<128>::kRegsProducer +
                    TcCfg<128>::kMmaWarps * TcCfg<128>::kRegsLaunch) <=
                  TcCfg<128>::kThreads * TcCfg<128>::kRegsLaunch,
              "register split within the registers the CTA is launched with");

// Barrier indices, laid out from the ring sizes; every ring of n slots has
// one barrier per slot, so that a parity wait never meets a phase n uses
// ahead.
template <int D>
struct TcBars {
  using C = TcCfg<D>;
  enum : int {
    kKFull = 0,
    kKEmpty = kKFull + C::kKStages,
    kVFull = kKEmpty + C::kKStages,
    kVEmpty = kVFull + C::kVStages,
    kSFull = kVEmpty + C::kVStages,
    kSFree = kSFull + 1,
    kPFull = kSFree + 1,        // [key half]
    kODone = kPFull + 2,        // [key half]
    kQFull = kODone + 2,
    kQTmem = kQFull + 1,
    kItemFull = kQTmem + 1,     // [item slot]
    kItemEmpty = kItemFull + 2,
    kDrain = kItemEmpty + 2,
    kXFull = kDrain + 1,        // [quarter][slot]: the two threads of a row published a value (epilogue)
    kORead = kXFull + 8,        // tree: the epilogue has read O
    kNumTcBars = kORead + 1
  };
};
// after the barriers: item ring, tensor-memory slot, abort flag, non-finite tree tokens
static_assert(TcBars<64>::kNumTcBars * 8 + 32 + 96 <= 512, "barrier region");
static_assert(TcBars<64>::kNumTcBars % 2 == 0 && TcBars<128>::kNumTcBars % 2 == 0, "the flags are read 16 bytes at a time");

template <typename T, int D, typename Params>
__global__ void __launch_bounds__(TcCfg<D>::kThreads, 1)
    rows_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params P) {
  using C = TcCfg<D>;
  using B = TcBars<D>;
  constexpr bool kTree = std::is_same<Params, TreeParams>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + C::kOffQ;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  volatile int* s_items = reinterpret_cast<volatile int*>(bar + B::kNumTcBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + B::kNumTcBars + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + B::kNumTcBars + 2);
  // tree: per item modulo 3, the tree tokens of the item whose V has NaN or infinities
  uint32_t (*s_bad)[8] = reinterpret_cast<uint32_t (*)[8]>(bar + B::kNumTcBars + 4);
  if (kTree && threadIdx.x < 24) s_bad[threadIdx.x >> 3][threadIdx.x & 7] = 0;
  int* err = &P.ws->error_bits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.G;
  if (tid == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&bar[B::kKFull + i], C::kProducerWarps);
      mbar_init(&bar[B::kKEmpty + i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&bar[B::kVFull + i], C::kProducerWarps);
      mbar_init(&bar[B::kVEmpty + i], 1);
    }
    mbar_init(&bar[B::kSFull], 1);
    mbar_init(&bar[B::kSFree], C::kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[B::kPFull + i], C::kSoftmaxWarps / 2);   // per key half
      mbar_init(&bar[B::kODone + i], 1);
      mbar_init(&bar[B::kItemFull + i], 1);
      // the other producers (3), MMA issuers (2), softmax (8)
      mbar_init(&bar[B::kItemEmpty + i], C::kProducerWarps - 1 + C::kMmaWarps + C::kSoftmaxWarps);
    }
    mbar_init(&bar[B::kQFull], 1);
    mbar_init(&bar[B::kQTmem], C::kSoftmaxWarps);
    mbar_init(&bar[B::kDrain], C::kMmaWarps);
    for (int i = 0; i < 8; ++i) mbar_init(&bar[B::kXFull + i], 2);
    mbar_init(&bar[B::kORead], C::kSoftmaxWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kProducerWarp0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  if constexpr (kTree) pdl_wait();   // the plan and everything before it
  const int n_entries = *reinterpret_cast<volatile int32_t*>(&P.ws->n_entries);
  const int n_work = n_entries * P.hkv;

  if (warp >= C::kProducerWarp0 && warp < C::kMmaWarp) {
    // ------------------------------------------------------------ producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsProducer));
    // Warp 8 takes items from the atomic counter and publishes them; all
    // four producer warps read block ids 32 at a time (one coalesced load)
    // and each issues the copies of blocks p and p + 4 of every chunk
    // (lanes 0..3: block p / p + 4, dims 0-63 / 64-127), arming the stage
    // barrier for its own 8 KB.
    const int pw = warp - C::kProducerWarp0;
    const int64_t y_oob = P.num_blocks * P.hkv * kBlock;
    uint32_t it = 0, cc = 0;
    bool ok = true;
    auto wait = [&](int idx, uint32_t parity) {
      if (ok) ok = mbar_wait(&bar[idx], parity, abort_flag, err);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    // tree: a CTA's first item is its own number, the counter starts past them;
    // its record is fetched beside the number of records
    TcItem first;
    if constexpr (kTree) {
      if (pw == 0) first = tc_item(P, blockIdx.x, 0);
    }
    const int my_blk = pw + 4 * (lane & 1), my_hf = (lane >> 1) & 1;
    while (ok) {
      const int slot = it & 1;
      int wi = 0;
      if (pw == 0) {
        if (kTree && it == 0) wi = blockIdx.x;
        else if (lane == 0) wi = atomicAdd(&P.ws->next_item, 1);
        wi = __shfl_sync(0xffffffffu, wi, 0);
        if (*abort_flag) wi = n_work;
        if (it >= 2 && !wait(B::kItemEmpty + slot, ((it >> 1) - 1) & 1)) break;
        if (lane == 0) {
          s_items[slot] = wi < n_work ? wi : -1;
          mbar_arrive(&bar[B::kItemFull + slot]);
        }
        if (wi >= n_work) {
          if constexpr (kTree) pdl_launch_dependents();   // the merge may be scheduled
          break;
        }
      } else {
        if (!wait(B::kItemFull + slot, (it >> 1) & 1)) break;
        wi = s_items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kItemEmpty + slot]);
        if (wi < 0) break;
      }
      TcItem item;
      if constexpr (kTree) item = pw == 0 && it == 0 ? first : tc_item(P, wi, n_entries);
      else item = tc_item(P, wi, n_entries);
      const int h = item.h, b = item.b, tile = item.tile, nkb = item.nkb;
      if (pw == 0) {
        // the softmax warps moved the previous item's Q into tensor memory
        if (it >= 1 && !wait(B::kQTmem, (it - 1) & 1)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[B::kQFull], C::kQBytes);
          const int z = item.q0 + tile * P.tile_tokens;
          tma_load_3d(sQ, &tm_q, 0, h * G, z, &bar[B::kQFull]);
          if constexpr (D == 128) tma_load_3d(sQ + C::kHalf, &tm_q, 64, h * G, z, &bar[B::kQFull]);
        }
      }
      const int32_t* trow = P.tables + static_cast<int64_t>(b) * P.max_blocks + item.c0 * C::kChunkBlocks;
      const int nch = (nkb + C::kChunkBlocks - 1) / C::kChunkBlocks;
      const int held = kTree && item.L == 0 ? 0 : nkb;   // a tree's item has a block at least, if an empty one
      // K runs one chunk ahead of V: S of chunk c needs K(c) one step before
      // O += P V needs V(c)
      int32_t ids = 0, yk = 0, yprev = 0;   // lanes 0..3: the row of this lane's block
      for (int c = 0; c <= nch && ok; ++c) {
        if (c < nch) {
          if ((c & 3) == 0) {   // ids of chunks c .. c + 3
            const int blk = c * C::kChunkBlocks + lane;
            int32_t id = blk < held ? trow[blk] : -1;   // past the tile's keys: zero fill
            if (blk < held && (id < 0 || id >= P.num_blocks)) {
              if (pw == 0) atomicOr(err, kErrBlockId);
              id = -1;
            }
            ids = id;
          }
          const int32_t id = __shfl_sync(0xffffffffu, ids, (c & 3) * C::kChunkBlocks + my_blk);
          yk = static_cast<int32_t>(id < 0 ? y_oob : (static_cast<int64_t>(id) * P.hkv + h) * kBlock);
          const uint32_t x = cc + c;
          const int ks = x % C::kKStages;
          if (x >= C::kKStages && !wait(B::kKEmpty + ks, ((x / C::kKStages) - 1) & 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar[B::kKFull + ks], C::kChunkBytes / C::kProducerWarps);
          __syncwarp();
          if (lane < 2 * C::kHalves)
            tma_load_2d(smem + C::kOffK + static_cast<size_t>(ks) * C::kChunkBytes + my_hf * C::kHalf + my_blk * 2048,
                        &tm_k, my_hf * 64, yk, &bar[B::kKFull + ks]);
        }
        if (c >= 1) {
          const uint32_t x = cc + c - 1;
          const int vs = x % C::kVStages;
          if (x >= C::kVStages && !wait(B::kVEmpty + vs, ((x / C::kVStages) - 1) & 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar[B::kVFull + vs], C::kChunkBytes / C::kProducerWarps);
          __syncwarp();
          if (lane < 2 * C::kHalves)
            tma_load_2d(smem + C::kOffV + static_cast<size_t>(vs) * C::kChunkBytes + my_hf * C::kHalf + my_blk * 2048,
                        &tm_v, my_hf * 64, yprev, &bar[B::kVFull + vs]);
        }
        yprev = yk;
      }
      cc += nch;
      ++it;
    }
  } else if (warp >= C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuers
    // lane 0 of warp 12 issues the S products, lane 0 of warp 13 the PV
    // products: issuing blocks a thread about as long as the product runs,
    // so with one issuer its waits and commits sat between the products;
    // with two, each one's bookkeeping overlaps the other's products
    if (lane == 0) {
      const bool pv_role = warp == C::kMmaWarp + 1;
      constexpr int kBf = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
      constexpr uint32_t id_s = umma_idesc_f16(kBf, 0, 128, 128);
      constexpr uint32_t id_o = umma_idesc_f16(kBf, 1, 128, D);
      // shared-memory descriptors of the K and V rings; an MMA's operand is
      // the base plus a constant byte offset (>> 4 in the start-address field)
      const uint64_t dK0 = umma_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      // V is MN-major (dims contiguous): one N = 128 product spans its two
      // 64-dim atoms, C::kHalf bytes apart (the leading byte offset); one
      // 128-wide product runs at the full rate where two 64-wide ones do not
      const uint64_t dV0 = umma_desc_sw128(smem_u32(smem + C::kOffV), C::kHalf, 1024);
      uint32_t it = 0, cc = 0;
      bool ok = true;
      auto wait = [&](int idx, uint32_t parity) {
        if (ok) ok = mbar_wait_sleep(&bar[idx], parity, abort_flag, err);
        return ok;
      };
      while (ok) {
        const int slot = it & 1;
        if (!wait(B::kItemFull + slot, (it >> 1) & 1)) break;
        const int wi = s_items[slot];
        mbar_arrive(&bar[B::kItemEmpty + slot]);
        if (wi < 0) break;
        const int nkb = tc_blocks(P, wi, n_entries);
        const int nch = (nkb + C::kChunkBlocks - 1) / C::kChunkBlocks;
        if (!pv_role) {
          // S of chunk x into the single S buffer once the softmax has read
          // S of chunk x - 1: A = Q from tensor memory (16 dims = 8 packed
          // columns per step), B = K (K-major, 32 bytes per step inside a
          // 128-byte row)
          if (!wait(B::kQTmem, it & 1)) break;   // this item's Q is in tensor memory
          for (int c = 0; c < nch && ok; ++c, ++cc) {
            const int kst = cc % C::kKStages;
            if (!wait(B::kKFull + kst, (cc / C::kKStages) & 1)) break;
            if (cc >= 1 && !wait(B::kSFree, (cc - 1) & 1)) break;
            tc_fence_after();
            const uint64_t dK = dK0 + (static_cast<uint64_t>(kst) * C::kChunkBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_f16_ts(tbase + C::kColS, tbase + C::kColQ + 8 * ks,
                          dK + (((ks >> 2) * C::kHalf + (ks & 3) * 32) >> 4), id_s, ks > 0);
            umma_commit(&bar[B::kSFull]);
            umma_commit(&bar[B::kKEmpty + kst]);
          }
        } else {
          // O += P V of chunk x: A = P from tensor memory (16 keys = 8
          // packed columns per step), B = V (MN-major)
          if constexpr (kTree) {
            // the first product overwrites O: every warp read the last item's
            if (it >= 1 && !wait(B::kORead, (it - 1) & 1)) break;
          }
          for (int c = 0; c < nch && ok; ++c, ++cc) {
            const int vs = cc % C::kVStages;
            if (!wait(B::kVFull + vs, (cc / C::kVStages) & 1)) break;
            const uint64_t dV = dV0 + (static_cast<uint64_t>(vs) * C::kChunkBytes >> 4);
            // key half hk: O_hk += P[:, 64 hk ..] V[64 hk .., :] once that half's
            // softmax warps wrote their P
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) {
              if (!wait(B::kPFull + hk, cc & 1)) break;
              tc_fence_after();
#pragma unroll
              for (int ks = 4 * hk; ks < 4 * hk + 4; ++ks)
                umma_f16_ts(tbase + C::kColO + D * hk, tbase + C::kColP + 8 * ks, dV + ((ks * 2048) >> 4),
                            id_o, c > 0 || ks > 4 * hk);
              umma_commit(&bar[B::kODone + hk]);
            }
            if (!ok) break;
            umma_commit(&bar[B::kVEmpty + vs]);
          }
        }
        ++it;
      }
      // every product issued has completed before tensor memory is freed
      umma_commit(&bar[B::kDrain]);
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(&bar[B::kDrain], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // two threads per query row: warp w (w < 4) takes keys 0-63 of every
    // chunk, warp w + 4 keys 64-127, in the same tensor-memory lane quarter.
    // Each keeps its own running maximum and sum and its own O (O0, O1), so
    // the two never wait for each other inside an item; at its end they
    // exchange (maximum, sum) once and each writes 64 of the 128 output
    // dims of the combined result.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int quarter = warp & 3, half = warp >> 2;
    const int row = 32 * quarter + lane;
    const uint32_t lane_addr = tbase + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t o_mine = lane_addr + C::kColO + D * half;
    // The running maximum moves when it grows by more than 2^kGrow.  Trees: an
    // fp16 weight of less than 2^-14 would be subnormal and lose bits, one of
    // 2^-25 all, so the weights are stored 2^kBias higher and the quotient
    // O / l drops it.  With kGrow 4 they end at 2^11: the 2^5 below fp16's
    // largest hold what the rounding of a maximum up to 2^26 can add.
    constexpr bool kLift = kTree && std::is_same<T, __half>::value;
    constexpr float kBias = kLift ? 7.f : 0.f, kGrow = kLift ? 4.f : 8.f;
    uint32_t it = 0, cc = 0, xk = 0;
    bool ok = true;
    auto wait = [&](int idx, uint32_t parity) {
      if (ok) ok = mbar_wait(&bar[idx], parity, abort_flag, err);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    // one value with the row's other thread, through two tensor-memory
    // columns of the S buffer (free at an epilogue: the next item's first S
    // waits for its Q, which these warps write after the epilogue); a slot
    // is rewritten two exchanges later, after the partner passed the
    // exchange between
    auto exchange = [&](float mine) -> float {
      const uint32_t xs = xk & 1;
      tmem_st1(lane_addr + C::kColS + 2 * xs + half, mine);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B::kXFull + 2 * quarter + xs]);
      wait(B::kXFull + 2 * quarter + xs, (xk >> 1) & 1);
      tc_fence_after();
      const float other = tmem_ld1(lane_addr + C::kColS + 2 * xs + (half ^ 1));
      ++xk;
      return other;
    };
    // This thread's 64 dims of item `at`'s Q row -> tensor memory (the products
    // that read the item before's Q are done).  The TMA box put row `row` at
    // row * 128 bytes of each 64-dim half, its 16-byte pieces permuted by the
    // 128-byte swizzle (piece j at j ^ (row & 7)).
    auto move_q = [&](uint32_t at) -> bool {
      if (!wait(B::kQFull, at & 1)) return false;
      if (D == 128 || half == 0) {   // 64 dims a thread
        uint32_t qw[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(sQ + half * C::kHalf + row * 128 + ((j ^ (row & 7)) << 4));
          qw[4 * j] = u.x;
          qw[4 * j + 1] = u.y;
          qw[4 * j + 2] = u.z;
          qw[4 * j + 3] = u.w;
        }
        tmem_st32u(lane_addr + C::kColQ + 32 * half, qw);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B::kQTmem]);
      return true;
    };
    // tree: the record and the Q of item `at` of this CTA
    auto take = [&](uint32_t at, TcItem* item) -> bool {
      const int slot = at & 1;
      if (!wait(B::kItemFull + slot, (at >> 1) & 1)) return false;
      const int wi = s_items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B::kItemEmpty + slot]);
      item->h = -1;
      if (wi < 0) return true;
      *item = tc_item(P, wi, n_entries);
      // the flags of this item are first set after every warp has moved its Q;
      // those of three items before were read before every warp moved the last's
      if (warp == 0 && lane < 8) s_bad[at % 3][lane] = 0;
      return move_q(at);
    };
    TcItem next;
    if constexpr (kTree) ok = take(0, &next);
    while (ok) {
      TcItem item;
      if constexpr (kTree) {
        item = next;
        if (item.h < 0) break;
      } else {
        const int slot = it & 1;
        if (!wait(B::kItemFull + slot, (it >> 1) & 1)) break;
        const int wi = s_items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kItemEmpty + slot]);
        if (wi < 0) break;
        item = tc_item(P, wi, n_entries);
      }
      const int h = item.h, b = item.b, tile = item.tile, nkb = item.nkb;
      const int nch = (nkb + C::kChunkBlocks - 1) / C::kChunkBlocks;
      const int tok = tile * P.tile_tokens + row / G;
      const int pos = item.before + tok;
      const bool valid = tok < item.rows && (kTree || pos >= 0);
      const int lim = valid ? pos : -1;
      const bool live = !kTree || __any_sync(0xffffffffu, valid);
      const int64_t* row_mask = nullptr;
      if constexpr (kTree)
        row_mask = P.masks + (static_cast<int64_t>(item.q0) + (valid ? tok : 0)) * P.mask_words;
      else if (!move_q(it)) break;
      // V rows past the sequence end (the last block's tail) may hold
      // anything, NaN included: zero them so that 0 * NaN never enters O.
      // Rows of a tree are seen by some queries only: their NaN and infinite
      // values are zeroed too, and the queries that see them get them back in
      // the epilogue.
      auto zero_tail = [&](int kc) -> bool {
        const int before = kTree ? item.before : item.L;   // keys that every row sees
        if (kc + 128 <= before) return true;
        // the chunk's V copies have landed before their rows are overwritten
        const int vs = cc % C::kVStages;
        if (!wait(B::kVFull + vs, (cc / C::kVStages) & 1)) return false;
        // this half's product reads only keys 64 half .. 64 half + 63 of the
        // chunk, and waits only for this half's warps: they zero those rows
        const int z0 = max(max(item.L, kc) - kc, 64 * half);
        const int z1 = min(min(kc + 128, (item.c0 * C::kChunkBlocks + nkb) * kBlock) - kc, 64 * half + 64);
        uint8_t* sV = smem + C::kOffV + static_cast<size_t>(vs) * C::kChunkBytes;
        for (int i = row; i < (z1 - z0) * (D / 8); i += 128) {   // 16-byte pieces of the key rows
          const int key = z0 + i / (D / 8), part = i % (D / 8);
          *reinterpret_cast<uint4*>(sV + (part >> 3) * C::kHalf + key * 128 + (part & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        if constexpr (kTree) {
          const int y0 = max(max(before, kc) - kc, 64 * half), y1 = min(min(item.L, kc + 128) - kc, 64 * half + 64);
          for (int i = row; i < (y1 - y0) * (D / 8); i += 128) {
            const int key = y0 + i / (D / 8), part = i % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(sV + (part >> 3) * C::kHalf + key * 128 + (part & 7) * 16);
            const uint4 x = *at;
            const uint4 n = make_uint4(nonfinite2<T>(x.x), nonfinite2<T>(x.y), nonfinite2<T>(x.z), nonfinite2<T>(x.w));
            if (n.x | n.y | n.z | n.w) {
              *at = make_uint4(x.x & ~n.x, x.y & ~n.y, x.z & ~n.z, x.w & ~n.w);
              const int token = kc + key - before;
              if (token < 256) atomicOr(&s_bad[it % 3][token >> 5], 1u << (token & 31));
            }
          }
        }
        fence_proxy_async_smem();   // the zeros before the tensor cores read V
        return true;
      };
      float m_ref = -INFINITY, l = 0.f;   // this key half's reference maximum and sum
      if constexpr (kTree) {
        // a warp with no query row keeps its barriers' phases and nothing else:
        // its rows of S, P and O hold anything, and no other row reads them
        if (!live) {
          for (int c = 0; c < nch; ++c, ++cc) {
            if (!wait(B::kSFull, cc & 1)) break;
            if (lane == 0) mbar_arrive(&bar[B::kSFree]);
            // the product before it is done, so every warp has arrived for it
            if (cc >= 1 && !wait(B::kODone + half, (cc - 1) & 1)) break;
            if (!zero_tail((item.c0 + c) * 128)) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B::kPFull + half]);
          }
        }
      }
      for (int c = live ? 0 : nch; c < nch; ++c, ++cc) {
        if (!wait(B::kSFull, cc & 1)) break;
        tc_fence_after();
        const int kc = (item.c0 + c) * 128, k0 = kc + 64 * half;
        float t[64];
        tmem_ld64(lane_addr + C::kColS + 64 * half, t);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kSFree]);
        if constexpr (kTree) {
          const int first = k0 - item.before;   // tree index of this half's first key
          if (first > -64) {                    // keys of the tree, or past it
            uint64_t win = valid ? tree_window(row_mask, P.mask_words, first) : 0ull;
            if (k0 + 64 > item.L) win &= k0 < item.L ? (1ull << (item.L - k0)) - 1 : 0ull;
#pragma unroll
            for (int i = 0; i < 64; ++i) t[i] = (win >> i) & 1 ? t[i] : -INFINITY;
          }
        } else if (!__all_sync(0xffffffffu, k0 + 63 <= lim)) {   // causal mask / tail: -inf
#pragma unroll
          for (int i = 0; i < 64; ++i) t[i] = k0 + i <= lim ? t[i] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // 4 chains for ILP
#pragma unroll
        for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], t[i]);
        // the scale is positive, so it commutes with the maximum
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * P.scale_log2;
        const bool need = mx > m_ref + kGrow;
        const float new_ref = need ? mx : m_ref;
        const float mu = new_ref == -INFINITY ? 0.f : new_ref;
        const float alpha = need ? exp2f(m_ref - new_ref) : 1.f;
        // p = 2^(s * scale - mu) as 16-bit, two per column, into this half's
        // 32 columns of P, once the previous chunk's product over this half
        // has read them; row sum in fp32 (pairs on the packed two-lane FMA/add).
        // The tensor cores take P in T, so each weight is rounded once, by half
        // a step of T; the sum keeps it in fp32.
        const float shift = kLift ? kBias - mu : -mu;
        const float2 sc2 = make_float2(P.scale_log2, P.scale_log2), nm2 = make_float2(shift, shift);
        float2 r2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 x = fma2(make_float2(t[2 * i], t[2 * i + 1]), sc2, nm2);
          const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          r2[i & 3] = add2(r2[i & 3], p);
          pk[i] = pack2<T>(p.x, p.y);
        }
        if (cc >= 1 && !wait(B::kODone + half, (cc - 1) & 1)) break;
        tc_fence_after();
        tmem_st32u(lane_addr + C::kColP + 32 * half, pk);
        r2[0] = add2(add2(r2[0], r2[1]), add2(r2[2], r2[3]));
        l = l * alpha + (r2[0].x + r2[0].y);
        if (c > 0 && __any_sync(0xffffffffu, need)) {
          // this half's O holds the previous chunk's product (waited above)
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            float o32[32];
            tmem_ld32(o_mine + cb * 32, o32);
#pragma unroll
            for (int i = 0; i < 32; ++i) o32[i] *= alpha;
            tmem_st32(o_mine + cb * 32, o32);
          }
        }
        if (!zero_tail(kc)) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kPFull + half]);
        m_ref = new_ref;
      }
      if (!ok) break;
      // epilogue: combine the halves, out = (O0 2^(m0 - m) + O1 2^(m1 - m)) /
      // (l0 2^(m0 - m) + l1 2^(m1 - m)) with m the larger maximum; each thread
      // writes 64 of the 128 dims, one rounding to T
      float m_other, l_other;
      if constexpr (kTree) {
        // The next item's Q goes to tensor memory now, so that its first S runs
        // beside this epilogue.  The state is exchanged through the columns
        // of P: each thread writes into its partner's half, which the partner
        // writes again only after it has read it here.
        if (!take(it + 1, &next)) break;
        if (nch > 0) {
          if (!wait(B::kODone + 0, (cc - 1) & 1)) break;
          if (!wait(B::kODone + 1, (cc - 1) & 1)) break;
        }
        tc_fence_after();
        tmem_st1(lane_addr + C::kColP + 32 * (half ^ 1), m_ref);
        tmem_st1(lane_addr + C::kColP + 32 * (half ^ 1) + 1, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kXFull + 2 * quarter]);
        if (!wait(B::kXFull + 2 * quarter, it & 1)) break;
        tc_fence_after();
        m_other = tmem_ld1(lane_addr + C::kColP + 32 * half);
        l_other = tmem_ld1(lane_addr + C::kColP + 32 * half + 1);
      } else {
        m_other = exchange(m_ref);
        l_other = exchange(l);
        if (!ok) break;
        if (nch > 0) {
          if (!wait(B::kODone + 0, (cc - 1) & 1)) break;
          if (!wait(B::kODone + 1, (cc - 1) & 1)) break;
        }
      }
      tc_fence_after();
      {
        const float m0 = half == 0 ? m_ref : m_other, m1 = half == 0 ? m_other : m_ref;
        const float l0 = half == 0 ? l : l_other, l1 = half == 0 ? l_other : l;
        const float mm = fmaxf(m0, m1);
        const float w0 = mm == -INFINITY ? 0.f : exp2f(m0 - mm);
        const float w1 = mm == -INFINITY ? 0.f : exp2f(m1 - mm);
        const float lsum = l0 * w0 + l1 * w1;
        const bool split = kTree && item.slot >= 0;   // the state goes to the merge as it is
        const float inv = split ? 1.f : (valid && lsum > 0.f) ? 1.0f / lsum : 0.f;
        const float a0 = w0 * inv, a1 = w1 * inv;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(P.out) +
                                              ((static_cast<int64_t>(item.q0) + tok) * P.hq + h * G + row % G) * D +
                                              D / 2 * half);
        float* part = nullptr;
        if constexpr (kTree) {
          if (split) {
            const int64_t prow = static_cast<int64_t>(item.slot) * 128 + row;
            part = P.acc + prow * D + D / 2 * half;
            if (tok < item.rows && half == 0) P.ml[prow] = make_float2(mm, lsum);
          }
        }
#pragma unroll 1
        for (int cb = 0; cb < D / 64; ++cb) {
          float x32[32], y32[32];
          if (nch > 0) {   // uniform over the warp: every lane takes part in the loads
            tmem_ld32(lane_addr + C::kColO + D / 2 * half + cb * 32, x32);
            tmem_ld32(lane_addr + C::kColO + D + D / 2 * half + cb * 32, y32);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x32[i] = y32[i] = 0.f;
          }
          if (tok < item.rows) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              float o8[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) o8[e] = fmaf(x32[8 * q4 + e], a0, y32[8 * q4 + e] * a1);
              if (kTree && split) {
                st_global_v8(part + cb * 32 + 8 * q4, o8);
                continue;
              }
              dst[cb * 4 + q4] = make_uint4(pack2<T>(o8[0], o8[1]), pack2<T>(o8[2], o8[3]),
                                            pack2<T>(o8[4], o8[5]), pack2<T>(o8[6], o8[7]));
            }
          }
        }
      }
      if constexpr (kTree) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B::kORead]);
        // every warp's flags are set: both halves' last products are done
        asm volatile("" ::: "memory");   // the rows above were stored as wider words
        const uint4* flags = reinterpret_cast<const uint4*>(s_bad[it % 3]);
        const uint4 f0 = flags[0], f1 = flags[1];
        const uint32_t bad[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
        const bool any = f0.x | f0.y | f0.z | f0.w | f1.x | f1.y | f1.z | f1.w;
        for (int w = 0; any && w < 8; ++w) {
          uint32_t left = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) left = k == w ? bad[k] : left;
          for (; left; left &= left - 1) {
            const int token = 32 * w + __ffs(left) - 1, at = item.before + token;
            if (tok >= item.rows || (token >> 6) >= P.mask_words || !((row_mask[token >> 6] >> (token & 63)) & 1)) continue;
            const int64_t id = P.tables[static_cast<int64_t>(b) * P.max_blocks + at / kBlock];
            const int d0 = D / 2 * half;
            const T* vrow = static_cast<const T*>(P.v_cache) + ((id * P.hkv + h) * kBlock + at % kBlock) * D + d0;
            const int64_t orow = (static_cast<int64_t>(item.q0) + tok) * P.hq + h * G + row % G;
            T* final = static_cast<T*>(P.out) + orow * D + d0;
            float* state = P.acc + (static_cast<int64_t>(item.slot) * 128 + row) * D + d0;
            for (int d = 0; d < D / 2; ++d) {   // a weight above 0 times NaN or infinity: itself
              const float x = to_float<T>(vrow[d]);
              if (isfinite(x)) continue;
              if (item.slot >= 0) state[d] += x;
              else final[d] = from_float<T>(to_float<T>(final[d]) + x);
            }
          }
        }
      }
      tc_fence_before();
      ++it;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // copies still in flight land before the CTA leaves: a copy takes
    // microseconds, so every thread waits 200 us of global time
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000ull) {
    }
  }
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// q [Tq][hq][D] as a 3-D tensor (dims, heads, tokens); one box = the G heads
// of a KV head for 128 / G tokens and 64 dims: 128 rows of 128 bytes in the
// order (token, head), 128-byte swizzle.
inline bool encode_q_map(CUtensorMap* m, const void* q, int64_t Tq, int hq, int G, int D,
                  std::string* why) {
  EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder(why));
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(hq),
                        static_cast<cuuint64_t>(Tq)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(hq) * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *why = "cuTensorMapEncodeTiled (q) failed with CUresult " + std::to_string(static_cast<int>(r));
    return false;
  }
  return true;
}

}  // namespace pa
