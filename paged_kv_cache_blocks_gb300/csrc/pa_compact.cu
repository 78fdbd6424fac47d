// Compaction of accepted draft-tree tokens for sm_103a.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Compaction after a draft tree was verified: the accepted tokens' rows move
// to consecutive positions, row(before + j) <- row(before + accepted[j]) with
// accepted ascending, in every layer's caches by one launch.
//
// A thread owns one 16-byte column of a (K or V, sequence, KV head) and walks
// its moves in order, kBatch at a time, in the layers of its CTA: a batch's
// loads come before its stores.  accepted[j] >= j, so a later batch's sources
// lie past every row an earlier batch wrote, and no two threads share a byte:
// no barrier is needed.  Tokens already in place are skipped.  A few rows per
// sequence move, so the chain of loads (lengths and accepted tokens, page ids,
// rows) bounds it: it is walked once for several layers, as many as leave
// about three CTAs for every SM.  32 layers, 64 sequences, 4 moves each at the
// 8B shape: 14 to 15 us for 67 MB (batches of 8 at two CTAs an SM 16.7; a chain per
// layer 18.6).
constexpr int kSms = 152;             // for the choice of a CTA's share only
constexpr int kCompactLayers = 128;   // layers of one launch (their pointers are kernel arguments)

struct CompactPtrs {
  uint4* k[kCompactLayers];
  uint4* v[kCompactLayers];
};

__global__ void __launch_bounds__(256, 4)
    cache_compact_kernel(const __grid_constant__ CompactPtrs C, int layers, bool report_here, int64_t threads,
                         int chunks_per_row, int hkv, int64_t num_blocks, const int32_t* __restrict__ tables,
                         int max_blocks, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ q_off,
                         const int32_t* __restrict__ accepted, const int32_t* __restrict__ num_accepted,
                         int max_accepted, int32_t* __restrict__ new_lens, int32_t* __restrict__ error_bits) {
  constexpr int kBatch = 4;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= threads) return;
  const int per_seq = chunks_per_row * hkv;
  const int b = static_cast<int>(i / per_seq);
  const int rem = static_cast<int>(i - static_cast<int64_t>(b) * per_seq);
  const int h = rem / chunks_per_row, c = rem - h * chunks_per_row;
  uint4* const* caches = blockIdx.z == 0 ? C.k : C.v;
  const int32_t* acc = accepted + static_cast<int64_t>(b) * max_accepted;
  const int32_t* row = tables + static_cast<int64_t>(b) * max_blocks;
  const int L = seq_lens[b], a = q_off[b], e = q_off[b + 1], want = num_accepted[b];
  int bad = 0, n = 0, take = 0, prev = -1, done = 0;
  do {
    // one round of loads each: the accepted tokens (the first beside the
    // lengths), their page ids, their rows
    int src[kBatch], from[kBatch], to[kBatch];   // tree tokens; rows of the cache, in units of one head's row
#pragma unroll
    for (int u = 0; u < kBatch; ++u) src[u] = done + u < max_accepted ? acc[done + u] : -1;
    if (done == 0) {
      const int64_t n64 = static_cast<int64_t>(e) - a;
      if (L < 0 || L > static_cast<int64_t>(max_blocks) * kBlock || a < 0 || n64 < 0 || n64 > L) {
        bad = kErrSeqLen;   // nothing of this sequence moves
      } else {
        n = static_cast<int>(n64);
        take = min(max(want, 0), min(max_accepted, n));
        if (take != want) bad = kErrTree;
      }
    }
    const int before = L - n;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = done + u;
      if (j < take && (src[u] <= prev || src[u] >= n)) {   // not ascending, or not in the tree: the list ends here
        bad |= kErrTree;
        take = j;
      }
      prev = src[u];
      if (j >= take || src[u] == j) src[u] = -1;           // nothing to move
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      from[u] = src[u] >= 0 ? row[(before + src[u]) / kBlock] : -1;
      to[u] = src[u] >= 0 ? row[(before + done + u) / kBlock] : -1;
    }
    bool any = false;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (from[u] < 0 || from[u] >= num_blocks || to[u] < 0 || to[u] >= num_blocks) {
        if (src[u] >= 0) bad |= kErrBlockId;               // this row stays where it is
        from[u] = -1;
      } else {
        from[u] = (from[u] * hkv + h) * kBlock + (before + src[u]) % kBlock;
        to[u] = (to[u] * hkv + h) * kBlock + (before + done + u) % kBlock;
        any = true;
      }
    }
    for (int layer = blockIdx.y; any && layer < layers; layer += gridDim.y) {
      uint4* cache = caches[layer] + c;
      uint4 r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (from[u] >= 0) r[u] = cache[static_cast<int64_t>(from[u]) * chunks_per_row];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (from[u] >= 0) cache[static_cast<int64_t>(to[u]) * chunks_per_row] = r[u];
    }
    done += kBatch;
  } while (done < take);
  if (report_here && rem == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    if (new_lens) new_lens[b] = max(0, L - n) + take;
    if (bad && error_bits) atomicOr(error_bits, bad);
  }
}

int cache_compact_launch(const CompactArgs& a, std::string* why) {
  const int chunks_per_row = a.head_dim * 2 / 16;
  const int64_t threads = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * chunks_per_row;
  for (int first = 0; first < a.num_layers; first += kCompactLayers) {
    const int layers = a.num_layers - first < kCompactLayers ? a.num_layers - first : kCompactLayers;
    CompactPtrs C = {};
    for (int i = 0; i < layers; ++i) {
      C.k[i] = static_cast<uint4*>(a.k_caches[first + i]);
      C.v[i] = static_cast<uint4*>(a.v_caches[first + i]);
    }
    const int64_t ctas = (threads + 255) / 256;
    if (ctas > INT32_MAX) {
      *why = "cache_compact: too many sequences for one call";
      return 3;
    }
    int64_t groups = (3 * kSms + 2 * ctas - 1) / (2 * ctas);   // of layers
    if (groups > layers) groups = layers;
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(groups), 2);
    cudaError_t e = launch_pdl(cache_compact_kernel, grid, dim3(256), 0, static_cast<cudaStream_t>(a.stream), C,
                               layers, first == 0, threads, chunks_per_row, static_cast<int>(a.num_kv_heads), a.num_blocks,
                               a.block_tables, static_cast<int>(a.max_blocks_per_seq), a.seq_lens, a.q_offsets,
                               a.accepted, a.num_accepted, static_cast<int>(a.max_accepted),
                               a.new_seq_lens, a.error_bits);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
      *why = std::string("cache_compact launch: ") + cudaGetErrorString(e);
      return 5;
    }
  }
  return 0;
}

}  // namespace pa
