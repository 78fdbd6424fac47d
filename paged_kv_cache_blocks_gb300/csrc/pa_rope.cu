// Per-head norm of q and k, position rotation and cache write in one pass.
//
// For each token at position p, with x a head of q or k:
//   y   = x * rsqrt(mean(x^2) + eps) * w            (a head of q or k with a weight)
//   z_a = f * (y_a cos(p w_i) - y_b sin(p w_i)),  z_b = f * (y_b cos(p w_i) + y_a sin(p w_i))
// for pair i = (a, b) of the rotated part: (i, i + r/2) or (2i, 2i + 1), r =
// rotary_dim; the rest of the head keeps y.  q goes to q_out, k and v to their
// cache slots.  fp32 throughout, one rounding where a value is stored.
//
// The angle is kept in turns as a 64-bit fraction: p * (2^64 w_i / 2 pi)
// wraps modulo one turn by itself, so a far position costs no accuracy (the
// frequency is off by less than 2^-53 of itself and 2^-64 of a turn per token)
// and no 64-bit floating point, of which an SM does two operations per clock.
//
// A head of D values is held by D / 16 threads, each with eight values from
// the first and eight from the second half of the rotated part (of the rest,
// past it): both members of a pair of either layout are in one thread, loads
// and stores are 16 bytes wide and every 128-byte line is used whole.  A CTA
// takes consecutive (token, head) rows, kRopeRows per thread, all loaded before the
// angles of its tokens are computed; a token's angles are shared by its heads
// through shared memory, laid out so that the threads of a row read
// consecutive words.  Memory should bound it and instructions nearly do: fp32
// pairs go through the packed two-lane operations, and a row's token and head
// follow from the last one's without a division.
//
// E4M3 caches hold V dimension-major ([128][16] bytes a page and head), a
// token's values 16 bytes apart: CTAs of their own take kVTokens consecutive
// tokens of a head, quantise them into shared memory and write each run of
// tokens that fills a page's 16 rows with one 16-byte store per dimension; the
// rest (a page's beginning or end, single tokens) byte by byte.  30000 tokens,
// 1168 MB: 195 us in runs of pages (0.88 of the copy rate), 260 us scattered;
// 256 single tokens 12.6 us (16-bit caches 4.1).
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Two fp32 lanes per instruction, each exactly the scalar product.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

namespace {

constexpr int kRopeThreads = 256;
// Rows a thread: they share the CTA's angles and index arithmetic, against the
// registers that keep four CTAs on an SM.  us for 3770 tokens at the 70B shape /
// 30000 to E4M3 in runs of pages / 256 tokens: 2 rows 26.0 / 210 / 4.2, 3 rows 24.7 / 201 / 4.1,
// 4 rows 25.1 / 212 / 4.1 (25.5 / 208 with three CTAs an SM).
constexpr int kRopeRows = 3;

struct RopeParams {
  const void *q, *k, *v;
  int q_stride, k_stride, v_stride;   // elements
  const int32_t* positions;
  const int64_t* slots;
  const double* inv_freq;
  const void *q_norm, *k_norm;
  void *q_out, *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  int64_t num_blocks;
  int tokens, rows;                   // rows = tokens * heads
  int row_ctas;                       // the CTAs past them write V of E4M3 caches
  int heads, hq, hkv, rotary;         // heads of a token: q, k and (16-bit caches) v
  int step_tokens, step_heads;        // rows-at-a-time / heads and the remainder
  float factor, eps;
};

}  // namespace

// 2^64 w / 2 pi modulo 2^64: the mantissa m (53 bits) times 2^64 * 2 / pi, whose
// upper word is m 2^11 (2 / pi), shifted to w's exponent.
__device__ __forceinline__ uint64_t turn_fraction(double w) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(w));
  const int e = static_cast<int>(bits >> 52 & 0x7ff);
  if (e == 0) return 0;                                   // zero (and subnormals: no turn within 2^64 tokens)
  const uint64_t m = (bits << 11) | (1ull << 63);         // w = m 2^(e - 1023 - 63)
  const uint64_t hi = __umul64hi(m, 11743562013128004906ull);   // times 2^64 * 2 / pi
  const int s = e - 1023 - 1;                             // 2^64 w / 2 pi = hi 2^s
  const uint64_t f = s >= 64 || s <= -64 ? 0 : s >= 0 ? hi << s : hi >> -s;
  return w < 0 ? 0 - f : f;
}

constexpr int kVTokens = 128;   // us for 30000 tokens in runs of pages: 32 tokens 215, 64 202, 128 198

// V rows of kVTokens tokens from t0 on, head h, into the E4M3 cache.
template <typename T>
__device__ void write_v8(const RopeParams& P, int t0, int h, uint8_t* smem) {
  constexpr int D = 128, kPitch = D + 16;                 // bytes; 16-byte aligned rows
  uint8_t* s_q = smem;                                    // [kVTokens][kPitch] codes
  int64_t* s_slot = reinterpret_cast<int64_t*>(smem + kVTokens * kPitch);
  int* s_run = reinterpret_cast<int*>(s_slot + kVTokens); // [kVTokens] (first token | tokens << 16) of each run
  __shared__ int s_runs;
  const int tid = threadIdx.x;
  const int n = min(kVTokens, P.tokens - t0);
  const int l = tid & 15, row = tid >> 4;                 // 16 threads a row, eight values each
  uint4 x[kVTokens / 16];
#pragma unroll
  for (int u = 0; u < kVTokens / 16; ++u) {
    const int i = row + 16 * u;
    const T* src = static_cast<const T*>(P.v) + static_cast<int64_t>(t0 + i) * P.v_stride + h * D + 8 * l;
    x[u] = i < n ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
  }
  const int64_t slot = tid < n ? P.slots[t0 + tid] : -1;
  if (tid < kVTokens) s_slot[tid] = slot;
  if (tid == 0) s_runs = 0;
  const float inv = 1.0f / P.v_scale[h];
#pragma unroll
  for (int u = 0; u < kVTokens / 16; ++u) {
    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = unpack2<T>(w[e]);
      q[e] = float2_to_e4m3x2(p.x * inv, p.y * inv);
    }
    *reinterpret_cast<uint2*>(s_q + (row + 16 * u) * kPitch + 8 * l) =
        make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
  }
  __syncthreads();
  // a run: tokens in consecutive rows of one page
  if (tid < n && slot >= 0 && slot / kBlock < P.num_blocks &&
      (tid == 0 || slot % kBlock == 0 || s_slot[tid - 1] != slot - 1)) {
    int len = 1;
    while (tid + len < n && (slot + len) % kBlock != 0 && s_slot[tid + len] == slot + len) ++len;
    s_run[atomicAdd(&s_runs, 1)] = tid | len << 16;
  }
  __syncthreads();
  for (int i = tid; i < s_runs * D; i += kRopeThreads) {
    const int first = s_run[i / D] & 0xffff, len = s_run[i / D] >> 16, d = i % D;
    const int64_t s = s_slot[first], blk = s / kBlock;
    uint8_t* dst = static_cast<uint8_t*>(P.v_cache) + ((blk * P.hkv + h) * D + d) * kBlock + (s - blk * kBlock);
    const uint8_t* src = s_q + first * kPitch + d;
    if (len == kBlock) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = src[(4 * e) * kPitch] | src[(4 * e + 1) * kPitch] << 8 | src[(4 * e + 2) * kPitch] << 16 |
               static_cast<uint32_t>(src[(4 * e + 3) * kPitch]) << 24;
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int j = 0; j < len; ++j) dst[j] = src[j * kPitch];
    }
  }
}

template <typename T, int D, bool kInter, bool kFp8, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_cache_write_kernel(const RopeParams P) {
  constexpr int kLanes = D / 16;                          // threads of a row
  constexpr int kGroups = kRopeThreads / kLanes;          // rows at a time
  constexpr int U = kRopeRows;
  // per token of the CTA [4][rotary / 16] (cos, cos, sin, sin) of two pairs
  extern __shared__ __align__(16) uint8_t s_raw[];
  float4* s_cs = reinterpret_cast<float4*>(s_raw);
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (kFp8) {
    const int w = static_cast<int>(blockIdx.x) - P.row_ctas;
    if (w >= 0) {
      write_v8<T>(P, w / P.hkv * kVTokens, w % P.hkv, s_raw);
      return;
    }
  }
  const int tid = threadIdx.x, l = tid % kLanes, g = tid / kLanes;
  const int row0 = static_cast<int>(blockIdx.x) * (kGroups * U);
  const int t0 = row0 / P.heads, r0 = row0 - t0 * P.heads;   // first token, and its heads in earlier CTAs
  const int nrows = min(kGroups * U, P.rows - row0);
  const int half = P.rotary >> 1, rl = P.rotary >> 4;     // rl: threads that hold rotated values
  // this thread's two runs of eight values
  const int ca = l < rl ? 8 * l : P.rotary + 8 * (l - rl);
  const int cb = l < rl ? half + 8 * l : P.rotary + ((D - P.rotary) >> 1) + 8 * (l - rl);
  uint4 xa[U], xb[U];
  int64_t slot[U];
  const int tok0 = (r0 + g) / P.heads, head0 = r0 + g - tok0 * P.heads;
  int tok = tok0, hd = head0;
  auto next = [&] {   // kGroups rows further
    tok += P.step_tokens;
    hd += P.step_heads;
    if (hd >= P.heads) {
      hd -= P.heads;
      ++tok;
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u, next()) {
    xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
    slot[u] = -1;
    if (g + u * kGroups >= nrows) continue;
    const bool is_q = hd < P.hq, is_v = hd >= P.hq + P.hkv;
    const T* src = static_cast<const T*>(is_q ? P.q : is_v ? P.v : P.k) +
                   static_cast<int64_t>(t0 + tok) * (is_q ? P.q_stride : is_v ? P.v_stride : P.k_stride) +
                   (hd - (is_q ? 0 : is_v ? P.hq + P.hkv : P.hq)) * D;
    xa[u] = *reinterpret_cast<const uint4*>(src + ca);
    xb[u] = *reinterpret_cast<const uint4*>(src + cb);
    if (!is_q) slot[u] = P.slots[t0 + tok];
  }
  // cos and sin of the CTA's tokens: a pair per thread of 64, four tokens at a time
  if ((tid & 63) < half) {
    const int f = tid & 63;
    const uint64_t frequency = turn_fraction(P.inv_freq[f]);
    // where the thread that turns this pair reads it: its eight pairs are
    // 8 l + e, or interleaved 4 l + e of the first run and of the second
    const int second = kInter && f >= half >> 1, h = f - (second ? half >> 1 : 0);
    const int fl = kInter ? h >> 2 : h >> 3, e = kInter ? 4 * second + (h & 3) : h & 7;
    float* at = reinterpret_cast<float*>(s_cs + (e >> 1) * rl + fl) + (e & 1);
    const int ntok = (r0 + nrows - 1) / P.heads + 1;
    for (int t = tid >> 6; t < ntok; t += kRopeThreads / 64) {
      const int64_t p = P.positions[t0 + t];
      const int32_t turn = static_cast<int32_t>((static_cast<uint64_t>(p) * frequency) >> 32);
      float sn, cs;
      sincospif(static_cast<float>(turn) * 0x1p-31f, &sn, &cs);   // signed: a half turn either way
      at[16 * rl * t] = cs * P.factor;
      at[16 * rl * t + 2] = sn * P.factor;
    }
  }
  __syncthreads();
  tok = tok0;
  hd = head0;
#pragma unroll
  for (int u = 0; u < U; ++u, next()) {
    const bool is_q = hd < P.hq, is_v = !kFp8 && hd >= P.hq + P.hkv;
    float2 a[4], b[4];
    a[0] = unpack2<T>(xa[u].x), a[1] = unpack2<T>(xa[u].y), a[2] = unpack2<T>(xa[u].z), a[3] = unpack2<T>(xa[u].w);
    b[0] = unpack2<T>(xb[u].x), b[1] = unpack2<T>(xb[u].y), b[2] = unpack2<T>(xb[u].z), b[3] = unpack2<T>(xb[u].w);
    if constexpr (kNorm) {
      // every row of the warp takes part, v too: shuffles that only some of
      // its rows reach are taken one by one
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(a[e], a[e], fma2(b[e], b[e], s2));
      float ss = s2.x + s2.y;
      __syncwarp();
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, kLanes);
      const T* norm = static_cast<const T*>(is_q ? P.q_norm : P.k_norm);
      if (norm && !is_v) {
        const uint4 na = *reinterpret_cast<const uint4*>(norm + ca), nb = *reinterpret_cast<const uint4*>(norm + cb);
        const uint32_t wa[4] = {na.x, na.y, na.z, na.w}, wb[4] = {nb.x, nb.y, nb.z, nb.w};
        const float rs = rsqrtf(ss * (1.0f / D) + P.eps);
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = mul2(a[e], mul2(unpack2<T>(wa[e]), rs2));
          b[e] = mul2(b[e], mul2(unpack2<T>(wb[e]), rs2));
        }
      }
    }
    if (g + u * kGroups >= nrows) continue;
    const int h = is_v ? hd - P.hq - P.hkv : hd - P.hq;   // the KV head
    if (!is_q && (slot[u] < 0 || slot[u] / kBlock >= P.num_blocks)) continue;   // padding, or outside the pool
    // where the row goes, in rows
    const int64_t to = is_q ? static_cast<int64_t>(t0 + tok) * P.hq + hd
                            : (slot[u] / kBlock * P.hkv + h) * kBlock + slot[u] % kBlock;
    if (is_v) {   // a bit copy
      T* dst = static_cast<T*>(P.v_cache) + to * D;
      *reinterpret_cast<uint4*>(dst + ca) = xa[u];
      *reinterpret_cast<uint4*>(dst + cb) = xb[u];
      continue;
    }
    if (l < rl) {
      const float4* cs = s_cs + tok * 4 * rl + l;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 c = cs[e * rl];
        if constexpr (kInter) {
          float2& x = e < 2 ? a[2 * e] : b[2 * e - 4];
          float2& y = e < 2 ? a[2 * e + 1] : b[2 * e - 3];
          x = make_float2(x.x * c.x - x.y * c.z, x.y * c.x + x.x * c.z);
          y = make_float2(y.x * c.y - y.y * c.w, y.y * c.y + y.x * c.w);
        } else {
          const float2 co = make_float2(c.x, c.y), si = make_float2(c.z, c.w), ns = make_float2(-c.z, -c.w);
          const float2 x = a[e];
          a[e] = fma2(x, co, mul2(b[e], ns));
          b[e] = fma2(b[e], co, mul2(x, si));
        }
      }
    }
    if (is_q || !kFp8) {
      T* dst = static_cast<T*>(is_q ? P.q_out : P.k_cache) + to * D;
      *reinterpret_cast<uint4*>(dst + ca) = make_uint4(pack2<T>(a[0].x, a[0].y), pack2<T>(a[1].x, a[1].y),
                                                       pack2<T>(a[2].x, a[2].y), pack2<T>(a[3].x, a[3].y));
      *reinterpret_cast<uint4*>(dst + cb) = make_uint4(pack2<T>(b[0].x, b[0].y), pack2<T>(b[1].x, b[1].y),
                                                       pack2<T>(b[2].x, b[2].y), pack2<T>(b[3].x, b[3].y));
    } else {
      const float inv = 1.0f / P.k_scale[h];
      uint32_t qa[4], qb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qa[e] = float2_to_e4m3x2(a[e].x * inv, a[e].y * inv);
        qb[e] = float2_to_e4m3x2(b[e].x * inv, b[e].y * inv);
      }
      uint8_t* dst = static_cast<uint8_t*>(P.k_cache) + to * D;
      *reinterpret_cast<uint2*>(dst + ca) = make_uint2(qa[0] | qa[1] << 16, qa[2] | qa[3] << 16);
      *reinterpret_cast<uint2*>(dst + cb) = make_uint2(qb[0] | qb[1] << 16, qb[2] | qb[3] << 16);
    }
  }
}

int rope_cache_write_launch(const RopeArgs& a, std::string* why) {
  const bool fp8 = a.k_scale != nullptr;
  const int64_t heads = a.num_q_heads + (fp8 ? 1 : 2) * static_cast<int64_t>(a.num_kv_heads);
  const int64_t v_ctas = fp8 ? (static_cast<int64_t>(a.num_tokens) + kVTokens - 1) / kVTokens * a.num_kv_heads : 0;
  const int64_t far = 1ll << 30;   // strides, rows and CTAs in 32 bits
  if (heads * a.num_tokens > far || v_ctas > far || a.q_stride > far || a.q_stride < -far || a.k_stride > far ||
      a.k_stride < -far || a.v_stride > far || a.v_stride < -far) {
    *why = "rope_cache_write: more than 2^30 (token, head) rows or a token stride past 2^30";
    return 3;
  }
  RopeParams P;
  P.q = a.q;
  P.k = a.k;
  P.v = a.v;
  P.q_stride = static_cast<int>(a.q_stride);
  P.k_stride = static_cast<int>(a.k_stride);
  P.v_stride = static_cast<int>(a.v_stride);
  P.positions = a.positions;
  P.slots = a.slot_mapping;
  P.inv_freq = a.inv_freq;
  P.q_norm = a.q_norm;
  P.k_norm = a.k_norm;
  P.q_out = a.q_out;
  P.k_cache = a.k_cache;
  P.v_cache = a.v_cache;
  P.k_scale = a.k_scale;
  P.v_scale = a.v_scale;
  P.num_blocks = a.num_blocks;
  P.heads = static_cast<int>(heads);
  P.tokens = a.num_tokens;
  P.rows = static_cast<int>(heads * a.num_tokens);
  P.hq = a.num_q_heads;
  P.hkv = a.num_kv_heads;
  P.rotary = a.rotary_dim;
  P.factor = a.attn_factor;
  P.eps = a.norm_eps;
  const int groups = kRopeThreads / (a.head_dim / 16);
  P.step_tokens = groups / P.heads;
  P.step_heads = groups % P.heads;
  const int rows = groups * kRopeRows;
  P.row_ctas = (P.rows + rows - 1) / rows;
  // a CTA's rows begin within a token: at most (rows - 2) / heads + 2 tokens
  size_t smem = static_cast<size_t>((rows - 2) / P.heads + 2) * (a.rotary_dim / 2) * sizeof(float2);
  constexpr size_t v_smem = kVTokens * (128 + 16 + sizeof(int64_t) + sizeof(int));
  if (fp8 && smem < v_smem) smem = v_smem;
  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(P.row_ctas + v_ctas)), dim3(kRopeThreads), smem, s, P);
  };
  auto pick = [&](auto t, auto inter, auto norm) {
    using T = decltype(t);
    constexpr bool kI = decltype(inter)::value, kN = decltype(norm)::value;
    return fp8                 ? go(rope_cache_write_kernel<T, 128, kI, true, kN>)
           : a.head_dim == 128 ? go(rope_cache_write_kernel<T, 128, kI, false, kN>)
                               : go(rope_cache_write_kernel<T, 64, kI, false, kN>);
  };
  auto pick_norm = [&](auto t, auto inter) {
    return a.q_norm || a.k_norm ? pick(t, inter, std::true_type()) : pick(t, inter, std::false_type());
  };
  auto pick_layout = [&](auto t) {
    return a.interleaved ? pick_norm(t, std::true_type()) : pick_norm(t, std::false_type());
  };
  cudaError_t e = a.dtype == 1 ? pick_layout(__nv_bfloat16()) : pick_layout(__half());
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("rope_cache_write launch: ") + cudaGetErrorString(e);
    return 5;
  }
  return 0;
}

}  // namespace pa
