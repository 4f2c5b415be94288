// What the attention kernels share: the line of key tiles that is cut into equal runs (Walk), the
// partial results of items cut by a border and their merge, and small device helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "attn.h"
#include "internal.h"
#include "kv_layout.h"
#include "mma_core.cuh"

namespace w4a16 {

// Most CTAs of a launch, which size the workspace: of the kernel for few rows, and of the one for many.
constexpr int kMaxCtas = 1024, kMaxManyCtas = 192;

// Partial results: two slots per CTA, the second for an item that begins in its run, the first for
// one that began before it.
struct Partials {
  struct Start {  // where CTA i's run starts
    int b, h, rt, tile;  // tile > 0: inside an item
    int first;           // the CTA in which that item begins
    int last;            // and the one in which it ends
  };
  Start* start;  // [grid]
  float* lse2;   // [2 * grid, rows]
  float* o;      // [2 * grid, rows, D], normalised
  int rows;

  static size_t bytes(int rows, int D, int ctas) {
    return ctas * sizeof(Start) + (size_t)2 * ctas * rows * (D + 1) * sizeof(float);
  }
  static Partials at(void* ws, int rows, int D, int ctas) {
    Partials p;
    p.o = static_cast<float*>(ws);
    p.lse2 = p.o + (size_t)2 * ctas * rows * D;
    p.start = reinterpret_cast<Start*>(p.lse2 + (size_t)2 * ctas * rows);
    p.rows = rows;
    return p;
  }
};

namespace attn {

// V scales enter the weights as p * scale * 2^bias with bias = kBias - (exponent field of the largest
// scale), which keeps the product below 2^15; the field is clamped so that float32 sums of p * 2^bias
// stay far from overflow (scales under 2^-56 lose bits, none above 2^74 are ever appended).
constexpr int kBias = 141;
constexpr int kMinScaleExp = 70, kMaxScaleExp = 200;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Transpose of an 8 x 8 matrix of 16-bit values held as MMA fragments (lane (g, t): row g, columns
// 2t, 2t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(a));
  return r;
}
// 2^x: relative error 2^-22, results under 2^-126 are zero.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// Bytes (multiple of 16, both addresses 16-byte aligned) from global to shared memory, completing on
// an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = mma::lds128(addr + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    static_assert(N == 1);
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w[0]) : "r"(addr));
  }
}
// Element i of packed bf16 values, as float32.
template <int N>
__device__ __forceinline__ float bf16_of(const uint32_t (&w)[N], int i) {
  return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = bf16_of(w, j);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
// (x, y) as fp16 pairs: one term, or hi + lo.
template <int TERMS>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[TERMS]) {
  const __half2 h = __floats2half2_rn(x, y);
  out[0] = *reinterpret_cast<const uint32_t*>(&h);
  if constexpr (TERMS == 2) {
    const float2 b = __half22float2(h);
    const __half2 lo = __floats2half2_rn(x - b.x, y - b.y);
    out[1] = *reinterpret_cast<const uint32_t*>(&lo);
  }
}
// Nibbles as fp16 bit patterns: n * 2^-24, or 16 n * 2^-24 for the odd ones (all under 0x0400:
// subnormals).
constexpr float kRawUnit = 16777216.0f;
__device__ __forceinline__ void raw_word(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t w8 = w >> 8;
  p[0] = w & 0x000F000Fu;
  p[1] = w & 0x00F000F0u;
  p[2] = w8 & 0x000F000Fu;
  p[3] = w8 & 0x00F000F0u;
}
// The operand order of mma::unpack_pair.
__device__ __forceinline__ void raw_pair(uint32_t wa, uint32_t wb, uint32_t (&a0)[4], uint32_t (&a1)[4]) {
  uint32_t x[4], y[4];
  raw_word(wa, x);
  raw_word(wb, y);
  a0[0] = x[0], a0[1] = y[0], a0[2] = x[1], a0[3] = y[1];
  a1[0] = x[2], a1[1] = y[2], a1[2] = x[3], a1[3] = y[3];
}
__device__ __forceinline__ float2 half2_of(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// (x, y) as three bf16 pairs whose sum is exact: 8 of the 24 bits each, cut off, not rounded.
__device__ __forceinline__ void split_pair3(float x, float y, uint32_t (&out)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    out[k] = prmt(__float_as_uint(x), __float_as_uint(y), 0x7632u);
    x -= __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    y -= __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
  }
}
// Word -> four bf16x2 registers of (nibble - 8): (n0, n4), (n1, n5), (n2, n6), (n3, n7).
__device__ __forceinline__ void unpack_word_bf16(uint32_t w, uint32_t (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(v) : "r"(w >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;\n" : "=r"(p[j]) : "r"(v), "r"(0x3F803F80u), "r"(0xC308C308u));
  }
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Exponent e of a row whose largest magnitude is amax: amax * 2^(14 - e) is in [2^14, 2^15), for
// amax from 2^-100 on (below, and for zero, e = -100).
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127;
  return e < -100 ? -100 : (e > 127 ? 127 : e);
}
__device__ __forceinline__ bool draft_bit(const AttnArgs& a, int token, int d) {
  return d < 32 * a.mask_words &&
         ((__ldg(a.mask + (long long)token * a.mask_words + (d >> 5)) >> (d & 31)) & 1u);
}

// An item's fixed cost, in tiles: its first loads, its queries and its merge take about as long as 12
// tiles of the CTA's stream (few rows), or 4 of the larger tiles (many rows). Without it a run of many
// short sequences took twice as long as one of a long sequence: 64 sequences of 100 .. 16384 keys took
// 97 us without, 71, 68, 64 and 68 us with 6, 10, 16 and 24.
constexpr int kItemCost = 12, kManyItemCost = 4;

// The line: sequences in order; within one, heads; within a head, row tiles; within a row tile, the
// tiles of keys that any of its rows sees (one empty tile where there are none, so that its rows are
// written), after kItemCost places that stand for the item's fixed cost. Sequences whose rows are not in
// (min_rows, max_rows] belong to another kernel. All threads of a CTA walk together: total() and seek() contain barriers.
template <int tile_keys, int R, int cost>
struct Walk {
  const AttnArgs& a;
  const int max_tokens, max_rows, min_rows, Hkv;
  unsigned int* err;
  int b = -1, h = 0, rt = 0;                 // position
  KvSeq s = {0, 0, 0};                       // sequence b
  int lo = 0, hi = 0, tiles = 0;             // of row tile rt: keys [lo, hi) that any of its rows may see
  long long tile0 = 0;                       // place of the item's tile 0 on the line

  __device__ Walk(const AttnArgs& a_, int page_size, int max_rows_, int min_rows_, int Hkv_, unsigned int* err_)
      : a(a_), max_tokens(a_.max_pages * page_size), max_rows(max_rows_), min_rows(min_rows_), Hkv(Hkv_),
        err(err_) {}

  // Sequence i, with n = 0 if it is not this kernel's.
  __device__ KvSeq sequence(int i) {
    bool bad = false;
    KvSeq q = kv_sequence(__ldg(a.q_starts + i), __ldg(a.q_starts + i + 1), __ldg(a.kv_lens + i),
                          a.T, max_tokens, &bad);
    if (q.n > a.max_q) {
      bad = true;
      q.n = 0;
    }
    if (bad && err) atomicCAS(err, 0u, 1u);  // W4A16_ERR_ARG
    const long long rows = (long long)q.n * a.G;
    if (rows > max_rows || rows <= min_rows) q.n = 0;
    return q;
  }
  __device__ int row_tiles(const KvSeq& q) const { return (q.n * a.G + R - 1) / R; }
  __device__ void range(const KvSeq& q, int r, int* lo, int* end) const {
    const int i0 = r * R / a.G, i1 = (min((r + 1) * R, q.n * a.G) - 1) / a.G;
    *lo = kv_lo(q, i0, a.window);
    *end = kv_hi(q, i1, a.causal, a.mask != nullptr);
  }
  static __device__ int first_key(int lo) { return lo & -tile_keys; }  // of tile 0
  __device__ int tiles_of(const KvSeq& q, int r) const {
    int lo, end;
    range(q, r, &lo, &end);
    lo = first_key(lo);
    return end > lo ? (end - lo + tile_keys - 1) / tile_keys : 1;
  }
  __device__ long long head_units(const KvSeq& q) const {
    long long u = 0;
    const int n = row_tiles(q);
    for (int r = 0; r < n; ++r) u += cost + tiles_of(q, r);
    return u;
  }

  // Sum over the CTA's threads, returned to all.
  static __device__ long long cta_sum(long long v) {
    __shared__ long long parts[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) parts[warp] = v;
    __syncthreads();
    long long r = 0;
    for (int i = 0; i < (int)(blockDim.x + 31) / 32; ++i) r += parts[i];
    __syncthreads();
    return r;
  }
  __device__ long long total() {
    long long u = 0;
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) u += head_units(sequence(i)) * Hkv;
    return cta_sum(u);
  }
  // Goes to the item at place `at` of the line (at < total()).
  __device__ void seek(long long at) {
    __shared__ long long found[2];
    long long base = 0;
    const int lane = threadIdx.x & 31;
    // one warp's worth of sequences at a time, every warp the same: no barrier until one is found
    for (int i0 = 0; i0 < a.B; i0 += 32) {
      const int i = i0 + lane;
      const long long u = i < a.B ? head_units(sequence(i)) * Hkv : 0;
      long long inc = u;
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, base + inc > at);
      if (past) {
        const int k = __ffs(past) - 1;
        if (threadIdx.x == k) found[0] = i0 + k, found[1] = base + inc - u;
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    __syncthreads();
    b = (int)found[0];
    long long u = found[1];
    s = sequence(b);
    const long long per_head = head_units(s);
    h = (int)((at - u) / per_head);
    u += h * per_head;
    rt = 0;
    for (;;) {
      tiles = tiles_of(s, rt);
      if (u + cost + tiles > at) break;
      u += cost + tiles;
      ++rt;
    }
    tile0 = u + cost;
    range(s, rt, &lo, &hi);
  }
  // To the item after this one (there is one).
  __device__ void next_item() {
    tile0 += tiles + cost;
    if (++rt == row_tiles(s)) {
      rt = 0;
      if (++h == Hkv) {
        h = 0;
        do s = sequence(++b);
        while (s.n == 0 && b + 1 < a.B);
      }
    }
    tiles = tiles_of(s, rt);
    range(s, rt, &lo, &hi);
  }
  // Tile of the item at or after place `at`.
  __device__ int tile_at(long long at) const {
    const long long t = at - tile0;
    return t < 0 ? 0 : (t > tiles ? tiles : (int)t);
  }
  __device__ Partials::Start start(long long at, long long per) const {
    return {b, h, rt, tile_at(at), (int)(tile0 / per), (int)((tile0 + tiles - 1) / per)};
  }
};

}  // namespace attn

// CTA column i merges the item that the run of CTA i starts inside of, if that item began in CTA
// i - 1 (so each cut item is merged once): the piece in slot 2 (i - 1) + 1, then those in slots 2 i,
// 2 (i + 1), ... One CTA per row (gridDim.y strides over them): its 128 threads first turn the
// pieces' statistics into weights, then every D/4 threads add a share of the pieces, and the shares
// are added in order. An item may be cut into hundreds of pieces (one sequence on the whole GPU):
// with a thread adding all of a row's 57 pieces one after the other this took 29 us.
constexpr int kMergeThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads)
    attn_merge_kernel(const AttnArgs a, const Partials p, const int D) {
  __shared__ float weight[kMergeThreads];
  __shared__ float red[2][kMergeThreads / 32];
  __shared__ float4 share[kMergeThreads];
  const Partials::Start st = p.start[blockIdx.x];
  if (st.tile == 0 || st.first != (int)blockIdx.x - 1) return;
  const int R = p.rows, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int q0 = max(__ldg(a.q_starts + st.b), 0), n = min(__ldg(a.q_starts + st.b + 1), a.T) - q0;
  const int r0 = st.rt * R, rows = min(R, n * a.G - r0);
  const int per_row = D / 4, shares = kMergeThreads / per_row;
  const int pieces = st.last - st.first + 1;
  auto slot = [&](int k) { return 2 * (st.first + k) + (k == 0 ? 1 : 0); };
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    // largest statistic of the row; a NaN row stays NaN
    float top = -CUDART_INF_F, bad = 0.0f;
    for (int k = tid; k < pieces; k += kMergeThreads) {
      const float v = p.lse2[(long long)slot(k) * R + r];
      top = fmaxf(top, v);
      if (v != v) bad = v;
    }
    for (int o = 16; o; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      bad += __shfl_xor_sync(0xFFFFFFFFu, bad, o);
    }
    __syncthreads();  // the previous row is done with shared memory
    if (lane == 0) red[0][warp] = top, red[1][warp] = bad;
    __syncthreads();
    for (int k = 0; k < kMergeThreads / 32; ++k) top = fmaxf(top, red[0][k]), bad += red[1][k];
    if (top == -CUDART_INF_F) top = 0.0f;
    top += bad;
    const int d4 = tid % per_row, part = tid / per_row;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int k0 = 0; k0 < pieces; k0 += kMergeThreads) {
      const int m = min(kMergeThreads, pieces - k0);
      if (k0) __syncthreads();
      if (tid < m) weight[tid] = attn::ex2(p.lse2[(long long)slot(k0 + tid) * R + r] - top);
      __syncthreads();
#pragma unroll 8
      for (int k = part; k < m; k += shares) {
        const float f = weight[k];
        const float4 x = reinterpret_cast<const float4*>(p.o)[((long long)slot(k0 + k) * R + r) * per_row + d4];
        sum += f;
        v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
      }
    }
    share[tid] = v;
    __syncthreads();
    weight[tid] = sum;
    __syncthreads();
    if (tid < per_row) {
      for (int k = 1; k < shares; ++k) {
        const float4 x = share[k * per_row + tid];
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        sum += weight[k * per_row + tid];
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
      const int i = (r0 + r) / a.G, hq = (r0 + r) - i * a.G;
      const long long at = (long long)(q0 + i) * a.Hq + st.h * a.G + hq;
      attn::store4(static_cast<T*>(a.out) + at * D + 4 * tid, v);
      if (tid == 0 && a.lse)
        a.lse[at] = (sum == 0.0f ? -CUDART_INF_F : top + log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

// The same for items of many rows and few pieces (the kernel for many rows has one CTA per SM): a warp per
// row, up to 128 dims. 256 rows x 151 cut items took 50 us with a CTA per row, 4096 tokens over 8192 keys.
template <typename T>
__global__ void __launch_bounds__(256) attn_merge_rows_kernel(const AttnArgs a, const Partials p, const int D) {
  const Partials::Start st = p.start[blockIdx.x];
  if (st.tile == 0 || st.first != (int)blockIdx.x - 1) return;
  const int R = p.rows, lane = threadIdx.x & 31, per_row = D / 4;
  const int q0 = max(__ldg(a.q_starts + st.b), 0), n = min(__ldg(a.q_starts + st.b + 1), a.T) - q0;
  const int r0 = st.rt * R, rows = min(R, n * a.G - r0);
  const int pieces = st.last - st.first + 1;
  auto slot = [&](int k) { return 2 * (st.first + k) + (k == 0 ? 1 : 0); };
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 8) {
    float top = -CUDART_INF_F, bad = 0.0f;  // (a NaN row stays NaN)
    for (int k = 0; k < pieces; ++k) {
      const float v = p.lse2[(long long)slot(k) * R + r];
      top = fmaxf(top, v);
      if (v != v) bad = v;
    }
    if (top == -CUDART_INF_F) top = 0.0f;
    top += bad;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int k = 0; k < pieces; ++k) {
      const float f = attn::ex2(p.lse2[(long long)slot(k) * R + r] - top);
      const float4 x = lane < per_row
                           ? reinterpret_cast<const float4*>(p.o)[((long long)slot(k) * R + r) * per_row + lane]
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      sum += f;
      v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y);
      v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    const int i = (r0 + r) / a.G, hq = (r0 + r) - i * a.G;
    const long long at = (long long)(q0 + i) * a.Hq + st.h * a.G + hq;
    if (lane < per_row) attn::store4(static_cast<T*>(a.out) + at * D + 4 * lane, v);
    if (lane == 0 && a.lse)
      a.lse[at] = (sum == 0.0f ? -CUDART_INF_F : top + log2f(sum)) * 0.69314718055994530942f;
  }
}

template <typename T>
cudaError_t launch_attn_merge_rows(const AttnArgs& a, const Partials& p, int grid, int D, cudaStream_t s) {
  attn_merge_rows_kernel<T><<<dim3(grid, 16), 256, 0, s>>>(a, p, D);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_attn_merge(const AttnArgs& a, const Partials& p, int grid, int D, cudaStream_t s) {
  attn_merge_kernel<T><<<dim3(grid, p.rows), kMergeThreads, 0, s>>>(a, p, D);
  return cudaGetLastError();
}

// Sequences of at most max_rows rows per key/value head; those of more than min_rows.
cudaError_t launch_attn_few(const AttnArgs& a, const KvCache& c, int max_rows, void* ws, cudaStream_t s);
cudaError_t launch_attn_many(const AttnArgs& a, const KvCache& c, int min_rows, void* ws, cudaStream_t s);

}  // namespace w4a16
