// Rotary positions: the cos/sin table and the rotation of query or key heads.
//
// Pair i of a head turns by theta = position * f_i, f_i = base^(-2 i / rot):
//   (a, b) -> (a cos - b sin, b cos + a sin), pairs (i, i + rot/2) or (2i, 2i + 1); dims from rot
// on are copied. Angles of far positions need more than float32 holds (position 100000 has 7 bits
// left for the fraction of a radian), so the table is computed in 64 bits, once, and rounded to
// float32; the rotation reads it.
// Bound: memory. 8192 tokens of 64 float32 heads, out of a fused projection: 78 us, 6.9 TB/s; one token is
// a launch (2.8 us).
#include <cuda_bf16.h>
#include <math.h>

#include "attn.h"
#include "internal.h"

namespace w4a16 {
namespace {

// Frequency of pair i. scaling 1 divides every frequency by `factor`; scaling 2 (YaRN, Peng et
// al., "YaRN: Efficient Context Window Extension of Large Language Models", 2023) keeps the pairs
// that turn more than beta_fast times within `original` positions, divides those that turn less
// than beta_slow times, and blends linearly in between.
// What depends on no pair is computed by the host: log2(base), and the ramp's borders.
struct RopeFreq {
  int rot, scaling;
  double log2_base, factor, low, high;
  __device__ double operator()(int i) const {
    const double f = exp2(-2.0 * i / rot * log2_base);
    if (scaling == 1) return f / factor;
    if (scaling != 2) return f;
    const double w = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
    return f * (1.0 - w) + f / factor * w;
  }
};
RopeFreq rope_freq(const RopeTableArgs& a) {
  RopeFreq r = {a.rot, a.scaling, log2(a.base), a.factor, 0.0, 0.0};
  if (a.scaling == 2) {
    const double two_pi = 6.283185307179586476925, l2 = 2.0 * log(a.base);
    r.low = fmax(floor(a.rot * log(a.original / (two_pi * a.beta_fast)) / l2), 0.0);
    r.high = fmin(ceil(a.rot * log(a.original / (two_pi * a.beta_slow)) / l2), (double)(a.rot - 1));
  }
  return r;
}

// A CTA fills kRun positions of kTablePairs pairs. A 64-bit sincos costs some 50 times what an entry may
// (FP64 runs at 1/64 of the FP32 rate here: one sincos per entry took 2317 us for 131072 x 32 entries, 5 us
// being the time to write them; this way 25 us), so only the run's first position and the angle of one position get one;
// the entries in between are products of rotations, e^(i (x + y)) = e^(i x) e^(i y):
//   fine[v] = rotation by v positions, v = 0 .. 32, and coarse[u] = gain * rotation by first + 32 u, u = 0 .. 15,
//   by doubling in 64 bits (chains of at most 10 products: error 2^-49);
//   entry (32 u + v) = coarse[u] * fine[v] in pairs of float32 (each factor hi + lo, products exact by FMA),
//   error about 2^-45 before the one rounding to float32.
constexpr int kTablePairs = 32, kFine = 32, kCoarse = 16, kRun = kFine * kCoarse;

__device__ __forceinline__ double2 turn_by(double2 a, double2 b) {
  return make_double2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}
// a b - c d, each given as hi + lo: products exact by FMA (Ogita, Rump, Oishi, "Accurate Sum and Dot Product", 2005),
// their difference by Knuth's exact sum ("The Art of Computer Programming", vol. 2, 4.2.2).
__device__ __forceinline__ float diff_of_products(float ah, float al, float bh, float bl, float ch, float cl, float dh,
                                                  float dl) {
  const float p = __fmul_rn(ah, bh), pl = fmaf(ah, bl, fmaf(al, bh, fmaf(ah, bh, -p)));
  const float q = __fmul_rn(ch, dh), ql = fmaf(ch, dl, fmaf(cl, dh, fmaf(ch, dh, -q)));
  const float d = __fsub_rn(p, q), t = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, t)), __fadd_rn(q, t));
  return __fadd_rn(d, __fadd_rn(e, __fsub_rn(pl, ql)));
}
__device__ __forceinline__ float4 split(double2 z) {  // (cos hi, cos lo, sin hi, sin lo)
  const float ch = (float)z.x, sh = (float)z.y;
  return make_float4(ch, (float)(z.x - ch), sh, (float)(z.y - sh));
}

__global__ void __launch_bounds__(256)
    rope_table_kernel(float2* __restrict__ table, const int P, const RopeFreq freq, const double gain) {
  __shared__ double2 fine[kFine + 1][kTablePairs], coarse[kCoarse][kTablePairs];
  __shared__ float4 coarse_f[kCoarse][kTablePairs];
  const int half = freq.rot / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = blockIdx.x * kRun, pair = blockIdx.y * kTablePairs + lane;
  if (warp < 2) {
    const double f = freq(min(pair, half - 1));
    double s, c;
    sincos(warp == 0 ? f : (double)first * f, &s, &c);
    if (warp == 0) {
      fine[0][lane] = make_double2(1.0, 0.0);
      fine[1][lane] = make_double2(c, s);
    } else {
      coarse[0][lane] = make_double2(c * gain, s * gain);
    }
  }
  __syncthreads();
  for (int k = 1; k < kFine; k *= 2) {
    for (int v = 1 + warp; v <= k; v += 8) fine[k + v][lane] = turn_by(fine[k][lane], fine[v][lane]);
    __syncthreads();
  }
  double2 step = fine[kFine][lane];  // rotation by 32 k positions
  for (int k = 1; k < kCoarse; k *= 2) {
    for (int u = warp; u < k; u += 8) coarse[k + u][lane] = turn_by(coarse[u][lane], step);
    step = turn_by(step, step);
    __syncthreads();
  }
  for (int u = warp; u < kCoarse; u += 8) coarse_f[u][lane] = split(coarse[u][lane]);
  __syncthreads();
  if (pair >= half) return;
  for (int v = warp; v < kFine; v += 8) {
    const float4 y = split(fine[v][lane]);
#pragma unroll 4
    for (int u = 0; u < kCoarse; ++u) {
      const int p = first + u * kFine + v;
      if (p >= P) break;
      const float4 x = coarse_f[u][lane];
      const float c = diff_of_products(x.x, x.y, y.x, y.y, x.z, x.w, y.z, y.w);
      const float s = diff_of_products(x.x, x.y, y.z, y.w, x.z, x.w, -y.x, -y.y);
      table[(long long)p * half + pair] = make_float2(c, s);
    }
  }
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  float v[4];
  __device__ void load(const float* p) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
  __device__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  float v[8];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ void store(__nv_bfloat16* p) const {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ void turn(float& a, float& b, float2 cs, float sign) {
  const float s = sign * cs.y;
  const float p = fmaf(a, cs.x, -(b * s));
  b = fmaf(b, cs.x, a * s);
  a = p;
}

enum RopeMode { kPairs, kHalvesVec, kHalvesScalar };

// A thread owns one slot of the head -- a 16-byte vector (pairs side by side), two vectors rot/2
// apart (halves), or one pair or element where rot/2 is no whole number of vectors -- for kHeads
// heads of a token, so the table's entries are read once for kHeads rotations and kHeads loads are
// in flight. Every element is read and written by the same thread, so y may be x. What is only copied goes
// through no arithmetic: a turn by (1, 0) would make infinity's partner NaN and lose the sign of zeros.
constexpr int kHeads = 4;

template <typename T, RopeMode MODE>
__global__ void __launch_bounds__(256)
    rope_kernel(const T* x, HeadStrides xs, T* y, HeadStrides ys, int tokens, int H, int D,
                RopeArgs r, float sign, unsigned int* err) {
  constexpr int N = Vec<T>::N;
  const int half = r.rot / 2;
  const int turned = MODE == kPairs ? (r.rot + N - 1) / N : MODE == kHalvesVec ? half / N : half;
  const int slots = MODE == kPairs ? D / N
                    : MODE == kHalvesVec ? turned + (D - r.rot) / N : D - half;
  const int hgroups = (H + kHeads - 1) / kHeads;
  const long long total = (long long)tokens * hgroups * slots;
  for (long long idx = blockIdx.x * (long long)blockDim.x + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * blockDim.x) {
    const long long th = idx / slots;
    const int slot = (int)(idx - th * slots);
    const long long t = th / hgroups;
    const int h0 = (int)(th - t * hgroups) * kHeads;
    int pos = r.positions[t];
    const bool bad = pos < 0 || pos >= r.P;
    if (bad) {
      if (slot == 0 && err) atomicCAS(err, 0u, 1u);  // W4A16_ERR_ARG: the token is copied as it is
      pos = 0;
    }
    const float2* tab = reinterpret_cast<const float2*>(r.table) + (long long)pos * half;
    const T* xp = x + t * xs.token + h0 * xs.head;
    T* yp = y + t * ys.token + h0 * ys.head;
    const bool rotate = slot < turned && !bad;
    if constexpr (MODE == kHalvesScalar) {
      const int d = slot < half ? slot : slot + half;  // second halves belong to the first's slot
      const float2 cs = rotate ? tab[slot] : make_float2(1.0f, 0.0f);
      for (int h = 0; h < kHeads && h0 + h < H; ++h) {
        if (slot < half) {
          float a = to_f(xp[h * xs.head + d]), b = to_f(xp[h * xs.head + d + half]);
          if (rotate) turn(a, b, cs, sign);
          yp[h * ys.head + d] = from_f<T>(a);
          yp[h * ys.head + d + half] = from_f<T>(b);
        } else {
          yp[h * ys.head + d] = xp[h * xs.head + d];
        }
      }
    } else if constexpr (MODE == kHalvesVec) {
      if (slot < turned) {
        const int d = slot * N;
        float2 cs[N];
#pragma unroll
        for (int j = 0; j < N; ++j) cs[j] = rotate ? tab[d + j] : make_float2(1.0f, 0.0f);
        Vec<T> a[kHeads], b[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (h0 + h < H) {
            a[h].load(xp + h * xs.head + d);
            b[h].load(xp + h * xs.head + d + half);
          }
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (h0 + h < H) {
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (rotate) turn(a[h].v[j], b[h].v[j], cs[j], sign);
            a[h].store(yp + h * ys.head + d);
            b[h].store(yp + h * ys.head + d + half);
          }
      } else {
        const int d = r.rot + (slot - turned) * N;
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (h0 + h < H) {
            Vec<T> a;
            a.load(xp + h * xs.head + d);
            a.store(yp + h * ys.head + d);
          }
      }
    } else {
      const int d = slot * N;
      float2 cs[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        cs[j] = rotate && d / 2 + j < half ? tab[d / 2 + j] : make_float2(1.0f, 0.0f);
      Vec<T> a[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h0 + h < H) a[h].load(xp + h * xs.head + d);
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h0 + h < H) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j)
            if (rotate && d / 2 + j < half) turn(a[h].v[2 * j], a[h].v[2 * j + 1], cs[j], sign);
          a[h].store(yp + h * ys.head + d);
        }
    }
  }
}

cudaError_t grid_for(long long total, int block, int* grid) {
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  long long b = (total + block - 1) / block;
  const long long cap = (long long)di.sm_count * 64;
  *grid = (int)(b > cap ? cap : b);
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_rope_t(const T* x, HeadStrides xs, T* y, HeadStrides ys, int tokens, int H,
                          int D, const RopeArgs& r, bool inverse, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int hgroups = (H + kHeads - 1) / kHeads;
  const float sign = inverse ? -1.0f : 1.0f;
  unsigned int* err = device_error_word();
  int grid = 0, slots;
  const bool vec = (r.rot / 2) % N == 0;
  if (r.interleaved) slots = D / N;
  else slots = vec ? r.rot / 2 / N + (D - r.rot) / N : D - r.rot / 2;
  const cudaError_t e = grid_for((long long)tokens * hgroups * slots, 256, &grid);
  if (e != cudaSuccess) return e;
  if (r.interleaved)
    rope_kernel<T, kPairs><<<grid, 256, 0, s>>>(x, xs, y, ys, tokens, H, D, r, sign, err);
  else if (vec)
    rope_kernel<T, kHalvesVec><<<grid, 256, 0, s>>>(x, xs, y, ys, tokens, H, D, r, sign, err);
  else
    rope_kernel<T, kHalvesScalar><<<grid, 256, 0, s>>>(x, xs, y, ys, tokens, H, D, r, sign, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(float* table, const RopeTableArgs& a, cudaStream_t s) {
  const dim3 grid((a.P + kRun - 1) / kRun, (a.rot / 2 + kTablePairs - 1) / kTablePairs);
  rope_table_kernel<<<grid, 256, 0, s>>>(reinterpret_cast<float2*>(table), a.P, rope_freq(a), a.gain);
  return cudaGetLastError();
}

cudaError_t launch_rope(const void* x, HeadStrides xs, void* y, HeadStrides ys, bool bf16, int T,
                        int H, int D, const RopeArgs& r, bool inverse, cudaStream_t s) {
  if (bf16)
    return launch_rope_t(static_cast<const __nv_bfloat16*>(x), xs, static_cast<__nv_bfloat16*>(y),
                         ys, T, H, D, r, inverse, s);
  return launch_rope_t(static_cast<const float*>(x), xs, static_cast<float*>(y), ys, T, H, D, r,
                       inverse, s);
}

}  // namespace w4a16
