// Appending keys and values to the paged 4-bit cache, the position rotation applied on the way, and
// reading tokens back.
//
// Per token, head and group of 32 dims: r = float32 of the rotated key (or the value as it is),
// scale = bf16(absmax / 7), code = clamp(rint(r / scale), -8, 7) -- the weights' quantizer with a
// 16-bit scale. A code is decided by r, so r must not depend on how it was computed: the rotation
// carries both products' rounding errors along (exact by FMA) and rounds once, which gives the
// float32 nearest to the exact value but for ties within 2^-45 or so.
//
// Bound: memory. A thread owns one packed word (8 dims), four neighbouring threads a group: the
// absmax takes two shuffles, a (token, head) row of codes is written as one contiguous 64-byte
// piece (D = 128), and nothing is staged. A thread keeps its (K or V, head, word) and walks over
// tokens, so that the index arithmetic is done once; quotients are reciprocal products, corrected
// where they are close to a border. 16384 tokens of 8 heads of 128 (bf16, rotated), append and read back: 107 us with
// 64-bit index divisions per word and IEEE quotients, 85 us now (52 + 34). Appending is bound by
// instruction issue (350 a warp and 32 words, most of them the rotation, the exact rounding and the packing,
// at 2.9 per SM cycle, 72 % of the slots) and its loads' latency, reading back by its float32 stores (134 MB, 4.6 TB/s with the loads).
#include <cuda_bf16.h>

#include "attn.h"
#include "internal.h"
#include "kv_layout.h"

namespace w4a16 {
namespace {

// Groups whose largest magnitude is not below this are stored as zeros and flagged: scales stay in
// a range in which attention's products cannot overflow float32.
constexpr uint32_t kKvLimitBits = (127u + 64u) << 23;  // 2^64 as float32

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
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// a * c + b * s, rounded once: products exact as (p + e), by FMA (Ogita, Rump, Oishi, "Accurate Sum and Dot Product",
// 2005), sum exact as (h + l) (Knuth, "The Art of Computer Programming", vol. 2, 4.2.2).
__device__ __forceinline__ float dot2_rn(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float q = __fmul_rn(b, s), qe = __fmaf_rn(b, s, -q);
  const float h = __fadd_rn(p, q);
  const float t = __fsub_rn(h, p);
  const float l = __fadd_rn(__fsub_rn(p, __fsub_rn(h, t)), __fsub_rn(q, t));
  return __fadd_rn(h, __fadd_rn(l, __fadd_rn(pe, qe)));  // (NaN where a product or the sum overflows)
}

// Codes rint(x / s) + 8 for |x / s| < 8, packed. The product with the rounded reciprocal is off by less
// than 2^-19, and the remainder x - n s is exact (n has 4 bits, s 8): only where it is that close to s / 2
// can n be wrong or a tie, and the remainder then tells (ties to even). A float32 quotient, which defines
// the code, never rounds onto a border it is not on: |x - (k + 1/2) s| is 0 or at least ulp(x), which
// moves the quotient by more than half its last place, as s has 8 bits.
__device__ __forceinline__ uint32_t pack_codes(const float (&x)[8], float s) {
  const float kMagic = 12582920.0f;  // 1.5 * 2^23 + 8: adding it rounds to an integer, ties to even
  const float inv = __frcp_rn(s), near = 0.499998f * s, h = 0.5f * s;
  uint32_t word = 0;
  bool close = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = __fmaf_rn(x[j], inv, kMagic);
    close |= fabsf(__fmaf_rn(kMagic - t, s, x[j])) > near;
    word |= (__float_as_uint(t) & 15u) << (4 * j);
  }
  if (close) {
    word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t = __fmaf_rn(x[j], inv, kMagic);
      const float r = __fmaf_rn(kMagic - t, s, x[j]), a = fabsf(r);
      if (a > h || (a == h && (__float_as_uint(t) & 1u))) t += copysignf(1.0f, r);
      word |= (__float_as_uint(t) & 15u) << (4 * j);
    }
  }
  return word;
}

constexpr int kAppendPerSm = 16, kReadPerSm = 32;  // (8 .. 32 and 16 .. 64 measure the same)

// What a thread works on: item (K or V, head, word) of every step-th token from the first. Blocks hold as
// many tokens as 256 threads give items (one, with the items on several block rows, for large heads).
struct TokenItems {
  int first, step;
  bool live;         // (idle threads take part in the shuffles)
  int is_v, head, word;
  __device__ TokenItems(int Hkv, int words_log2) {
    const int items = (2 * Hkv) << words_log2;
    const int row = items < 256 ? items : 256, tokens = 256 / row;
    const int tok = threadIdx.x / row, item = blockIdx.y * 256 + (threadIdx.x - tok * row);
    live = tok < tokens && item < items;
    first = blockIdx.x * tokens + tok;
    step = gridDim.x * tokens;
    const int rest = live ? item : 0;
    is_v = rest >= (Hkv << words_log2);
    const int hw = rest - (is_v ? Hkv << words_log2 : 0);
    head = hw >> words_log2;
    word = hw & ((1 << words_log2) - 1);
  }
};
// Its grid: enough blocks for every token, at most `per_sm` per SM.
cudaError_t token_grid(int T, int Hkv, int D, int per_sm, dim3* grid) {
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int items = 2 * Hkv * (D / 8), tokens = items < 256 ? 256 / items : 1, rows = (items + 255) / 256;
  const int need = (T + tokens - 1) / tokens, cap = di.sm_count * per_sm / (rows < per_sm ? rows : per_sm);
  *grid = dim3(need < cap ? need : cap, rows);
  return cudaSuccess;
}

template <typename T>
__global__ void __launch_bounds__(256, 6)
    kv_append_kernel(const T* __restrict__ k, HeadStrides ks, const T* __restrict__ v,
                     HeadStrides vs, int tokens, const int64_t* __restrict__ slots, RopeArgs r,
                     KvCache c, int words_log2, int page_log2, unsigned int* err) {
  const TokenItems it(c.Hkv, words_log2);
  const int is_v = it.is_v, h = it.head, u = it.word;  // u: word of the head in dim order
  const long long cap = (long long)c.num_pages * c.page_size;
  const int half = r.rot / 2;
  // Whole warps go round together: as often as the block's first token asks for. The next token's slot and
  // position are on their way while one is worked on: nothing but latency bounds this loop.
  auto slot_of = [&](int t) { return it.live && t < tokens ? __ldg(slots + t) : -1ll; };
  auto pos_of = [&](int t) { return r.rot && it.live && t < tokens ? __ldg(r.positions + t) : 0; };
  long long next_slot = slot_of(it.first);
  int next_pos = pos_of(it.first);
  for (int t0 = it.first, left = (tokens - blockIdx.x * (it.step / gridDim.x) + it.step - 1) / it.step; left > 0;
       --left, t0 += it.step) {
    const bool live = it.live && t0 < tokens;
    const long long t = live ? t0 : 0;
    const long long slot = next_slot;
    int pos = next_pos;
    next_slot = slot_of(t0 + it.step);
    next_pos = pos_of(t0 + it.step);
    bool write = slot >= 0;
    bool bad = slot >= cap;
    if (r.rot && (pos < 0 || pos >= r.P)) {
      bad = bad || write;
      pos = 0;
    }
    if (bad) write = false;
    float x[8];
    if (is_v) {
      load8(v + t * vs.token + h * vs.head + 8 * u, x);
    } else {
      const T* kp = k + t * ks.token + h * ks.head;
      load8(kp + 8 * u, x);
      if (8 * u < r.rot) {
        const float2* tab = reinterpret_cast<const float2*>(r.table) + (long long)pos * half;
        if (r.interleaved) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (4 * u + j < half) {
              const float2 cs = __ldg(tab + 4 * u + j);
              const float a = x[2 * j], b = x[2 * j + 1];
              x[2 * j] = dot2_rn(a, cs.x, -b, cs.y);
              x[2 * j + 1] = dot2_rn(b, cs.x, a, cs.y);
            }
          }
        } else if (half % 8 == 0) {
          const bool second = 8 * u >= half;
          const int i0 = second ? 8 * u - half : 8 * u;
          float y[8];
          load8(kp + (second ? i0 : i0 + half), y);
          const float4* tab4 = reinterpret_cast<const float4*>(tab + i0);  // rows of 8 pairs and more
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float4 cs = __ldg(tab4 + j / 2);
            x[j] = dot2_rn(x[j], cs.x, second ? y[j] : -y[j], cs.y);
            x[j + 1] = dot2_rn(x[j + 1], cs.z, second ? y[j + 1] : -y[j + 1], cs.w);
          }
        } else {  // halves that do not fall on whole words
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int d = 8 * u + j;
            if (d < r.rot) {
              const bool second = d >= half;
              const int i = second ? d - half : d;
              const float y = load1(kp + (second ? i : i + half));
              const float2 cs = __ldg(tab + i);
              x[j] = dot2_rn(x[j], cs.x, second ? y : -y, cs.y);
            }
          }
        }
      }
    }
    uint32_t amax_bits = 0;  // of magnitudes, whose bits order as they do; NaN comes out on top
#pragma unroll
    for (int j = 0; j < 8; ++j) amax_bits = max(amax_bits, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    amax_bits = max(amax_bits, __shfl_xor_sync(0xFFFFFFFFu, amax_bits, 1));
    amax_bits = max(amax_bits, __shfl_xor_sync(0xFFFFFFFFu, amax_bits, 2));
    const bool zeroed = amax_bits >= kKvLimitBits;
    if (write && zeroed) bad = true;
    const __nv_bfloat16 sb =
        __float2bfloat16_rn(zeroed ? 0.0f : __fdiv_rn(__uint_as_float(amax_bits), 7.0f));
    const float s = __bfloat162float(sb);
    uint32_t word = 0x88888888u;
    if (s >= 1e-30f) {
      word = pack_codes(x, s);
    } else if (s > 0.0f) {  // scales whose reciprocal or half may not be a normal number
      word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(x[j], s)), -8.0f), 7.0f);  // half to even
        word |= (uint32_t)((int)q + 8) << (4 * j);
      }
    }
    if (bad && err) atomicCAS(err, 0u, 1u);  // W4A16_ERR_ARG
    if (write) {
      const int off = (int)slot & (c.page_size - 1), row = off % kKvBlock, i = u / 4, w = u % 4;
      char* block = static_cast<char*>(c.data) +
                    kv_block_addr(c.D, c.page_size, c.Hkv, slot >> page_log2, h, off);
      *reinterpret_cast<uint32_t*>(block + kv_codes_off(c.D, is_v) +
                                   kv_word_off(c.D, row, w, i)) = word;
      if (w == 0)
        *reinterpret_cast<__nv_bfloat16*>(block + kv_scales_off(c.D, is_v) +
                                          kv_scale_off(c.D, row, i)) = sb;
    }
  }
}

// A thread per packed word again: 8 values of k or v as float32. Slots outside the cache read as zeros.
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvCache c, const int64_t* __restrict__ slots, int tokens, float* __restrict__ k,
                   float* __restrict__ v, int words_log2, int page_log2, unsigned int* err) {
  const TokenItems it(c.Hkv, words_log2);
  const long long cap = (long long)c.num_pages * c.page_size;
  if (!it.live) return;
  float* out = it.is_v ? v : k;
#pragma unroll 4
  for (int t = it.first; t < tokens; t += it.step) {
    const long long slot = __ldg(slots + t);
    uint32_t word = 0x88888888u;
    float s = 0.0f;
    if (slot >= 0 && slot < cap) {
      const int off = (int)slot & (c.page_size - 1), row = off % kKvBlock;
      const char* block = static_cast<const char*>(c.data) +
                          kv_block_addr(c.D, c.page_size, c.Hkv, slot >> page_log2, it.head, off);
      word = __ldg(reinterpret_cast<const uint32_t*>(block + kv_codes_off(c.D, it.is_v) +
                                                     kv_word_off(c.D, row, it.word % 4, it.word / 4)));
      s = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
          block + kv_scales_off(c.D, it.is_v) + kv_scale_off(c.D, row, it.word / 4)));
    } else if (slot >= cap && it.head == 0 && it.word == 0 && err) {
      atomicCAS(err, 0u, 1u);  // W4A16_ERR_ARG
    }
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (float)((int)((word >> (4 * j)) & 15u) - 8) * s;
    float4* dst = reinterpret_cast<float4*>(out + ((((long long)t * c.Hkv + it.head) << words_log2) + it.word) * 8);
    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
  }
}

int log2_of(int v) {  // of a power of two
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

}  // namespace

cudaError_t launch_kv_append(const void* k, HeadStrides ks, const void* v, HeadStrides vs,
                             bool bf16, int T, const int64_t* slots, const RopeArgs& r,
                             const KvCache& c, cudaStream_t s) {
  dim3 grid;
  const cudaError_t e = token_grid(T, c.Hkv, c.D, kAppendPerSm, &grid);
  if (e != cudaSuccess) return e;
  unsigned int* err = device_error_word();
  const int wl = log2_of(c.D / 8), pl = log2_of(c.page_size);
  if (bf16)
    kv_append_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(k), ks,
                                          static_cast<const __nv_bfloat16*>(v), vs, T, slots, r, c, wl, pl,
                                          err);
  else
    kv_append_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(k), ks, static_cast<const float*>(v), vs, T,
                                          slots, r, c, wl, pl, err);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvCache& c, const int64_t* slots, int T, float* k, float* v,
                           cudaStream_t s) {
  dim3 grid;
  const cudaError_t e = token_grid(T, c.Hkv, c.D, kReadPerSm, &grid);
  if (e != cudaSuccess) return e;
  kv_read_kernel<<<grid, 256, 0, s>>>(c, slots, T, k, v, log2_of(c.D / 8), log2_of(c.page_size), device_error_word());
  return cudaGetLastError();
}

}  // namespace w4a16
