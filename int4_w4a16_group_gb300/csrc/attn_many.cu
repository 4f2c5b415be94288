// Attention over the paged 4-bit cache for many query rows per key/value head (prompts, large
// drafts), bf16 activations, on the 5th-generation tensor cores.
//
// An item is (sequence, head, tile of 256 rows = two row tiles of 128), a row being one (query token,
// query head) of the key/value head's group; it walks its visible keys 128 at a time:
//   S = Q K'^T (128 x 128, into TMEM), softmax of S by one thread per row, P back into S's columns,
//   O += P V' (TMEM). While one row tile is in the softmax the tensor core works on the other.
// K' and V' are codes times scales as fp16: a code has 4 bits and a scale 8, so the product is exact;
// a power of two per tile of keys (K) and per item (V, kept until a larger scale comes) holds them
// below 2^15 whatever the scales are. Queries are exact in fp16 after a power of two per row. P is
// fp16 below 2^15: the maximum that is subtracted lags by up to 8 binades (2^7 .. 2^15 at the top), so
// O (and the tile's earlier P, by a factor rounded to fp16 and rounded once more, 2 x 2^-11, where the output's
// own rounding is 2^-8; the sum takes the exact factor) is rescaled only when a row's maximum has grown
// by more than that. Weights under 2^-31 of a row's largest lose bits. Sums are float32.
//
// Roles (640 threads, one CTA per SM, persistent over an equal run of the line of key tiles):
//   warps 0-7   softmax, four per row tile (TMEM lane = row); queries in, outputs out;
//   warps 8-15  dequantize: raw blocks -> K' (key rows) and V'^T (dim rows), both K-major with the
//               128-byte swizzle, into a ring of three 128 x D tiles (K0 V0 K1 V1 ...);
//   warp 16     bulk copies of raw blocks (one contiguous piece per 16 keys) into a ring of three stages,
//               and each tile's largest scales;
//   warp 17     issues the MMAs: per key tile and row tile P V' of this tile, then S of the next, which
//               overwrites the P just used (MMAs of one thread run in order).
//
// What bounds it: the chain of hand-offs. 4096 tokens over 8192 keys, 64 query and 8 key/value heads of 128: 799 us,
// 1032 TFLOP/s, 0.54 of the measured bf16 rate; the tensor pipe is busy for 45 % of the cycles. A key tile takes some
// 4200 cycles where its MMAs take 2050: a row tile's softmax (2600) and its MMAs with their two hand-offs (1700)
// follow one another, and only the other row tile's overlap them. 59 % of the issue slots are used; of the 8.5 cycles
// that a warp takes per instruction, 2.8 go to loads of long latency, 1.2 to the latency of the instruction before, 0.9
// to barriers, 0.35 to fetching instructions. A change of items takes 11000 cycles,
// of which the queries' loads are 4600.
// The dims of K' and Q are stored in the order the nibbles unpack in (0 4 1 5 2 6 3 7), and the keys of
// V' and P rotated within each 8 by the chunk's index, so that neither side reorders anything and the
// reads of V's rows fall on different banks.
#include <limits.h>
#include <math_constants.h>

#include "attn_core.cuh"
#include "tc_core.cuh"

namespace w4a16 {
namespace {

using namespace mma;
using namespace attn;

constexpr int kRows = 128;       // rows of a row tile (TMEM lanes)
constexpr int kKeys = 128;       // keys of a tile
constexpr int kSoftWarps = 8, kDeqWarps = 8;
constexpr int kDeqWarp0 = kSoftWarps;
constexpr int kCopyWarp = kDeqWarp0 + kDeqWarps;
constexpr int kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = (kMmaWarp + 3) * 32;  // whole groups of four warps share a register count
// Registers a thread: 96 at launch (640 threads), then moved from the other warps to the softmax.
constexpr int kRegsLaunch = 96, kRegsSoft = 128, kRegsDeq = 64, kRegsRest = 96;
static_assert(kSoftWarps * kRegsSoft + kDeqWarps * kRegsDeq + 4 * kRegsRest <= kThreads / 32 * kRegsLaunch,
              "the warps' shares come out of the launch's registers");
constexpr int kRawStages = 3, kOps = 3, kInfos = 8;
constexpr float kLag = 8.0f;     // binades a row's maximum may grow before O is rescaled
constexpr float kTop = 7.0f;     // P's largest value when it has not grown: 2^7
// Products are below 2^37, so with factors up to this scores stay below 2^20, and the weights multiply and subtract
// in one rounding. With larger ones the unrounded product and the rounded maximum could differ by more binades than a
// weight has room for, so the scores are rounded first, in a pass of their own. (Two roundings for all cost 841 .. 859
// us where one takes 795, the test for this pass 802: 4096 tokens over 8192 keys.)
constexpr float kFusedFactor = 0x1p-17f;

template <int NG>
struct Smem {
  static constexpr int D = 32 * NG;
  static constexpr int q = 0;                                   // 2 x [D/64 slabs][128 rows][128 B]
  static constexpr int q_tile = kRows * D * 2;
  static constexpr int ops = 2 * q_tile;                        // 3 x K' or V'
  static constexpr int op_tile = kKeys * D * 2;
  static constexpr int raw = ops + kOps * op_tile;              // 3 x 8 blocks
  static constexpr int block = kKvBlock * (D + D / 8);
  static constexpr int raw_tile = kKeys / kKvBlock * block;
  static constexpr int bars = raw + kRawStages * raw_tile;
  static constexpr int info = bars + 256;
  static constexpr int bytes = info + kInfos * 16 + 16;
  static constexpr int alloc = bytes + 1024;                    // for the 1024-byte alignment
};
static_assert(Smem<4>::alloc <= 227 * 1024, "shared memory of a CTA");
// barriers
constexpr int kRawFull = 0, kRawSeen = kRawFull + kRawStages, kRawEmpty = kRawSeen + kRawStages,
              kOpFull = kRawEmpty + kRawStages, kKFreed = kOpFull + kOps, kVFreed = kKFreed + 2, kQFull = kVFreed + 2,
              kSFull = kQFull + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2, kDrain = kPvDone + 2,
              kNumBars = kDrain + 1;
static_assert(kNumBars * 8 <= 256);

// What a key tile's softmax needs to know about it.
struct TileInfo {
  int k_exp, v_exp;  // exponent fields of the largest K scale (tile) and V scale (item so far)
  uint32_t there;    // blocks that were copied
  int flags;
};
// The tile is its item's first or last, the CTA's last, and the item has rows for the second row tile.
enum { kFirst = 1, kLast = 2, kEnd = 4, kBoth = 8 };

// Scales enter K' and V' as scale * 2^(138 - field): below 2^12, times a code below 2^15.
constexpr int kNorm = 138;
__device__ __forceinline__ int clamp_exp(int e) { return e < 40 ? 40 : (e > 250 ? 250 : e); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr));
  return v;
}
// Bits [a, b) of a word, the borders clamped to 0 .. 32.
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0), b = min(b, 32);
  if (a >= 32 || b <= a) return 0u;
  return (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (32 - b));
}
// Which of the 32 keys from draft index d0 on (negative: before the drafts) the row's mask shows.
__device__ __forceinline__ uint32_t draft_bits(const AttnArgs& a, int token, int d0) {
  if (d0 <= -32) return 0xFFFFFFFFu;
  const uint32_t* w = a.mask + (long long)token * a.mask_words;
  auto word = [&](int i) { return i < a.mask_words ? __ldg(w + i) : 0u; };
  if (d0 < 0) return (word(0) << -d0) | ((1u << -d0) - 1u);
  return __funnelshift_r(word(d0 >> 5), word((d0 >> 5) + 1), d0 & 31);
}

// The part of a wait that does not succeed at once: polls until the phase completes, another role gave
// up, or kPolls polls (a second or more) have passed. Kept short: it is inlined at every wait.
constexpr int kPolls = 1 << 24;
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort_at, unsigned int* err) {
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i) {
    if (mbar_try_wait_poll(bar, parity)) return true;
    uint32_t gone;
    asm volatile("ld.volatile.shared.u32 %0, [%1];\n" : "=r"(gone) : "r"(abort_at));
    if (gone) return false;
  }
  if (err) atomicCAS(err, 0u, 8u);  // W4A16_ERR_TIMEOUT
  asm volatile("st.volatile.shared.u32 [%0], %1;\n" ::"r"(abort_at), "r"(1u) : "memory");
  return false;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// (dec to more, or inc to fewer, than the launch's count is an illegal instruction)
template <int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > kRegsLaunch)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
  else if constexpr (N < kRegsLaunch)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// Two float32 operations in one instruction (lo in the low word).
__device__ __forceinline__ uint64_t pair64(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair64(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = __uint_as_float(x[k]);
#pragma unroll
  for (int k = 4; k < 32; ++k) m[k & 3] = fmaxf(m[k & 3], __uint_as_float(x[k]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// 32 scores -> weights 2^(x ft - off), added to the sums, packed as fp16 in V's key order: position k of
// 8 keys holds key (k + their index within 64 keys) & 7 of them. C0: index of the first 8.
template <int C0>
__device__ __forceinline__ void chunk_weights(const uint32_t (&x)[32], uint32_t (&p)[16], float ft, float off,
                                              uint64_t& s0, uint64_t& s1) {
  const uint64_t f2 = pair64(ft, ft), o2 = pair64(-off, -off);
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint64_t y =
          fma_f32x2(pair64(__uint_as_float(x[8 * ch + k]), __uint_as_float(x[8 * ch + k + 1])), f2, o2);
      unpair64(y, v[k], v[k + 1]);
      v[k] = ex2(v[k]);
      v[k + 1] = ex2(v[k + 1]);
      if (k & 2) s1 = add_f32x2(s1, pair64(v[k], v[k + 1]));
      else s0 = add_f32x2(s0, pair64(v[k], v[k + 1]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      p[4 * ch + k] = pack_half2(v[(2 * k + C0 + ch) & 7], v[(2 * k + 1 + C0 + ch) & 7]);
  }
}
// Multiplies 16 weights (8 columns) of a row by f.
__device__ __forceinline__ void scale_weights(uint32_t taddr, uint32_t f2) {
  uint32_t r[8];
  asm volatile("tcgen05.wait::st.sync.aligned;\n tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               " tcgen05.wait::ld.sync.aligned;\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = hmul2_u32(r[k], f2);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Multiplies a row's scores by f where they lie. Out of line: it hardly ever runs (inlined, every tile pays: 817 us).
__device__ __noinline__ void scale_scores(uint32_t taddr, float f) {
#pragma unroll 1
  for (int q = 0; q < kKeys / 16; ++q) {
    uint32_t x[16];
    tmem_ld16(taddr + 16 * q, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__fmul_rn(__uint_as_float(x[k]), f));
    tmem_st16(taddr + 16 * q, x);
  }
  tmem_wait_st();
}

template <int NG>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const AttnArgs a, const KvCache c, const int min_rows, const Partials part,
                     unsigned int* err) {
  using L = Smem<NG>;
  constexpr int D = L::D;
  extern __shared__ __align__(1024) char smem_raw[];
  char* sm = align1024(smem_raw);
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + L::bars + 8u * (uint32_t)i; };
  TileInfo* info = reinterpret_cast<TileInfo*>(sm + L::info);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + L::info + kInfos * 16);

  Walk<kKeys, 2 * kRows, kManyItemCost> w(a, c.page_size, INT_MAX, min_rows, c.Hkv, err);
  const long long total = w.total();
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kManyItemCost + 1) per = kManyItemCost + 1;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  const bool any = begin < total;
  if (any) w.seek(begin);
  if (threadIdx.x == 0) part.start[blockIdx.x] = any ? w.start(begin, per) : Partials::Start{0, 0, 0, 0, 0, 0};
  if (!any) return;
  while (w.tile_at(begin) == w.tile_at(end)) {  // only (part of) an item's fixed cost: on to one with tiles
    if (w.tile0 + w.tiles >= end) return;
    w.next_item();
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(bar(kRawFull + s), 1);
      mbar_init(bar(kRawSeen + s), 1);
      mbar_init(bar(kRawEmpty + s), kDeqWarps);
    }
    for (int s = 0; s < kOps; ++s) {
      mbar_init(bar(kOpFull + s), kDeqWarps);
    }
    for (int r = 0; r < 2; ++r) {
      mbar_init(bar(kQFull + r), 4);
      mbar_init(bar(kSFull + r), 1);
      mbar_init(bar(kPFull + r), 4);
      mbar_init(bar(kPvDone + r), 1);
    }
    mbar_init(bar(kDrain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFreed + i), 1);
      mbar_init(bar(kVFreed + i), 1);
    }
    misc[1] = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     sb + (uint32_t)(L::info + kInfos * 16))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = misc[0];
  // columns: S (and P) of the two row tiles, then their O
  auto s_col = [&](int r) { return tmem + (uint32_t)(r * kKeys); };
  auto o_col = [&](int r) { return tmem + (uint32_t)(2 * kKeys + r * D); };

  const uint32_t abort_at = sb + (uint32_t)(L::info + kInfos * 16) + 4u;
  // for whole warps: all lanes go on, or none
  auto wait_warp = [&](int b, uint32_t parity) {
    bool ok = mbar_try_wait_poll(bar(b), parity);
    if (!ok) ok = wait_slow(bar(b), parity, abort_at, err);
    return __all_sync(0xFFFFFFFFu, ok) != 0;
  };

  if (warp >= kCopyWarp) set_regs<kRegsRest>();
  if (warp == kCopyWarp) {
    // ---- raw blocks in; one tile behind, the tile's largest scales
    const int page_shift = 31 - __clz(c.page_size);
    int n = 0;           // tiles issued
    int ve = 0;          // item's running V exponent field
    bool wrote = false;  // this lane changed scales since the last copy
    uint32_t pend_ok[2] = {0, 0};  // of the two tiles issued last: blocks copied,
    uint32_t pend_seen[2] = {0, 0};  // its keys that a row of the item sees (lane q: keys 32 (q % 4) ..),
    int pend_flags[2] = {0, 0};
    bool ok = true;
    auto look = [&](int i, uint32_t copied, uint32_t seen, int flags) {
      const int s = i % kRawStages;
      if (!wait_warp(kRawFull + s, (i / kRawStages) & 1)) return false;
      const uint32_t st = sb + L::raw + s * L::raw_tile;
      uint32_t mk = 0, mv = 0;
#pragma unroll 1
      for (int p = 0; p < kKeys / 32; ++p) {
        const int key = p * 32 + lane, blk = key / kKvBlock, r = key % kKvBlock;
        uint32_t ks[NG / 2], vs[NG / 2];
        lds_words<NG / 2>(st + blk * L::block + kv_scales_off(D, 0) + r * NG * 2, ks);
        lds_words<NG / 2>(st + blk * L::block + kv_scales_off(D, 1) + r * NG * 2, vs);
        if ((__shfl_sync(0xFFFFFFFFu, seen, p) >> lane) & 1u) {
#pragma unroll
          for (int k = 0; k < NG / 2; ++k) {
            mk = __vmaxu2(mk, ks[k] & 0x7FFF7FFFu);
            mv = __vmaxu2(mv, vs[k] & 0x7FFF7FFFu);
          }
        } else {
          wrote = true;  // whatever the bytes are: K' and V' of keys that no row sees are zeros
#pragma unroll
          for (int k = 0; k < NG / 2; ++k) {
            sts32(st + blk * L::block + kv_scales_off(D, 0) + r * NG * 2 + 4 * k, 0u);
            sts32(st + blk * L::block + kv_scales_off(D, 1) + r * NG * 2 + 4 * k, 0u);
          }
        }
      }
      __syncwarp();
      mk = __reduce_max_sync(0xFFFFFFFFu, max(mk & 0xFFFFu, mk >> 16)) >> 7;
      mv = __reduce_max_sync(0xFFFFFFFFu, max(mv & 0xFFFFu, mv >> 16)) >> 7;
      ve = (flags & kFirst) ? clamp_exp((int)mv) : max(ve, clamp_exp((int)mv));
      if (lane == 0) {
        info[i % kInfos] = TileInfo{clamp_exp((int)mk), ve, copied, flags};
        tc::mbar_arrive(bar(kRawSeen + s));
      }
      __syncwarp();
      return true;
    };
    // Step n issues tile n and looks at tile n - 2; two more steps after the last tile.
    int t = w.tile_at(begin), t1 = w.tile_at(end), after = 0;
    auto page_of = [&](int tile) {
      const int key = w.first_key(w.lo) + tile * kKeys + lane * kKvBlock;
      return lane < kKeys / kKvBlock && tile < t1 && key + kKvBlock > w.lo && key < w.hi
                 ? __ldg(a.block_table + (size_t)w.b * a.max_pages + (key >> page_shift)) : -1;
    };
    int next_page = page_of(t), steps = 0;
    bool first = true;
    for (;; ++steps) {
      if (steps > 1 && !look(steps - 2, pend_ok[1], pend_seen[1], pend_flags[1])) {
        ok = false;
        break;
      }
      pend_ok[1] = pend_ok[0], pend_seen[1] = pend_seen[0], pend_flags[1] = pend_flags[0];
      if (after) {  // no tile left to issue
        if (++after == 3) break;
        continue;
      }
      const int base = w.first_key(w.lo) + t * kKeys, key = base + lane * kKvBlock;
      const bool want = lane < kKeys / kKvBlock && key + kKvBlock > w.lo && key < w.hi;
      const int page = next_page;
      const bool good = want && page >= 0 && page < c.num_pages;
      const uint32_t okm = __ballot_sync(0xFFFFFFFFu, good);
      if (__any_sync(0xFFFFFFFFu, want && !good) && lane == 0 && err) atomicCAS(err, 0u, 1u);
      const int s = n % kRawStages;
      if (n >= kRawStages && !wait_warp(kRawEmpty + s, ((n / kRawStages) & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (wrote) fence_proxy_async_shared();  // look() wrote where copies go
      wrote = false;
      if (lane == 0) mbar_expect_tx(bar(kRawFull + s), (uint32_t)__popc(okm) * L::block);
      __syncwarp();
      if (good)
        bulk_load(sb + L::raw + s * L::raw_tile + lane * L::block,
                  static_cast<const char*>(c.data) +
                      kv_block_addr(D, c.page_size, c.Hkv, page, w.h, key & (c.page_size - 1)),
                  L::block, bar(kRawFull + s));
      ++n;
      const bool item_ends = t + 1 == t1, run_ends = item_ends && w.tile0 + w.tiles + kManyItemCost >= end;
      pend_ok[0] = okm;
      const int k0 = base + 32 * (lane & 3);
      uint32_t seen = bit_range(w.lo - k0, w.hi - k0) & ((okm >> (2 * (lane & 3)) & 1u ? 0x0000FFFFu : 0u) |
                                                         (okm >> (2 * (lane & 3)) & 2u ? 0xFFFF0000u : 0u));
      const int dbase = w.s.len - w.s.n;
      if (a.mask != nullptr && base + kKeys > dbase) {  // drafts: those that the mask shows to one of the item's tokens
        const int r0 = w.rt * 2 * kRows, i_last = (min(r0 + 2 * kRows, w.s.n * a.G) - 1) / a.G;
        uint32_t any = 0;
#pragma unroll 4
        for (int i = r0 / a.G + (lane >> 2); i <= i_last; i += 8) any |= draft_bits(a, w.s.q0 + i, k0 - dbase);
        any |= __shfl_xor_sync(0xFFFFFFFFu, any, 4);
        any |= __shfl_xor_sync(0xFFFFFFFFu, any, 8);
        any |= __shfl_xor_sync(0xFFFFFFFFu, any, 16);
        seen &= any;
      }
      pend_seen[0] = seen;
      pend_flags[0] = (first ? kFirst : 0) | (item_ends ? kLast : 0) | (run_ends ? kEnd : 0) |
                      (w.s.n * a.G - w.rt * 2 * kRows > kRows ? kBoth : 0);
      first = item_ends;
      if (run_ends) {
        after = 1;
      } else if (item_ends) {
        w.next_item();
        t = w.tile_at(begin);
        t1 = w.tile_at(end);
        next_page = page_of(t);
      } else {
        next_page = page_of(++t);
      }
    }
    if (!ok)  // copies still under way write into this CTA's memory: see them land
      for (int i = max(0, n - kRawStages); i < n; ++i)
        (void)mbar_wait(bar(kRawFull + i % kRawStages), (i / kRawStages) & 1, kWaitLimitNs / 16);
  } else if (warp >= kDeqWarp0 && warp < kCopyWarp) {
    // ---- raw blocks -> K' and V'^T
    set_regs<kRegsDeq>();
    const int dw = warp - kDeqWarp0;
    int s = 0, slot = 0;  // raw stage, operand slot
    uint32_t ph = 0;
    for (int n = 0;; ++n) {
      if (!wait_warp(kRawFull + s, ph) || !wait_warp(kRawSeen + s, ph)) break;
      const TileInfo ti = info[n % kInfos];
      const uint32_t st = sb + L::raw + s * L::raw_tile;
      // K': a thread takes word w of every group of a key
      // K's slot held V of tile n - 2, V's slot K of tile n - 1. Even and odd tiles have barriers of
      // their own: the one waited on cannot move on another phase before this tile is handed over.
      if (n >= 2 && !wait_warp(kVFreed + (n & 1), ((n >> 1) & 1) ^ 1)) break;
      uint32_t op = sb + L::ops + slot * L::op_tile;
      {
        const float f = exp2i(kNorm - ti.k_exp);
        const int word = lane >> 3;
#pragma unroll 1
        for (int p = 0; p < kKeys / (8 * kDeqWarps); ++p) {
          const int key = (p * kDeqWarps + dw) * 8 + (lane & 7);
          const uint32_t blk = st + (key / kKvBlock) * L::block;
          const int r = key % kKvBlock;
          uint32_t cw[NG], sw[NG / 2];
          lds_words<NG>(blk + r * (D / 2) + ((word ^ (r & 2)) * NG) * 4, cw);
          lds_words<NG / 2>(blk + kv_scales_off(D, 0) + r * NG * 2, sw);
          const uint32_t row = op + (uint32_t)(key >> 3) * 1024u + (uint32_t)(key & 7) * 128u;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float sc = bf16_of(sw, i) * f;
            const uint32_t s2 = pack_half2(sc, sc);
            uint32_t x[4];
            unpack_word(cw[i], x);
            const int chunk = 4 * i + word;
            sts128(row + (chunk >> 3) * (kKeys * 128) + (((chunk & 7) ^ (key & 7)) << 4),
                   hmul2_u32(x[0], s2), hmul2_u32(x[1], s2), hmul2_u32(x[2], s2), hmul2_u32(x[3], s2));
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kOpFull + slot));
      if (++slot == kOps) slot = 0;
      // V'^T: a thread takes one word of 8 keys (rotated by its chunk) and writes 8 dim rows
      if (n >= 1 && !wait_warp(kKFreed + ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
      op = sb + L::ops + slot * L::op_tile;
      {
        const float f = exp2i(kNorm - ti.v_exp);
        const int word = dw & 3, ch = dw >> 2, cc = lane & 7, i = lane >> 3;
        if (i < NG) {
          uint32_t cw[8];
          float sc[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int key = ch * 64 + cc * 8 + ((k + cc) & 7);
            const uint32_t blk = st + (key / kKvBlock) * L::block;
            const int r = key % kKvBlock;
            asm volatile("ld.shared.u32 %0, [%1];\n"
                         : "=r"(cw[k])
                         : "r"(blk + kv_codes_off(D, 1) + r * (D / 2) + ((word ^ (r & 2)) * NG + i) * 4));
            const uint32_t b = lds_u16(blk + kv_scales_off(D, 1) + (r * NG + i) * 2);
            sc[k] = __uint_as_float(b << 16) * f;
          }
          uint32_t s2[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) s2[q] = pack_half2(sc[2 * q], sc[2 * q + 1]);
          const uint32_t row = op + ch * (D * 128) + (uint32_t)(4 * i + word) * 1024u;
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {  // dims 0 .. 3, then 4 .. 7 of the word
            const uint32_t sel = hf ? 0x7632u : 0x5410u;
            uint32_t o[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t x[4];
              unpack_word(prmt(cw[2 * q], cw[2 * q + 1], sel), x);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j][q] = hmul2_u32(x[j], s2[q]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sts128(row + (4 * hf + j) * 128u + ((cc ^ (4 * hf + j)) << 4), o[j][0], o[j][1], o[j][2], o[j][3]);
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(bar(kOpFull + slot));
        tc::mbar_arrive(bar(kRawEmpty + s));
      }
      if (++slot == kOps) slot = 0;
      if (++s == kRawStages) s = 0, ph ^= 1u;
      if (ti.flags & kEnd) break;
    }
  } else if (warp == kMmaWarp) {
    // ---- MMAs. The whole warp walks along and one elected lane issues: descriptors then stay in uniform
    // registers (under lane == 0 every MMA took about 90 cycles to issue, whatever its size). One warp
    // for both row tiles: the tensor core finishes row tile 0's P V' and S before it begins row tile
    // 1's, which keeps the two half a tile apart; with a warp each they fell into step, softmax and
    // tensor core taking turns (939 -> 1016 us for 4096 tokens over 8192 keys).
    constexpr uint32_t idesc_s = tc::idesc_f16(false, kRows, kKeys);
    constexpr uint32_t idesc_o = tc::idesc_f16(false, kRows, D);
    int slot = 0;                        // operand slot
    uint32_t par = 0;                    // parity of its present use
    uint32_t q_par = 0, p_par = 0;       // bit r: parity of row tile r's next Q and P
    bool ok = true;
    const uint64_t q_desc = tc::sw128_desc(sb + L::q), op_desc = tc::sw128_desc(sb + L::ops);
    auto next_slot = [&]() {
      if (++slot == kOps) slot = 0, par ^= 1u;
    };
    auto scores = [&](int r, int at, int frees) {
      const uint64_t qd = q_desc + (uint64_t)(r * (L::q_tile >> 4));
      const uint64_t kd = op_desc + (uint64_t)(at * (L::op_tile >> 4));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
          mma_ss(s_col(r), qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        commit(bar(kSFull + r));  // (a commit costs some 150 .. 400 cycles: as few as possible)
        if (frees >= 0) commit(bar(kKFreed + (frees & 1)));
      }
      __syncwarp();
    };
    auto outputs = [&](int r, int at, bool first, bool last, int frees) {
      const uint64_t vd = op_desc + (uint64_t)(at * (L::op_tile >> 4));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * (D * 128) + (kk & 3) * 32) >> 4);
          mma_ts(o_col(r), s_col(r) + kk * 8, vd + off, idesc_o, !first || kk > 0 ? 1u : 0u);
        }
        if (frees >= 0) commit(bar(kVFreed + (frees & 1)));
        if (last) commit(bar(kPvDone + r));
      }
      __syncwarp();
    };
    // One tile after the other, by its flags; K of the tile is in `slot`, and its scores are under way
    // unless it is an item's first.
    bool have_k = false;  // K has been waited for (a second wait could come after the slot's next phase)
    for (int n = 0;; ++n) {
      ok = have_k || wait_warp(kOpFull + slot, par);
      if (!ok) break;
      const int flags = info[n % kInfos].flags;
      const int nr = (flags & kBoth) ? 2 : 1;
      have_k = !(flags & kLast);
      if (flags & kFirst) {
        for (int r = 0; ok && r < nr; ++r) {
          ok = wait_warp(kQFull + r, (q_par >> r) & 1u);
          q_par ^= 1u << r;
          tc::fence_after();
          if (ok) scores(r, slot, r == nr - 1 ? n : -1);
        }
      }
      next_slot();
      const int v = slot;
      ok = ok && wait_warp(kOpFull + v, par);
      next_slot();
      for (int r = 0; ok && r < nr; ++r) {
        ok = wait_warp(kPFull + r, (p_par >> r) & 1u);
        p_par ^= 1u << r;
        if (!ok) break;
        tc::fence_after();
        outputs(r, v, flags & kFirst, flags & kLast, r == nr - 1 ? n : -1);
        if (!(flags & kLast)) {
          if (r == 0) ok = wait_warp(kOpFull + slot, par);
          if (!ok) break;
          tc::fence_after();
          scores(r, slot, r == nr - 1 ? n + 1 : -1);
        }
      }
      if (!ok || (flags & kEnd)) break;
    }
    // every MMA issued here has finished before TMEM is given back
    if (elect_one()) commit(bar(kDrain));
    __syncwarp();
    (void)mbar_wait(bar(kDrain), 0, kWaitLimitNs);
  } else if (warp < kDeqWarp0) {
    set_regs<kRegsSoft>();
    // ---- softmax warps: row tile r, TMEM lanes 32 * (warp % 4) ..
    const int r = warp >> 2, row_in = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t S = s_col(r) + lane_base, O = o_col(r) + lane_base;
    int n = 0;      // tiles seen by the CTA
    int cnt = 0;    // tiles of this row tile
    int items = 0;  // items of this row tile
    bool ok = true;
    // The row's result of the item before, still in O: written after the next item's queries have been
    // handed over, so that its first scores do not wait for it.
    bool held = false, h_live = false, h_whole = false;
    float h_inv = 0.0f, h_lse2 = 0.0f;
    long long h_row = 0;  // row of the output, or of the partial results
    auto write_held = [&]() {
      if (!wait_warp(kPvDone + r, (items++) & 1)) return false;
      tc::fence_after();
#pragma unroll 1
      for (int q = 0; q < D; q += 16) {
        uint32_t x[16];
        tmem_ld16(O + q, x);
        if (h_live) {
#pragma unroll
          for (int k = 0; k < 16; ++k)  // (0: no key was seen, O may hold anything)
            x[k] = h_inv == 0.0f ? 0u : __float_as_uint(__uint_as_float(x[k]) * h_inv);
          if (h_whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + h_row * D + q);
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 b2 =
                  __floats2bfloat162_rn(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
              h[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(part.o + h_row * D + q);
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
        __syncwarp();  // the next load is for the whole warp
      }
      if (h_live) {
        if (!h_whole) part.lse2[h_row] = h_lse2;
        else if (a.lse) a.lse[h_row] = h_lse2 * 0.69314718055994530942f;
      }
      tc::fence_before();
      held = false;
      return true;
    };
    for (;; w.next_item()) {
      const int t0 = w.tile_at(begin), t1 = w.tile_at(end);
      const bool last = w.tile0 + w.tiles + kManyItemCost >= end;
      const int rows = min(2 * kRows, w.s.n * a.G - w.rt * 2 * kRows);
      if (t0 < t1 && r * kRows >= rows) n += t1 - t0;  // no rows for this tile: the MMA warp skips it too
      if (t0 < t1 && r * kRows < rows) {
        const KvSeq sq = w.s;
        const int row = w.rt * 2 * kRows + r * kRows + row_in;  // token * G + head
        const bool live = r * kRows + row_in < rows;
        const int row_last = w.rt * 2 * kRows + min((r + 1) * kRows, rows) - 1;
        const int i = (live ? row : row_last) / a.G, hq = (live ? row : row_last) - i * a.G;
        const int i_first = (w.rt * 2 * kRows + r * kRows) / a.G, i_last = row_last / a.G;
        const bool masked = a.mask != nullptr;
        const int dbase = sq.len - sq.n;
        const int full_hi = masked ? dbase : kv_hi(sq, i_first, a.causal, false);
        const int full_lo = kv_lo(sq, i_last, a.window);
        const int hi_r = kv_hi(sq, i, a.causal, masked), lo_r = kv_lo(sq, i, a.window);
        const int key_end = w.hi;

        // queries: row exponent, then fp16 chunks of 8 dims in the nibbles' order
        float f_row;
        {
          const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                                    (long long)(sq.q0 + i) * a.qs.token + (long long)(w.h * a.G + hq) * a.qs.head;
          // Into their places as they are, D/8 lanes a row (a thread reading its own row touches 32 lines a
          // load), then each thread scales its row there.
          constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
          const unsigned long long own = live ? reinterpret_cast<unsigned long long>(qp) : 0ull;
          const uint32_t tile = sb + L::q + r * L::q_tile;
          const int k_in = lane % kLanes;
#pragma unroll 8
          for (int j = 0; j < kLanes; ++j) {
            const int from = j * kRowsAtOnce + lane / kLanes, to = (warp & 3) * 32 + from;
            const uint4* src = reinterpret_cast<const uint4*>(__shfl_sync(0xFFFFFFFFu, own, from));
            const uint4 v = src ? __ldg(src + k_in) : make_uint4(0, 0, 0, 0);
            sts128(tile + (uint32_t)(to >> 3) * 1024u + (uint32_t)(to & 7) * 128u + (k_in >> 3) * (kRows * 128) +
                       (((k_in & 7) ^ (to & 7)) << 4), v.x, v.y, v.z, v.w);
          }
          __syncwarp();
          const uint32_t dst = tile + (uint32_t)(row_in >> 3) * 1024u + (uint32_t)(row_in & 7) * 128u;
          auto place = [&](int k) { return dst + (k >> 3) * (kRows * 128) + (((k & 7) ^ (row_in & 7)) << 4); };
          uint32_t big = 0;
#pragma unroll 4
          for (int k = 0; k < D / 8; ++k) {
            const uint4 v = lds128(place(k));
            big = __vmaxu2(big, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                         __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
          }
          const int e = row_exponent(__uint_as_float(max(big & 0xFFFFu, big >> 16) << 16));
          const float up = exp2i(14 - e);
          f_row = a.scale * 1.44269504088896340736f * exp2i(e - 14);
#pragma unroll 1
          for (int k = 0; k < D / 8; ++k) {
            const uint4 q8 = lds128(place(k));
            const uint32_t x[4] = {q8.x, q8.y, q8.z, q8.w};
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = bf16_of(x, j) * up;
            sts128(place(k), pack_half2(y[0], y[4]), pack_half2(y[1], y[5]), pack_half2(y[2], y[6]),
                   pack_half2(y[3], y[7]));
          }
        }
        tc::fence_proxy_async();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(kQFull + r));
        if (held && !write_held()) {
          ok = false;
          break;
        }

        float m = -CUDART_INF_F, l = 0.0f;
        int ve = 0;
        for (int t = t0; t < t1; ++t, ++n, ++cnt) {
          if (!wait_warp(kSFull + r, cnt & 1)) {
            ok = false;
            break;
          }
          tc::fence_after();
          const TileInfo ti = info[n % kInfos];
          const int kbase = w.first_key(w.lo) + t * kKeys;
          const bool full = ti.there == (1u << (kKeys / kKvBlock)) - 1u && kbase + kKeys <= min(full_hi, key_end) &&
                            kbase >= full_lo;
          uint32_t vis[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
          if (!full) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k0 = kbase + 32 * q;
              vis[q] = bit_range(lo_r - k0, min(hi_r, key_end) - k0);
              if (!((ti.there >> (2 * q)) & 1u)) vis[q] &= 0xFFFF0000u;
              if (!((ti.there >> (2 * q + 1)) & 1u)) vis[q] &= 0x0000FFFFu;
              if (masked) vis[q] &= draft_bits(a, sq.q0 + i, k0 - dbase);
            }
          }
          // never 0, which would turn hidden keys' -inf into NaN: zero queries over small keys reach 2^-215
          // (scores are below 2^37 in these units, so a larger ft leaves them at 0 all the same)
          float ft = fmaxf(f_row * exp2i(ti.k_exp - kNorm), 0x1p-126f);
          if (!full) {  // hidden keys' scores become -inf, in TMEM
#pragma unroll 1
            for (int q = 0; q < kKeys / 16; ++q) {
              uint32_t x[16];
              tmem_ld16(S + 16 * q, x);
              const uint32_t v = (q < 4 ? (q < 2 ? vis[0] : vis[1]) : (q < 6 ? vis[2] : vis[3])) >> (16 * (q & 1));
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (!((v >> k) & 1u)) x[k] = 0xFF800000u;
              tmem_st16(S + 16 * q, x);
            }
            tmem_wait_st();
          }
          if (__any_sync(0xFFFFFFFFu, ft > kFusedFactor)) {  // such a row's scores become what they are, in TMEM
            scale_scores(S, ft > kFusedFactor ? ft : 1.0f);
            ft = ft > kFusedFactor ? 1.0f : ft;  // (a row's result does not depend on its neighbours)
          }
          // Weights under the maximum so far, 32 keys at a time, over S's columns (always behind what has
          // been read). Where a row's maximum is too low (8 binades; on an item's first keys) it is
          // raised first, and the tile's earlier weights are scaled down where they lie.
          float fo = 1.0f;  // what O has to be multiplied by
          uint64_t s0 = 0, s1 = 0;  // sums, two zeros each
          uint32_t x[32];
          tc::tmem_ld32(S, x);
#pragma unroll 1
          for (int q = 0; q < kKeys / 32; q += 2) {
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              tc::tmem_wait_ld(x);
              float mx = max32(x);
              mx *= ft;  // (-inf stays: ft > 0)
              const bool grow = mx > m + kLag;
              if (__any_sync(0xFFFFFFFFu, grow)) {
                const float f = grow && m != -CUDART_INF_F ? ex2(m - mx) : 1.0f;
                const uint64_t f2 = pair64(f, f);
                s0 = mul_f32x2(s0, f2);
                s1 = mul_f32x2(s1, f2);
                fo *= f;
                if (grow) m = mx;
                const uint32_t h2 = pack_half2(f, f);
#pragma unroll 1
                for (int k = 0; k < 2 * (q + o); ++k) scale_weights(S + 8 * k, h2);
              }
              const float off = (m == -CUDART_INF_F ? 0.0f : m) - kTop;
              uint32_t p[16];
              if (o == 0) chunk_weights<0>(x, p, ft, off, s0, s1);
              else chunk_weights<4>(x, p, ft, off, s0, s1);
              if (o == 0 || q + 2 < kKeys / 32) tc::tmem_ld32(S + 32 * (q + o + 1), x);
              tmem_st16(S + 16 * (q + o), p);
            }
          }
          {
            float u0, u1;
            unpair64(add_f32x2(s0, s1), u0, u1);
            l = l * fo + (u0 + u1);
          }
          if (t > t0) {
            if (ti.v_exp != ve) fo *= exp2i(max(ve - ti.v_exp, -126));
            if (__any_sync(0xFFFFFFFFu, fo != 1.0f)) {
              // (P V' of the tile before is complete: its MMAs were issued before this tile's scores)
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t y[16];
                tmem_ld16(O + 16 * q, y);
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * fo);
                tmem_st16(O + 16 * q, y);
              }
            }
          }
          ve = ti.v_exp;
          tmem_wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(kPFull + r));
        }
        if (!ok) break;
        held = true;
        h_live = live;
        h_whole = t0 == 0 && t1 == w.tiles;
        h_inv = l == 0.0f ? 0.0f : exp2i(ve - kNorm) / l;
        h_lse2 = l == 0.0f ? -CUDART_INF_F : (m == -CUDART_INF_F ? 0.0f : m) - kTop + log2f(l);
        h_row = h_whole ? (long long)(sq.q0 + i) * a.Hq + w.h * a.G + hq
                        : (long long)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * (2 * kRows) + r * kRows + row_in;
      }
      if (last || !ok) break;
    }
    if (ok && held) (void)write_held();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
}

template <int NG>
cudaError_t launch_many_t(const AttnArgs& a, const KvCache& c, int min_rows, void* ws, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce<int> once;
  const int* unused = nullptr;
  e = once.get(di.device, [&](int&) {
    return cudaFuncSetAttribute(attn_many_kernel<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<NG>::alloc);
  }, &unused);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count < kMaxManyCtas ? di.sm_count : kMaxManyCtas;
  const Partials p = Partials::at(ws, 2 * kRows, 32 * NG, kMaxManyCtas);
  attn_many_kernel<NG><<<grid, kThreads, Smem<NG>::alloc, s>>>(a, c, min_rows, p, device_error_word());
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attn_merge_rows<__nv_bfloat16>(a, p, grid, 32 * NG, s);
}

}  // namespace

cudaError_t launch_attn_many(const AttnArgs& a, const KvCache& c, int min_rows, void* ws, cudaStream_t s) {
  return c.D == 64 ? launch_many_t<2>(a, c, min_rows, ws, s) : launch_many_t<4>(a, c, min_rows, ws, s);
}

}  // namespace w4a16
