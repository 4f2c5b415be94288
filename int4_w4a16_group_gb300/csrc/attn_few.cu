// Attention over the paged 4-bit cache for few query rows per key/value head: decoding, and small
// drafts.
//
// A row is one (query token, query head). Rows that share a key/value head share its keys, so an
// item is (sequence, head, tile of 8 NB rows); it walks the visible keys in tiles of 32. Both
// products run on mma.sync m16n8k16 with the CODES as the 16-row operand, so 8 query rows cost one
// column block:
//   S^T[16 keys, 8 rows] = K codes x Q^T  per group of 32 dims, times the key's group scale in float32;
//   O^T[16 dims, 8 rows] += V codes^T x P'^T, P' = p times the key's group scale.
// Codes are exact in fp16, so scores lose nothing to the 4-bit form. Numerics:
//   * Q: each row scaled by a power of two so that its largest value is just below 2^15, then fp16:
//     one term holds bf16 queries exactly (down to 2^-28 of the row's largest), hi + lo terms hold 22
//     bits of float32 queries.
//   * P', bf16 calls: one fp16 term (2^-11 a weight, below the output's own rounding). The running
//     maximum is moved by the exponent of the largest V scale seen so far, which keeps p * scale below
//     2^15 whatever the scales are, with 39 bits of range under it.
//   * P', float32 calls: three bf16 terms, exact, with float32's own range (fp16 hi + lo lost weights
//     2^-30 below a row's largest, which show where the large weights meet codes of zero).
//   * Sums and accumulators are float32.
//   * bf16 calls do not turn K's codes into numbers: a masked nibble n read as an fp16 bit pattern is
//     the subnormal n * 2^-24 (16 n * 2^-24 one nibble up), exact, and the offset of 8 comes back as the
//     accumulator's initial value -8 sum(q), which saves 8 of 18 unpacking instructions. The float32
//     form keeps signed codes, whose sums cancel less inside the tensor core; so does V, where the
//     offset's share can be far larger than an output.
//
// Work: all items' key tiles form one line that is cut into equal runs, one per CTA, whatever the
// lengths of the sequences; an item cut by a border is merged afterwards (attn_merge_kernel) from the
// normalised partial results, in the order of the CTAs. The 4 warps of a CTA take a run's tiles in
// turn, each with its own ring of bulk copies (a tile is one contiguous piece of a page) and its own
// running softmax, merged through shared memory at the end of an item: no barrier in the loop.
//
// What bounds it: latency, with few warps to hide it. A tile of 32 keys (D = 128, 8 rows) is a chain of some 500
// instructions a warp (load, unpack, product, scale, maximum, exponential, product), and the registers leave 2.8 warps
// per scheduler (float32, 16 rows: 2): 55 % (48 %) of the issue slots are used, and the most frequent reason for a warp
// to wait is the fixed latency of the instruction before. DRAM reads are the cache's bytes once (205.6 MB for
// 205.5). One token of 64 sequences of 100 .. 16384 tokens, 64 query and 8 key/value heads, bf16: 64 us, 3.2 TB/s; one
// of 131071 tokens, float32 (twice the products, three terms of P'): 62 us, 2.4 TB/s; one of 333: 14 us, of which two
// launches are 5: its warps wait at the barriers of the walk and the merge and for instructions that run for the first
// time; 16 draft tokens of 4 sequences, float32, 8 row tiles over the same keys: 174 us. Three CTAs per SM (168 registers)
// beat four (128, spilling) by 5 to 10 us for the bf16 form with 8 rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "attn_core.cuh"

namespace w4a16 {
namespace {

using namespace mma;
using namespace attn;

constexpr int kWarps = 4;
constexpr int kTile = 32;     // keys per tile
constexpr int kMinRun = kItemCost + kWarps;  // shortest run of a CTA: one tile per warp

// Stages of a warp's ring: about 14 KB in flight per warp, and room for the merge (R x D floats).
constexpr int ring_stages(int NG) { return NG == 2 ? 4 : NG == 4 ? 3 : 2; }
constexpr int tile_bytes(int NG) { return kTile * 36 * NG; }
constexpr int warp_smem(int NG) { return ring_stages(NG) * tile_bytes(NG); }
constexpr int kBarBytes = 256;
constexpr int few_smem(int NG) { return kWarps * warp_smem(NG) + kBarBytes + kWarps * 16 * 8; }

// C row rho of a 16-key S^T block holds key key_of(rho): chosen so that the rows of V that a lane
// pair needs (C rows 2t, 2t + 1) lie in different halves of a 128-byte line.
__device__ __forceinline__ int key_of(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

template <typename T, int NG, int NB>
__global__ void __launch_bounds__(kWarps * 32, NG <= 4 && NB == 1 && sizeof(T) == 2 ? 3 : 1)
    attn_few_kernel(const AttnArgs a, const KvCache c, const int max_rows, const Partials part,
                    unsigned int* err) {
  constexpr int D = 32 * NG, R = 8 * NB, S = ring_stages(NG), TB = tile_bytes(NG);
  constexpr int BB = TB / 2;  // bytes of a 16-token block
  constexpr bool kTwo = sizeof(T) == 4;  // float32: hi and lo terms
  constexpr int TERMS = kTwo ? 2 : 1;
  static_assert(R * D * 4 <= warp_smem(NG), "the merge uses a warp's ring");
  extern __shared__ __align__(128) char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  char* ring = smem + warp * warp_smem(NG);
  const uint32_t ring_u = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + kWarps * warp_smem(NG)) + 8u * (warp * S);
  float2* stats = reinterpret_cast<float2*>(smem + kWarps * warp_smem(NG) + kBarBytes);

  if (lane < S) mbar_init(bar0 + 8u * lane, 1);
  mbar_fence_init();
  __syncwarp();

  // ---- this CTA's run of the line
  Walk<kTile, R, kItemCost> w(a, c.page_size, max_rows, 0, c.Hkv, err);
  const long long total = w.total();
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMinRun) per = kMinRun;
  const long long begin = per * blockIdx.x;
  const bool any = begin < total;
  if (any) w.seek(begin);
  if (threadIdx.x == 0) part.start[blockIdx.x] = any ? w.start(begin, per) : Partials::Start{0, 0, 0, 0, 0, 0};
  if (!any) return;
  const long long end = min(begin + per, total);

  uint32_t phases = 0, armed = 0;  // per stage: parity bit, copies under way
  bool failed = false;             // a wait ran out: this warp copies and computes no more
  for (;; w.next_item()) {
    const KvSeq sq = w.s;
    const int ntiles = w.tiles;           // of the item
    const int t_begin = w.tile_at(begin), t_end = w.tile_at(end);
    const bool last = w.tile0 + ntiles >= end;
    if (t_begin == t_end) {  // only (part of) the item's fixed cost lies in this run
      if (last) break;
      continue;
    }
    const int rows = min(R, sq.n * a.G - w.rt * R);
    const int r0 = w.rt * R;              // first row of the item: row = token * G + head
    const int key0 = w.first_key(w.lo);   // first key of tile 0
    const int i_first = r0 / a.G, i_last = (r0 + rows - 1) / a.G;
    const bool masked = a.mask != nullptr;
    const int dbase = sq.len - sq.n;      // first draft key
    // keys that every row of the item sees
    const int full_hi = masked ? dbase : kv_hi(sq, i_first, a.causal, false);
    const int full_lo = kv_lo(sq, i_last, a.window);
    const int key_lo = w.lo, key_end = w.hi;  // (blocks wholly outside are not looked at)

    // ---- the ring: tiles t_begin + warp + 4 k of this warp
    const int* bt = a.block_table + (size_t)w.b * a.max_pages;
    const int page_shift = 31 - __clz(c.page_size);
    // page of lane's block (lane 0, 1) of a tile, or -1
    auto page_id = [&](int tile) {
      const int key = key0 + tile * kTile + (lane & 1) * kKvBlock;
      return (lane < 2 && tile < t_end && key + kKvBlock > key_lo && key < key_end) ? __ldg(bt + (key >> page_shift))
                                                                                    : -1;
    };
    uint32_t valid = 0;  // two bits per stage: the tile's blocks that were copied
    auto issue = [&](int tile, int stage, int page) {
      if (failed || tile >= t_end) return;
      const int key = key0 + tile * kTile + (lane & 1) * kKvBlock;
      const bool want = lane < 2 && key + kKvBlock > key_lo && key < key_end;
      const bool ok = want && page >= 0 && page < c.num_pages;
      const uint32_t okm = __ballot_sync(0xFFFFFFFFu, ok);
      if (__any_sync(0xFFFFFFFFu, want && !ok) && lane == 0 && err) atomicCAS(err, 0u, 1u);
      armed |= 1u << stage;
      valid = (valid & ~(3u << (2 * stage))) | (okm << (2 * stage));
      if (lane == 0) mbar_expect_tx(bar0 + 8u * stage, (uint32_t)__popc(okm) * BB);
      __syncwarp();
      if (ok) {
        const char* src = static_cast<const char*>(c.data) +
                          kv_block_addr(D, c.page_size, c.Hkv, page, w.h, key & (c.page_size - 1));
        bulk_load(ring_u + stage * TB + lane * BB, src, BB, bar0 + 8u * stage);
      }
    };
    int tile = t_begin + warp;
#pragma unroll
    for (int s = 0; s < S; ++s) issue(tile + kWarps * s, s, page_id(tile + kWarps * s));
    int next_page = page_id(tile + kWarps * S);

    // ---- queries as B fragments: lane (g, t) holds dims 8t .. 8t + 7 of every group of row g
    uint32_t qf[NB][NG][2][2][TERMS];  // k-step, register, term
    float qc[NB][NG][4];               // bf16 calls: what the raw codes' offset of 8 adds to a score
    float f0[NB], f1[NB];              // score factor of the lane's accumulator columns 2t, 2t + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g;
      float x[NG][8];
      float amax = 0.0f;
      if (r < rows) {
        const int i = (r0 + r) / a.G, hq = (r0 + r) - i * a.G;
        const T* qp = static_cast<const T*>(a.q) + (long long)(sq.q0 + i) * a.qs.token +
                      (long long)(w.h * a.G + hq) * a.qs.head + 8 * t;
#pragma unroll
        for (int i2 = 0; i2 < NG; ++i2) load8(qp + 32 * i2, x[i2]);
#pragma unroll
        for (int i2 = 0; i2 < NG; ++i2)
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[i2][j]));
      } else {
#pragma unroll
        for (int i2 = 0; i2 < NG; ++i2)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[i2][j] = 0.0f;
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int e = row_exponent(amax);
      const float up = exp2i(14 - e);
#pragma unroll
      for (int i2 = 0; i2 < NG; ++i2)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int rg = 0; rg < 2; ++rg) {
            const int j = 2 * ks + rg;  // nibbles j and j + 4 share a register
            // raw codes: odd nibbles stand 4 bits higher
            const float us = !kTwo && rg ? up * 0.0625f : up;
            split_pair<TERMS>(x[i2][j] * us, x[i2][j + 4] * us, qf[nb][i2][ks][rg]);
          }
      float f = a.scale * 1.44269504088896340736f * exp2i(e - 14);  // to log2 units
      if constexpr (!kTwo) {
#pragma unroll
        for (int i2 = 0; i2 < NG; ++i2) {  // -8 * sum of the group's queries, in the raw codes' units
          float v = 0.0f;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const float2 x0 = half2_of(qf[nb][i2][ks][0][0]), x1 = half2_of(qf[nb][i2][ks][1][0]);
            v += x0.x + x0.y + 16.0f * (x1.x + x1.y);
          }
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
          v *= -8.0f / kRawUnit;
          qc[nb][i2][0] = qc[nb][i2][2] = __shfl_sync(0xFFFFFFFFu, v, 8 * t);
          qc[nb][i2][1] = qc[nb][i2][3] = __shfl_sync(0xFFFFFFFFu, v, 8 * t + 4);
        }
      }
      f0[nb] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);
      f1[nb] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
    }

    // ---- running softmax of columns 2t, 2t + 1, and accumulators
    float m[NB][2], off[NB][2], l[NB][2], o[NB][NG][2][4];
    int ve = kTwo ? kBias : kMinScaleExp;  // exponent field of the largest V scale so far (bf16 calls)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[nb][k] = -CUDART_INF_F;
        off[nb][k] = 0.0f;
        l[nb][k] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nb][i][u][k] = 0.0f;
    }
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t half_sel = (g >> 2) ? 0x7632u : 0x5410u;
    const int kkey = key_of(g);
    const uint32_t k_off = kkey * (D / 2) + ((t ^ (kkey & 2)) * NG) * 4;
    const uint32_t v_off = 8 * D + ((g & 3) ^ (t & 2)) * NG * 4;
    const uint32_t ks_off = 16 * D + kkey * NG * 2, vs_off = ks_off + 16 * NG * 2;

    int stage = 0;
    for (; !failed && tile < t_end; tile += kWarps) {
      const bool landed = mbar_wait_poll(bar0 + 8u * stage, (phases >> stage) & 1u, kWaitLimitNs);
      if (__any_sync(0xFFFFFFFFu, !landed)) {
        failed = true;
        if (lane == 0 && err) atomicCAS(err, 0u, 8u);  // W4A16_ERR_TIMEOUT
        for (int s = 0; s < S; ++s)  // what is still under way writes into this CTA's memory
          if ((armed >> s) & 1u) (void)mbar_wait(bar0 + 8u * s, (phases >> s) & 1u, kWaitLimitNs / 16);
        break;
      }
      phases ^= 1u << stage;
      armed &= ~(1u << stage);
      const uint32_t okm = (valid >> (2 * stage)) & 3u;
      const int kbase = key0 + tile * kTile;
      const bool full = okm == 3u && kbase + kTile <= full_hi && kbase >= full_lo;
      const uint32_t st = ring_u + stage * TB;

      // scores, and the V scales of the lane's keys (C rows g and g + 8 of both blocks)
      float sc[2][NB][4];
      uint32_t vs[2][2][NG / 2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t sb = st + blk * BB;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[blk][nb][k] = 0.0f;
        uint32_t wa[NG], wb[NG], sa[NG / 2], sbk[NG / 2];
        lds_words<NG>(sb + k_off, wa);
        lds_words<NG>(sb + k_off + 4 * D, wb);
        lds_words<NG / 2>(sb + ks_off, sa);
        lds_words<NG / 2>(sb + ks_off + 16 * NG, sbk);
        lds_words<NG / 2>(sb + vs_off, vs[blk][0]);
        lds_words<NG / 2>(sb + vs_off + 16 * NG, vs[blk][1]);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          uint32_t a0[4], a1[4];
          if constexpr (kTwo)
            unpack_pair(wa[i], wb[i], a0, a1);
          else
            raw_pair(wa[i], wb[i], a0, a1);
          const float s0 = bf16_of(sa, i), s1 = bf16_of(sbk, i);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float d[4];
            if constexpr (kTwo)
              mma_f16_zc(d, a0, qf[nb][i][0][0][0], qf[nb][i][0][1][0], zero);
            else
              mma_f16_zc(d, a0, qf[nb][i][0][0][0], qf[nb][i][0][1][0], qc[nb][i]);
            mma_f16(d, a1, qf[nb][i][1][0][0], qf[nb][i][1][1][0]);
            if constexpr (kTwo) {
              mma_f16(d, a0, qf[nb][i][0][0][TERMS - 1], qf[nb][i][0][1][TERMS - 1]);
              mma_f16(d, a1, qf[nb][i][1][0][TERMS - 1], qf[nb][i][1][1][TERMS - 1]);
            }
            sc[blk][nb][0] = fmaf(d[0], s0, sc[blk][nb][0]);
            sc[blk][nb][1] = fmaf(d[1], s0, sc[blk][nb][1]);
            sc[blk][nb][2] = fmaf(d[2], s1, sc[blk][nb][2]);
            sc[blk][nb][3] = fmaf(d[3], s1, sc[blk][nb][3]);
          }
        }
      }
      if (!kTwo) {  // (the factor times the raw codes' unit would pass float32's range for queries of 2^121)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[0][nb][k] *= kRawUnit, sc[1][nb][k] *= kRawUnit;
      }
      float mx[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          sc[blk][nb][0] *= f0[nb];
          sc[blk][nb][2] *= f0[nb];
          sc[blk][nb][1] *= f1[nb];
          sc[blk][nb][3] *= f1[nb];
        }
      }
      if (!full) {  // a border, a draft or a missing page is in this tile
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = kbase + blk * 16 + hf * 8 + kkey;
            const bool there = ((okm >> blk) & 1u) && key >= key_lo && key < key_end;
            bool seen = false;  // by a row of the lane's columns
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int i = min(r0 + nb * 8 + 2 * t + k, r0 + rows - 1) / a.G;
                bool see = there && key < kv_hi(sq, i, a.causal, masked) &&
                           key >= kv_lo(sq, i, a.window);
                if (see && masked && key >= dbase) see = draft_bit(a, sq.q0 + i, key - dbase);
                if (!see) sc[blk][nb][2 * hf + k] = -CUDART_INF_F;
                seen = seen || see;
              }
            // whatever the bytes of a key are that no row sees, they take no part
            const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, seen);
            if (!((lanes >> (lane & 28)) & 15u)) {
#pragma unroll
              for (int k = 0; k < NG / 2; ++k) vs[blk][hf][k] = 0u;
            }
          }
      }
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v = fmaxf(fmaxf(sc[0][nb][k], sc[0][nb][2 + k]), fmaxf(sc[1][nb][k], sc[1][nb][2 + k]));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
          mx[nb][k] = fmaxf(m[nb][k], v);
          grow = grow || mx[nb][k] != m[nb][k];
        }
      int ve2 = ve;
      if constexpr (!kTwo) {
        uint32_t big = 0;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) big = __vmaxu2(big, vs[blk][hf][k] & 0x7FFF7FFFu);
        big = __reduce_max_sync(0xFFFFFFFFu, max(big & 0xFFFFu, big >> 16));
        ve2 = max(ve, min((int)(big >> 7), kMaxScaleExp));
      }
      if (__any_sync(0xFFFFFFFFu, grow || ve2 != ve)) {
        ve = ve2;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // p' = 2^(score - off), off = max - bias: p' * scale < 2^15
            const float on = (mx[nb][k] == -CUDART_INF_F ? 0.0f : mx[nb][k]) - (float)(kBias - ve);
            const float f = m[nb][k] == -CUDART_INF_F ? 0.0f : ex2(off[nb][k] - on);
            off[nb][k] = on;
            m[nb][k] = mx[nb][k];
            l[nb][k] *= f;
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                o[nb][i][u][k] *= f;
                o[nb][i][u][2 + k] *= f;
              }
          }
      }
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc[blk][nb][k] = ex2(sc[blk][nb][k] - off[nb][k & 1]);
            l[nb][k & 1] += sc[blk][nb][k];
          }
      // O^T += V^T P'^T
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t sv = st + blk * BB + v_off;
        uint32_t w0[NG], w1[NG], w2[NG], w3[NG];  // the rows of C rows 2t, 2t + 1, 2t + 8, 2t + 9
        lds_words<NG>(sv + t * (D / 2), w0);
        lds_words<NG>(sv + (4 + (t ^ 1)) * (D / 2), w1);
        lds_words<NG>(sv + (8 + t) * (D / 2), w2);
        lds_words<NG>(sv + (12 + (t ^ 1)) * (D / 2), w3);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          uint32_t px[4], py[4];
          if constexpr (kTwo) {
            unpack_word_bf16(prmt(w0[i], w1[i], half_sel), px);
            unpack_word_bf16(prmt(w2[i], w3[i], half_sel), py);
          } else {
            unpack_word(prmt(w0[i], w1[i], half_sel), px);
            unpack_word(prmt(w2[i], w3[i], half_sel), py);
          }
          const uint32_t A0[4] = {px[0], px[1], py[0], py[1]};
          const uint32_t A1[4] = {px[2], px[3], py[2], py[3]};
          const float s0 = bf16_of(vs[blk][0], i), s1 = bf16_of(vs[blk][1], i);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if constexpr (kTwo) {
              uint32_t pa[3], pb[3];
              split_pair3(sc[blk][nb][0] * s0, sc[blk][nb][1] * s0, pa);
              split_pair3(sc[blk][nb][2] * s1, sc[blk][nb][3] * s1, pb);
              // The terms' products first, small ones before large, then one float32 addition: the tensor
              // core cuts off what falls below its accumulator, and hundreds of products added straight to
              // a running output lost 2.8e-6 of it (draft trees over 9000 keys) where this loses 3.9e-7.
              float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int k = 2; k >= 0; --k) {
                const uint32_t b0 = transpose8x8(pa[k]), b1 = transpose8x8(pb[k]);
                mma_bf16(d0, A0, b0, b1);
                mma_bf16(d1, A1, b0, b1);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[nb][i][0][k] += d0[k];
                o[nb][i][1][k] += d1[k];
              }
            } else {
              uint32_t pa[1], pb[1];
              split_pair<1>(sc[blk][nb][0] * s0, sc[blk][nb][1] * s0, pa);
              split_pair<1>(sc[blk][nb][2] * s1, sc[blk][nb][3] * s1, pb);
              const uint32_t b0 = transpose8x8(pa[0]), b1 = transpose8x8(pb[0]);
              mma_f16(o[nb][i][0], A0, b0, b1);
              mma_f16(o[nb][i][1], A1, b0, b1);
            }
          }
        }
      }
      __syncwarp();  // every lane is done with the stage
      const int ahead = tile + kWarps * S;
      issue(ahead, stage, next_page);
      next_page = page_id(ahead + kWarps);
      stage = stage + 1 == S ? 0 : stage + 1;
    }

    // ---- merge the warps: each writes its rows into its ring (nothing is in flight there)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = l[nb][k];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
        const int r = nb * 8 + 2 * t + k;
        if (g == 0) stats[warp * R + r] = make_float2(v > 0.0f || v != v ? off[nb][k] : -CUDART_INF_F, v);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          float4* dst = reinterpret_cast<float4*>(ring) + r * (D / 4) + 8 * i + 2 * (g & 3) + (g >> 2);
          *dst = make_float4(o[nb][i][0][k], o[nb][i][0][2 + k], o[nb][i][1][k], o[nb][i][1][2 + k]);
        }
      }
    }
    __syncwarp();
    __syncthreads();
    const bool whole = t_begin == 0 && t_end == ntiles;
    const int slot = 2 * blockIdx.x + (t_begin == 0 ? 1 : 0);
    for (int q = threadIdx.x; q < rows * (D / 4); q += kWarps * 32) {
      const int r = q / (D / 4), d4 = q % (D / 4);
      float top = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stats[k * R + r].x);
      float sum = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 sk = stats[k * R + r];
        if (sk.x == -CUDART_INF_F) continue;
        const float f = ex2(sk.x - top);
        const float4 x = reinterpret_cast<const float4*>(smem + k * warp_smem(NG))[r * (D / 4) + d4];
        sum = fmaf(f, sk.y, sum);
        v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
      const float lse2 = sum == 0.0f ? -CUDART_INF_F : top + log2f(sum);
      if (whole) {
        const int i = (r0 + r) / a.G, hq = (r0 + r) - i * a.G;
        const long long at = (long long)(sq.q0 + i) * a.Hq + w.h * a.G + hq;
        store4(static_cast<T*>(a.out) + at * D + 4 * d4, v);
        if (d4 == 0 && a.lse) a.lse[at] = lse2 * 0.69314718055994530942f;
      } else {
        reinterpret_cast<float4*>(part.o)[((long long)slot * R + r) * (D / 4) + d4] = v;
        if (d4 == 0) part.lse2[slot * R + r] = lse2;
      }
    }
    fence_proxy_async_shared();  // the next item's copies overwrite what was just read and written
    __syncthreads();
    if (last) break;
  }
}

template <typename T, int NG, int NB>
cudaError_t launch_few_t(const AttnArgs& a, const KvCache& c, int max_rows, void* ws, cudaStream_t s) {
  constexpr int smem = few_smem(NG);
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce<int> cache;
  const int* occ = nullptr;
  e = cache.get(di.device, [&](int& n) {
    cudaError_t r = cudaFuncSetAttribute(attn_few_kernel<T, NG, NB>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) return r;
    r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_few_kernel<T, NG, NB>, kWarps * 32, smem);
    if (n < 1) n = 1;
    return r;
  }, &occ);
  if (e != cudaSuccess) return e;
  int grid = di.sm_count * *occ;  // (twice as many CTAs only cut more items: 75 us against 64)
  if (grid > kMaxCtas) grid = kMaxCtas;
  const Partials p = Partials::at(ws, 8 * NB, 32 * NG, kMaxCtas);
  attn_few_kernel<T, NG, NB><<<grid, kWarps * 32, smem, s>>>(a, c, max_rows, p, device_error_word());
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attn_merge<T>(a, p, grid, 32 * NG, s);
}

template <typename T>
cudaError_t launch_few(const AttnArgs& a, const KvCache& c, int max_rows, void* ws, cudaStream_t s) {
  // 16 rows a tile where a sequence may bring more than 8: the codes are unpacked once for both column
  // blocks. Heads of 256 dims keep to 8 rows: the accumulators of 16 would not fit in registers.
  const bool wide = (long long)a.max_q * a.G > 8;
  if (c.D == 64)
    return wide ? launch_few_t<T, 2, 2>(a, c, max_rows, ws, s) : launch_few_t<T, 2, 1>(a, c, max_rows, ws, s);
  if (c.D == 128)
    return wide ? launch_few_t<T, 4, 2>(a, c, max_rows, ws, s) : launch_few_t<T, 4, 1>(a, c, max_rows, ws, s);
  return launch_few_t<T, 8, 1>(a, c, max_rows, ws, s);
}

}  // namespace

cudaError_t launch_attn_few(const AttnArgs& a, const KvCache& c, int max_rows, void* ws,
                            cudaStream_t s) {
  return a.bf16 ? launch_few<__nv_bfloat16>(a, c, max_rows, ws, s)
                : launch_few<float>(a, c, max_rows, ws, s);
}

}  // namespace w4a16
