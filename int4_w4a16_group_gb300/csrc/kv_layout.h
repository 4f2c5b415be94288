// Layout of the paged 4-bit key/value cache and the index arithmetic of its readers, shared by the
// kernels and by host code (every function here is plain integer arithmetic, tested on the CPU).
//
// cache [num_pages][Hkv][page_size / 16 blocks]; a block holds 16 consecutive tokens of one head:
//   K codes 16 x D/2 B | V codes 16 x D/2 B | K scales 16 x D/32 bf16 | V scales 16 x D/32 bf16
// so any run of whole blocks inside a page is one contiguous piece with everything attention needs.
// In a token's row of codes (r = token in the block) the 32-bit word (w ^ (r & 2)) * D/32 + i holds
// dims 32 i + 8 w .. + 7, lowest nibble first, code = nibble - 8: the D/32 words that one lane of an
// MMA fragment needs are adjacent (one wide shared-memory load), and the XOR spreads the rows that
// eight neighbouring lanes read over all banks.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define W4A16_HD __host__ __device__ __forceinline__
#else
#define W4A16_HD inline
#endif

namespace w4a16 {

constexpr int kKvBlock = 16;  // tokens per block
constexpr int kKvGroup = 32;  // dims per scale

W4A16_HD bool kv_head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }
W4A16_HD bool kv_page_size_ok(int S) { return S == 16 || S == 32 || S == 64 || S == 128; }

// Bytes of one block, and the parts' offsets inside it.
W4A16_HD int kv_block_bytes(int D) { return kKvBlock * (D + D / 8); }
W4A16_HD int kv_codes_off(int D, int is_v) { return is_v * kKvBlock * D / 2; }
W4A16_HD int kv_scales_off(int D, int is_v) {
  return kKvBlock * D + is_v * kKvBlock * (D / kKvGroup) * 2;
}
// Byte offset of word w of group i in the row of token r (0..15) of a block's codes.
W4A16_HD int kv_word_off(int D, int r, int w, int i) {
  return r * (D / 2) + ((w ^ (r & 2)) * (D / kKvGroup) + i) * 4;
}
W4A16_HD int kv_scale_off(int D, int r, int i) { return (r * (D / kKvGroup) + i) * 2; }

// Byte offset of the block that holds token `off` (0 .. page_size - 1) of a page and head.
W4A16_HD size_t kv_block_addr(int D, int page_size, int Hkv, long long page, int head, int off) {
  return ((size_t)page * Hkv + head) * ((size_t)(page_size / kKvBlock) * kv_block_bytes(D)) +
         (size_t)(off / kKvBlock) * kv_block_bytes(D);
}

// Query tokens and visible keys of one sequence, from device data that may be malformed: counts
// are clamped to what the arrays hold; *bad is set when anything had to be.
struct KvSeq {
  int q0, n;   // first query token, query tokens
  int len;     // cached tokens (the queries' own among them)
};
W4A16_HD KvSeq kv_sequence(int q_begin, int q_end, int kv_len, int T, int max_tokens, bool* bad) {
  KvSeq s;
  int b = q_begin < 0 ? 0 : (q_begin > T ? T : q_begin);
  int e = q_end < b ? b : (q_end > T ? T : q_end);
  int l = kv_len < 0 ? 0 : (kv_len > max_tokens ? max_tokens : kv_len);
  if (b != q_begin || e != q_end || l != kv_len) *bad = true;
  s.q0 = b;
  s.n = e - b;
  s.len = l;
  return s;
}

// Keys [lo, hi) that query token i of a sequence may see by position (a draft mask takes out more).
W4A16_HD int kv_hi(const KvSeq& s, int i, int causal, bool masked) {
  if (masked || !causal) return s.len;
  const int p = s.len - s.n + i + 1;
  return p < 0 ? 0 : p;
}
W4A16_HD int kv_lo(const KvSeq& s, int i, int window) {
  if (window <= 0) return 0;
  const int p = s.len - s.n + i + 1;
  return p <= window ? 0 : p - window;  // (p - window first would overflow for p < 0 and the largest windows)
}

}  // namespace w4a16
