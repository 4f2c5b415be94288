// C ABI of the attention operators (declared in include/w4a16.h): argument checks and dispatch to
// the launchers in rope.cu, kv_cache.cu and attn.cu.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/w4a16.h"
#include "attn.h"
#include "internal.h"
#include "kv_layout.h"

using namespace w4a16;

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline w4a16_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return W4A16_OK;
  set_last_cuda_error((int)e);
  return W4A16_ERR_CUDA;
}

inline bool dtype_ok(int dtype) { return dtype == W4A16_F32 || dtype == W4A16_BF16; }

// Strides keep every head 16-byte aligned.
inline bool strides_ok(int dtype, int64_t token, int64_t head) {
  const int64_t n = dtype == W4A16_BF16 ? 8 : 4;
  return token % n == 0 && head % n == 0;
}

// The cache's kernels step through tokens with 32-bit counters, up to a whole grid (below 2^24) past the last one.
constexpr int kMaxCacheTokens = INT_MAX - (1 << 24);
// They have a thread for every 8 dims of a token's keys and values, in at most 65535 rows of blocks of 256.
inline bool cache_grid_ok(int T, int Hkv, int D) {
  return T <= kMaxCacheTokens && (long long)Hkv * (D / 4) <= 65535ll * 256;
}

inline w4a16_status check_cache(const void* cache, int num_pages, int page_size, int Hkv, int D) {
  if (Hkv <= 0 || num_pages < 0 || D <= 0) return W4A16_ERR_ARG;
  if (!kv_head_dim_ok(D) || !kv_page_size_ok(page_size)) return W4A16_ERR_UNSUPPORTED;
  if (num_pages > 0 && !cache) return W4A16_ERR_ARG;
  if (!aligned16(cache)) return W4A16_ERR_ALIGN;
  return W4A16_OK;
}

}  // namespace

extern "C" {

w4a16_status w4a16_rope_table(float* table, int P, int rot, double base, int scaling,
                              double factor, int original, double beta_fast, double beta_slow,
                              double gain, w4a16_stream_t stream) {
  if (P < 0 || rot <= 0 || rot % 2 != 0 || !(base > 1.0) || !isfinite(base) || !isfinite(gain))
    return W4A16_ERR_ARG;
  if (scaling < W4A16_ROPE_NONE || scaling > W4A16_ROPE_YARN) return W4A16_ERR_ARG;
  if (scaling != W4A16_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor))) return W4A16_ERR_ARG;
  if (scaling == W4A16_ROPE_YARN &&
      (original <= 0 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !isfinite(beta_fast)))
    return W4A16_ERR_ARG;
  if (P > (1 << 30) || rot > 65536) return W4A16_ERR_UNSUPPORTED;
  if (P == 0) return W4A16_OK;
  if (!table) return W4A16_ERR_ARG;
  if (!aligned16(table)) return W4A16_ERR_ALIGN;
  const RopeTableArgs a = {P, rot, scaling, original, base, factor, beta_fast, beta_slow, gain};
  return cuda_status(launch_rope_table(table, a, (cudaStream_t)stream));
}

w4a16_status w4a16_rope(const void* x, int64_t x_token, int64_t x_head, int dtype, int T, int H,
                        int D, const int32_t* positions, const float* table, int P, int rot,
                        int interleaved, int inverse, void* y, int64_t y_token, int64_t y_head,
                        w4a16_stream_t stream) {
  if (!dtype_ok(dtype) || T < 0 || H < 0 || D <= 0 || D % 8 != 0) return W4A16_ERR_ARG;
  if (rot <= 0 || rot % 2 != 0 || rot > D || P <= 0) return W4A16_ERR_ARG;
  if (T == 0 || H == 0) return W4A16_OK;
  if (!x || !y || !positions || !table) return W4A16_ERR_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(table) || ((uintptr_t)positions & 3u))
    return W4A16_ERR_ALIGN;
  if (!strides_ok(dtype, x_token, x_head) || !strides_ok(dtype, y_token, y_head))
    return W4A16_ERR_ALIGN;
  if (x == y && (x_token != y_token || x_head != y_head)) return W4A16_ERR_ARG;
  if (!heads_disjoint(T, H, {y_token, y_head}, D)) return W4A16_ERR_ARG;
  const RopeArgs r = {positions, table, P, rot, interleaved ? 1 : 0};
  return cuda_status(launch_rope(x, {x_token, x_head}, y, {y_token, y_head}, dtype == W4A16_BF16,
                                 T, H, D, r, inverse != 0, (cudaStream_t)stream));
}

size_t w4a16_kv_page_bytes(int Hkv, int D, int page_size) {
  if (Hkv <= 0 || !kv_head_dim_ok(D) || !kv_page_size_ok(page_size)) return 0;
  return (size_t)Hkv * (page_size / kKvBlock) * kv_block_bytes(D);
}

w4a16_status w4a16_kv_append(const void* k, int64_t k_token, int64_t k_head, const void* v,
                             int64_t v_token, int64_t v_head, int dtype, int T, int Hkv, int D,
                             const int64_t* slots, const int32_t* positions, const float* table,
                             int P, int rot, int interleaved, void* cache, int num_pages,
                             int page_size, w4a16_stream_t stream) {
  const w4a16_status st = check_cache(cache, num_pages, page_size, Hkv, D);
  if (st != W4A16_OK) return st;
  if (!dtype_ok(dtype) || T < 0 || rot < 0 || rot % 2 != 0 || rot > D) return W4A16_ERR_ARG;
  if (rot > 0 && P <= 0) return W4A16_ERR_ARG;
  if (!cache_grid_ok(T, Hkv, D)) return W4A16_ERR_UNSUPPORTED;
  if (T == 0) return W4A16_OK;
  if (!k || !v || !slots || (rot > 0 && (!positions || !table))) return W4A16_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 7u)) return W4A16_ERR_ALIGN;
  if (rot > 0 && (!aligned16(table) || ((uintptr_t)positions & 3u))) return W4A16_ERR_ALIGN;
  if (!strides_ok(dtype, k_token, k_head) || !strides_ok(dtype, v_token, v_head))
    return W4A16_ERR_ALIGN;
  const RopeArgs r = {positions, table, P, rot, interleaved ? 1 : 0};
  const KvCache c = {cache, num_pages, page_size, Hkv, D};
  return cuda_status(launch_kv_append(k, {k_token, k_head}, v, {v_token, v_head},
                                      dtype == W4A16_BF16, T, slots, r, c, (cudaStream_t)stream));
}

w4a16_status w4a16_kv_read(const void* cache, int num_pages, int page_size, int Hkv, int D,
                           const int64_t* slots, int T, float* k, float* v,
                           w4a16_stream_t stream) {
  const w4a16_status st = check_cache(cache, num_pages, page_size, Hkv, D);
  if (st != W4A16_OK) return st;
  if (T < 0) return W4A16_ERR_ARG;
  if (!cache_grid_ok(T, Hkv, D)) return W4A16_ERR_UNSUPPORTED;
  if (T == 0) return W4A16_OK;
  if (!slots || !k || !v) return W4A16_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 7u)) return W4A16_ERR_ALIGN;
  const KvCache c = {const_cast<void*>(cache), num_pages, page_size, Hkv, D};
  return cuda_status(launch_kv_read(c, slots, T, k, v, (cudaStream_t)stream));
}

size_t w4a16_attention_workspace_size(int T, int B, int Hkv, int G, int D, int max_q) {
  if (T < 0 || B < 0 || Hkv <= 0 || G <= 0 || !kv_head_dim_ok(D) || max_q < 0) return 0;
  return attn_workspace_size(T, B, Hkv, G, D, max_q);
}

w4a16_status w4a16_attention(const void* q, int64_t q_token, int64_t q_head, int dtype, int T,
                             int Hq, const void* cache, int num_pages, int page_size, int Hkv,
                             int D, const int32_t* block_table, int max_pages, int B,
                             const int32_t* kv_lens, const int32_t* q_starts, int max_q,
                             float scale, int causal, int window, const uint32_t* tree_mask,
                             int mask_words, void* out, float* lse, void* workspace,
                             size_t ws_bytes, w4a16_stream_t stream) {
  const w4a16_status st = check_cache(cache, num_pages, page_size, Hkv, D);
  if (st != W4A16_OK) return st;
  if (!dtype_ok(dtype) || T < 0 || Hq <= 0 || Hq % Hkv != 0 || B < 0) return W4A16_ERR_ARG;
  if (max_pages < 0 || max_pages > (1 << 30) / page_size || max_q < 0 || window < 0)
    return W4A16_ERR_ARG;
  if (Hq / Hkv > 128 || (long long)T * Hq > (1ll << 31) - 1) return W4A16_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !isfinite(scale)) return W4A16_ERR_ARG;
  // a draft mask says by itself what a draft token sees; a window or a non-causal call beside it
  // would have no meaning
  if (tree_mask && (window > 0 || !causal || mask_words <= 0)) return W4A16_ERR_ARG;
  if (window > 0 && !causal) return W4A16_ERR_ARG;
  if (T == 0) return W4A16_OK;
  if (B == 0 || !q || !out || !kv_lens || !q_starts || (max_pages > 0 && !block_table))
    return W4A16_ERR_ARG;
  if (!aligned16(q) || !aligned16(out)) return W4A16_ERR_ALIGN;
  if (((uintptr_t)kv_lens | (uintptr_t)q_starts | (uintptr_t)block_table | (uintptr_t)tree_mask |
       (uintptr_t)lse) & 3u)
    return W4A16_ERR_ALIGN;
  if (!strides_ok(dtype, q_token, q_head)) return W4A16_ERR_ALIGN;
  const size_t need = attn_workspace_size(T, B, Hkv, Hq / Hkv, D, max_q);
  if (!workspace || ws_bytes < need) return W4A16_ERR_WORKSPACE;
  if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
  AttnArgs a = {};
  a.q = q;
  a.qs = {q_token, q_head};
  a.bf16 = dtype == W4A16_BF16;
  a.T = T, a.B = B, a.Hq = Hq, a.G = Hq / Hkv;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.kv_lens = kv_lens;
  a.q_starts = q_starts;
  a.max_q = max_q;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.window = window;
  a.mask = tree_mask;
  a.mask_words = mask_words;
  a.out = out;
  a.lse = lse;
  const KvCache c = {const_cast<void*>(cache), num_pages, page_size, Hkv, D};
  return cuda_status(launch_attention(a, c, workspace, ws_bytes, (cudaStream_t)stream));
}

}  // extern "C"
