// Internal interface of the attention operators (rotary positions, paged 4-bit cache, attention
// over it): launchers, called by attn_abi.cu with validated arguments.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "heads.h"

namespace w4a16 {

struct RopeTableArgs {
  int P, rot, scaling, original;
  double base, factor, beta_fast, beta_slow, gain;
};
cudaError_t launch_rope_table(float* table, const RopeTableArgs& a, cudaStream_t s);

struct RopeArgs {
  const int32_t* positions;
  const float* table;
  int P, rot, interleaved;
};
cudaError_t launch_rope(const void* x, HeadStrides xs, void* y, HeadStrides ys, bool bf16, int T,
                        int H, int D, const RopeArgs& r, bool inverse, cudaStream_t s);

struct KvCache {
  void* data;
  int num_pages, page_size, Hkv, D;
};
// r.rot == 0: keys are stored as they come.
cudaError_t launch_kv_append(const void* k, HeadStrides ks, const void* v, HeadStrides vs,
                             bool bf16, int T, const int64_t* slots, const RopeArgs& r,
                             const KvCache& c, cudaStream_t s);
cudaError_t launch_kv_read(const KvCache& c, const int64_t* slots, int T, float* k, float* v,
                           cudaStream_t s);

struct AttnArgs {
  const void* q;
  HeadStrides qs;
  bool bf16;
  int T, B, Hq, G;             // G = Hq / Hkv query heads per key/value head
  const int32_t* block_table;  // [B, max_pages]
  int max_pages;
  const int32_t* kv_lens;      // [B]
  const int32_t* q_starts;     // [B + 1]
  int max_q;
  float scale;
  int causal, window;
  const uint32_t* mask;        // [T, mask_words] or null
  int mask_words;
  void* out;                   // [T, Hq, D], the type of q
  float* lse;                  // [T, Hq] or null
};
size_t attn_workspace_size(int T, int B, int Hkv, int G, int D, int max_q);
cudaError_t launch_attention(const AttnArgs& a, const KvCache& c, void* ws, size_t ws_bytes,
                             cudaStream_t s);

// Records the CUDA error behind a W4A16_ERR_CUDA of this thread (abi.cu).
void set_last_cuda_error(int e);

}  // namespace w4a16
