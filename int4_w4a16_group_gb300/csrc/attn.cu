// Attention over the paged 4-bit cache: which kernel takes which sequences, and the workspace.
#include <limits.h>

#include "attn_core.cuh"

namespace w4a16 {
namespace {

// bf16 sequences of more rows per key/value head than this go to the tcgen05 kernel. 8 rows a token, heads of 128
// (few / many, us): 4 sequences of 6000 tokens: 24 rows 34 / 41, 32 rows 34 / 41, 48 rows 43 / 43, 64 rows 52 / 43,
// 128 rows 91 / 45, 256 rows 163 / 55; 32 of 2000: 24 rows 71 / 81, 32 rows 74 / 84, 48 rows 100 / 85, 64 rows 129 /
// 85; one of 6000: 32 rows 22 / 25, 64 rows 25 / 26, 128 rows 35 / 28. float32 calls and heads of 256 dims have no such kernel:
// their rows go through the other in tiles of 16 (8), which read the keys from L2 again.
constexpr int kManyRows = 32;

bool many(bool bf16, int D, int G, int max_q) {
  return bf16 && D <= 128 && (long long)max_q * G > kManyRows;
}

}  // namespace

// The two kernels run one after the other and share the workspace.
size_t attn_workspace_size(int T, int B, int Hkv, int G, int D, int max_q) {
  const size_t few = Partials::bytes(16, D, kMaxCtas);
  const size_t big = many(true, D, G, max_q) ? Partials::bytes(256, D, kMaxManyCtas) : 0;
  return few > big ? few : big;
}

cudaError_t launch_attention(const AttnArgs& a, const KvCache& c, void* ws, size_t ws_bytes,
                             cudaStream_t s) {
  if (!many(a.bf16, c.D, a.G, a.max_q)) return launch_attn_few(a, c, INT_MAX, ws, s);
  // one sequence goes to one kernel, whatever its rows turn out to be
  if (a.B == 1) return launch_attn_many(a, c, 0, ws, s);
  const cudaError_t e = launch_attn_many(a, c, kManyRows, ws, s);
  if (e != cudaSuccess) return e;
  return launch_attn_few(a, c, kManyRows, ws, s);
}

}  // namespace w4a16
