// Strided [tokens, heads, D] activations: the strides, and whether a layout's heads lie apart. Plain host code.
#pragma once
#include <stdint.h>

namespace w4a16 {

// Strides in elements of a [tokens, heads, D] tensor whose last dimension is contiguous.
struct HeadStrides {
  long long token, head;
};

// Whether no two of the T x H heads of D elements share one. Heads (t, h) and (t + dt, h + dh) are dt * token +
// dh * head apart, so for each dh the possible dt closest to -dh * head / token decide.
inline bool heads_disjoint(int T, int H, HeadStrides s, int D) {
  const __int128 far = D, st = s.token, sh = s.head;
  if ((H == 1 || sh >= far) && (T == 1 || st >= (H - 1) * sh + far)) return true;  // tokens of whole heads, as usual
  auto apart = [&](__int128 dt, __int128 dh) {
    if (dt > T - 1 || dt < -(T - 1)) return true;  // no such pair
    const __int128 x = dt * st + dh * sh;
    return x >= far || -x >= far;
  };
  if (T > 1 && !apart(1, 0)) return false;
  for (int dh = 1; dh < H; ++dh) {
    __int128 dt = st ? -(dh * sh) / st : 0;
    dt = dt > T - 1 ? T - 1 : (dt < -(T - 1) ? -(T - 1) : dt);
    if (!apart(dt, dh) || !apart(dt - 1, dh) || !apart(dt + 1, dh)) return false;
  }
  return true;
}

}  // namespace w4a16
