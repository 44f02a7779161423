// Parts of the kernels that norm and turn rows of heads (norm_rope.hip, paged_append.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace trsc {

constexpr int kRowElts = 4;  // elements of either half of a row in a lane

// (cos, sin) of this lane's pair at token t into the wave's table.
__device__ __forceinline__ void turn_table(int32_t p, double freq_turns, bool turns, int lane, float2* table) {
  float2 cs = make_float2(1.f, 0.f);
  if (turns) {
    const double t = double(p) * freq_turns;
    const float f = float(t - rint(t));
    sincospif(2.f * f, &cs.y, &cs.x);
  }
  table[lane] = cs;
}

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Lanes that share a row: a power of two, dim / (2 kRowElts) or more.
inline int group_lanes(int dim) {
  const int lanes = dim / (2 * kRowElts);
  int g = 1;
  while (g < lanes) g <<= 1;
  return g;
}

}  // namespace trsc
