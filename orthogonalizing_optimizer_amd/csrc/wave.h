// Reductions over the lanes of a wave without LDS.
//
// A value that is equal in all lanes of a group of O lanes is exchanged with
// the neighbouring group's by a DPP move (one vector instruction, against a
// round trip through LDS for a shuffle): inside a quad by its permutations,
// between quads and eights by mirrors of half a row and of a row, which reach
// another lane of the right group.  Every lane of the wave must be active.
#pragma once

#include <hip/hip_runtime.h>

namespace dion3 {
namespace {

// The value of the other group of O lanes, O = 1, 2, 4, 8; v is equal in groups of O.
template <int O>
__device__ __forceinline__ float other(float v) {
  constexpr int ctrl = O == 1 ? 0xB1 : O == 2 ? 0x4E : O == 4 ? 0x141 : 0x140;
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl,
                                                               0xF, 0xF, true));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// op over groups of G lanes (a power of two), the same bits in every lane of one.
template <class F>
__device__ __forceinline__ float group_reduce(float v, int G, F op) {
  if (G > 1) v = op(v, other<1>(v));
  if (G > 2) v = op(v, other<2>(v));
  if (G > 4) v = op(v, other<4>(v));
  if (G > 8) v = op(v, other<8>(v));
  if (G > 16) v = op(v, __shfl_xor(v, 16, 64));
  if (G > 32) v = op(v, __shfl_xor(v, 32, 64));
  return v;
}

// op over the wave.
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F op) {
  v = op(v, other<1>(v));
  v = op(v, other<2>(v));
  v = op(v, other<4>(v));
  v = op(v, other<8>(v));
  return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ float wave_add(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
}  // namespace dion3
