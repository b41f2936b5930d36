// Reductions over a wave (device functions).
#pragma once

#include <hip/hip_runtime.h>

namespace muon {

// The maximum and the sum over a wave, in every lane; all lanes take part.
// Quads, then halves and mirrors of 16 lanes, then the rows of 16 into the last
// one: no LDS, and a fixed order.
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ float max_step(float v) {
  const int w = __float_as_int(v);
  return fmaxf(v, __int_as_float(dpp<CTRL, ROWS>(w, w)));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double sum_step(double v) {
  return v + __hiloint2double(dpp<CTRL, ROWS>(0, __double2hiint(v)), dpp<CTRL, ROWS>(0, __double2loint(v)));
}
constexpr int kQuad1 = 0xb1, kQuad2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140, kLane15 = 0x142, kLane31 = 0x143;
__device__ __forceinline__ float wave_max(float v) {
  v = max_step<kQuad1, 0xf>(v);
  v = max_step<kQuad2, 0xf>(v);
  v = max_step<kHalfMirror, 0xf>(v);
  v = max_step<kMirror, 0xf>(v);
  v = max_step<kLane15, 0xa>(v);
  v = max_step<kLane31, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
  v = sum_step<kQuad1, 0xf>(v);
  v = sum_step<kQuad2, 0xf>(v);
  v = sum_step<kHalfMirror, 0xf>(v);
  v = sum_step<kMirror, 0xf>(v);
  v = sum_step<kLane15, 0xa>(v);
  v = sum_step<kLane31, 0xc>(v);
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                          __builtin_amdgcn_readlane(__double2loint(v), 63));
}

}  // namespace muon
