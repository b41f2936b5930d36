// Gradients of an 8-bit linear layer: out = op(y) diag(scale) q, with y in bf16
// and q the 8-bit rows, both with the contraction index as a memory row:
//   weights: sum over tokens of grad_y (columns) and the kept activations,
//   inputs:  sum over channels of grad_y (rows) and the weights.
#include "linear8.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kTile = 64, kStep = 16, kPitch = kTile + 4;

// Sums in fp32 of exact values, for any addresses and strides.
template <typename T>
__global__ __launch_bounds__(256) void grad8_simple_kernel(Grad8Args a) {
  __shared__ float ty[kStep * kPitch], tq[kStep * kPitch];
  const bf16_t* y = reinterpret_cast<const bf16_t*>(a.y.p);
  const int64_t tiles_n = (a.n + kTile - 1) / kTile;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) / tiles_n * kTile, n0 = static_cast<int64_t>(blockIdx.x) % tiles_n * kTile;
  const int jx = threadIdx.x & 15, ix = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t c0 = 0; c0 < a.c; c0 += kStep) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      const int i = a.of_columns ? e % kTile : e / kStep, ci = a.of_columns ? e / kTile : e % kStep;
      float v = 0.0f;
      if (m0 + i < a.m && c0 + ci < a.c)
        v = muon::bf16_to_f32(a.of_columns ? y[(c0 + ci) * a.y.ld + m0 + i] : y[(m0 + i) * a.y.ld + c0 + ci]);
      ty[ci * kPitch + i] = v;
      const int j = e % kTile, cj = e / kTile;
      v = 0.0f;
      if (n0 + j < a.n && c0 + cj < a.c) v = a.q.scale[c0 + cj] * static_cast<float>(a.q.p[(c0 + cj) * a.q.ld + n0 + j]);
      tq[cj * kPitch + j] = v;
    }
    __syncthreads();
    for (int c = 0; c < kStep; ++c) {
      float vy[4], vq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) vy[i] = ty[c * kPitch + ix + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) vq[j] = tq[c * kPitch + jx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(vy[i], vq[j], acc[i][j]);
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ix + 16 * i, n = n0 + jx + 16 * j;
      if (m >= a.m || n >= a.n) continue;
      T* at = reinterpret_cast<T*>(a.out.p) + m * a.out.ld + n;
      muon::Elem<T>::store(at, a.accumulate ? muon::Elem<T>::load(at) + acc[i][j] : acc[i][j]);
    }
}

}  // namespace

hipError_t launch_grad8(hipStream_t s, const Grad8Args& a) {
  if (a.m == 0 || a.n == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>(((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile));
  if (a.out.bf16) grad8_simple_kernel<bf16_t><<<grid, 256, 0, s>>>(a);
  else grad8_simple_kernel<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
