// Products of 8-bit rows: out = (a b^T) times the scales of a row and a column.
//
// Mathematics.  The integers' sum is exact in 32 bits (at most 131071 products
// of at most 2^14); it is rounded to fp32 once and multiplied by the product of
// the two scales.
#include "linear8.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kTile = 64, kStep = 64, kPitch = kStep + 4;

template <typename T>
__global__ __launch_bounds__(256) void matmul8_simple_kernel(Matmul8Args a) {
  __shared__ int8_t ta[kTile * kPitch], tb[kTile * kPitch];
  const int64_t tiles_n = (a.n + kTile - 1) / kTile;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) / tiles_n * kTile, n0 = static_cast<int64_t>(blockIdx.x) % tiles_n * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.k; k0 += kStep) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      const int r = e / kStep, c = e % kStep;
      const bool in = k0 + c < a.k;
      ta[r * kPitch + c] = in && m0 + r < a.m ? a.a.p[(m0 + r) * a.a.ld + k0 + c] : 0;
      tb[r * kPitch + c] = in && n0 + r < a.n ? a.b.p[(n0 + r) * a.b.ld + k0 + c] : 0;
    }
    __syncthreads();
    for (int c = 0; c < kStep; c += 4) {
      int va[4], vb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) va[i] = *reinterpret_cast<const int*>(ta + (ty + 16 * i) * kPitch + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) vb[j] = *reinterpret_cast<const int*>(tb + (tx + 16 * j) * kPitch + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_sdot4(va[i], vb[j], acc[i][j], false);
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.m && n < a.n)
        muon::Elem<T>::store(reinterpret_cast<T*>(a.out.p) + m * a.out.ld + n,
                             static_cast<float>(acc[i][j]) * (a.a.scale[m] * a.b.scale[n]));
    }
}

}  // namespace

hipError_t launch_matmul8(hipStream_t s, const Matmul8Args& a) {
  if (a.m == 0 || a.n == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>(((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile));
  if (a.out.bf16) matmul8_simple_kernel<bf16_t><<<grid, 256, 0, s>>>(a);
  else matmul8_simple_kernel<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
