// Rows of values in 8 bits, a scale per row, and back.
//
// Mathematics.  s = max |x| / 127 in binary32; q is the integer nearest to the
// exact x / s, ties to even.  x / s is formed as x (1 / s): its error, below
// 2^-22 of the quotient (|q| <= 127: 2^-15), matters only next to a half, where
// the remainder x - q s (exact as one fused multiply-add: |x - q s| <= s, and
// both are multiples of the smaller's last place) is compared with s / 2.
#include "linear8.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kThreads = 256;
constexpr float kMostScale = 0x1.020406p+121f;  // 127 times the next larger number overflows

// x / s to the nearest integer, ties to even, given an estimate of it.
__device__ __forceinline__ float nearest(float x, float s, float estimate) {
  float q = rintf(estimate);
  const float r = __builtin_fmaf(-q, s, x);  // exact
  const float over = 2.0f * fabsf(r);
  if (over >= s) {
    // at or past the half: the neighbour on r's side, or of two the even one
    const float next = q + copysignf(1.0f, r);
    const bool odd = (static_cast<int>(q) & 1) != 0;
    if (over > s || odd) q = next;
  }
  return fminf(fmaxf(q, -127.0f), 127.0f);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                                                            int64_t rows, int cols) {
  __shared__ float wave_top[kThreads / 64];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* row = x + r * ldx;
    // the largest magnitude by its bits: NaN and infinity come out on top
    uint32_t top = 0;
    for (int c = threadIdx.x; c < cols; c += kThreads)
      top = max(top, __float_as_uint(muon::Elem<T>::load(row + c)) & 0x7fffffffu);
    for (int d = 32; d > 0; d /= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = __uint_as_float(top);
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) top = max(top, __float_as_uint(wave_top[w]));
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : fminf(__uint_as_float(top) / 127.0f, kMostScale);
    if (threadIdx.x == 0) scale[r] = s;
    const bool zero = bad || s == 0.0f;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
      const float v = muon::Elem<T>::load(row + c);
      // (1 / s overflows where s is denormal: the quotient itself then)
      q[r * ldq + c] = zero ? 0 : static_cast<int8_t>(nearest(v, s, s < 1.2e-38f ? v / s : v * (1.0f / s)));
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const int8_t* q, int64_t ldq, const float* scale, T* out,
                                                              int64_t ldo, int64_t rows, int cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float s = scale[r];
    for (int c = threadIdx.x; c < cols; c += kThreads)
      muon::Elem<T>::store(out + r * ldo + c, s * static_cast<float>(q[r * ldq + c]));
  }
}

unsigned row_grid(int64_t rows) { return static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20)); }

}  // namespace

hipError_t launch_quantize_rows(hipStream_t s, Values x, Bytes q, int64_t rows, int cols) {
  if (rows == 0) return hipSuccess;
  if (x.bf16)
    quantize_kernel<bf16_t><<<row_grid(rows), kThreads, 0, s>>>(reinterpret_cast<const bf16_t*>(x.p), x.ld, q.p, q.ld, q.scale, rows, cols);
  else
    quantize_kernel<float><<<row_grid(rows), kThreads, 0, s>>>(reinterpret_cast<const float*>(x.p), x.ld, q.p, q.ld, q.scale, rows, cols);
  return hipGetLastError();
}

hipError_t launch_dequantize_rows(hipStream_t s, Bytes q, Values out, int64_t rows, int cols) {
  if (rows == 0) return hipSuccess;
  if (out.bf16)
    dequantize_kernel<bf16_t><<<row_grid(rows), kThreads, 0, s>>>(q.p, q.ld, q.scale, reinterpret_cast<bf16_t*>(out.p), out.ld, rows, cols);
  else
    dequantize_kernel<float><<<row_grid(rows), kThreads, 0, s>>>(q.p, q.ld, q.scale, reinterpret_cast<float*>(out.p), out.ld, rows, cols);
  return hipGetLastError();
}
