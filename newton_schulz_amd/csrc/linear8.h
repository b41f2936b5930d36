// Host-side declarations of the launchers of 8-bit rows, their products and
// gradients (rows8.hip, matmul8.hip, grad8.hip) and of draft verification
// (verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "loss_kernels.h"
#include "muon.h"

struct Values {  // rows of bf16 or fp32, ld elements apart
  char* p;
  int bf16;
  int64_t ld;
};
struct Bytes {  // 8-bit rows, ld bytes apart (a multiple of 16)
  int8_t* p;
  float* scale;
  int64_t ld;
};

hipError_t launch_quantize_rows(hipStream_t s, Values x, Bytes q, int64_t rows, int cols);
hipError_t launch_dequantize_rows(hipStream_t s, Bytes q, Values out, int64_t rows, int cols);

// out[m][n] = sum_k a[m][k] b[n][k] * (sa[m] sb[n])
struct Matmul8Args {
  Bytes a, b;
  Values out;
  int64_t m, n;
  int k;
  int cus;
};
hipError_t launch_matmul8(hipStream_t s, const Matmul8Args& a);

// out[i][j] (+)= sum_c y(i, c) scale[c] q[c][j]; y(i, c) at y[i][c], or, of_columns, at y[c][i]
struct Grad8Args {
  Values y;
  int of_columns;
  Bytes q;
  Values out;
  int64_t m, n, c;
  int accumulate;
  int cus;
};
hipError_t launch_grad8(hipStream_t s, const Grad8Args& a);

struct VerifyArgs {
  RowsRef x;       // target: batch x (draft + 1) rows
  int x_bf16;
  RowsRef d;       // draft: batch x draft rows; base nullptr: deterministic
  int d_bf16;
  int batch, draft, vocab;
  const int64_t* drafted;
  const float* uniforms;
  double inv_t;    // 1 / temperature; 0: greedy
  int64_t* tokens;
  int64_t* accepted;
  float* logps;
};
hipError_t launch_verify(hipStream_t s, const VerifyArgs& a);
