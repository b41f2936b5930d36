// Host-side declarations of the loss kernels' launchers (loss.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

// Rows of scores: row r = (r / seq, r % seq) starts bs, rs bytes apart.
struct RowsRef {
  char* base;
  int64_t bs, rs;
};

struct LossArgs {
  RowsRef x;
  int bf16;
  int rows, seq, vocab;
  int row0;          // first row of this launch (set by the launchers)
  const int64_t* labels;
  float temperature;
  int splits;        // workgroups a row's statistics are split over
  float2* part;      // [rows][splits] (maximum, sum around it) of each split
  double* lp;        // [rows]
  float* logps;      // [rows] or nullptr
  float2* stats;     // [rows] (maximum, sum) of the whole row
};

// Workgroups to split each row's statistics over.
int loss_splits(int64_t rows, int64_t vocab, int bf16, int cus);

// stats, lp and logps of every row (logps of tokens left out: 0).
hipError_t launch_row_stats(hipStream_t s, const LossArgs& a);

// grad row r = g[r] / temperature * ([v = y] - softmax); zeros for tokens left out.
hipError_t launch_logits_grad(hipStream_t s, const LossArgs& a, RowsRef grad, const float* g);

// The policy loss of given log-probabilities: out[4] and (g not null) the
// gradient of weight * loss in each of them.
struct PolicyArgs {
  muon_policy_params_t p;
  int batch, seq;
  const int64_t* labels;
  const double* lp;
  const float* adv;
  const float* old_lp;
  const float* ref_lp;
  float* out;
  float* g;
  int* counts;   // [batch]
  double* sums;  // three per workgroup of launch_policy_rows
};
hipError_t launch_policy_terms(hipStream_t s, const PolicyArgs& a);

// Loss and gradient in one pass over rows that a workgroup's registers hold.
bool policy_rows_fit(const LossArgs& a);
hipError_t launch_policy_rows(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p, int cus);

struct PreferenceArgs {
  muon_preference_params_t p;
  int batch, seq;
  const int64_t* labels;
  const double* lp;
  const float* ref_lp;
  float* out;
  float* rewards;
  float* g;
  double* score;  // [batch]
  int* counts;    // [batch]
};
hipError_t launch_preference_terms(hipStream_t s, const PreferenceArgs& a);

// ---------------------------------------------------------------------------
// gradient norm and scaling (grad_clip.hip)
// ---------------------------------------------------------------------------

// Elements of a chunk (one workgroup, one partial sum) for tensors of `total`
// elements together, and the chunks that one tensor takes.
int64_t clip_chunk(int64_t total);
int64_t clip_chunks(const muon_tensor_t& t, int64_t chunk);

hipError_t launch_grad_norm(hipStream_t s, const muon_tensor_t* t, int64_t count, int64_t chunk,
                            double* partial, double max_norm, double eps, double* norm);
hipError_t launch_clip_coef(hipStream_t s, double max_norm, double eps, double* norm);
hipError_t launch_scale_grads(hipStream_t s, const muon_tensor_t* t, const muon_tensor_t* out,
                              int64_t count, int64_t chunk, const double* norm);
