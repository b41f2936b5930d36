// Host-side declarations of the launchers of loss.hip and grad_clip.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"

// Rows of scores: row r = (r / seq, r % seq) starts bs, rs bytes apart.
struct RowsRef {
  char* base;
  int64_t bs, rs;
};

// Words of a context through which workgroups of one launch exchange what they
// found (pairs of slices, weights of tokens, counts of those that are through).
// They are zero between calls: each call leaves them so, so none has to clear
// them first.  Calls that need more take their workspace and a launch more.
// Counters of a call's workgroups lie behind them, in different channels.
constexpr int kExchangeWords = 32768;
// Calls of so few workgroups are one launch, whose last workgroup does what is
// left.  Against a launch more: 480 workgroups of log-probabilities 8.5 and 10.3 us
// (12.7 if all count themselves at one address), 564 of the policy loss 10.4 and
// 13.6, 198 of the preference loss 14.0 and 16.9, 536 of it 16.8 and 16.9.
constexpr int kArriveGroups = 1024;
constexpr int kCountedTogether = 32, kCounters = 1 + kArriveGroups / kCountedTogether, kCounterWords = 32;
struct Exchange {
  uint64_t* words = nullptr;
  bool dirty = false;  // a call failed between its launches
};
// Empties the words if a call failed half way; recorded into a graph it leaves
// `dirty` as it is, so that calls before the first replay empty them too.
hipError_t clear_exchange(hipStream_t s, Exchange& x);

struct LossArgs {
  RowsRef x;
  int bf16;
  int rows, seq, vocab;
  int row0;          // first row of this launch (set by the launchers)
  const int64_t* labels;
  float k, k_rest;   // log2 e / temperature = k + k_rest, k rounded to fp32
  float none;        // a difference of scores whose exponential is 0: 2^-256
  float k_each[8];   // its neighbours in fp32, of mean k over the 8 or 4 scores of 16 bytes
  double inv_t;      // 1 / temperature
  int slices;        // workgroups that a row is cut over
  int spin;          // polls before a slice computes its neighbours' pairs itself
  uint64_t* part;    // [rows][slices] pairs of the slices
  float* chosen;     // [rows] the labels' scores, of rows in several slices
  double* lp;        // [rows] or nullptr
  float* logps;      // [rows] or nullptr
  float2* stats;     // [rows] (maximum, sum - 1) of the whole row, or nullptr
  uint64_t* arrived; // a call's counters if it is one launch, else nullptr
};

// Slices of each row (at most 60 within MUON_MAX_VOCAB).
int loss_slices(int64_t rows, int64_t vocab, int bf16, int cus);

// stats, lp and logps of every row (logps of tokens left out: 0).
hipError_t launch_row_stats(hipStream_t s, const LossArgs& a, Exchange& x);

// grad row r = g / temperature * ([v = y] - softmax), g[r] or g[sequence];
// zeros for tokens left out.  Needs a.stats.
hipError_t launch_logits_grad(hipStream_t s, const LossArgs& a, RowsRef grad, const float* g, bool per_sequence);

constexpr int kPolicySums = 64;  // workgroups that add up a policy loss's tokens
struct PolicyArgs {
  muon_policy_params_t p;
  int batch, seq;
  const int64_t* labels;
  const float* adv;
  const float* old_lp;
  const float* ref_lp;
  float* out;
  uint64_t* weights;  // [batch] weight of a sequence's tokens (binary64), or one for all
  uint64_t* terms;    // [rows][2] words of pg and kl, and of clipped
  uint64_t* scores;   // [rows] the label's score, where the workgroup of its slice stopped waiting
  double* sums;       // [kPolicySums][3]
  // set by the launcher
  int count_here;     // the slices count the tokens and publish the weights
  int clear;          // exchange words to empty afterwards
};

// Loss, and gradient where grad.base is set, in one pass over the scores.
hipError_t launch_policy(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p, Exchange& x);

struct PreferenceArgs {
  muon_preference_params_t p;
  int batch, seq;
  const float* ref_lp;
  float* out;
  float* rewards;
  float* g;       // [batch] gradient in each log-probability of a sequence
  double* terms;  // [pairs][3] loss, margin, won
};
hipError_t launch_preference(hipStream_t s, const LossArgs& a, RowsRef grad, const PreferenceArgs& p, Exchange& x);

// ---------------------------------------------------------------------------
// gradient norm and scaling (grad_clip.hip)
// ---------------------------------------------------------------------------

// Elements of a chunk (one workgroup, one partial sum) for tensors of `total`
// elements together, and the chunks that one tensor takes.
int64_t clip_chunk(int64_t total);
int64_t clip_chunks(const muon_tensor_t& t, int64_t chunk);
constexpr int kClipJoin = 32;  // workgroups that add up many partials; room for their sums follows the partials

hipError_t launch_grad_norm(hipStream_t s, const muon_tensor_t* t, int64_t count, int64_t chunk,
                            double* partial, double max_norm, double eps, double* norm, Exchange& x);
hipError_t launch_clip_coef(hipStream_t s, double max_norm, double eps, double* norm);
hipError_t launch_scale_grads(hipStream_t s, const muon_tensor_t* t, const muon_tensor_t* out,
                              int64_t count, int64_t chunk, const double* norm);
