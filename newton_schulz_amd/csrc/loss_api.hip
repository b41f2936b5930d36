// C entry points of the losses and of gradient clipping: argument checks,
// workspace layout, launches.  Arguments are checked before the context, so
// that a refusal names the argument also where no context exists
// (muon_last_error(NULL)).
#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "api_checks.h"
#include "loss_kernels.h"
#include "muon_ctx.h"

namespace {

// What the kernels of one loss call hand each other, for the finest slicing
// that `cus` compute units can ask for.
struct LossLayout {
  size_t part, stats, lp, terms, weights, pairs, sums, total;  // (lp: in the policy loss the labels' scores)
};

LossLayout loss_layout(int64_t batch, int64_t seq, int slices) {
  const size_t rows = static_cast<size_t>(batch * seq), b = static_cast<size_t>(batch);
  LossLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += up256(bytes);
    return p;
  };
  l.part = take(sizeof(uint64_t) * rows * static_cast<size_t>(slices));
  l.stats = take(sizeof(float2) * rows);
  l.lp = take(sizeof(double) * rows);
  l.terms = take(sizeof(uint64_t) * 2 * rows);
  l.weights = take(sizeof(double) * (b + 1));
  l.pairs = take(sizeof(double) * 3 * (b / 2));
  l.sums = take(sizeof(double) * 3 * kPolicySums);
  l.total = at;
  return l;
}

bool same_place(const muon_logits_t& a, const muon_logits_t& b) {
  return a.data == b.data && (a.batch <= 1 || a.batch_stride == b.batch_stride) &&
         (a.seq <= 1 || a.row_stride == b.row_stride);
}

muon_status_t check_grad(muon_ctx* c, const muon_logits_t* x, const muon_logits_t* g, size_t* bytes) {
  *bytes = 0;
  if (g == nullptr) return MUON_OK;
  const muon_status_t st = check_logits(c, g, bytes);
  if (st != MUON_OK) return st;
  if (g->dtype != x->dtype) return fail(c, MUON_EDTYPE, "gradient and logits differ in dtype");
  if (g->batch != x->batch || g->seq != x->seq || g->vocab != x->vocab)
    return fail(c, MUON_ESHAPE, "gradient and logits differ in shape");
  if (!rows_disjoint(*g)) return fail(c, MUON_EINVAL, "rows of the gradient overlap");
  return MUON_OK;
}

constexpr double kLog2e = 1.44269504088896340736;
int slices_of(const muon_ctx* c, const muon_logits_t& x) {
  return loss_slices(x.batch * x.seq, x.vocab, x.dtype == MUON_BF16, c ? c->cus : 256);
}

LossArgs loss_args(const muon_ctx* c, const LossLayout& l, const muon_logits_t& x, const int64_t* labels,
                   double temperature) {
  LossArgs a = {};
  a.x = rows_ref(x);
  a.bf16 = x.dtype == MUON_BF16;
  a.rows = static_cast<int>(x.batch * x.seq);
  a.seq = static_cast<int>(x.seq > 0 ? x.seq : 1);
  a.vocab = static_cast<int>(x.vocab);
  a.labels = labels;
  const double k = kLog2e / temperature;
  a.k = static_cast<float>(k);
  a.k_rest = static_cast<float>(k - static_cast<double>(a.k));
  a.none = static_cast<float>(-256.0 / k);  // (finite: k is above 1e-30)
  // k lies between two fp32 numbers: the mean over a piece of the two is k
  k_neighbours(k, a.bf16 ? 8 : 4, a.k_each);
  a.inv_t = 1.0 / temperature;
  a.slices = slices_of(c, x);
  a.spin = c->loss_spin;
  a.part = reinterpret_cast<uint64_t*>(c->ws + l.part);
  a.chosen = reinterpret_cast<float*>(c->ws + l.terms);
  a.lp = reinterpret_cast<double*>(c->ws + l.lp);
  a.stats = reinterpret_cast<float2*>(c->ws + l.stats);
  return a;
}

}  // namespace

extern "C" {

size_t muon_loss_workspace_bytes(int64_t batch, int64_t seq, int64_t vocab, int32_t dtype) {
  const muon_logits_t x = {nullptr, dtype, batch, seq, vocab, 0, 0};
  size_t bytes = 0;
  // (an address is no part of the size; every other argument is checked)
  const muon_status_t st = check_logits(nullptr, &x, &bytes);
  if (st != MUON_OK && !(st == MUON_EINVAL && bytes)) return 0;
  return loss_layout(batch, seq, slices_of(nullptr, x)).total;
}

muon_status_t muon_loss_set_polls(muon_ctx_t* c, int32_t polls) {
  if (polls < 0) return fail(c, MUON_EINVAL, "polls < 0");
  if (c == nullptr) return fail(c, MUON_EINVAL, "context NULL");
  c->loss_spin = polls;
  return MUON_OK;
}

muon_status_t muon_token_logps(muon_ctx_t* c, void* stream, const muon_logits_t* logits,
                               const int64_t* labels, double temperature, float* logps,
                               float* row_stats) {
  size_t xb = 0;
  muon_status_t st = check_logits(c, logits, &xb);
  if (st != MUON_OK) return st;
  if (!good_temperature(temperature)) return fail(c, MUON_EINVAL, "temperature");
  const size_t rows = static_cast<size_t>(logits->batch * logits->seq);
  const Span spans[] = {{logits->data, xb, 1, false, true, "logits"},
                        {labels, rows * 8, 8, false, true, "labels"},
                        {logps, rows * 4, 4, true, true, "logps"},
                        {row_stats, rows * 8, 8, true, false, "row_stats"}};
  st = check_spans(c, spans, 4, false);
  if (st != MUON_OK) return st;
  const LossLayout l = loss_layout(logits->batch, logits->seq, slices_of(c, *logits));
  st = check_ctx(c, l.total);
  if (st != MUON_OK || rows == 0) return st;
  DeviceGuard g(c->device);
  LossArgs a = loss_args(c, l, *logits, labels, temperature);
  a.lp = nullptr;
  a.logps = logps;
  a.stats = reinterpret_cast<float2*>(row_stats);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_LOSS, "row statistics launch", [&] { return launch_row_stats(s, a, c->exchange); });
}

muon_status_t muon_token_logps_backward(muon_ctx_t* c, void* stream, const muon_logits_t* logits,
                                        const int64_t* labels, double temperature,
                                        const float* row_stats, const float* grad_logps,
                                        const muon_logits_t* grad_logits) {
  size_t xb = 0, gb = 0;
  muon_status_t st = check_logits(c, logits, &xb);
  if (st != MUON_OK) return st;
  if (grad_logits == nullptr) return fail(c, MUON_EINVAL, "grad_logits NULL");
  st = check_grad(c, logits, grad_logits, &gb);
  if (st != MUON_OK) return st;
  if (!good_temperature(temperature)) return fail(c, MUON_EINVAL, "temperature");
  const size_t rows = static_cast<size_t>(logits->batch * logits->seq);
  const Span spans[] = {{logits->data, xb, 1, false, true, "logits"},
                        {grad_logits->data, gb, 1, true, true, "grad_logits"},
                        {labels, rows * 8, 8, false, true, "labels"},
                        {row_stats, rows * 8, 8, false, true, "row_stats"},
                        {grad_logps, rows * 4, 4, false, true, "grad_logps"}};
  st = check_spans(c, spans, 5, same_place(*logits, *grad_logits));
  if (st != MUON_OK) return st;
  st = check_ctx(c, 0);
  if (st != MUON_OK || rows == 0) return st;
  DeviceGuard g(c->device);
  LossArgs a = loss_args(c, LossLayout{}, *logits, labels, temperature);
  a.stats = reinterpret_cast<float2*>(const_cast<float*>(row_stats));
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_LOSS, "gradient launch",
               [&] { return launch_logits_grad(s, a, rows_ref(*grad_logits), grad_logps, false); });
}

muon_status_t muon_policy_loss(muon_ctx_t* c, void* stream, const muon_logits_t* logits,
                               const int64_t* labels, const muon_policy_params_t* p,
                               const float* advantages, const float* old_logps,
                               const float* ref_logps, float* out, float* logps,
                               const muon_logits_t* grad_logits) {
  size_t xb = 0, gb = 0;
  muon_status_t st = check_logits(c, logits, &xb);
  if (st != MUON_OK) return st;
  st = check_grad(c, logits, grad_logits, &gb);
  if (st != MUON_OK) return st;
  if (p == nullptr) return fail(c, MUON_EINVAL, "params NULL");
  if (!good_temperature(p->temperature)) return fail(c, MUON_EINVAL, "temperature");
  if (!(p->clip_low >= 0.0f && p->clip_low <= 1.0f) || !(p->clip_high >= 0.0f))
    return fail(c, MUON_EINVAL, "clip range");
  if (!(p->kl_coef >= 0.0f) || !std::isfinite(p->kl_coef) || !std::isfinite(p->weight))
    return fail(c, MUON_EINVAL, "kl_coef or weight");
  if (p->reduce < MUON_REDUCE_TOKEN || p->reduce > MUON_REDUCE_SUM) return fail(c, MUON_EINVAL, "reduce");
  const size_t batch = static_cast<size_t>(logits->batch), rows = batch * static_cast<size_t>(logits->seq);
  if (p->kl_coef > 0.0f && ref_logps == nullptr && rows) return fail(c, MUON_EINVAL, "kl_coef needs ref_logps");
  const Span spans[] = {{logits->data, xb, 1, false, true, "logits"},
                        {grad_logits ? grad_logits->data : nullptr, gb, 1, true, false, "grad_logits"},
                        {labels, rows * 8, 8, false, true, "labels"},
                        {advantages, (p->advantage_per_token ? rows : batch) * 4, 4, false, true, "advantages"},
                        {old_logps, rows * 4, 4, false, false, "old_logps"},
                        {ref_logps, rows * 4, 4, false, false, "ref_logps"},
                        {out, 16, 4, true, true, "out"},
                        {logps, rows * 4, 4, true, false, "logps"}};
  st = check_spans(c, spans, 8, grad_logits && same_place(*logits, *grad_logits));
  if (st != MUON_OK) return st;
  const LossLayout l = loss_layout(logits->batch, logits->seq, slices_of(c, *logits));
  st = check_ctx(c, l.total);
  if (st != MUON_OK) return st;
  DeviceGuard dg(c->device);
  LossArgs a = loss_args(c, l, *logits, labels, p->temperature);
  a.logps = logps;
  PolicyArgs t = {};
  t.p = *p;
  t.batch = static_cast<int>(logits->batch);
  t.seq = static_cast<int>(logits->seq);
  t.labels = labels;
  t.adv = advantages;
  t.old_lp = old_logps;
  t.ref_lp = ref_logps;
  t.out = out;
  t.weights = reinterpret_cast<uint64_t*>(c->ws + l.weights);
  t.terms = reinterpret_cast<uint64_t*>(c->ws + l.terms);
  t.scores = reinterpret_cast<uint64_t*>(c->ws + l.lp);
  t.sums = reinterpret_cast<double*>(c->ws + l.sums);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_LOSS, "policy loss launch",
               [&] { return launch_policy(s, a, grad_logits && rows ? rows_ref(*grad_logits) : RowsRef{}, t, c->exchange); });
}

muon_status_t muon_preference_loss(muon_ctx_t* c, void* stream, const muon_logits_t* logits,
                                   const int64_t* labels, const muon_preference_params_t* p,
                                   const float* ref_logps, float* out, float* rewards,
                                   float* logps, const muon_logits_t* grad_logits) {
  size_t xb = 0, gb = 0;
  muon_status_t st = check_logits(c, logits, &xb);
  if (st != MUON_OK) return st;
  if (logits->batch % 2) return fail(c, MUON_ESHAPE, "an odd number of sequences makes no pairs");
  st = check_grad(c, logits, grad_logits, &gb);
  if (st != MUON_OK) return st;
  if (p == nullptr) return fail(c, MUON_EINVAL, "params NULL");
  if (!good_temperature(p->temperature)) return fail(c, MUON_EINVAL, "temperature");
  if (!(p->beta > 0.0f) || !std::isfinite(p->beta) || !std::isfinite(p->weight))
    return fail(c, MUON_EINVAL, "beta or weight");
  if (p->kind != MUON_PREFERENCE_SIGMOID && p->kind != MUON_PREFERENCE_IPO) return fail(c, MUON_EINVAL, "kind");
  if (!(p->label_smoothing >= 0.0f && p->label_smoothing <= 0.5f) ||
      (p->kind != MUON_PREFERENCE_SIGMOID && p->label_smoothing != 0.0f))
    return fail(c, MUON_EINVAL, "label_smoothing");
  const size_t batch = static_cast<size_t>(logits->batch), rows = batch * static_cast<size_t>(logits->seq);
  const Span spans[] = {{logits->data, xb, 1, false, true, "logits"},
                        {grad_logits ? grad_logits->data : nullptr, gb, 1, true, false, "grad_logits"},
                        {labels, rows * 8, 8, false, true, "labels"},
                        {ref_logps, rows * 4, 4, false, false, "ref_logps"},
                        {out, 12, 4, true, true, "out"},
                        {rewards, batch * 4, 4, true, false, "rewards"},
                        {logps, rows * 4, 4, true, false, "logps"}};
  st = check_spans(c, spans, 7, grad_logits && same_place(*logits, *grad_logits));
  if (st != MUON_OK) return st;
  const LossLayout l = loss_layout(logits->batch, logits->seq, slices_of(c, *logits));
  st = check_ctx(c, l.total);
  if (st != MUON_OK) return st;
  DeviceGuard dg(c->device);
  LossArgs a = loss_args(c, l, *logits, labels, p->temperature);
  a.logps = logps;
  PreferenceArgs t = {};
  t.p = *p;
  t.batch = static_cast<int>(logits->batch);
  t.seq = static_cast<int>(logits->seq);
  t.ref_lp = ref_logps;
  t.out = out;
  t.rewards = rewards;
  t.g = reinterpret_cast<float*>(c->ws + l.weights);
  t.terms = reinterpret_cast<double*>(c->ws + l.pairs);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_LOSS, "preference loss launch",
               [&] { return launch_preference(s, a, grad_logits && rows ? rows_ref(*grad_logits) : RowsRef{}, t, c->exchange); });
}

}  // extern "C"

// ---------------------------------------------------------------------------
// gradient norm and clipping
// ---------------------------------------------------------------------------
namespace {

constexpr int64_t kMostElements = int64_t{1} << 40;
// Of one tensor, which is one launch: its chunks (8192 elements in lists that
// large, and one more for where it starts) are workgroups of 256 threads, and a grid
// holds fewer than 2^32 threads.
constexpr int64_t kMostInTensor = ((int64_t{1} << 24) - 2) * 8192;

// Each entry on its own; *total receives the elements of all.
muon_status_t check_list(muon_ctx* c, const muon_tensor_t* t, int64_t count, int64_t* total) {
  *total = 0;
  if (count < 0) return fail(c, MUON_EINVAL, "count < 0");
  if (count > 0 && t == nullptr) return fail(c, MUON_EINVAL, "tensor list NULL");
  for (int64_t i = 0; i < count; ++i) {
    if (!is_dtype(t[i].dtype)) return fail(c, MUON_EDTYPE, "tensor dtype");
    if (t[i].numel < 0 || t[i].numel > kMostInTensor) return fail(c, MUON_ESHAPE, "tensor numel");
    if (t[i].numel && t[i].data == nullptr) return fail(c, MUON_EINVAL, "tensor data NULL");
    if (reinterpret_cast<uintptr_t>(t[i].data) % esize(t[i].dtype)) return fail(c, MUON_EINVAL, "misaligned tensor");
    *total += t[i].numel;
    if (*total > kMostElements) return fail(c, MUON_ESHAPE, "too many elements");
  }
  return MUON_OK;
}

size_t norm_bytes(const muon_tensor_t* t, int64_t count, int64_t total) {
  const int64_t chunk = clip_chunk(total);
  size_t n = kClipJoin;
  for (int64_t i = 0; i < count; ++i) n += static_cast<size_t>(clip_chunks(t[i], chunk));
  return up256(n * 8);
}

muon_status_t check_norm(muon_ctx* c, const double* norm) {
  if (norm == nullptr) return fail(c, MUON_EINVAL, "norm NULL");
  if (reinterpret_cast<uintptr_t>(norm) % 8) return fail(c, MUON_EINVAL, "misaligned norm");
  return MUON_OK;
}

muon_status_t check_limits(muon_ctx* c, double max_norm, double eps) {
  if (!(max_norm > 0.0)) return fail(c, MUON_EINVAL, "max_norm must be positive");
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(c, MUON_EINVAL, "eps");
  return MUON_OK;
}

}  // namespace

extern "C" {

size_t muon_grad_norm_workspace_bytes(const muon_tensor_t* grads, int64_t count) {
  int64_t total = 0;
  if (count <= 0 || check_list(nullptr, grads, count, &total) != MUON_OK) return 0;
  return norm_bytes(grads, count, total);
}

muon_status_t muon_grad_norm(muon_ctx_t* c, void* stream, const muon_tensor_t* grads,
                             int64_t count, double max_norm, double eps, double* norm) {
  int64_t total = 0;
  muon_status_t st = check_list(c, grads, count, &total);
  if (st == MUON_OK) st = check_limits(c, max_norm, eps);
  if (st == MUON_OK) st = check_norm(c, norm);
  if (st != MUON_OK) return st;
  for (int64_t i = 0; i < count; ++i)
    if (ranges_overlap(norm, 24, grads[i].data, static_cast<size_t>(grads[i].numel) * esize(grads[i].dtype)))
      return fail(c, MUON_EINVAL, "norm overlaps a tensor");
  st = check_ctx(c, norm_bytes(grads, count, total));
  if (st != MUON_OK) return st;
  DeviceGuard g(c->device);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_CLIP, "gradient norm launch", [&] {
    return launch_grad_norm(s, grads, count, clip_chunk(total), reinterpret_cast<double*>(c->ws), max_norm, eps,
                            norm, c->exchange);
  });
}

muon_status_t muon_clip_coef(muon_ctx_t* c, void* stream, double max_norm, double eps,
                             double* norm) {
  muon_status_t st = check_limits(c, max_norm, eps);
  if (st == MUON_OK) st = check_norm(c, norm);
  if (st == MUON_OK) st = check_ctx(c, 0);
  if (st != MUON_OK) return st;
  DeviceGuard g(c->device);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_CLIP, "clip coefficient launch", [&] { return launch_clip_coef(s, max_norm, eps, norm); });
}

muon_status_t muon_scale_grads(muon_ctx_t* c, void* stream, const muon_tensor_t* grads,
                               const muon_tensor_t* out, int64_t count, const double* norm) {
  int64_t total = 0;
  muon_status_t st = check_list(c, grads, count, &total);
  if (st == MUON_OK) st = check_norm(c, norm);
  if (st != MUON_OK) return st;
  if (out != nullptr) {
    int64_t same = 0;
    st = check_list(c, out, count, &same);
    if (st != MUON_OK) return st;
    for (int64_t i = 0; i < count; ++i)
      if (out[i].numel != grads[i].numel) return fail(c, MUON_ESHAPE, "out and grads differ in numel");
  }
  // Nothing written that is read or written elsewhere (an output that is its own
  // input counts once); what is only read may overlap.
  try {
    struct Range {
      uintptr_t from, to;
      bool written;
    };
    std::vector<Range> v;
    v.reserve(static_cast<size_t>(2 * count + 1));
    auto add = [&](const void* p, size_t bytes, bool written) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      if (bytes) v.push_back({at, at + bytes, written});
    };
    add(norm, 24, false);
    for (int64_t i = 0; i < count; ++i) {
      const size_t n = static_cast<size_t>(grads[i].numel);
      const bool in_place = !out || (out[i].data == grads[i].data && out[i].dtype == grads[i].dtype);
      add(grads[i].data, n * esize(grads[i].dtype), in_place);
      if (!in_place) add(out[i].data, n * esize(out[i].dtype), true);
    }
    std::sort(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;  // ends of what came before
    for (const Range& r : v) {
      if (r.from < (r.written ? any : written)) return fail(c, MUON_EINVAL, "tensors overlap");
      any = std::max(any, r.to);
      if (r.written) written = std::max(written, r.to);
    }
  } catch (...) {
    return fail(c, MUON_ENOMEM, "host memory");
  }
  st = check_ctx(c, 0);
  if (st != MUON_OK || total == 0) return st;
  DeviceGuard g(c->device);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return timed(c, s, MUON_K_CLIP, "gradient scaling launch", [&] {
    return launch_scale_grads(s, grads, out ? out : grads, count, clip_chunk(total), norm);
  });
}

}  // extern "C"
