// Checks of arguments and helpers that the C entry points share.
#pragma once

#include <cmath>

#include "loss_kernels.h"
#include "muon_ctx.h"

constexpr int64_t kMostTokens = int64_t{1} << 30;

inline size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Bytes from the first to past the last element of x; false: does not fit 2^62.
inline bool extent(const muon_logits_t& x, size_t* bytes) {
  *bytes = 0;
  if (x.batch == 0 || x.seq == 0) return true;
  const __int128 n = static_cast<__int128>(x.batch - 1) * (x.batch > 1 ? x.batch_stride : 0) +
                     static_cast<__int128>(x.seq - 1) * (x.seq > 1 ? x.row_stride : 0) + x.vocab;
  if (n > (static_cast<__int128>(1) << 59)) return false;
  *bytes = static_cast<size_t>(n) * esize(x.dtype);
  return true;
}

inline muon_status_t check_logits(muon_ctx* c, const muon_logits_t* x, size_t* bytes) {
  if (x == nullptr) return fail(c, MUON_EINVAL, "logits NULL");
  if (!is_dtype(x->dtype)) return fail(c, MUON_EDTYPE, "logits dtype");
  if (x->batch < 0 || x->seq < 0 || x->vocab < 1 || x->vocab > MUON_MAX_VOCAB || x->batch > kMostTokens ||
      x->seq > kMostTokens || x->batch * x->seq > kMostTokens)
    return fail(c, MUON_ESHAPE, "batch, seq or vocab out of range");
  if ((x->batch > 1 && x->batch_stride < 0) || (x->seq > 1 && x->row_stride < 0))
    return fail(c, MUON_ESHAPE, "negative stride");
  if (!extent(*x, bytes)) return fail(c, MUON_ESHAPE, "strides out of range");
  if (*bytes && x->data == nullptr) return fail(c, MUON_EINVAL, "logits data NULL");
  if (reinterpret_cast<uintptr_t>(x->data) % esize(x->dtype)) return fail(c, MUON_EINVAL, "misaligned logits");
  return MUON_OK;
}

inline bool rows_disjoint(const muon_logits_t& x) {
  if (x.batch * x.seq < 2) return true;
  if (x.batch == 1) return x.row_stride >= x.vocab;
  if (x.seq == 1) return x.batch_stride >= x.vocab;
  return (x.row_stride >= x.vocab && x.batch_stride / x.row_stride >= x.seq - 1 &&
          x.batch_stride - (x.seq - 1) * x.row_stride >= x.vocab) ||
         (x.batch_stride >= x.vocab && x.row_stride / x.batch_stride >= x.batch - 1 &&
          x.row_stride - (x.batch - 1) * x.batch_stride >= x.vocab);
}

// The memory of one argument.
struct Span {
  const void* p;
  size_t bytes;
  size_t align;
  bool written;
  bool required;
  const char* name;
};

// Every pointer there that has to be, aligned, and nothing written that the
// call reads or writes elsewhere.
inline muon_status_t check_spans(muon_ctx* c, const Span* s, int n, bool in_place) {
  for (int i = 0; i < n; ++i) {
    if (s[i].required && s[i].bytes && s[i].p == nullptr) return fail(c, MUON_EINVAL, "null pointer");
    if (reinterpret_cast<uintptr_t>(s[i].p) % s[i].align) return fail(c, MUON_EINVAL, "misaligned pointer");
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!(s[i].written || s[j].written) || s[i].p == nullptr || s[j].p == nullptr) continue;
      if (in_place && i == 0 && j == 1) continue;  // logits and their gradient
      if (ranges_overlap(s[i].p, s[i].bytes, s[j].p, s[j].bytes))
        return fail(c, MUON_EINVAL, "an output overlaps another argument");
    }
  return MUON_OK;
}

// also 1 / t and log2 e / t, which the kernels take in fp32, have to be finite
inline bool good_temperature(double t) { return t > 1e-30 && t < 1e30; }

// Neighbours of k in fp32 whose mean over `vec` scores is k to half a step / vec.
inline void k_neighbours(double k, int vec, float (&each)[8]) {
  const float near = static_cast<float>(k);
  const float down = static_cast<double>(near) <= k ? near : std::nextafterf(near, 0.0f);
  const float up = std::nextafterf(down, INFINITY);
  const double ups = vec * (k - down) / (static_cast<double>(up) - down);
  for (int i = 0; i < 8; ++i) each[i] = i % vec < static_cast<int>(ups + 0.5) ? up : down;
}

inline muon_status_t check_ctx(muon_ctx* c, size_t need) {
  if (c == nullptr) return fail(c, MUON_EINVAL, "context NULL");
  if (c->ws_bytes < need) return fail(c, MUON_EWORKSPACE, "the call needs more workspace than the context holds");
  return MUON_OK;
}

inline RowsRef rows_ref(const muon_logits_t& x) {
  const int64_t e = static_cast<int64_t>(esize(x.dtype));
  return RowsRef{static_cast<char*>(x.data), x.batch > 1 ? x.batch_stride * e : 0, x.seq > 1 ? x.row_stride * e : 0};
}

// Runs a launcher under the timing events of its class.
template <typename F> muon_status_t timed(muon_ctx* c, hipStream_t s, int cls, const char* what, F launch) {
  const long k = tstart(c, s, cls);
  const hipError_t e = launch();
  tstop(c, s, k);
  return e == hipSuccess ? MUON_OK : hip_fail(c, e, what);
}
