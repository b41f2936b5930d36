// The context behind the C ABI and the small host helpers that every entry
// point uses: error text, timed launches, device selection, range checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <vector>

#include "loss_kernels.h"
#include "muon.h"
#include "muon_internal.h"

constexpr int kTabSlots = 4;
constexpr int64_t kTabCap = 65536;  // pointers per table (per in/out) per slot

struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) prev = -1;
    ok = hipSetDevice(dev) == hipSuccess;
  }
  ~DeviceGuard() {
    if (prev >= 0) (void)hipSetDevice(prev);
  }
};

struct muon_ctx {
  int device = 0;
  int cus = 256;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  uint64_t* host_tab = nullptr;  // pinned staging, kTabSlots * 2 * kTabCap
  uint64_t* dev_tab = nullptr;   // device tables, same layout
  hipEvent_t tab_ev[kTabSlots] = {};
  bool tab_used[kTabSlots] = {};
  int tab_next = 0;
  // polls (a microsecond or so each) before a slice of a row stops waiting for
  // its neighbours and computes their pairs itself (loss.hip)
  int loss_spin = 1 << 14;
  Exchange exchange;
  // timing
  bool timing = false;
  uint32_t tmask = (1u << MUON_K_COUNT) - 1;  // classes that record events
  std::vector<hipEvent_t> tev;
  std::vector<int> tcls;
  size_t tused = 0;  // events recorded (pairs * 2)
  std::string err;
};

// Text of the calling thread's last refusal of a call without a context
// (muon_last_error(NULL)); static strings only.
extern thread_local const char* muon_thread_err;

// The context's text is assigned under a handler: no exception may leave a C
// entry point, and a text that cannot be kept is no reason to fail otherwise.
inline muon_status_t fail(muon_ctx* c, muon_status_t s, const char* what) {
  if (c == nullptr) {
    muon_thread_err = what;
    return s;
  }
  try {
    c->err = what;
  } catch (...) {
  }
  return s;
}

inline muon_status_t hip_fail(muon_ctx* c, hipError_t e, const char* where) {
  if (c) {
    try {
      c->err = std::string(where) + ": " + hipGetErrorString(e);
    } catch (...) {
    }
  }
  return MUON_EHIP;
}

// Record the start event of a timed launch; returns the pair index or -1.
inline long tstart(muon_ctx* c, hipStream_t s, int cls) {
  if (!c->timing || !((c->tmask >> cls) & 1u) || c->tused + 2 > c->tev.size()) return -1;
  // launches recorded into a graph are not timed (the events would be
  // re-recorded by every replay)
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(s, &cs) != hipSuccess || cs != hipStreamCaptureStatusNone) return -1;
  const long k = static_cast<long>(c->tused);
  if (hipEventRecord(c->tev[k], s) != hipSuccess) return -1;
  c->tcls[k / 2] = cls;
  return k;
}
inline void tstop(muon_ctx* c, hipStream_t s, long k) {
  if (k < 0) return;
  if (hipEventRecord(c->tev[k + 1], s) == hipSuccess) c->tused = static_cast<size_t>(k) + 2;
}

inline bool is_dtype(int32_t d) { return d == MUON_F32 || d == MUON_BF16; }
inline size_t esize(int32_t d) { return d == MUON_BF16 ? 2 : 4; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return na && nb && x < y + nb && y < x + na;
}
