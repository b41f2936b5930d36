// Verification of drafted tokens against the target's probabilities.
//
// Mathematics.  Keeping a token x drawn from q with probability min(1, p(x) /
// q(x)), and drawing from max(p - q, 0) where it is not kept, gives a token
// distributed as p: q min(1, p / q) + (1 - sum_v min(p, q)) max(p - q, 0) /
// sum_v max(p - q, 0) = min(p, q) + max(p - q, 0) = p.  Everything that decides
// is binary64: a drawn index moves when the running sum of the weights moves
// past u times their total, and tokens of probability 1e-6 lie that close.
#include "linear8.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

struct Row {
  const char* p;
  int bf16;
  __device__ __forceinline__ float at(int v) const {
    return bf16 ? muon::bf16_to_f32(reinterpret_cast<const bf16_t*>(p)[v]) : reinterpret_cast<const float*>(p)[v];
  }
};

__device__ double block_sum(double v, double* lds) {
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kWaves; ++w) v += lds[w];
  return v;
}

// Of a row: the largest score, the lowest index that has it, and the sum of
// exp((x - m) / T).  A sum that is not finite: no distribution.
struct Pair {
  float m;
  double s;
  int best;
  __device__ __forceinline__ bool ok() const { return s < static_cast<double>(INFINITY); }
};
__device__ Pair row_pair(const Row& x, int vocab, double inv_t, double* lds) {
  __shared__ float top[kWaves];
  __shared__ int where[kWaves];
  float m = -INFINITY;
  int best = vocab;
  for (int v = threadIdx.x; v < vocab; v += kThreads) {
    const float z = x.at(v);
    if (z > m) m = z, best = v;
  }
  for (int d = 32; d > 0; d /= 2) {
    const float om = __shfl_xor(m, d);
    const int ob = __shfl_xor(best, d);
    if (om > m || (om == m && ob < best)) m = om, best = ob;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m, where[threadIdx.x >> 6] = best;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w)
    if (top[w] > m || (top[w] == m && where[w] < best)) m = top[w], best = where[w];
  double s = 0.0;
  for (int v = threadIdx.x; v < vocab; v += kThreads) s += exp((static_cast<double>(x.at(v)) - static_cast<double>(m)) * inv_t);
  return {m, block_sum(s, lds), best};
}

__global__ __launch_bounds__(kThreads) void verify_simple_kernel(VerifyArgs a) {
  __shared__ double lds[kWaves];
  __shared__ double weight[kThreads];
  __shared__ int found;
  const int b = blockIdx.x, t = threadIdx.x, V = a.vocab;
  const bool greedy = a.inv_t == 0.0;
  const double k = greedy ? 1.0 : a.inv_t;
  const int64_t* drafted = a.drafted + static_cast<int64_t>(b) * a.draft;
  int64_t* tokens = a.tokens + static_cast<int64_t>(b) * (a.draft + 1);
  float* logps = a.logps ? a.logps + static_cast<int64_t>(b) * (a.draft + 1) : nullptr;
  int r = 0;
  int64_t next = -1;
  double next_lp = __longlong_as_double(0x7ff8000000000000ll);
  for (;; ++r) {
    const Row x = {a.x.base + b * a.x.bs + r * a.x.rs, a.x_bf16};
    const Pair P = row_pair(x, V, k, lds);
    const int64_t y = r < a.draft ? drafted[r] : -1;
    const bool named = y >= 0 && y < V;
    if (!P.ok()) break;
    auto lp = [&](int64_t v) { return (static_cast<double>(x.at(static_cast<int>(v))) - static_cast<double>(P.m)) * k - log(P.s); };
    bool keep;
    Row d = {nullptr, 0};
    Pair Q = {0.0f, 1.0, 0};
    if (greedy) {
      keep = named && y == P.best;
    } else {
      double qx = 1.0;
      if (y >= 0 && a.d.base) {
        d = {a.d.base + b * a.d.bs + r * a.d.rs, a.d_bf16};
        Q = row_pair(d, V, k, lds);
        qx = named && Q.ok() ? exp((static_cast<double>(d.at(static_cast<int>(y))) - static_cast<double>(Q.m)) * k) / Q.s : 1.0;
      }
      keep = named && Q.ok() && static_cast<double>(a.uniforms[static_cast<int64_t>(b) * (a.draft + 1) + r]) * qx < exp(lp(y));
    }
    if (keep) {
      if (t == 0) {
        tokens[r] = y;
        if (logps) logps[r] = static_cast<float>(lp(y));
      }
      continue;
    }
    if (greedy) {
      next = P.best;
    } else {
      bool rest = y >= 0 && Q.ok();  // weights max(p - q, 0), else p
      auto w = [&](int v) {
        const double p = exp((static_cast<double>(x.at(v)) - static_cast<double>(P.m)) * k) / P.s;
        if (!rest) return p;
        const double q = d.p ? exp((static_cast<double>(d.at(v)) - static_cast<double>(Q.m)) * k) / Q.s : (v == y ? 1.0 : 0.0);
        return fmax(p - q, 0.0);
      };
      double total = 0.0;
      for (;;) {
        double s = 0.0;
        for (int v = t; v < V; v += kThreads) s += w(v);
        total = block_sum(s, lds);
        if (total > 0.0 || !rest) break;
        rest = false;
      }
      const double want = static_cast<double>(a.uniforms[static_cast<int64_t>(b) * (a.draft + 1) + a.draft]) * total;
      double before = 0.0;
      int last = -1;
      if (t == 0) found = -1;
      for (int v0 = 0; v0 < V; v0 += kThreads) {
        const double mine = v0 + t < V ? w(v0 + t) : 0.0;
        __syncthreads();
        weight[t] = mine;
        __syncthreads();
        if (t == 0) {
          for (int i = 0; i < kThreads; ++i) {
            if (!(weight[i] > 0.0)) continue;
            before += weight[i];
            last = v0 + i;
            if (before > want) {
              found = last;
              break;
            }
          }
        }
        __syncthreads();
        if (found >= 0) break;
      }
      if (t == 0 && found < 0) found = last;
      __syncthreads();
      next = found;
    }
    next_lp = lp(next);
    break;
  }
  if (t == 0) {
    a.accepted[b] = r;
    for (int i = r; i <= a.draft; ++i) {
      tokens[i] = i == r ? next : -1;
      if (logps) logps[i] = i == r ? static_cast<float>(next_lp) : 0.0f;
    }
  }
}

}  // namespace

hipError_t launch_verify(hipStream_t s, const VerifyArgs& a) {
  if (a.batch == 0) return hipSuccess;
  verify_simple_kernel<<<static_cast<unsigned>(a.batch), kThreads, 0, s>>>(a);
  return hipGetLastError();
}
