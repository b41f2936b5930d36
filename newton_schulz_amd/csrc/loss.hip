// Log-probabilities of chosen tokens, the policy and preference losses on
// them, and the gradients of the scores.
//
// Mathematics.  With z = x / T, M = max z and S = sum_v exp(z_v - M):
//   lp = z_y - M - log S,   d lp / d x_v = ([v = y] - exp(z_v - M) / S) / T,
// so a row needs two numbers, (max x, S), beyond itself.  They are found in
// one pass: each thread keeps the maximum m and the sum s around it of what it
// has seen, and a larger maximum m' turns s into s exp(m - m').  Partial pairs
// join the same way, in a fixed order.
//
// Precision.  Scores are widened to fp32 and subtracted before they are
// scaled: (x - m) * (log2 e / T) is exact in the subtraction for bf16 and has
// no large cancelling terms at any magnitude of x, where x * k - m * k loses
// |m| k 2^-24 (and overflows for masks of the type's lowest value).  m starts
// at the lowest finite number, not at -infinity, so that a masked score gives
// exp2(-inf) = 0 and never inf - inf.  The log-probability is formed from
// (x_y - M), S in binary64: what follows takes differences of two of them.
//
// All kernels are bound by HBM: the statistics read each row once, the
// gradient reads and writes it once.
#include <cfloat>

#include "loss_kernels.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -FLT_MAX;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // 16 bytes at an element's alignment

template <typename T> constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // scores per 16 bytes

// 16 bytes of scores as fp32.
template <typename T> struct Scores;
template <> struct Scores<bf16_t> {
  static __device__ __forceinline__ void unpack(u32x4 w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* v) {
    return u32x4{muon::pack_bf16x2(v[0], v[1]), muon::pack_bf16x2(v[2], v[3]),
                 muon::pack_bf16x2(v[4], v[5]), muon::pack_bf16x2(v[6], v[7])};
  }
  static constexpr uint32_t kMasked = 0xff80ff80u;  // two -infinities
};
template <> struct Scores<float> {
  static __device__ __forceinline__ void unpack(u32x4 w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* v) {
    return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                 __float_as_uint(v[3])};
  }
  static constexpr uint32_t kMasked = 0xff800000u;
};

// A row is walked in pieces of 16 bytes that start at 16-byte addresses: piece
// i holds scores [i * kVec - lead, ...), lead = scores of the first piece that
// lie before the row (rows of an odd vocabulary start at odd addresses).  The
// first and the last piece may be partial.
template <typename T> __device__ __forceinline__ int row_lead(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}
template <typename T> __device__ __forceinline__ int row_pieces(int vocab, int lead) {
  return (vocab + lead + kVec<T> - 1) / kVec<T>;
}

// Piece with first score e0; scores outside [0, vocab) read as -infinity.
template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* row, int e0, int vocab) {
  if (e0 >= 0 && e0 + kVec<T> <= vocab) return *reinterpret_cast<const u32x4*>(row + e0);
  u32x4 w = {Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked};
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    const int e = e0 + i;
    if (e >= 0 && e < vocab) {
      if (sizeof(T) == 4) {
        w[i] = reinterpret_cast<const uint32_t*>(row)[e];
      } else {
        const uint32_t h = reinterpret_cast<const bf16_t*>(row)[e];
        w[i / 2] = (i & 1) ? (w[i / 2] & 0xffffu) | (h << 16) : (w[i / 2] & 0xffff0000u) | h;
      }
    }
  }
  return w;
}

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int e0, int vocab, u32x4 w) {
  if (e0 >= 0 && e0 + kVec<T> <= vocab) {
    *reinterpret_cast<u32x4_any*>(row + e0) = w;  // the gradient's rows have their own alignment
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    const int e = e0 + i;
    if (e >= 0 && e < vocab) {
      if (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[e] = w[i];
      else reinterpret_cast<bf16_t*>(row)[e] = static_cast<bf16_t>((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    }
  }
}

template <typename T> __device__ __forceinline__ T* row_at(const RowsRef& x, int r, int seq) {
  const int b = r / seq;
  return reinterpret_cast<T*>(x.base + static_cast<int64_t>(b) * x.bs +
                              static_cast<int64_t>(r - b * seq) * x.rs);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// (m, s) joined with (mo, so); k = log2 e / T.
__device__ __forceinline__ void join(float& m, float& s, float mo, float so, float k) {
  const float mn = fmaxf(m, mo);
  s = s * exp2_fast((m - mn) * k) + so * exp2_fast((mo - mn) * k);
  m = mn;
}

// The pair of all threads of the workgroup, in every thread.
template <int NT> __device__ __forceinline__ void block_join(float& m, float& s, float k) {
  constexpr int W = NT / 64;
  __shared__ float2 wave[W];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const float mo = __shfl_xor(m, d, 64), so = __shfl_xor(s, d, 64);
    // both partners join in the same order: lower lane's pair first
    if (threadIdx.x & d) {
      float m2 = mo, s2 = so;
      join(m2, s2, m, s, k);
      m = m2;
      s = s2;
    } else {
      join(m, s, mo, so, k);
    }
  }
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = make_float2(m, s);
  __syncthreads();
  m = wave[0].x;
  s = wave[0].y;
#pragma unroll
  for (int w = 1; w < W; ++w) join(m, s, wave[w].x, wave[w].y, k);
}

// What the row's pair makes of token r (one thread).
template <typename T>
__device__ __forceinline__ void finish_row(const LossArgs& a, int r, int64_t y, float m, float s) {
  double lp = 0.0;
  if (y >= a.vocab) {
    lp = __longlong_as_double(0x7ff8000000000000ll);
  } else if (y >= 0) {
    const float z = muon::Elem<T>::load(row_at<const T>(a.x, r, a.seq) + y) - m;
    lp = static_cast<double>(z) / static_cast<double>(a.temperature) - log(static_cast<double>(s));
  }
  if (a.lp) a.lp[r] = lp;
  if (a.logps) a.logps[r] = static_cast<float>(lp);
  if (a.stats) a.stats[r] = make_float2(m, s);
}

constexpr int kStatsThreads = 256;
constexpr int kStatsUnroll = 8;  // pieces in flight per thread

// Statistics of row blockIdx / splits, pieces of split blockIdx % splits.
template <typename T>
__global__ __launch_bounds__(kStatsThreads) void row_stats_kernel(LossArgs a) {
  const int r = a.row0 + static_cast<int>(blockIdx.x) / a.splits, sp = static_cast<int>(blockIdx.x) % a.splits;
  const int64_t y = a.labels[r];
  if (y < 0 || y >= a.vocab) {
    if (a.splits == 1 && threadIdx.x == 0) finish_row<T>(a, r, y, 0.0f, 1.0f);
    return;
  }
  const float k = kLog2e / a.temperature;
  const T* row = row_at<const T>(a.x, r, a.seq);
  const int lead = row_lead(row), pieces = row_pieces<T>(a.vocab, lead);
  const int per = (pieces + a.splits - 1) / a.splits;
  const int p0 = sp * per, p1 = min(pieces, p0 + per);
  float m = kLowest, s = 0.0f;
  for (int p = p0 + static_cast<int>(threadIdx.x); p < p1; p += kStatsThreads * kStatsUnroll) {
    u32x4 w[kStatsUnroll];
#pragma unroll
    for (int u = 0; u < kStatsUnroll; ++u) {
      const int q = p + u * kStatsThreads;
      w[u] = load_piece<T>(row, q < p1 ? q * kVec<T> - lead : a.vocab, a.vocab);
    }
#pragma unroll
    for (int u = 0; u < kStatsUnroll; ++u) {
      float v[kVec<T>];
      Scores<T>::unpack(w[u], v);
      float mn = m;
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i) mn = fmaxf(mn, v[i]);
      s *= exp2_fast((m - mn) * k);
      m = mn;
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i) s += exp2_fast((v[i] - m) * k);
    }
  }
  block_join<kStatsThreads>(m, s, k);
  if (threadIdx.x == 0) {
    if (a.splits == 1) finish_row<T>(a, r, y, m, s);
    else a.part[static_cast<int64_t>(r) * a.splits + sp] = make_float2(m, s);
  }
}

// Joins the splits of each row in index order; one thread per row.
template <typename T> __global__ __launch_bounds__(64) void row_join_kernel(LossArgs a) {
  const int r = blockIdx.x * 64 + threadIdx.x;
  if (r >= a.rows) return;
  const int64_t y = a.labels[r];
  float m = 0.0f, s = 1.0f;
  if (y >= 0 && y < a.vocab) {
    const float k = kLog2e / a.temperature;
    m = kLowest;
    s = 0.0f;
    for (int i = 0; i < a.splits; ++i) {
      const float2 q = a.part[static_cast<int64_t>(r) * a.splits + i];
      join(m, s, q.x, q.y, k);
    }
  }
  finish_row<T>(a, r, y, m, s);
}

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;

// Gradient of row blockIdx / chunks, pieces of chunk blockIdx % chunks.
template <typename T>
__global__ __launch_bounds__(kGradThreads) void logits_grad_kernel(LossArgs a, RowsRef grad,
                                                                   const float* __restrict__ g, int chunks) {
  const int r = a.row0 + static_cast<int>(blockIdx.x) / chunks, c = static_cast<int>(blockIdx.x) % chunks;
  const int64_t y = a.labels[r];
  const T* row = row_at<const T>(a.x, r, a.seq);
  T* out = row_at<T>(grad, r, a.seq);
  const int lead = row_lead(row), pieces = row_pieces<T>(a.vocab, lead);
  const int p0 = c * kGradThreads * kGradUnroll + static_cast<int>(threadIdx.x);
  if (y < 0) {
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int p = p0 + u * kGradThreads;
      if (p < pieces) store_piece<T>(out, p * kVec<T> - lead, a.vocab, u32x4{0, 0, 0, 0});
    }
    return;
  }
  const float k = kLog2e / a.temperature;
  const float2 st = a.stats[r];
  float G = g[r] / a.temperature;
  if (y >= a.vocab) G = __uint_as_float(0x7fc00000u);  // the label names no score
  const float scale = -G / st.y;
  u32x4 w[kGradUnroll];
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int p = p0 + u * kGradThreads;
    if (p < pieces) w[u] = load_piece<T>(row, p * kVec<T> - lead, a.vocab);
  }
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int p = p0 + u * kGradThreads;
    if (p >= pieces) continue;
    const int e0 = p * kVec<T> - lead;
    float v[kVec<T>];
    Scores<T>::unpack(w[u], v);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = scale * exp2_fast((v[i] - st.x) * k);
    const int64_t at = y - e0;
    if (at >= 0 && at < kVec<T>) {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i)
        if (i == at) v[i] += G;
    }
    store_piece<T>(out, e0, a.vocab, Scores<T>::pack(v));
  }
}

// ---------------------------------------------------------------------------
// per-token terms
// ---------------------------------------------------------------------------
constexpr int kTermThreads = 1024;

// Sum over the workgroup in a fixed order, in every thread.
__device__ __forceinline__ double block_total(double v) {
  __shared__ double wave[kTermThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();  // the last call's values have been read
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kTermThreads / 64; ++w) t += wave[w];
  return t;
}

// Tokens that count of each sequence, one wave per sequence in turn.
__device__ __forceinline__ void count_tokens(const int64_t* labels, int batch, int seq, int* counts) {
  const int lane = threadIdx.x & 63;
  for (int b = threadIdx.x >> 6; b < batch; b += kTermThreads / 64) {
    int n = 0;
    for (int t0 = 0; t0 < seq; t0 += 64)
      n += __popcll(__ballot(t0 + lane < seq && labels[static_cast<int64_t>(b) * seq + t0 + lane] >= 0));
    if (lane == 0) counts[b] = n;
  }
  __syncthreads();
}

// max(a, b) that hands a NaN on, as the formula does.
__device__ __forceinline__ double max_nan(double a, double b) { return (a > b || a != a) ? a : b; }

__global__ __launch_bounds__(kTermThreads) void policy_terms_kernel(PolicyArgs a) {
  const int rows = a.batch * a.seq;
  count_tokens(a.labels, a.batch, a.seq, a.counts);
  double n = 0.0;
  for (int b = threadIdx.x; b < a.batch; b += kTermThreads) n += a.counts[b];
  n = block_total(n);
  double sum_pg = 0.0, sum_kl = 0.0, sum_clip = 0.0;
  for (int t = threadIdx.x; t < rows; t += kTermThreads) {
    if (a.labels[t] < 0) {
      if (a.g) a.g[t] = 0.0f;
      continue;
    }
    const int b = t / a.seq;
    const double w = a.p.reduce == MUON_REDUCE_TOKEN      ? 1.0 / n
                     : a.p.reduce == MUON_REDUCE_SEQUENCE ? 1.0 / (static_cast<double>(a.counts[b]) * a.batch)
                                                          : 1.0;
    const double lp = a.lp[t], A = a.adv[a.p.advantage_per_token ? t : b];
    // without an old policy it is the policy itself: ratio 1 (NaN when lp is)
    const double ratio = a.old_lp ? exp(lp - a.old_lp[t]) : lp == lp ? 1.0 : lp;
    const double lo = 1.0 - static_cast<double>(a.p.clip_low), hi = 1.0 + static_cast<double>(a.p.clip_high);
    const double held = -A * (ratio < lo ? lo : ratio > hi ? hi : ratio);
    const double free = -A * ratio;
    sum_pg += w * max_nan(free, held);
    if (held > free) sum_clip += w;
    double g = held > free ? 0.0 : free;
    if (a.ref_lp) {
      const double e = static_cast<double>(a.ref_lp[t]) - lp, em = expm1(e);
      sum_kl += w * (em - e);
      if (a.p.kl_coef != 0.0f) g -= static_cast<double>(a.p.kl_coef) * em;
    }
    if (a.g) a.g[t] = static_cast<float>(static_cast<double>(a.p.weight) * w * g);
  }
  const double pg = block_total(sum_pg), kl = block_total(sum_kl), clipped = block_total(sum_clip);
  if (threadIdx.x == 0) {
    double loss = pg;
    if (a.p.kl_coef != 0.0f) loss += static_cast<double>(a.p.kl_coef) * kl;
    a.out[0] = static_cast<float>(static_cast<double>(a.p.weight) * loss);
    a.out[1] = static_cast<float>(pg);
    a.out[2] = static_cast<float>(kl);
    a.out[3] = static_cast<float>(clipped);
  }
}

// -log sigma(h) and sigma(h), without overflow.
__device__ __forceinline__ double neg_log_sigmoid(double h) {
  return (h < 0.0 ? -h : 0.0) + log1p(exp(-fabs(h)));
}
__device__ __forceinline__ double sigmoid(double h) {
  const double q = exp(-fabs(h));
  return (h < 0.0 ? q : 1.0) / (1.0 + q);
}

__global__ __launch_bounds__(kTermThreads) void preference_terms_kernel(PreferenceArgs a) {
  const int lane = threadIdx.x & 63;
  // one wave per sequence in turn
  for (int b = threadIdx.x >> 6; b < a.batch; b += kTermThreads / 64) {
    double sum = 0.0;
    int n = 0;
    for (int t0 = 0; t0 < a.seq; t0 += 64) {
      const int64_t t = static_cast<int64_t>(b) * a.seq + t0 + lane;
      const bool counts = t0 + lane < a.seq && a.labels[t] >= 0;
      n += __popcll(__ballot(counts));
      if (counts) sum += a.lp[t] - (a.ref_lp ? static_cast<double>(a.ref_lp[t]) : 0.0);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) {
      a.counts[b] = n;
      const double s = a.p.average ? (n ? sum / n : 0.0) : sum;
      a.score[b] = s;
      if (a.rewards) a.rewards[b] = static_cast<float>(static_cast<double>(a.p.beta) * s);
    }
  }
  __syncthreads();
  const int pairs = a.batch / 2;
  const double beta = a.p.beta, eps = a.p.label_smoothing;
  double loss = 0.0, margin = 0.0, won = 0.0;
  for (int i = threadIdx.x; i < pairs; i += kTermThreads) {
    const double m = a.score[i] - a.score[i + pairs], h = beta * m;
    if (a.p.kind == MUON_PREFERENCE_SIGMOID) {
      loss += (1.0 - eps) * neg_log_sigmoid(h) + eps * neg_log_sigmoid(-h);
    } else {
      const double d = m - 0.5 / beta;
      loss += d * d;
    }
    margin += h;
    won += m > 0.0 ? 1.0 : 0.0;
  }
  loss = block_total(loss);
  margin = block_total(margin);
  won = block_total(won);
  if (threadIdx.x == 0) {
    const double n = pairs > 0 ? pairs : 1;
    a.out[0] = static_cast<float>(static_cast<double>(a.p.weight) * loss / n);
    a.out[1] = static_cast<float>(margin / n);
    a.out[2] = static_cast<float>(won / n);
  }
  if (a.g == nullptr) return;
  for (int t = threadIdx.x; t < a.batch * a.seq; t += kTermThreads) {
    float g = 0.0f;
    if (a.labels[t] >= 0) {
      const int b = t / a.seq, i = b < pairs ? b : b - pairs;
      const double m = a.score[i] - a.score[i + pairs], h = beta * m;
      double d = a.p.kind == MUON_PREFERENCE_SIGMOID ? beta * (eps * sigmoid(h) - (1.0 - eps) * sigmoid(-h))
                                                     : 2.0 * (m - 0.5 / beta);
      if (b >= pairs) d = -d;
      if (a.p.average) d /= a.counts[b];
      g = static_cast<float>(static_cast<double>(a.p.weight) * d / pairs);
    }
    a.g[t] = g;
  }
}

}  // namespace

int loss_splits(int64_t rows, int64_t vocab, int bf16, int cus) {
  // Rows that leave compute units idle are split, down to one trip of a
  // workgroup's loads per split.
  const int64_t trip = static_cast<int64_t>(kStatsThreads) * kStatsUnroll * (bf16 ? 8 : 4);
  int64_t want = (2 * static_cast<int64_t>(cus) + rows - 1) / (rows > 0 ? rows : 1);
  const int64_t most = (vocab + trip - 1) / trip;
  if (want > most) want = most;
  return static_cast<int>(want < 1 ? 1 : want > 32 ? 32 : want);
}

// Rows of one launch when each takes `per` workgroups: a grid holds fewer than
// 2^32 threads.
static int rows_per_launch(int64_t per) {
  const int64_t n = 0xff0000 / per;  // of 256 threads
  return static_cast<int>(n > 1 ? n : 1);
}

hipError_t launch_row_stats(hipStream_t s, const LossArgs& a) {
  LossArgs c = a;
  const int step = rows_per_launch(a.splits);
  for (c.row0 = 0; c.row0 < a.rows; c.row0 += step) {
    const int n = a.rows - c.row0 < step ? a.rows - c.row0 : step;
    const unsigned grid = static_cast<unsigned>(n) * static_cast<unsigned>(a.splits);
    if (a.bf16) row_stats_kernel<bf16_t><<<grid, kStatsThreads, 0, s>>>(c);
    else row_stats_kernel<float><<<grid, kStatsThreads, 0, s>>>(c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.splits > 1 && a.rows > 0) {
    const unsigned blocks = static_cast<unsigned>((a.rows + 63) / 64);
    if (a.bf16) row_join_kernel<bf16_t><<<blocks, 64, 0, s>>>(a);
    else row_join_kernel<float><<<blocks, 64, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_logits_grad(hipStream_t s, const LossArgs& a, RowsRef grad, const float* g) {
  const int vec = a.bf16 ? 8 : 4;
  // pieces of a row that starts as late in a piece as it can
  const int64_t pieces = (static_cast<int64_t>(a.vocab) + 2 * vec - 2) / vec;
  const int chunks = static_cast<int>((pieces + kGradThreads * kGradUnroll - 1) / (kGradThreads * kGradUnroll));
  LossArgs c = a;
  const int step = rows_per_launch(chunks);
  for (c.row0 = 0; c.row0 < a.rows; c.row0 += step) {
    const int n = a.rows - c.row0 < step ? a.rows - c.row0 : step;
    const unsigned grid = static_cast<unsigned>(n) * static_cast<unsigned>(chunks);
    if (a.bf16) logits_grad_kernel<bf16_t><<<grid, kGradThreads, 0, s>>>(c, grad, g, chunks);
    else logits_grad_kernel<float><<<grid, kGradThreads, 0, s>>>(c, grad, g, chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_policy_terms(hipStream_t s, const PolicyArgs& a) {
  policy_terms_kernel<<<1, kTermThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_preference_terms(hipStream_t s, const PreferenceArgs& a) {
  preference_terms_kernel<<<1, kTermThreads, 0, s>>>(a);
  return hipGetLastError();
}
