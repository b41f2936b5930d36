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
#include <algorithm>
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

// A row is walked in pieces of 16 bytes at 16-byte addresses.  What lies
// before the first and after the last of them (rows of an odd vocabulary start
// at odd addresses) are edges: at most 2 (kVec - 1) single scores, taken by as
// many threads of the first wave.
struct RowShape {
  int head;   // scores before the first piece
  int full;   // pieces
  int edges;  // single scores in all
};
template <typename T> __device__ __forceinline__ RowShape row_shape(const T* row, int vocab) {
  RowShape s;
  s.head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(T));
  if (s.head > vocab) s.head = vocab;
  s.full = (vocab - s.head) / kVec<T>;
  s.edges = vocab - s.full * kVec<T>;
  return s;
}
// The score that edge i < edges is.
template <typename T> __device__ __forceinline__ int edge_score(const RowShape& s, int i) {
  return i < s.head ? i : i + s.full * kVec<T>;
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

// The pair of N neighbouring lanes, in each of them.
template <int N = 64> __device__ __forceinline__ void wave_join(float& m, float& s, float k) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) {
    const float mo = __shfl_xor(m, d, 64), so = __shfl_xor(s, d, 64);
    const float mn = fmaxf(m, mo);
    // a + b commutes: both partners form the same sum
    const float a = s * exp2_fast((m - mn) * k), b = so * exp2_fast((mo - mn) * k);
    s = a + b;
    m = mn;
  }
}

// The pair of all threads of the workgroup, in every thread.
template <int NT> __device__ __forceinline__ void block_join(float& m, float& s, float k) {
  constexpr int W = NT / 64;
  __shared__ float2 wave[W];
  wave_join(m, s, k);
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = make_float2(m, s);
  __syncthreads();
  m = wave[0].x;
  s = wave[0].y;
#pragma unroll
  for (int w = 1; w < W; ++w) join(m, s, wave[w].x, wave[w].y, k);
}

// z_y - M - log S with T = 1 / inv_t, xm = x_y - max x.  log S = ln 2 (e +
// log2 f), S = 2^e f with f in [1/2, 1): the large part is exact, so the
// absolute error is that of log2 f, below 2^-23, at any S.
__device__ __forceinline__ double token_lp(float xm, float s, double inv_t) {
  int e = 0;
  const float f = frexpf(s, &e);
  const double log2s = static_cast<double>(e) + static_cast<double>(__builtin_amdgcn_logf(f));
  return static_cast<double>(xm) * inv_t - log2s * 0.69314718055994530942;
}

// What the row's pair makes of token r (one thread).
template <typename T>
__device__ __forceinline__ void finish_row(const LossArgs& a, int r, int64_t y, float m, float s) {
  double lp = 0.0;
  if (y >= a.vocab) {
    lp = __longlong_as_double(0x7ff8000000000000ll);
  } else if (y >= 0) {
    const float xm = muon::Elem<T>::load(row_at<const T>(a.x, r, a.seq) + y) - m;
    lp = token_lp(xm, s, 1.0 / static_cast<double>(a.temperature));
  }
  if (a.lp) a.lp[r] = lp;
  if (a.logps) a.logps[r] = static_cast<float>(lp);
  if (a.stats) a.stats[r] = make_float2(m, s);
}

constexpr int kStatsThreads = 256;
constexpr int kStatsUnroll = 4;  // pieces in flight per thread, twice

// (m, s) with the scores of one piece.
template <typename T> __device__ __forceinline__ void take_piece(u32x4 w, float& m, float& s, float k) {
  float v[kVec<T>];
  Scores<T>::unpack(w, v);
  float mn = m;
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) mn = fmaxf(mn, v[i]);
  s *= exp2_fast((m - mn) * k);
  m = mn;
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) s += exp2_fast((v[i] - m) * k);
}
__device__ __forceinline__ void take_score(float v, float& m, float& s, float k) {
  const float mn = fmaxf(m, v);
  s = s * exp2_fast((m - mn) * k) + exp2_fast((v - mn) * k);
  m = mn;
}

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
  const RowShape sh = row_shape(row, a.vocab);
  const u32x4* body = reinterpret_cast<const u32x4*>(row + sh.head);
  const int per = (sh.full + a.splits - 1) / a.splits;
  const int p0 = sp * per, p1 = min(sh.full, p0 + per);
  constexpr int U = kStatsUnroll, step = kStatsThreads * U;
  const u32x4 masked = {Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked};
  float m = kLowest, s = 0.0f;
  const int t = static_cast<int>(threadIdx.x);
  auto load = [&](u32x4* w, int base) {
    if (base + step <= p1) {
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = body[base + u * kStatsThreads + t];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = base + u * kStatsThreads + t;
        w[u] = masked;
        if (q < p1) w[u] = body[q];
      }
    }
  };
  // two sets of loads: one in flight while the other is taken
  u32x4 w[2][U];
  load(w[0], p0);
  for (int base = p0; base < p1; base += 2 * step) {
    load(w[1], base + step);
#pragma unroll
    for (int u = 0; u < U; ++u) take_piece<T>(w[0][u], m, s, k);
    load(w[0], base + 2 * step);
#pragma unroll
    for (int u = 0; u < U; ++u) take_piece<T>(w[1][u], m, s, k);
  }
  if (sp == 0 && t < sh.edges) take_score(muon::Elem<T>::load(row + edge_score<T>(sh, t)), m, s, k);
  block_join<kStatsThreads>(m, s, k);
  if (t == 0) {
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

// Gradient of row blockIdx / chunks, pieces of chunk blockIdx % chunks (the
// first chunk takes the edges).
template <typename T>
__global__ __launch_bounds__(kGradThreads) void logits_grad_kernel(LossArgs a, RowsRef grad,
                                                                   const float* __restrict__ g, int chunks) {
  const int r = a.row0 + static_cast<int>(blockIdx.x) / chunks, c = static_cast<int>(blockIdx.x) % chunks;
  const int64_t y = a.labels[r];
  const T* row = row_at<const T>(a.x, r, a.seq);
  T* out = row_at<T>(grad, r, a.seq);
  const RowShape sh = row_shape(row, a.vocab);
  const u32x4* body = reinterpret_cast<const u32x4*>(row + sh.head);
  // the gradient's rows have an alignment of their own
  u32x4_any* obody = reinterpret_cast<u32x4_any*>(out + sh.head);
  const int t = static_cast<int>(threadIdx.x), p0 = c * kGradThreads * kGradUnroll + t;
  const bool edge = c == 0 && t < sh.edges;
  if (y < 0) {
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int p = p0 + u * kGradThreads;
      if (p < sh.full) obody[p] = u32x4{0, 0, 0, 0};
    }
    if (edge) muon::Elem<T>::store(out + edge_score<T>(sh, t), 0.0f);
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
    if (p < sh.full) w[u] = body[p];
  }
  // the label's place: piece py, score iy of it (no piece when it is an edge)
  const int ly = static_cast<int>(y < a.vocab ? y : 0) - sh.head;
  const int py = ly >= 0 ? ly / kVec<T> : -1, iy = ly - py * kVec<T>;
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int p = p0 + u * kGradThreads;
    if (p >= sh.full) continue;
    float v[kVec<T>];
    Scores<T>::unpack(w[u], v);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = scale * exp2_fast((v[i] - st.x) * k);
    if (p == py) {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i)
        if (i == iy) v[i] += G;
    }
    obody[p] = Scores<T>::pack(v);
  }
  if (edge) {
    const int e = edge_score<T>(sh, t);
    float v = scale * exp2_fast((muon::Elem<T>::load(row + e) - st.x) * k);
    if (e == y) v += G;
    muon::Elem<T>::store(out + e, v);
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
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

// exp(e) - 1 - e.  Below 1 by its series e^2 (1/2! + e/3! + ...), which keeps
// the relative accuracy that the difference loses; the term after the last is
// e^12 / 14! < 2e-11 of the first.
__device__ __forceinline__ float exp_excess(float e) {
  if (fabsf(e) < 1.0f) {
    float q = 1.6059044e-10f;  // 1 / 13!
    q = q * e + 2.0876757e-9f;
    q = q * e + 2.5052108e-8f;
    q = q * e + 2.7557319e-7f;
    q = q * e + 2.7557319e-6f;
    q = q * e + 2.4801587e-5f;
    q = q * e + 1.9841270e-4f;
    q = q * e + 1.3888889e-3f;
    q = q * e + 8.3333333e-3f;
    q = q * e + 4.1666667e-2f;
    q = q * e + 1.6666667e-1f;
    q = q * e + 0.5f;
    return q * e * e;
  }
  return expf(e) - 1.0f - e;
}

// One token of the policy loss: its terms and the gradient of pg + kl_coef kl
// in lp.  The differences of log-probabilities are formed in binary64; what
// follows has no cancellation left and is done in fp32 (a few roundings, far
// below the error of lp itself).
struct TokenTerms {
  float pg, kl, clipped, g;
};
__device__ __forceinline__ TokenTerms policy_token(const PolicyArgs& a, int t, int b, double lp) {
  TokenTerms o;
  const float A = a.adv[a.p.advantage_per_token ? t : b];
  // without an old policy it is the policy itself: ratio 1 (NaN when lp is)
  const float ratio = a.old_lp ? expf(static_cast<float>(lp - a.old_lp[t])) : lp == lp ? 1.0f : __uint_as_float(0x7fc00000u);
  const float lo = 1.0f - a.p.clip_low, hi = 1.0f + a.p.clip_high;
  const float held = -A * (ratio < lo ? lo : ratio > hi ? hi : ratio);
  const float free = -A * ratio;
  o.pg = max_nan(free, held);
  o.clipped = held > free ? 1.0f : 0.0f;
  o.g = held > free ? 0.0f : free;
  o.kl = 0.0f;
  if (a.ref_lp) {
    const float e = static_cast<float>(static_cast<double>(a.ref_lp[t]) - lp);
    o.kl = exp_excess(e);
    if (a.p.kl_coef != 0.0f) o.g -= a.p.kl_coef * (o.kl + e);  // kl + e = exp(e) - 1
  }
  return o;
}

__device__ __forceinline__ void write_policy(const PolicyArgs& a, double pg, double kl, double clipped) {
  double loss = pg;
  if (a.p.kl_coef != 0.0f) loss += static_cast<double>(a.p.kl_coef) * kl;
  a.out[0] = static_cast<float>(static_cast<double>(a.p.weight) * loss);
  a.out[1] = static_cast<float>(pg);
  a.out[2] = static_cast<float>(kl);
  a.out[3] = static_cast<float>(clipped);
}

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
    const TokenTerms o = policy_token(a, t, b, a.lp[t]);
    sum_pg += w * static_cast<double>(o.pg);
    sum_kl += w * static_cast<double>(o.kl);
    sum_clip += w * static_cast<double>(o.clipped);
    if (a.g) a.g[t] = static_cast<float>(static_cast<double>(a.p.weight) * w * static_cast<double>(o.g));
  }
  const double pg = block_total(sum_pg), kl = block_total(sum_kl), clipped = block_total(sum_clip);
  if (threadIdx.x == 0) write_policy(a, pg, kl, clipped);
}

// ---------------------------------------------------------------------------
// rows held in registers
// ---------------------------------------------------------------------------
// One workgroup holds a whole row (NV pieces a thread: 304 KB of the 512 KB of
// a compute unit's registers at 151936 bf16 scores), so the policy loss, whose
// gradient of a token needs nothing of other rows but their number, reads
// every score once and writes every gradient once.  The workgroup walks rows
// blockIdx, + gridDim, ...; as soon as a piece's gradient has gone out, the
// same registers receive the next row's piece, so loads are in flight through
// the whole second half of a row.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT, 4) void policy_rows_kernel(LossArgs a, RowsRef grad, PolicyArgs p) {
  constexpr int W = NT / 64;
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, wave = t >> 6;
  const int stride = static_cast<int>(gridDim.x);
  const float k = kLog2e / a.temperature;
  const u32x4 masked = {Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked, Scores<T>::kMasked};
  __shared__ float2 part[2][W];
  __shared__ int found[2][W];
  __shared__ float coef[2][3];
  __shared__ double weight, sums[3];  // of wave 0

  // The next row from r on that counts; rows left out on the way get their zeros.
  auto next_row = [&](int r) {
    for (; r < a.rows && a.labels[r] < 0; r += stride) {
      if (t == 0 && a.logps) a.logps[r] = 0.0f;
      if (grad.base == nullptr) continue;
      T* out = row_at<T>(grad, r, a.seq);
      const RowShape sh = row_shape(row_at<const T>(a.x, r, a.seq), a.vocab);
      u32x4_any* body = reinterpret_cast<u32x4_any*>(out + sh.head);
      for (int q = t; q < sh.full; q += NT) body[q] = u32x4{0, 0, 0, 0};
      if (t < sh.edges) muon::Elem<T>::store(out + edge_score<T>(sh, t), 0.0f);
    }
    return r;
  };

  u32x4 w[NV];
  float we = -INFINITY;  // this thread's edge
  int r = next_row(static_cast<int>(blockIdx.x));
  const T* row = row_at<const T>(a.x, r < a.rows ? r : 0, a.seq);
  RowShape sh = row_shape(row, a.vocab);
  if (r < a.rows) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      w[i] = masked;
      if (i * NT + t < sh.full) w[i] = reinterpret_cast<const u32x4*>(row + sh.head)[i * NT + t];
    }
    if (t < sh.edges) we = muon::Elem<T>::load(row + edge_score<T>(sh, t));
  }
  int counted = -1;  // the sequence (or 0: all) whose tokens the weight goes by
  if (t == 0) sums[0] = sums[1] = sums[2] = 0.0;
  const double inv_t = 1.0 / static_cast<double>(a.temperature);
  for (int parity = 0; r < a.rows; parity ^= 1) {
    const int b = r / a.seq;
    const int64_t y = a.labels[r];
    const bool named = y < a.vocab;
    const float xy = muon::Elem<T>::load(row + (named ? y : 0));
    // tokens that share the loss's mean with this one
    const int set = p.p.reduce == MUON_REDUCE_SEQUENCE ? b : 0;
    const bool count = set != counted;
    if (count && p.p.reduce != MUON_REDUCE_SUM) {
      const int lo = p.p.reduce == MUON_REDUCE_SEQUENCE ? b * a.seq : 0;
      const int hi = p.p.reduce == MUON_REDUCE_SEQUENCE ? lo + a.seq : a.rows;
      int n = 0;
      for (int j = lo + t; j - t < hi; j += NT) n += __popcll(__ballot(j < hi && a.labels[j < hi ? j : lo] >= 0));
      if (lane == 0) found[parity][wave] = n;
    }
    counted = set;
    float m = kLowest, s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      take_piece<T>(w[i], m, s, k);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (t < sh.edges) take_score(we, m, s, k);
    wave_join(m, s, k);
    if (lane == 0) part[parity][wave] = make_float2(m, s);
    const int rn = next_row(r + stride);
    __syncthreads();
    if (wave == 0) {
      const float2 q = part[parity][lane % W];
      m = q.x;
      s = q.y;
      wave_join<W>(m, s, k);
      if (count && lane == 0) {
        double n = 0.0;
        for (int i = 0; i < W; ++i) n += found[parity][i];
        weight = p.p.reduce == MUON_REDUCE_TOKEN      ? 1.0 / n
                 : p.p.reduce == MUON_REDUCE_SEQUENCE ? 1.0 / (n * p.batch)
                                                      : 1.0;
      }
      double lp = token_lp(xy - m, s, inv_t);
      if (!named) lp = __longlong_as_double(0x7ff8000000000000ll);
      const TokenTerms o = policy_token(p, r, b, lp);
      if (lane == 0) {
        const double wt = weight;
        sums[0] += wt * static_cast<double>(o.pg);
        sums[1] += wt * static_cast<double>(o.kl);
        sums[2] += wt * static_cast<double>(o.clipped);
        const float G = static_cast<float>(static_cast<double>(p.p.weight) * wt * static_cast<double>(o.g)) / a.temperature;
        coef[parity][0] = m;
        coef[parity][1] = -G / s;
        coef[parity][2] = G;
        if (a.logps) a.logps[r] = static_cast<float>(lp);
      }
    }
    __syncthreads();
    const float M = coef[parity][0], scale = coef[parity][1], G = coef[parity][2];
    // The pieces are unpacked again: as far as the compiler knows they may
    // have changed, so it keeps 4 registers a piece across the join, not 8
    // more of widened scores.
#pragma unroll
    for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(w[i]));
    const T* nrow = row_at<const T>(a.x, rn < a.rows ? rn : r, a.seq);
    const RowShape nsh = row_shape(nrow, a.vocab);
    const u32x4* nbody = reinterpret_cast<const u32x4*>(nrow + nsh.head);
    const int nfull = rn < a.rows ? nsh.full : 0;
    if (grad.base) {
      T* out = row_at<T>(grad, r, a.seq);
      u32x4_any* obody = reinterpret_cast<u32x4_any*>(out + sh.head);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[kVec<T>];
        Scores<T>::unpack(w[i], v);
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) v[e] = scale * exp2_fast((v[e] - M) * k);
        if (i * NT + t < sh.full) obody[i * NT + t] = Scores<T>::pack(v);
        w[i] = masked;
        if (i * NT + t < nfull) w[i] = nbody[i * NT + t];
        __builtin_amdgcn_sched_barrier(0);
      }
      if (t < sh.edges) muon::Elem<T>::store(out + edge_score<T>(sh, t), scale * exp2_fast((we - M) * k));
      // the label's score, by the thread whose piece or edge has just gone out
      if (named) {
        const int ly = static_cast<int>(y) - sh.head;
        const bool in_piece = ly >= 0 && ly < sh.full * kVec<T>;
        const int owner = in_piece ? (ly / kVec<T>) % NT : ly < 0 ? static_cast<int>(y) : ly - sh.full * kVec<T> + sh.head;
        if (t == owner) muon::Elem<T>::store(out + y, scale * exp2_fast((xy - M) * k) + G);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        w[i] = masked;
        if (i * NT + t < nfull) w[i] = nbody[i * NT + t];
      }
    }
    if (rn < a.rows && t < nsh.edges) we = muon::Elem<T>::load(nrow + edge_score<T>(nsh, t));
    r = rn;
    row = nrow;
    sh = nsh;
  }
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) p.sums[static_cast<int64_t>(blockIdx.x) * 3 + i] = sums[i];
  }
}

// The losses of `n` workgroups, in index order per thread.
__global__ __launch_bounds__(kTermThreads) void policy_sums_kernel(PolicyArgs p, int n) {
  double v[3] = {0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < n; i += kTermThreads)
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] += p.sums[static_cast<int64_t>(i) * 3 + j];
#pragma unroll
  for (int j = 0; j < 3; ++j) v[j] = block_total(v[j]);
  if (threadIdx.x == 0) write_policy(p, v[0], v[1], v[2]);
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
  const int pieces = a.vocab / vec;  // the most a row can have
  const int chunks = std::max(1, (pieces + kGradThreads * kGradUnroll - 1) / (kGradThreads * kGradUnroll));
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

namespace {

template <typename T, int NT, int NV>
hipError_t run_policy_rows(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p, int cus) {
  const int grid = std::min(a.rows, cus * (1024 / NT));
  policy_rows_kernel<T, NT, NV><<<static_cast<unsigned>(grid), NT, 0, s>>>(a, grad, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  policy_sums_kernel<<<1, kTermThreads, 0, s>>>(p, grid);
  return hipGetLastError();
}

template <typename T>
hipError_t policy_rows(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p, int cus) {
  const int pieces = a.vocab / kVec<T>;
  if (pieces <= 256 * 5) return run_policy_rows<T, 256, 5>(s, a, grad, p, cus);
  if (pieces <= 256 * 10) return run_policy_rows<T, 256, 10>(s, a, grad, p, cus);
  if (pieces <= 256 * 15) return run_policy_rows<T, 256, 15>(s, a, grad, p, cus);
  if (pieces <= 256 * 19) return run_policy_rows<T, 256, 19>(s, a, grad, p, cus);
  if (pieces <= 512 * 15) return run_policy_rows<T, 512, 15>(s, a, grad, p, cus);
  if (pieces <= 512 * 19) return run_policy_rows<T, 512, 19>(s, a, grad, p, cus);
  if (pieces <= 1024 * 15) return run_policy_rows<T, 1024, 15>(s, a, grad, p, cus);
  return run_policy_rows<T, 1024, 19>(s, a, grad, p, cus);
}

}  // namespace

bool policy_rows_fit(const LossArgs& a) { return a.vocab / (a.bf16 ? 8 : 4) <= 1024 * 19; }

hipError_t launch_policy_rows(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p, int cus) {
  return a.bf16 ? policy_rows<bf16_t>(s, a, grad, p, cus) : policy_rows<float>(s, a, grad, p, cus);
}

hipError_t launch_preference_terms(hipStream_t s, const PreferenceArgs& a) {
  preference_terms_kernel<<<1, kTermThreads, 0, s>>>(a);
  return hipGetLastError();
}
