// Verification of drafted tokens against the target's probabilities.
//
// Mathematics.  Keeping a token x drawn from q with probability min(1, p(x) /
// q(x)), and drawing from max(p - q, 0) where it is not kept, gives a token
// distributed as p: min(p, q) + max(p - q, 0) = p.
//
// Arithmetic.  Whether a token is kept is one comparison of two probabilities
// with a random number: fp32 exponentials added in binary64 leave it wrong once
// in some 10^7 times, and every row has to be read for it.  Which token is
// drawn depends on running sums over the vocabulary: an error d of those
// moves some of V borders past u, V d in all, so that fp32 (d = 3e-8, V =
// 151936) would draw another token every few hundred times.  The one or two
// rows that are drawn from are therefore read again with exponentials good to
// 2^-45 and everything in binary64.
//
// Shape.  Rows are cut into slices, a workgroup each.
//   verify_pairs_kernel: maximum and sum of every row that may be needed (the
//     bound: HBM and the exponentials);
//   verify_sums_kernel: which place ends the sequence, and that row's sums;
//   verify_weights_kernel: the sums of max(p - q, 0) (with draft scores only);
//   verify_take_kernel: the slice that u falls into, the token, the outputs.
#include <cfloat>

#include "linear8.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kRun = 4, kMostCuts = 64 * kRun;  // slices of the second reading that a lane holds, and of a row
constexpr float kLowest = -FLT_MAX;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T> constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// Scores [i, i + kVec) of a row, those at or past `end` -infinity.
template <typename T>
__device__ __forceinline__ void piece(const T* row, int i, int end, float (&v)[kVec<T>]) {
  if (i + kVec<T> <= end) {
    const u32x4 w = *reinterpret_cast<const u32x4_any*>(row + i);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[j] = i + j < end ? muon::Elem<T>::load(row + i + j) : -INFINITY;
  }
}

__device__ __forceinline__ float wave_max(float v) {
  for (int d = 32; d > 0; d /= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
  for (int d = 32; d > 0; d /= 2) v = min(v, __shfl_xor(v, d));
  return v;
}

// What a slice, or a row, leaves: the largest score, the lowest index that has
// it (greedy), the sum of exp((x - m) / T).
struct Part {
  float m;
  int best;
  double s;
};

// log2 e / T = k + rest.  Of the scores of 16 bytes some take k's upper and some
// its lower neighbour in fp32, so that their mean is right to 2^-27: k rounded
// once is another temperature, and puts every sum off the same way.
struct Scale {
  float k, rest;
  const float (&each)[8];
  __device__ __forceinline__ explicit Scale(const VerifyArgs& a) : k(a.k), rest(a.k_rest), each(a.k_each) {}
  __device__ __forceinline__ double exp(float d) const {  // exp(d / T), d <= 0, between maxima
    const float f = fmaxf(d, -256.0f / k);                // (2^-256: 0)
    return static_cast<double>(__builtin_amdgcn_exp2f(__builtin_fmaf(f, k, f * rest)));
  }
};

// 2^t for t <= 0, to 2^-45: t = n / 32 + f with a table of 2^(j / 32), and a
// polynomial of degree 5 in f log 2 (|f log 2| <= 0.0109: the rest is 2^-48).
struct Exp2 {
  const double* table;  // LDS
  __device__ __forceinline__ double operator()(double t) const {
    t = fmax(t, -1080.0);
    const double n = rint(t * 32.0);
    const double f = __builtin_fma(n, -1.0 / 32.0, t) * 0.69314718055994530942;
    const int i = static_cast<int>(n);
    double p = __builtin_fma(f, 1.0 / 120.0, 1.0 / 24.0);
    p = __builtin_fma(f, p, 1.0 / 6.0);
    p = __builtin_fma(f, p, 0.5);
    p = __builtin_fma(f, p, 1.0);
    p = __builtin_fma(f, p, 1.0);
    return ldexp(p * table[i & 31], i >> 5);
  }
};
__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < 32) table[threadIdx.x] = exp2(static_cast<double>(threadIdx.x) / 32.0);
}

template <typename T> __device__ __forceinline__ const T* row_of(const RowsRef& x, int b, int i) {
  return reinterpret_cast<const T*>(x.base + b * x.bs + i * x.rs);
}

// Places that sequence b drafts; every thread of a wave takes part.
__device__ __forceinline__ int drafted_places(const VerifyArgs& a, int b) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < a.draft; i0 += 64) {
    const bool ends = i0 + lane < a.draft && a.drafted[static_cast<int64_t>(b) * a.draft + i0 + lane] < 0;
    const uint64_t any = __ballot(ends);
    if (any) return i0 + __builtin_ctzll(any);
  }
  return a.draft;
}

constexpr int kPieces = 8;  // of 16 bytes that a thread holds

// (m, best, s) of scores [lo, hi) of a row, hi - lo <= kThreads kPieces kVec; in thread 0.
template <typename T, bool GREEDY>
__device__ __forceinline__ Part slice_part(const T* row, int lo, int hi, const Scale& q) {
  __shared__ float wm[kWaves];
  __shared__ double ws[kWaves];
  __shared__ int wb[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float v[kPieces][kVec<T>];
  float m = kLowest;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int i = lo + (p * kThreads + static_cast<int>(threadIdx.x)) * kVec<T>;
    if (lo + p * kThreads * kVec<T> < hi) piece(row, i, hi, v[p]);
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
    if (lo + p * kThreads * kVec<T> < hi) {
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) m = fmaxf(m, v[p][j]);
    }
  m = wave_max(m);
  double s = 0.0;
  int best = INT32_MAX;
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
    if (lo + p * kThreads * kVec<T> < hi) {
      float e[kVec<T>];
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) e[j] = __builtin_amdgcn_exp2f((v[p][j] - m) * q.each[j]);
#pragma unroll
      for (int w = kVec<T> / 2; w > 0; w /= 2)
#pragma unroll
        for (int j = 0; j < w; ++j) e[j] += e[j + w];
      s += static_cast<double>(e[0]);
      if (GREEDY) {
#pragma unroll
        for (int j = kVec<T> - 1; j >= 0; --j)
          if (v[p][j] == m) best = min(best, lo + (p * kThreads + static_cast<int>(threadIdx.x)) * kVec<T> + j);
      }
    }
  s = wave_sum(s);
  if (GREEDY) best = wave_min(best);
  if (lane == 0) wm[wave] = m, ws[wave] = s, wb[wave] = best;
  __syncthreads();
  Part r = {kLowest, INT32_MAX, 0.0};
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWaves; ++w) r.m = fmaxf(r.m, wm[w]);
    for (int w = 0; w < kWaves; ++w) {
      r.s += ws[w] * q.exp(wm[w] - r.m);
      if (GREEDY && wm[w] == r.m) r.best = min(r.best, wb[w]);
    }
    if (r.m == INFINITY) r.s = static_cast<double>(NAN);
  }
  return r;
}

template <typename TX, typename TD, bool GREEDY>
__global__ __launch_bounds__(kThreads) void verify_pairs_kernel(VerifyArgs a) {
  const int j = blockIdx.x, b = blockIdx.z, i = blockIdx.y;  // rows 0 .. draft: the target's, beyond: the draft's
  const int len = drafted_places(a, b);
  const bool target = i <= a.draft;
  const int place = target ? i : i - a.draft - 1;
  if (target ? place > len : place >= len) return;
  const Scale q(a);
  const int lo = j * a.slice, hi = min(lo + a.slice, a.vocab);
  const Part r = target ? slice_part<TX, GREEDY>(row_of<TX>(a.x, b, place), lo, hi, q)
                        : slice_part<TD, GREEDY>(row_of<TD>(a.d, b, place), lo, hi, q);
  if (threadIdx.x == 0) a.parts[(static_cast<int64_t>(b) * a.rows + i) * a.slices + j] = {r.m, r.best, r.s};
}

// A row's part from its slices', in every lane of the wave.
__device__ __forceinline__ Part row_part(const VerifyArgs& a, int b, int i, const Scale& q) {
  const int lane = threadIdx.x & 63;
  Part r = {kLowest, INT32_MAX, 0.0};
  if (lane < a.slices) {
    const VerifyPart p = a.parts[(static_cast<int64_t>(b) * a.rows + i) * a.slices + lane];
    r = {p.m, p.best, p.s};
  }
  const float m = wave_max(r.m);
  r.s = r.s == 0.0 ? 0.0 : r.s * q.exp(r.m - m);
  r.s = wave_sum(r.s);
  r.best = wave_min(r.m == m ? r.best : INT32_MAX);
  r.m = m;
  return r;
}
__device__ __forceinline__ bool has_distribution(const Part& p) { return p.s > 0.0 && p.s < static_cast<double>(INFINITY); }

// How sequence b ends, found by a whole workgroup: the place r and the row's
// parts there; with `out` the kept tokens and their log-probabilities are
// written.
struct End {
  int r;        // place that takes its token
  int y;        // the token drafted there, -1: none (or past the vocabulary: -2)
  int mode;     // 0: no distribution, 1: from p, 2: from max(p - q, 0)
  float mp, mq;
  int best;
  double sp;
};
template <typename TX, typename TD>
__device__ __forceinline__ End find_end(const VerifyArgs& a, int b, bool out) {
  __shared__ int first[kWaves];
  __shared__ End end;
  __shared__ float kept[MUON_MAX_DRAFT];
  const bool greedy = a.inv_t == 0.0;
  const Scale q(a);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int len = drafted_places(a, b);
  End mine = {INT32_MAX, -1, 0, 0.0f, 0.0f, 0, 0.0};
  // each wave takes every kWaves-th place, up to the first that is not kept
  for (int i = wave; i <= len; i += kWaves) {
    const Part P = row_part(a, b, i, q);
    const int64_t y = i < len ? a.drafted[static_cast<int64_t>(b) * a.draft + i] : -1;
    const bool named = y >= 0 && y < a.vocab;
    const bool ok = has_distribution(P);
    Part Q = {0.0f, 0, 1.0};
    bool near = true;
    double lp = 0.0;
    bool keep = false;
    if (ok && named) {
      const float xy = muon::Elem<TX>::load(row_of<TX>(a.x, b, i) + y);
      lp = (static_cast<double>(xy) - static_cast<double>(P.m)) * (greedy ? 1.0 : a.inv_t) - log(P.s);
    }
    if (greedy) {
      keep = ok && named && y == P.best;
    } else if (ok && y >= 0) {
      double qx = 1.0;
      if (a.d.base) {
        Q = row_part(a, b, a.draft + 1 + i, q);
        near = has_distribution(Q);
        if (near && named) qx = exp((static_cast<double>(muon::Elem<TD>::load(row_of<TD>(a.d, b, i) + y)) - static_cast<double>(Q.m)) * a.inv_t) / Q.s;
      }
      keep = named && near && static_cast<double>(a.uniforms[static_cast<int64_t>(b) * (a.draft + 1) + i]) * qx < exp(lp);
    }
    if (keep) {
      if (lane == 0) kept[i] = static_cast<float>(lp);
      continue;
    }
    mine = {i, named ? static_cast<int>(y) : y >= 0 ? -2 : -1, !ok ? 0 : (y >= 0 && near && !greedy ? 2 : 1), P.m, Q.m, P.best, P.s};
    break;
  }
  __syncthreads();
  if (lane == 0) first[wave] = mine.r;
  __syncthreads();
  int r = INT32_MAX;
  for (int w = 0; w < kWaves; ++w) r = min(r, first[w]);
  if (mine.r == r && lane == 0) end = mine;
  if (out)
    for (int i = threadIdx.x; i < r; i += kThreads) {
      const int64_t at = static_cast<int64_t>(b) * (a.draft + 1) + i;
      a.tokens[at] = a.drafted[static_cast<int64_t>(b) * a.draft + i];
      if (a.logps) a.logps[at] = kept[i];
    }
  __syncthreads();
  return end;
}

// Scores [lo, hi) of a row through f(index, score), a thread's in ascending order.
template <typename T, typename F>
__device__ __forceinline__ void each_score(const T* row, int lo, int hi, F&& f) {
  for (int i = lo + static_cast<int>(threadIdx.x) * kVec<T>; i < hi; i += kThreads * kVec<T>) {
    float v[kVec<T>];
    piece(row, i, hi, v);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) f(i + j, v[j]);
  }
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double lds[kWaves];
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kWaves; ++w) v += lds[w];
  return v;
}

// Sums over a slice of the row that is drawn from, around its maximum: of
// exp(x), and of exp of the draft's scores, or, without those, of exp(x) without
// the drafted token.
template <typename TX, typename TD>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs a) {
  __shared__ double table[32];
  fill_table(table);
  const int b = blockIdx.y, j = blockIdx.x;
  const End e = find_end<TX, TD>(a, b, j == 0);
  if (j == 0 && threadIdx.x == 0) a.ends[b] = {e.r, e.y, e.mode, e.mp, e.mq, e.best, e.sp};
  if (e.mode == 0) return;
  const Exp2 ex = {table};
  const int lo = j * a.cut, hi = min(lo + a.cut, a.vocab);
  double sp = 0.0, sq = 0.0;
  const double mp = e.mp, mq = e.mq;
  each_score(row_of<TX>(a.x, b, e.r), lo, hi, [&](int v, float x) {
    const double p = ex((static_cast<double>(x) - mp) * a.kd);
    sp += p;
    if (v != e.y) sq += p;
  });
  if (e.mode == 2 && a.d.base) {
    sq = 0.0;
    each_score(row_of<TD>(a.d, b, e.r), lo, hi, [&](int, float x) { sq += ex((static_cast<double>(x) - mq) * a.kd); });
  }
  sp = block_sum(sp);
  sq = block_sum(sq);
  if (threadIdx.x == 0) a.sums[static_cast<int64_t>(b) * a.cuts + j] = make_double2(sp, sq);
}

// The sum of column c (0: p, 1: q) of a sequence's sums, in every lane of the wave.
__device__ __forceinline__ double2 all_sums(const VerifyArgs& a, int b) {
  double2 t = make_double2(0.0, 0.0);
  for (int j = threadIdx.x & 63; j < a.cuts; j += 64) {
    const double2 s = a.sums[static_cast<int64_t>(b) * a.cuts + j];
    t.x += s.x;
    t.y += s.y;
  }
  return make_double2(wave_sum(t.x), wave_sum(t.y));
}

// max(p - q, 0) of one token.
struct Weight {
  double mp, mq, kd, ip, iq;
  Exp2 ex;
  __device__ __forceinline__ double operator()(float x, float d) const {
    const double p = ex((static_cast<double>(x) - mp) * kd) * ip, q = ex((static_cast<double>(d) - mq) * kd) * iq;
    return fmax(p - q, 0.0);
  }
};

template <typename TX, typename TD>
__global__ __launch_bounds__(kThreads) void verify_weights_kernel(VerifyArgs a) {
  __shared__ double table[32];
  fill_table(table);
  __syncthreads();
  const int b = blockIdx.y, j = blockIdx.x;
  const VerifyEnd e = a.ends[b];
  if (e.mode != 2) return;
  const double2 t = all_sums(a, b);
  const Weight w = {e.mp, e.mq, a.kd, 1.0 / t.x, 1.0 / t.y, {table}};
  const int lo = j * a.cut, hi = min(lo + a.cut, a.vocab);
  const TX* x = row_of<TX>(a.x, b, e.r);
  const TD* d = row_of<TD>(a.d, b, e.r);
  constexpr int N = kVec<TX> > kVec<TD> ? kVec<TX> : kVec<TD>;
  double s = 0.0;
  for (int i = lo + static_cast<int>(threadIdx.x) * N; i < hi; i += kThreads * N) {
    float vx[N], vd[N];
#pragma unroll
    for (int c = 0; c < N; c += kVec<TX>) piece(x, i + c, hi, *reinterpret_cast<float(*)[kVec<TX>]>(vx + c));
#pragma unroll
    for (int c = 0; c < N; c += kVec<TD>) piece(d, i + c, hi, *reinterpret_cast<float(*)[kVec<TD>]>(vd + c));
#pragma unroll
    for (int c = 0; c < N; ++c) s += w(vx[c], vd[c]);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) a.weights[static_cast<int64_t>(b) * a.cuts + j] = s;
}

// The token at the end of each sequence, and the outputs behind the kept ones.
template <typename TX, typename TD>
__global__ __launch_bounds__(kThreads) void verify_take_kernel(VerifyArgs a) {
  __shared__ double table[32], before[kWaves];
  __shared__ int chosen, last;
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool greedy = a.inv_t == 0.0;
  End e;
  double sum = 0.0;
  int64_t next = -1;
  fill_table(table);
  if (threadIdx.x == 0) chosen = INT32_MAX, last = -1;
  if (greedy) {
    e = find_end<TX, TD>(a, b, true);
    if (e.mode) next = e.best;
    sum = e.sp;
  } else {
    const VerifyEnd s = a.ends[b];
    e = {s.r, s.y, s.mode, s.mp, s.mq, s.best, s.sp};
    __syncthreads();
  }
  if (!greedy && e.mode) {
    const double2 t = all_sums(a, b);
    sum = t.x;
    // the slices' weights: one of three forms; a lane holds kRun of them
    enum { P, LESS, REST };
    int form = e.mode == 1 ? P : a.d.base ? REST : LESS;
    double held[kRun], upto;
    auto take_form = [&] {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int j = kRun * lane + i;
        const int64_t at = static_cast<int64_t>(b) * a.cuts + j;
        held[i] = j >= a.cuts ? 0.0 : form == REST ? a.weights[at] : form == LESS ? a.sums[at].y : a.sums[at].x;
        s += held[i];
      }
      upto = s;  // inclusive over the lanes
      for (int k = 1; k < 64; k *= 2) {
        const double o = __shfl_up(upto, k);
        if (lane >= k) upto += o;
      }
      return __shfl(upto, 63);
    };
    double total = take_form();
    if (!(total > 0.0)) form = P, total = take_form();
    const double want = static_cast<double>(a.uniforms[static_cast<int64_t>(b) * (a.draft + 1) + a.draft]) * total;
    // the first slice whose running sum exceeds it, else the last with weight
    double own = 0.0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) own += held[i];
    double run = upto - own;
    const uint64_t over = __ballot(own > 0.0 && upto > want), some = __ballot(own > 0.0);
    const int src = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
    int at = -1;
    double its = 0.0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (!(held[i] > 0.0) || (at >= 0 && run + its > want)) continue;
      run += its;  // the sum in front of slice `at`
      its = held[i];
      at = kRun * lane + i;
    }
    at = __shfl(at, src);
    run = __shfl(run, src);
    // `at` holds the token, unless rounding puts u past its last weight; then its last
    const TX* x = row_of<TX>(a.x, b, e.r);
    const TD* d = form == REST ? row_of<TD>(a.d, b, e.r) : nullptr;
    const Weight w = {e.mp, e.mq, a.kd, 1.0 / t.x, 1.0 / t.y, {table}};
    const int lo = at * a.cut, hi = min(lo + a.cut, a.vocab);
    // a contiguous run of tokens per thread
    const int per = (hi - lo + kThreads - 1) / kThreads, first = min(lo + per * static_cast<int>(threadIdx.x), hi), past = min(first + per, hi);
    auto weight = [&](int v) {
      const float xv = muon::Elem<TX>::load(x + v);
      if (form == REST) return w(xv, muon::Elem<TD>::load(d + v));
      if (form == LESS && v == e.y) return 0.0;
      return w.ex((static_cast<double>(xv) - w.mp) * a.kd);
    };
    double mine = 0.0;
    int my_last = -1;
    for (int v = first; v < past; ++v) {
      const double s = weight(v);
      if (s > 0.0) my_last = v;
      mine += s;
    }
    double scan = mine;  // inclusive over the wave
    for (int k = 1; k < 64; k *= 2) {
      const double o = __shfl_up(scan, k);
      if (lane >= k) scan += o;
    }
    if (lane == 63) before[wave] = scan;
    __syncthreads();
    double base = run;
    for (int k = 0; k < wave; ++k) base += before[k];
    double here = base + (scan - mine);
    if (my_last >= 0) atomicMax(&last, my_last);
    if (mine > 0.0 && here + mine > want) {
      for (int v = first; v < past; ++v) {
        const double s = weight(v);
        here += s;
        if (s > 0.0 && here > want) {
          atomicMin(&chosen, v);
          break;
        }
      }
    }
    __syncthreads();
    next = chosen != INT32_MAX ? chosen : last;
  }
  if (threadIdx.x == 0) {
    double lp = __longlong_as_double(0x7ff8000000000000ll);
    if (next >= 0) lp = (static_cast<double>(muon::Elem<TX>::load(row_of<TX>(a.x, b, e.r) + next)) - static_cast<double>(e.mp)) * (greedy ? 1.0 : a.inv_t) - log(sum);
    a.accepted[b] = e.r;
    a.tokens[static_cast<int64_t>(b) * (a.draft + 1) + e.r] = next;
    if (a.logps) a.logps[static_cast<int64_t>(b) * (a.draft + 1) + e.r] = static_cast<float>(lp);
  }
  for (int i = e.r + 1 + static_cast<int>(threadIdx.x); i <= a.draft; i += kThreads) {
    a.tokens[static_cast<int64_t>(b) * (a.draft + 1) + i] = -1;
    if (a.logps) a.logps[static_cast<int64_t>(b) * (a.draft + 1) + i] = 0.0f;
  }
}

// Sequences of one launch: the grid's third dimension, and the second of others.
constexpr int kMostBatch = 65535;

template <typename TX, typename TD>
hipError_t go(hipStream_t s, VerifyArgs a, int b0, int n) {
  a.x.base += b0 * a.x.bs;
  if (a.d.base) a.d.base += b0 * a.d.bs;
  const int64_t places = static_cast<int64_t>(b0) * (a.draft + 1);
  a.drafted += static_cast<int64_t>(b0) * a.draft;
  if (a.uniforms) a.uniforms += places;
  a.tokens += places;
  a.accepted += b0;
  if (a.logps) a.logps += places;
  const unsigned nb = static_cast<unsigned>(n);
  const dim3 grid(static_cast<unsigned>(a.slices), static_cast<unsigned>(a.rows), nb), cuts(static_cast<unsigned>(a.cuts), nb);
  if (a.inv_t == 0.0) {
    verify_pairs_kernel<TX, TD, true><<<grid, kThreads, 0, s>>>(a);
  } else {
    verify_pairs_kernel<TX, TD, false><<<grid, kThreads, 0, s>>>(a);
    verify_sums_kernel<TX, TD><<<cuts, kThreads, 0, s>>>(a);
    if (a.d.base) verify_weights_kernel<TX, TD><<<cuts, kThreads, 0, s>>>(a);
  }
  verify_take_kernel<TX, TD><<<nb, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

VerifyPlan verify_plan(int64_t batch, int64_t draft, int64_t vocab, int bytes) {
  VerifyPlan p;
  const int64_t most = kThreads * kPieces * 16 / bytes;  // scores of a slice
  p.slices = static_cast<int>((vocab + most - 1) / most);
  // whole pieces of 16 bytes
  p.slice = static_cast<int>(((vocab + p.slices - 1) / p.slices + 7) / 8 * 8);
  p.launch = static_cast<int>(batch < kMostBatch ? batch : kMostBatch);
  // the second reading: as many workgroups as fill the card, of 2048 scores at least
  int64_t cuts = (vocab + 2047) / 2048;
  static_assert(MUON_MAX_VOCAB / 2048 <= kMostCuts, "a wave holds a row's sums");
  const int64_t enough = (2048 + p.launch - 1) / (p.launch > 0 ? p.launch : 1);
  if (cuts > enough) cuts = enough;
  p.cut = static_cast<int>(((vocab + cuts - 1) / cuts + 7) / 8 * 8);
  p.cuts = static_cast<int>((vocab + p.cut - 1) / p.cut);
  p.rows = static_cast<int>(2 * draft + 1);
  size_t at = 0;
  auto take = [&](size_t bytes_) {
    const size_t was = at;
    at += (bytes_ + 255) & ~static_cast<size_t>(255);
    return was;
  };
  p.parts = take(sizeof(VerifyPart) * static_cast<size_t>(p.launch) * static_cast<size_t>(p.rows) * static_cast<size_t>(p.slices));
  p.ends = take(sizeof(VerifyEnd) * static_cast<size_t>(p.launch));
  p.sums = take(sizeof(double2) * static_cast<size_t>(p.launch) * static_cast<size_t>(p.cuts));
  p.weights = take(sizeof(double) * static_cast<size_t>(p.launch) * static_cast<size_t>(p.cuts));
  p.total = at;
  return p;
}

hipError_t launch_verify(hipStream_t s, VerifyArgs a, int64_t batch, const VerifyPlan& p, char* ws) {
  a.slices = p.slices;
  a.slice = p.slice;
  a.cut = p.cut;
  a.cuts = p.cuts;
  a.rows = a.d.base ? 2 * a.draft + 1 : a.draft + 1;
  a.parts = reinterpret_cast<VerifyPart*>(ws + p.parts);
  a.ends = reinterpret_cast<VerifyEnd*>(ws + p.ends);
  a.sums = reinterpret_cast<double2*>(ws + p.sums);
  a.weights = reinterpret_cast<double*>(ws + p.weights);
  for (int64_t b0 = 0; b0 < batch; b0 += kMostBatch) {
    const int n = static_cast<int>(batch - b0 < kMostBatch ? batch - b0 : kMostBatch), b = static_cast<int>(b0);
    hipError_t e;
    if (a.x_bf16) e = a.d_bf16 || !a.d.base ? go<bf16_t, bf16_t>(s, a, b, n) : go<bf16_t, float>(s, a, b, n);
    else e = a.d_bf16 ? go<float, bf16_t>(s, a, b, n) : go<float, float>(s, a, b, n);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
