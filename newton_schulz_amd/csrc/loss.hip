// Log-probabilities of chosen tokens, the policy and preference losses on
// them, and the gradients of the scores.
//
// Mathematics.  With z = x / T, M = max z and S = sum_v exp(z_v - M):
//   lp = z_y - M - log S,   d lp / d x_v = ([v = y] - exp(z_v - M) / S) / T,
// so a row needs two numbers, (max x, S), beyond itself.  They are found in
// one pass: a maximum m and sums s around it of what has been seen; a larger
// maximum m' turns s into s exp(m - m').  Partial pairs join the same way, in a
// fixed order.
//
// Arithmetic.  Scores are widened to fp32; with k = log2 e / T, exp(z - m / T) is
// exp2((x - m) k): the subtraction is exact for bf16 of like size, nothing large
// cancels at any magnitude of x, and the largest score gives exactly 1.  k rounded
// to fp32 is another temperature: every log-probability would be off the same way,
// by up to 2^-24 of the scores' mean distance from their maximum (5 over 151936
// normal ones: 3e-7), and the sum over a sequence by as much as there are tokens.
// So k is rounded up for some of the scores of a piece and down for the others,
// as many as make its mean right to 2^-27 (fp32 scores, 4 a piece: 2^-26), which
// costs nothing (a second multiply-add with the rest at every score took scoring
// 6%).  The mean over 1024 rows of 50257 or 151936 scores is then off by 1e-8
// (bf16) and 3e-8 (fp32) at T = 0.83 and 1, and by 4.4e-8 and 6.6e-8 where k lies
// half a step from fp32, next to 1.
// Factors between two maxima take the rest along.
// m is the running maximum of a wave; it is raised, and s scaled, only when some
// lane has met a larger score, and the lanes' sums then join without further
// exponentials.  (With a maximum per lane nearly every piece raised some lane's,
// and joins of pairs made 3/10 of the VALU instructions, which bound scoring:
// 2044 rows of 151936 bf16 took 95 us, 88.5 so.)  It starts at the lowest finite
// number, so that a masked score (-infinity) gives 0 and a row of nothing but
// the lowest number is uniform.
//
// A token that the policy is sure of has S = 1 + u with a small u, and lp = -u
// to first order: rounding S to fp32 would leave lp with an error of 2^-24
// whatever its size.  So the 8 exponentials of a piece are added pairwise in
// fp32 and everything beyond in binary64, and what is stored of S is u = S - 1.
// The label's own gradient is G (1 - p) = -G expm1(lp).
//
// The gradient takes p as exp2(x k - c) / S with c = m k rounded, one fused
// multiply-add a score; the rounding of c (far below 1 where |c| < 2^16) goes
// into the factor that p is multiplied by anyway.  Rows of larger |c| take
// exp2((x - m) k) there too.
//
// Shape of the kernels.  The statistics issue VALU instructions most of the time
// they read; the gradients are bound by HBM (a pass that only reads reaches
// 6.1-6.3 TB/s on MI355X, one that reads and writes alike 5.7-6.0), and HBM is
// fastest when the workgroups in flight cover a compact, moving window of
// addresses: copying in 16 KB pieces per workgroup reaches 6.0 TB/s, in 300 KB
// rows per workgroup 4.9.  So a row is cut into slices, one workgroup of 256
// threads each, in address order; a slice is held in registers.
#include <algorithm>
#include <cfloat>

#include "exchange.h"
#include "loss_kernels.h"
#include "muon_device.h"
#include "wave_ops.h"

using muon::bf16_t;
using muon::last_to_arrive;
using muon::publish;
using muon::published;
using muon::wave_max;
using muon::wave_sum;

namespace {

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

// Piece `base` + t of a row: a uniform base in scalar registers and one 32-bit
// offset per thread, whatever the base (indexing with base + t keeps a 64-bit
// address alive for every piece of an unrolled loop).
__device__ __forceinline__ const u32x4* piece_at(const u32x4* body, int base, int t) {
  return reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(body + base) + static_cast<uint32_t>(t) * 16u);
}
__device__ __forceinline__ u32x4_any* piece_at(u32x4_any* body, int base, int t) {
  return reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(body + base) + static_cast<uint32_t>(t) * 16u);
}

template <typename T> __device__ __forceinline__ T* row_at(const RowsRef& x, int r, int seq) {
  const int b = r / seq;
  return reinterpret_cast<T*>(x.base + static_cast<int64_t>(b) * x.bs +
                              static_cast<int64_t>(r - b * seq) * x.rs);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// log2 e / T = k + rest; exp(d / T) for d <= 0.  What is below `none`, -infinity too,
// is taken as that: exp2(none k) is 0, and the product with the rest, which exceeds
// 1 for k above 2^24, is far from overflow.
struct Scale {
  float k, rest, none;
  const float (&each)[8];  // for the scores of a piece
  __device__ __forceinline__ explicit Scale(const LossArgs& a) : k(a.k), rest(a.k_rest), none(a.none), each(a.k_each) {}
  __device__ __forceinline__ float exp(float d) const {
    const float f = fmaxf(d, none);
    return exp2_fast(__builtin_fmaf(f, k, f * rest));
  }
};

// (m, s) joined with (mo, so).
__device__ __forceinline__ void join(float& m, double& s, float mo, double so, const Scale& q) {
  const float mn = fmaxf(m, mo);
  s = s * static_cast<double>(q.exp(m - mn)) + so * static_cast<double>(q.exp(mo - mn));
  m = mn;
}

// The pair of a wave's lanes, in each of them.
__device__ __forceinline__ void wave_join(float& m, double& s, const Scale& q) {
  const float mn = wave_max(m);
  s = wave_sum(s * static_cast<double>(q.exp(m - mn)));
  m = mn;
}

// The pair of a workgroup whose waves have one maximum each, in wave 0.
template <int NT> __device__ __forceinline__ void block_join(float& m, double& s, const Scale& q) {
  constexpr int W = NT / 64;
  __shared__ float wave_m[W];
  __shared__ double wave_s[W];
  const int lane = static_cast<int>(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  s = wave_sum(s);
  __syncthreads();  // an earlier call's values have been read
  if (lane == 0) {
    wave_m[wave] = m;
    wave_s[wave] = s;
  }
  __syncthreads();
  if (wave) return;
  m = wave_m[lane & (W - 1)];
  s = lane < W ? wave_s[lane] : 0.0;
  wave_join(m, s, q);
}

// (m, s) with N = 1, 4 or 8 more scores from every lane; m is the wave's, s the
// lane's.
template <int N> __device__ __forceinline__ void take_scores(const float (&v)[N], float& m, double& s, const Scale& q) {
  float mn = m;
#pragma unroll
  for (int i = 0; i < N; ++i) mn = fmaxf(mn, v[i]);
  if (__any(mn > m)) {
    mn = wave_max(mn);
    s *= static_cast<double>(q.exp(m - mn));
    m = mn;
    asm volatile("" : "+v"(s));  // stays a branch
  }
  float e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = exp2_fast((v[i] - m) * (N == 1 ? q.k : q.each[i]));
#pragma unroll
  for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
    for (int i = 0; i < w; ++i) e[i] += e[i + w];
  s += static_cast<double>(e[0]);
}
template <typename T> __device__ __forceinline__ void take_piece(u32x4 w, float& m, double& s, const Scale& q) {
  float v[kVec<T>];
  Scores<T>::unpack(w, v);
  take_scores(v, m, s, q);
}

// log s to a few units of binary64, also next to 1: s = 2^e f with f in [3/4,
// 3/2), log f = 2 (t + t^3 / 3 + ...), t = (f - 1) / (f + 1), |t| <= 1/5.
__device__ __forceinline__ double log_sum(double s) {
  if (!(s > 0.0)) return s == 0.0 ? -static_cast<double>(INFINITY) : s;  // no score left, or NaN
  int e = 0;
  double f = frexp(s, &e);
  if (f < 0.75) {
    f *= 2.0;
    --e;
  }
  const double t = (f - 1.0) / (f + 1.0), q = t * t;
  double r = 1.0 / 19.0;
  r = r * q + 1.0 / 17.0;
  r = r * q + 1.0 / 15.0;
  r = r * q + 1.0 / 13.0;
  r = r * q + 1.0 / 11.0;
  r = r * q + 1.0 / 9.0;
  r = r * q + 1.0 / 7.0;
  r = r * q + 1.0 / 5.0;
  r = r * q + 1.0 / 3.0;
  r = r * q + 1.0;
  return static_cast<double>(e) * 0.69314718055994530942 + 2.0 * t * r;
}

// lp of score xy in a row of pair (m, s).
__device__ __forceinline__ double token_lp(const LossArgs& a, float xy, float m, double s) {
  return (static_cast<double>(xy) - static_cast<double>(m)) * a.inv_t - log_sum(s);
}

// What the row's pair and the label's score make of token r (one thread).
__device__ __forceinline__ double finish_row(const LossArgs& a, int r, int64_t y, float xy, float m, double s) {
  double lp = 0.0;
  if (y >= a.vocab) lp = __longlong_as_double(0x7ff8000000000000ll);
  else if (y >= 0) lp = token_lp(a, xy, m, s);
  if (a.lp) a.lp[r] = lp;
  if (a.logps) a.logps[r] = static_cast<float>(lp);
  if (a.stats) a.stats[r] = make_float2(m, static_cast<float>(s - 1.0));
  return lp;
}

// The gradient of a row's scores: scale * p for every score, p = exp2(x k - c)
// or, far, exp2((x - m) k).
struct RowGrad {
  float scale, c, m;
  bool far;
  __device__ __forceinline__ float at(float x, float k) const {
    return scale * exp2_fast(far ? (x - m) * k : __builtin_fmaf(x, k, -c));
  }
};
__device__ __forceinline__ RowGrad row_grad(float G, float m, float u, float k) {
  RowGrad g;
  g.m = m;
  g.c = m * k;
  g.far = !(fabsf(g.c) < 65536.0f);
  g.scale = -G / (1.0f + u);
  if (!g.far) {
    // exp2(x k - c) is 2^d times what it should be, d = m k - c (exact, below
    // 2^-8): 2^-d = 1 - h + h^2 / 2, h = d log 2
    const float h = __builtin_fmaf(m, k, -g.c) * 0.69314718f;
    g.scale *= 1.0f - h * (1.0f - 0.5f * h);
  }
  return g;
}
// The label's own gradient.
__device__ __forceinline__ float label_grad(float G, double lp) { return -G * expm1f(static_cast<float>(lp)); }

// ---------------------------------------------------------------------------
// slices of a row
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
// Pieces a thread may hold.  Finer slices read in a tighter window but exchange
// more pairs: 2048 x 151936 bf16 policy loss with at most 4, 6, 8, 10, 12, 16
// pieces a thread: 307, 252, 228, 220, 223, 223 us; 512 threads of 10: 242 us.
constexpr int kMostPieces = 10;

// Slice j of a row: pieces [first, first + count), and with slice 0 the edges.
struct Slice {
  int first, count;
};
__device__ __forceinline__ Slice slice_of(const RowShape& sh, int slices, int j) {
  const int per = (sh.full + slices - 1) / slices, first = min(sh.full, j * per);
  return {first, min(per, sh.full - first)};
}

// The pair of slice j read from memory, in wave 0: the sums of slice_kernel in
// its order, so the same bits.
template <typename T>
__device__ __forceinline__ void slice_pair(const T* row, const RowShape& sh, int slices, int j, const Scale& scale, float& m,
                                           double& s) {
  const Slice sl = slice_of(sh, slices, j);
  const u32x4* body = reinterpret_cast<const u32x4*>(row + sh.head) + sl.first;
  const int t = static_cast<int>(threadIdx.x);
  m = kLowest;
  s = 0.0;
#pragma unroll 1
  for (int q = 0; q < sl.count; q += kThreads) {
    const uint32_t none = Scores<T>::kMasked;
    u32x4 w = {none, none, none, none};
    if (q + t < sl.count) w = body[q + t];
    take_piece<T>(w, m, s, scale);
  }
  if (j == 0 && t < 64) {
    const float v[1] = {t < sh.edges ? muon::Elem<T>::load(row + edge_score<T>(sh, t)) : -INFINITY};
    take_scores(v, m, s, scale);
  }
  block_join<kThreads>(m, s, scale);
}

// Two numbers as one 64-bit word.
__device__ __forceinline__ uint64_t word_of(float lo, float hi) {
  return (static_cast<uint64_t>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float word_lo(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ __forceinline__ float word_hi(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }

// A pair as a word that is never 0 and whose highest bit is clear: m (a zero with
// its sign set) and s - 1, which is 0 or more, as the largest score itself adds 1,
// or a NaN.  Without any score left, m is -infinity, whose factor in a join is 0.
__device__ __forceinline__ uint64_t pair_word(float m, double s) {
  if (s == 0.0) return word_of(-INFINITY, 0.0f);
  return word_of(m == 0.0f ? -0.0f : m, fabsf(static_cast<float>(s - 1.0)));
}
__device__ __forceinline__ float word_max(uint64_t w) { return word_lo(w); }
__device__ __forceinline__ double word_sum(uint64_t w) { return 1.0 + static_cast<double>(word_hi(w)); }
// The highest bit of a pair's word: a mark (slice_work).
constexpr uint64_t kMark = 1ull << 63;

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

// Sum over the workgroup in a fixed order, in every thread.
template <int NT> __device__ __forceinline__ double block_total(double v) {
  __shared__ double wave[NT / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();  // an earlier call's values have been read
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t += wave[w];
  return t;
}

__device__ __forceinline__ void write_policy(const PolicyArgs& p, double pg, double kl, double clipped) {
  double loss = pg;
  if (p.p.kl_coef != 0.0f) loss += static_cast<double>(p.p.kl_coef) * kl;
  p.out[0] = static_cast<float>(static_cast<double>(p.p.weight) * loss);
  p.out[1] = static_cast<float>(pg);
  p.out[2] = static_cast<float>(kl);
  p.out[3] = static_cast<float>(clipped);
}

// The same of three values at once.
template <int NT> __device__ __forceinline__ void block_totals(double (&v)[3]) {
  __shared__ double wave[3][NT / 64];
#pragma unroll
  for (int j = 0; j < 3; ++j)
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v[j] += __shfl_xor(v[j], d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int j = 0; j < 3; ++j) wave[j][threadIdx.x >> 6] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    v[j] = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v[j] += wave[j][w];
  }
}

// The token weight that a word of the weights holds.
__device__ __forceinline__ double word_weight(uint64_t w) { return __longlong_as_double(static_cast<long long>(w)); }

// Labels in [lo, hi) that count, in every thread of the workgroup.
template <int NT> __device__ __forceinline__ double count_labels(const int64_t* labels, int64_t lo, int64_t hi) {
  int count = 0;
  constexpr int U = 8;
  for (int64_t i = lo + threadIdx.x; i < hi; i += U * NT) {
    int64_t y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = i + u * NT < hi ? labels[i + u * NT] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) count += y[u] >= 0;
  }
  return block_total<NT>(count);  // whole numbers: exact
}

// Weight of a token of sequence b in the loss.
template <int NT> __device__ __forceinline__ double token_weight(const PolicyArgs& p, int b) {
  if (p.p.reduce == MUON_REDUCE_SUM) return 1.0;
  if (p.p.reduce == MUON_REDUCE_TOKEN)
    return 1.0 / count_labels<NT>(p.labels, 0, static_cast<int64_t>(p.batch) * p.seq);
  const int64_t lo = static_cast<int64_t>(b) * p.seq;
  return 1.0 / (count_labels<NT>(p.labels, lo, lo + p.seq) * p.batch);
}

// The weighted sums of the terms of tokens [lo, hi), in every thread; SAME: by
// the launch that formed them.
template <int NT, bool SAME>
__device__ __forceinline__ void sum_terms(const PolicyArgs& p, int64_t lo, int64_t hi, double (&v)[3]) {
  v[0] = v[1] = v[2] = 0.0;
  auto word = [](const uint64_t* from) { return SAME ? published(from) : *from; };
  for (int64_t i = lo + threadIdx.x; i < hi; i += NT) {
    const int64_t y = p.labels[i];
    const uint64_t weight = word(p.weights + (p.p.reduce == MUON_REDUCE_SEQUENCE ? i / p.seq : 0));
    const uint64_t term = word(p.terms + 2 * i), clipped = word(p.terms + 2 * i + 1);
    if (y < 0) continue;  // (nothing was formed)
    const double w = word_weight(weight);
    v[0] += w * static_cast<double>(word_lo(term));
    v[1] += w * static_cast<double>(word_hi(term));
    v[2] += w * static_cast<double>(word_lo(clipped));
  }
  block_totals<NT>(v);
}

// What a slice is read for.
enum SliceUse : int {
  USE_STATS = 0,   // the row's pair alone
  USE_POLICY = 1   // the policy loss and its gradient
};

// Workgroup: slice blockIdx % slices of row blockIdx / slices, NV pieces a
// thread.
//
// USE_STATS leaves the slice's pair in a.part (whole rows: finishes the token).
//
// USE_POLICY reads every score once and writes every gradient once, which is
// all the traffic the loss needs: a token's gradient depends on nothing of
// other rows but their number, so a slice only lacks the pairs of its row's
// other slices.  It publishes its own as one 64-bit word (an agent-scope
// atomic store: no other data has to be made visible with it) and waits for
// theirs, its scores staying in registers.  The slices of a row are
// neighbours in the order in which workgroups start, so the wait is that of a
// few microseconds' skew, and other workgroups of the compute unit run
// meanwhile.  It is bounded: after a.spin polls the workgroup computes the
// missing pairs itself from memory, so it ends whether or not its neighbours
// ever run beside it.
// In place, a slice's scores are overwritten by its own workgroup alone, and
// only after what that publishes has arrived.  So a pair computed here from a
// neighbour's scores is used only if the neighbour's is still missing
// afterwards.  The label's score, which every workgroup reads at its start,
// may be overwritten by then only if the workgroup of its slice has stopped
// waiting (else it waited for all pairs, and a pair is published after the
// label's score is read).  That one publishes the score first and then its pair
// again with a mark; whoever finds the mark takes the published score.
// (Exchanging the score in every call instead, one word a row more to wait for,
// took 2048 tokens x 151936 bf16 scores from 218 to 249 us.)
// Against a workgroup per row with the row in its registers (1024 threads of 19
// pieces): 2048 tokens x 151936 bf16 scores took 267 us there.
template <typename T, int NV, int USE>
__device__ __forceinline__ void slice_work(const LossArgs& a, const RowsRef& grad, const PolicyArgs& p) {
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r = a.row0 + static_cast<int>(blockIdx.x) / a.slices, j = static_cast<int>(blockIdx.x) % a.slices;
  const int b = r / a.seq;
  if (USE == USE_POLICY && p.count_here && j == 0) {
    // the first workgroup of those that share a mean publishes its weight
    if (p.p.reduce == MUON_REDUCE_SEQUENCE ? r == b * a.seq : r == 0) {
      const double weight = token_weight<kThreads>(p, b);
      if (t == 0)
        publish(p.weights + (p.p.reduce == MUON_REDUCE_SEQUENCE ? b : 0),
                static_cast<uint64_t>(__double_as_longlong(weight)));
    }
  }
  const int64_t y = a.labels[r];
  const T* row = row_at<const T>(a.x, r, a.seq);
  const RowShape sh = row_shape(row, a.vocab);
  const Slice sl = slice_of(sh, a.slices, j);
  const bool edge = j == 0 && t < sh.edges;
  const float k = a.k;
  const Scale scale(a);
  T* out = USE == USE_POLICY ? row_at<T>(grad, r, a.seq) : nullptr;
  // the gradient's rows have an alignment of their own
  u32x4_any* obody = USE == USE_POLICY ? reinterpret_cast<u32x4_any*>(out + sh.head) + sl.first : nullptr;
  if (y < 0 || (USE == USE_STATS && y >= a.vocab)) {  // left out; or names no score, and its row is not needed
    if (USE == USE_POLICY && grad.base) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t < sl.count - i * kThreads) *piece_at(obody, i * kThreads, t) = u32x4{0, 0, 0, 0};
      if (edge) muon::Elem<T>::store(out + edge_score<T>(sh, t), 0.0f);
    }
    if (j == 0 && t == 0) {
      if (USE == USE_POLICY && a.logps) a.logps[r] = 0.0f;
      if (USE == USE_STATS && a.slices == 1 && a.arrived == nullptr) finish_row(a, r, y, 0.0f, 0.0f, 1.0);
    }
    return;
  }
  u32x4 w[NV];
  {
    const u32x4* body = reinterpret_cast<const u32x4*>(row + sh.head) + sl.first;
    const uint32_t none = Scores<T>::kMasked;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      w[i] = u32x4{none, none, none, none};
      if (t < sl.count - i * kThreads) w[i] = *piece_at(body, i * kThreads, t);
    }
  }
  const float we = edge ? muon::Elem<T>::load(row + edge_score<T>(sh, t)) : -INFINITY;
  const bool named = y < a.vocab;
  float xy = 0.0f;
  if (USE == USE_POLICY || j == 0) xy = muon::Elem<T>::load(row + (named ? y : 0));
  // From the wave's first lane on.  Slices seldom fill the last pieces, and the
  // statistics alone are bound by VALU: skipping what a wave has nothing of took
  // 2048 rows of 50257 bf16 scores and their gradient from 107.2 to 105.4 us; in
  // the policy loss, which waits for memory, the branches cost more (32000
  // scores: 50.5, 50.1 us without).
  const int own_pieces = sl.count - wave * 64;
  float m = kLowest;
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    // A piece is unpacked where it is used and never earlier, and its
    // exponentials are summed there and never later: as far as the compiler
    // knows the piece may have changed just before and the sum is read just
    // after, so it keeps 4 registers a piece and not 8 more of widened scores.
    asm volatile("" : "+v"(w[i]));
    if (USE == USE_POLICY || i * kThreads < own_pieces) take_piece<T>(w[i], m, s, scale);
    asm volatile("" : "+v"(s));
  }
  if (wave == 0) {  // threads without an edge hold -infinity
    const float v[1] = {we};
    take_scores(v, m, s, scale);
  }
  if (USE == USE_POLICY) asm volatile("" : "+v"(xy));  // read before this slice is published
  block_join<kThreads>(m, s, scale);
  if (USE == USE_STATS) {
    if (t == 0) {
      if (a.slices == 1 && a.arrived == nullptr) finish_row(a, r, y, xy, m, s);
      else publish(a.part + static_cast<int64_t>(r) * a.slices + j, pair_word(m, s));
      if (a.slices > 1 && j == 0 && a.arrived == nullptr) a.chosen[r] = xy;
    }
    return;
  }
  __shared__ RowGrad coef;
  __shared__ float own_grad;
  __shared__ uint64_t missing, own[64];
  constexpr int kWeightLane = 63;  // (a row has at most 60 slices)
  // wave 0: the row's pair from a slice's word in each lane, and what follows
  auto settle = [&](uint64_t word) {
    const double wt = word_weight(__shfl(word, kWeightLane, 64));
    if (__any(lane < a.slices && (word & kMark))) {  // xy may have been read too late
      xy = word_lo(published(p.scores + r));
      word &= ~kMark;
    }
    m = lane < a.slices ? word_max(word) : kLowest;
    s = lane < a.slices ? word_sum(word) : 0.0;
    wave_join(m, s, scale);
    double lp = token_lp(a, xy, m, s);
    if (!named) lp = __longlong_as_double(0x7ff8000000000000ll);
    const TokenTerms o = policy_token(p, r, b, lp);
    const float G = static_cast<float>(static_cast<double>(p.p.weight) * wt * static_cast<double>(o.g) * a.inv_t);
    if (lane == 0) {
      coef = row_grad(G, m, static_cast<float>(s - 1.0), k);
      own_grad = label_grad(G, lp);
      if (j == 0) {
        if (a.logps) a.logps[r] = static_cast<float>(lp);
        publish(p.terms + 2 * static_cast<int64_t>(r), word_of(o.pg, o.kl));
        publish(p.terms + 2 * static_cast<int64_t>(r) + 1, __float_as_uint(o.clipped));
      }
    }
  };
  uint64_t* slot = a.part + static_cast<int64_t>(r) * a.slices;
  const uint64_t word = pair_word(m, s);
  if (a.slices > 1 && t == 0) publish(slot + j, word);
  if (grad.base == nullptr && j > 0) return;  // evaluation: slice 0 has it all
  if (wave == 0) {
    // lanes 0 .. slices - 1: the slices' pairs, the last lane: the weight
    const uint64_t* from = lane == kWeightLane ? p.weights + (p.p.reduce == MUON_REDUCE_SEQUENCE ? b : 0) : slot + lane;
    const bool asks = lane == kWeightLane || (a.slices > 1 && lane < a.slices);
    uint64_t v = word;
    bool ready = true;
    for (int n = 0;; ++n) {
      if (asks) v = published(from);
      ready = __all(v != 0);
      if (ready || n >= a.spin) break;
      __builtin_amdgcn_s_sleep(1);
    }
    const uint64_t lack = __ballot(v == 0);
    if (lane == 0) missing = lack;
    own[lane] = v;
    if (ready) {
      settle(v);
    } else {
      // in place, what this workgroup overwrites may be read by others that start later
      const int ly = static_cast<int>(named ? y : 0) - sh.head, q = ly >= 0 ? ly / kVec<T> : sh.full;
      const bool holds = q < sh.full ? q >= sl.first && q < sl.first + sl.count : j == 0;
      if (lane == 0 && named && holds && a.slices > 1) {
        publish(p.scores + r, __float_as_uint(xy));
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        publish(slot + j, word | kMark);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
  }
  __syncthreads();
  if (const uint64_t lack = missing) {
    for (int i = 0; i < a.slices; ++i) {
      if (!((lack >> i) & 1)) continue;
      float mi;
      double si;
      slice_pair(row, sh, a.slices, i, scale, mi, si);
      if (t == 0) {
        const uint64_t v = published(slot + i);
        own[i] = v ? v : pair_word(mi, si);
      }
    }
    if ((lack >> kWeightLane) & 1) {
      const double weight = token_weight<kThreads>(p, b);
      if (t == 0) own[kWeightLane] = static_cast<uint64_t>(__double_as_longlong(weight));
    }
    __syncthreads();
    if (wave == 0) settle(own[lane]);
    __syncthreads();
  }
  if (grad.base == nullptr) return;
  const RowGrad g = coef;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[kVec<T>];
    asm volatile("" : "+v"(w[i]));
    Scores<T>::unpack(w[i], v);
    if (g.far) {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) v[e] = g.scale * exp2_fast((v[e] - g.m) * k);
    } else {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) v[e] = g.scale * exp2_fast(__builtin_fmaf(v[e], k, -g.c));
    }
    if (t < sl.count - i * kThreads)
      __builtin_nontemporal_store(Scores<T>::pack(v), piece_at(obody, i * kThreads, t));
  }
  if (edge) muon::Elem<T>::store(out + edge_score<T>(sh, t), g.at(we, k));
  // the label's score, by the thread whose piece or edge has just gone out
  if (named) {
    const int ly = static_cast<int>(y) - sh.head, q = ly >= 0 ? ly / kVec<T> : -1;
    bool mine = q >= sl.first && q < sl.first + sl.count && (q - sl.first) % kThreads == t;
    if (edge) mine = mine || edge_score<T>(sh, t) == y;
    if (mine) muon::Elem<T>::store(out + y, own_grad);
  }
}

// Every row of a small call joined by its last workgroup, a thread per row, and
// the exchange words left as they were found, all zero.
template <typename T> __device__ __forceinline__ void join_rows(const LossArgs& a) {
  __shared__ uint64_t words[kArriveGroups];
  const int t = static_cast<int>(threadIdx.x), slots = a.rows * a.slices;
  for (int i = t; i < slots; i += kThreads) {
    words[i] = published(a.part + i);
    a.part[i] = 0;
  }
  __syncthreads();
  const Scale scale(a);
  for (int r = t; r < a.rows; r += kThreads) {
    const int64_t y = a.labels[r];
    float m = 0.0f, xy = 0.0f;
    double s = 1.0;
    if (y >= 0 && y < a.vocab) {
      xy = muon::Elem<T>::load(row_at<const T>(a.x, r, a.seq) + y);
      const uint64_t* w = words + r * a.slices;
      m = kLowest;
      s = 0.0;
#pragma unroll 4
      for (int i = 0; i < a.slices; ++i) m = fmaxf(m, word_max(w[i]));
#pragma unroll 4
      for (int i = 0; i < a.slices; ++i) s += word_sum(w[i]) * static_cast<double>(scale.exp(word_max(w[i]) - m));
    }
    finish_row(a, r, y, xy, m, s);
  }
}

template <typename T, int NV, int USE>
__global__ __launch_bounds__(kThreads) void slice_kernel(LossArgs a, RowsRef grad, PolicyArgs p) {
  slice_work<T, NV, USE>(a, grad, p);
  // A small call is one launch: its last workgroup does the rest.
  if (a.arrived == nullptr || !last_to_arrive(a.arrived)) return;
  if (USE == USE_STATS) {
    join_rows<T>(a);
    return;
  }
  double v[3];
  sum_terms<kThreads, true>(p, 0, a.rows, v);
  if (threadIdx.x == 0) write_policy(p, v[0], v[1], v[2]);
  for (int i = threadIdx.x; i < p.clear; i += kThreads) a.part[i] = 0;
}

// Joins the slices of each row; one wave per row.
__global__ __launch_bounds__(kThreads) void row_join_kernel(LossArgs a) {
  const int r = a.row0 + static_cast<int>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= a.rows) return;
  const int64_t y = a.labels[r];
  float m = 0.0f;
  double s = 1.0;
  if (y >= 0 && y < a.vocab) {
    m = kLowest;
    s = 0.0;
    if (lane < a.slices) {
      const uint64_t v = a.part[static_cast<int64_t>(r) * a.slices + lane];
      m = word_max(v);
      s = word_sum(v);
    }
    wave_join(m, s, Scale(a));
  }
  if (lane == 0) finish_row(a, r, y, a.chosen[r], m, s);
}

constexpr int kGradUnroll = 4;

// Gradient of row blockIdx / chunks, pieces of chunk blockIdx % chunks (the
// first chunk takes the edges).
template <typename T>
__global__ __launch_bounds__(kThreads) void logits_grad_kernel(LossArgs a, RowsRef grad,
                                                                   const float* __restrict__ g, int per_sequence,
                                                                   int chunks) {
  const int block = static_cast<int>(gridDim.x - 1 - blockIdx.x);
  const int r = a.row0 + block / chunks, c = block % chunks;
  const int64_t y = a.labels[r];
  const T* row = row_at<const T>(a.x, r, a.seq);
  T* out = row_at<T>(grad, r, a.seq);
  const RowShape sh = row_shape(row, a.vocab);
  const u32x4* body = reinterpret_cast<const u32x4*>(row + sh.head);
  // the gradient's rows have an alignment of their own
  u32x4_any* obody = reinterpret_cast<u32x4_any*>(out + sh.head);
  const int t = static_cast<int>(threadIdx.x), p0 = c * kThreads * kGradUnroll + t;
  const bool edge = c == 0 && t < sh.edges;
  if (y < 0) {
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int p = p0 + u * kThreads;
      if (p < sh.full) obody[p] = u32x4{0, 0, 0, 0};
    }
    if (edge) muon::Elem<T>::store(out + edge_score<T>(sh, t), 0.0f);
    return;
  }
  const float k = a.k;
  const float2 st = a.stats[r];
  float G = static_cast<float>(static_cast<double>(g[per_sequence ? r / a.seq : r]) * a.inv_t);
  if (y >= a.vocab) G = __uint_as_float(0x7fc00000u);  // the label names no score
  const RowGrad rg = row_grad(G, st.x, st.y, k);
  u32x4 w[kGradUnroll];
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int p = p0 + u * kThreads;
    if (p < sh.full) w[u] = body[p];
  }
  // the label's place: piece py, score iy of it (no piece when it is an edge)
  const int ly = static_cast<int>(y < a.vocab ? y : 0) - sh.head;
  const int py = ly >= 0 ? ly / kVec<T> : -1, iy = ly - py * kVec<T>;
  auto own = [&](float xy) {
    return label_grad(G, token_lp(a, xy, st.x, 1.0 + static_cast<double>(st.y)));
  };
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int p = p0 + u * kThreads;
    if (p >= sh.full) continue;
    float v[kVec<T>];
    Scores<T>::unpack(w[u], v);
    float xy = 0.0f;
    if (p == py) {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i) xy = i == iy ? v[i] : xy;
    }
    if (rg.far) {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i) v[i] = rg.scale * exp2_fast((v[i] - rg.m) * k);
    } else {
#pragma unroll
      for (int i = 0; i < kVec<T>; ++i) v[i] = rg.scale * exp2_fast(__builtin_fmaf(v[i], k, -rg.c));
    }
    __builtin_nontemporal_store(Scores<T>::pack(v), obody + p);
    if (p == py && y < a.vocab) muon::Elem<T>::store(out + y, own(xy));
  }
  if (edge) {
    const int e = edge_score<T>(sh, t);
    const float x = muon::Elem<T>::load(row + e);
    muon::Elem<T>::store(out + e, e == y ? own(x) : rg.at(x, k));
  }
}

// ---------------------------------------------------------------------------
// sums over tokens
// ---------------------------------------------------------------------------
constexpr int kTermThreads = 1024;

// Before the slices of a policy loss too large for the exchange words: the
// weights (workgroup b: sequence first + b, or all tokens), and empty slots for
// the slices' pairs.
__global__ __launch_bounds__(kTermThreads) void policy_prepare_kernel(PolicyArgs p, uint64_t* slots, int64_t n, int first) {
  const int t = static_cast<int>(threadIdx.x), b = first + static_cast<int>(blockIdx.x);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kTermThreads + t; i < n; i += static_cast<int64_t>(gridDim.x) * kTermThreads)
    slots[i] = 0;
  if (b >= (p.p.reduce == MUON_REDUCE_SEQUENCE ? p.batch : 1)) return;
  const double weight = token_weight<kTermThreads>(p, b);
  if (t == 0) p.weights[b] = static_cast<uint64_t>(__double_as_longlong(weight));
}

// After the slices: workgroup b of n adds the b-th run of tokens.  One
// workgroup writes the losses, and empties the exchange words (`clear` of
// them from `words`) for the next call; several leave their sums.
__global__ __launch_bounds__(kTermThreads) void policy_sums_kernel(PolicyArgs p, int64_t rows, uint64_t* words) {
  const int64_t per = (rows + gridDim.x - 1) / gridDim.x, lo = static_cast<int64_t>(blockIdx.x) * per;
  double v[3];
  sum_terms<kTermThreads, false>(p, lo, lo + per < rows ? lo + per : rows, v);
  if (gridDim.x == 1) {  // (the sums' barriers lie after every read of the weights)
    for (int i = threadIdx.x; i < p.clear; i += kTermThreads) words[i] = 0;
    if (threadIdx.x == 0) write_policy(p, v[0], v[1], v[2]);
  } else if (threadIdx.x == 0) {
#pragma unroll
    for (int j = 0; j < 3; ++j) p.sums[3 * blockIdx.x + j] = v[j];
  }
}
__global__ __launch_bounds__(kTermThreads) void clear_words_kernel(uint64_t* words, int n) {
  for (int i = static_cast<int>(blockIdx.x) * kTermThreads + threadIdx.x; i < n; i += gridDim.x * kTermThreads) words[i] = 0;
}
__global__ void policy_total_kernel(PolicyArgs p, int n) {
  double v[3] = {0.0, 0.0, 0.0};
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] += p.sums[3 * i + j];
  write_policy(p, v[0], v[1], v[2]);
}

// -log sigma(h) and sigma(h), without overflow.
__device__ __forceinline__ double neg_log_sigmoid(double h) {
  return (h < 0.0 ? -h : 0.0) + log1p(exp(-fabs(h)));
}
__device__ __forceinline__ double sigmoid(double h) {
  const double q = exp(-fabs(h));
  return (h < 0.0 ? q : 1.0) / (1.0 + q);
}

__device__ __forceinline__ void write_preference(const PreferenceArgs& p, double loss, double margin, double won) {
  const double n = p.batch > 1 ? p.batch / 2 : 1;
  p.out[0] = static_cast<float>(static_cast<double>(p.p.weight) * loss / n);
  p.out[1] = static_cast<float>(margin / n);
  p.out[2] = static_cast<float>(won / n);
}

constexpr int kFewPairs = 8;  // handled by one workgroup, which then needs no launch to add them up

// The score of token q of sequence b (0 for tokens left out), its row finished.
__device__ __forceinline__ double token_score(const LossArgs& a, const PreferenceArgs& p, int b, int q, bool* counts) {
  const int r = b * p.seq + q;
  const int64_t y = a.labels[r];
  *counts = y >= 0;
  const float ref = p.ref_lp ? p.ref_lp[r] : 0.0f;  // (anything where the token is left out)
  double lp;
  if (a.slices == 1) {
    lp = a.lp[r];
  } else {
    const float xy = a.chosen[r];
    float m = 0.0f;
    double s = 1.0;
    if (y >= 0 && y < a.vocab) {
      const uint64_t* v = a.part + static_cast<int64_t>(r) * a.slices;
      m = kLowest;
      s = 0.0;
      constexpr int U = 8;  // words in flight
      for (int x0 = 0; x0 < a.slices; x0 += U) {
        uint64_t w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = x0 + u < a.slices ? v[x0 + u] : pair_word(kLowest, 0.0);
#pragma unroll
        for (int u = 0; u < U; ++u) join(m, s, word_max(w[u]), word_sum(w[u]), Scale(a));
      }
    }
    lp = finish_row(a, r, y, xy, m, s);
  }
  return *counts ? lp - static_cast<double>(ref) : 0.0;
}

// Scores of the pairs [first, first + n) (n = 1, or all of at most kFewPairs):
// half of the workgroup per sequence; then a thread per pair: its loss, and the
// gradient that every token of each sequence has.  Who has all pairs writes the
// losses; others leave their pairs' terms.
template <int NT>
__device__ __forceinline__ void pairs_work(const LossArgs& a, const PreferenceArgs& p, int first, int n) {
  constexpr int kHalf = NT / 2, W = kHalf / 64;
  const int pairs = p.batch / 2;
  const int side = __builtin_amdgcn_readfirstlane(threadIdx.x / kHalf);
  const int t = static_cast<int>(threadIdx.x) % kHalf, wave = t >> 6;
  __shared__ double scores[kFewPairs][2][W], terms[kFewPairs][3];
  __shared__ int tokens[kFewPairs][2][W];
  for (int i = 0; i < n; ++i) {
    double sum = 0.0;
    int count = 0;
    for (int q = t; q < p.seq; q += kHalf) {
      bool counts;
      sum += token_score(a, p, first + i + side * pairs, q, &counts);
      count += counts;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      sum += __shfl_xor(sum, d, 64);
      count += __shfl_xor(count, d, 64);
    }
    if ((t & 63) == 0) {
      scores[i][side][wave] = sum;
      tokens[i][side][wave] = count;
    }
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < n) {
    const int l = static_cast<int>(threadIdx.x), i = first + l;
    const double beta = p.p.beta, eps = p.p.label_smoothing;
    double score[2] = {0.0, 0.0};
    int count[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        score[k] += scores[l][k][w];
        count[k] += tokens[l][k][w];
      }
      if (p.p.average) score[k] = count[k] ? score[k] / count[k] : 0.0;
    }
    const double margin = score[0] - score[1], h = beta * margin;
    double loss, d;
    if (p.p.kind == MUON_PREFERENCE_SIGMOID) {
      loss = (1.0 - eps) * neg_log_sigmoid(h);
      if (eps != 0.0) loss += eps * neg_log_sigmoid(-h);  // infinite where the rejected answer is impossible
      d = beta * (eps * sigmoid(h) - (1.0 - eps) * sigmoid(-h));
    } else {
      const double off = margin - 0.5 / beta;
      loss = off * off;
      d = 2.0 * off;
    }
    terms[l][0] = loss;
    terms[l][1] = h;
    terms[l][2] = margin > 0.0 ? 1.0 : 0.0;
#pragma unroll
    for (int k = 0; k < 3; ++k) p.terms[3 * static_cast<int64_t>(i) + k] = terms[l][k];
    d *= static_cast<double>(p.p.weight) / pairs;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = i + k * pairs;
      if (p.rewards) p.rewards[b] = static_cast<float>(beta * score[k]);
      const double g = k ? -d : d;
      p.g[b] = static_cast<float>(p.p.average && count[k] ? g / count[k] : g);
    }
  }
  if (n < pairs) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total[3] = {0.0, 0.0, 0.0};
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k) total[k] += terms[i][k];
    write_preference(p, total[0], total[1], total[2]);
  }
}

__global__ __launch_bounds__(kTermThreads) void preference_pairs_kernel(LossArgs a, PreferenceArgs p, int first, int n) {
  pairs_work<kTermThreads>(a, p, first + static_cast<int>(blockIdx.x) * n, n);
}

// A small call of few pairs: its last workgroup joins the rows and scores them.
template <typename T, int NV>
__global__ __launch_bounds__(kThreads) void slice_pairs_kernel(LossArgs a, PreferenceArgs p) {
  slice_work<T, NV, USE_STATS>(a, RowsRef{}, PolicyArgs{});
  if (!last_to_arrive(a.arrived)) return;
  join_rows<T>(a);
  __syncthreads();
  a.slices = 1;  // (the rows' log-probabilities are whole)
  pairs_work<kThreads>(a, p, 0, p.batch / 2);
}

__global__ __launch_bounds__(kTermThreads) void preference_sums_kernel(PreferenceArgs p) {
  double v[3] = {0.0, 0.0, 0.0};
  for (int64_t i = threadIdx.x; i < p.batch / 2; i += kTermThreads)
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] += p.terms[3 * i + j];
  block_totals<kTermThreads>(v);
  if (threadIdx.x == 0) write_preference(p, v[0], v[1], v[2]);
}

}  // namespace

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
int loss_slices(int64_t rows, int64_t vocab, int bf16, int cus) {
  const int64_t pieces = vocab / (bf16 ? 8 : 4);
  const int64_t least = (pieces + kThreads * kMostPieces - 1) / (kThreads * kMostPieces);
  // rows that leave compute units idle are cut finer, down to one piece a thread
  const int64_t idle = rows > 0 ? 2 * static_cast<int64_t>(cus) / rows : 1;
  const int64_t most = std::min<int64_t>(60, (pieces + kThreads - 1) / kThreads);
  return static_cast<int>(std::max<int64_t>(1, std::max(least, std::min(idle, most))));
}

// A grid holds fewer than 2^32 threads; more rows, sequences or pairs are several
// launches.
constexpr int kMostTermGroups = 1 << 20;  // workgroups of kTermThreads in one launch

// Rows of one launch when each takes `per` workgroups.
static int rows_per_launch(int64_t per) {
  const int64_t n = 0xff0000 / per;  // of 256 threads
  return static_cast<int>(n > 1 ? n : 1);
}

namespace {

// Every pair's loss by the same launch as the rows' statistics.
struct PairsRef {
  const PreferenceArgs* p;
};

template <typename T, int NV, int USE>
hipError_t run_slices(hipStream_t s, const LossArgs& a, RowsRef, const PairsRef& pairs) {
  slice_pairs_kernel<T, NV><<<static_cast<unsigned>(a.rows * a.slices), kThreads, 0, s>>>(a, *pairs.p);
  return hipGetLastError();
}

template <typename T, int NV, int USE>
hipError_t run_slices(hipStream_t s, const LossArgs& a, RowsRef grad, const PolicyArgs& p) {
  LossArgs c = a;
  const int step = rows_per_launch(a.slices);
  for (c.row0 = 0; c.row0 < a.rows; c.row0 += step) {
    const int n = a.rows - c.row0 < step ? a.rows - c.row0 : step;
    slice_kernel<T, NV, USE><<<static_cast<unsigned>(n) * static_cast<unsigned>(a.slices), kThreads, 0, s>>>(c, grad, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int USE, typename P>
hipError_t slices(hipStream_t s, const LossArgs& a, RowsRef grad, const P& p) {
  const int per = (a.vocab / kVec<T> + a.slices - 1) / a.slices;
  if (per <= 1 * kThreads) return run_slices<T, 1, USE>(s, a, grad, p);
  if (per <= 2 * kThreads) return run_slices<T, 2, USE>(s, a, grad, p);
  if (per <= 4 * kThreads) return run_slices<T, 4, USE>(s, a, grad, p);
  if (per <= 6 * kThreads) return run_slices<T, 6, USE>(s, a, grad, p);
  if (per <= 8 * kThreads) return run_slices<T, 8, USE>(s, a, grad, p);
  return run_slices<T, kMostPieces, USE>(s, a, grad, p);
}

}  // namespace

hipError_t clear_exchange(hipStream_t s, Exchange& x) {
  if (!x.dirty) return hipSuccess;
  clear_words_kernel<<<8, kTermThreads, 0, s>>>(x.words, kExchangeWords + kCounters * kCounterWords);
  const hipError_t e = hipGetLastError();
  // a launch that only goes into a graph has emptied nothing yet
  hipStreamCaptureStatus c = hipStreamCaptureStatusNone;
  if (e == hipSuccess && hipStreamIsCapturing(s, &c) == hipSuccess && c == hipStreamCaptureStatusNone) x.dirty = false;
  return e;
}

static hipError_t launch_slice_stats(hipStream_t s, const LossArgs& a) {
  return a.bf16 ? slices<bf16_t, USE_STATS>(s, a, RowsRef{}, PolicyArgs{})
                : slices<float, USE_STATS>(s, a, RowsRef{}, PolicyArgs{});
}

// `a` with its pairs in the exchange words, to be joined by the last workgroup.
static LossArgs in_one_launch(const LossArgs& a, const Exchange& x) {
  LossArgs c = a;
  c.part = x.words;
  c.arrived = x.words + kExchangeWords;
  return c;
}

hipError_t launch_row_stats(hipStream_t s, const LossArgs& a, Exchange& x) {
  if (a.rows == 0 || a.slices == 1) return launch_slice_stats(s, a);
  if (static_cast<int64_t>(a.rows) * a.slices <= kArriveGroups) {
    const hipError_t e = clear_exchange(s, x);
    return e == hipSuccess ? launch_slice_stats(s, in_one_launch(a, x)) : e;
  }
  hipError_t e = launch_slice_stats(s, a);
  if (e != hipSuccess) return e;
  LossArgs c = a;
  constexpr int kRows = kThreads / 64;  // of a workgroup
  const int step = rows_per_launch(1) * kRows;
  for (c.row0 = 0; c.row0 < a.rows; c.row0 += step) {
    row_join_kernel<<<static_cast<unsigned>((std::min(step, a.rows - c.row0) + kRows - 1) / kRows), kThreads, 0, s>>>(c);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_logits_grad(hipStream_t s, const LossArgs& a, RowsRef grad, const float* g, bool per_sequence) {
  const int vec = a.bf16 ? 8 : 4;
  const int pieces = a.vocab / vec;  // the most a row can have
  const int chunks = std::max(1, (pieces + kThreads * kGradUnroll - 1) / (kThreads * kGradUnroll));
  LossArgs c = a;
  const int step = rows_per_launch(chunks);
  const int each = per_sequence ? 1 : 0;
  for (c.row0 = 0; c.row0 < a.rows; c.row0 += step) {
    const int n = a.rows - c.row0 < step ? a.rows - c.row0 : step;
    const unsigned grid = static_cast<unsigned>(n) * static_cast<unsigned>(chunks);
    if (a.bf16) logits_grad_kernel<bf16_t><<<grid, kThreads, 0, s>>>(c, grad, g, each, chunks);
    else logits_grad_kernel<float><<<grid, kThreads, 0, s>>>(c, grad, g, each, chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_policy(hipStream_t s, const LossArgs& args, RowsRef grad, const PolicyArgs& policy,
                         Exchange& x) {
  LossArgs a = args;
  PolicyArgs p = policy;
  const int64_t slots = static_cast<int64_t>(a.rows) * a.slices;
  const int64_t sets = p.p.reduce == MUON_REDUCE_SEQUENCE ? p.batch : 1;
  const bool kept = slots + sets <= kExchangeWords;
  hipError_t e = hipSuccess;
  // words that a launch has filled and none after it will empty
  auto failed = [&](hipError_t why) {
    if (kept) {
      x.dirty = true;
      (void)clear_exchange(s, x);  // now if that is possible: a recorded call would not ask
    }
    return why;
  };
  if (kept) {
    e = clear_exchange(s, x);
    if (e != hipSuccess) return e;
    a.part = x.words;
    p.weights = x.words + slots;
    p.count_here = 1;
    p.clear = static_cast<int>(slots + sets);
    if (a.rows > 0 && slots <= kArriveGroups) a = in_one_launch(a, x);
  } else {
    const int64_t clear = std::min<int64_t>(128, (slots + kTermThreads - 1) / kTermThreads);
    const int64_t groups = std::max(clear, sets);
    for (int64_t first = 0; first < groups && e == hipSuccess; first += kMostTermGroups) {
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>(groups - first, kMostTermGroups));
      policy_prepare_kernel<<<grid, kTermThreads, 0, s>>>(p, a.part, first ? 0 : slots, static_cast<int>(first));
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  e = a.bf16 ? slices<bf16_t, USE_POLICY>(s, a, grad, p) : slices<float, USE_POLICY>(s, a, grad, p);
  if (e != hipSuccess) return failed(e);
  if (a.arrived == nullptr) {
    const int n = kept ? 1 : std::min(kPolicySums, std::max(1, a.rows / 8192));
    policy_sums_kernel<<<static_cast<unsigned>(n), kTermThreads, 0, s>>>(p, a.rows, a.part);
    e = hipGetLastError();
    if (e != hipSuccess) return failed(e);
    if (n > 1) policy_total_kernel<<<1, 1, 0, s>>>(p, n);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_preference(hipStream_t s, const LossArgs& a, RowsRef grad, const PreferenceArgs& p, Exchange& x) {
  const int pairs = p.batch / 2;
  hipError_t e;
  if (a.rows > 0 && pairs <= kFewPairs && static_cast<int64_t>(a.rows) * a.slices <= kArriveGroups) {
    e = clear_exchange(s, x);
    if (e != hipSuccess) return e;
    const LossArgs c = in_one_launch(a, x);
    e = a.bf16 ? slices<bf16_t, USE_STATS>(s, c, RowsRef{}, PairsRef{&p})
               : slices<float, USE_STATS>(s, c, RowsRef{}, PairsRef{&p});
  } else {
    e = launch_slice_stats(s, a);
    if (e != hipSuccess) return e;
    if (pairs <= kFewPairs) {
      preference_pairs_kernel<<<1, kTermThreads, 0, s>>>(a, p, 0, pairs);
      e = hipGetLastError();
    }
    for (int first = 0; pairs > kFewPairs && first < pairs && e == hipSuccess; first += kMostTermGroups) {
      preference_pairs_kernel<<<static_cast<unsigned>(std::min(pairs - first, kMostTermGroups)), kTermThreads, 0, s>>>(a, p, first, 1);
      e = hipGetLastError();
    }
    if (e == hipSuccess && pairs > kFewPairs) {
      preference_sums_kernel<<<1, kTermThreads, 0, s>>>(p);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || grad.base == nullptr) return e;
  return launch_logits_grad(s, a, grad, p.g, true);
}
