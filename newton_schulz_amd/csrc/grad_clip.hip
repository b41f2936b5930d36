// Global gradient norm over a list of tensors, and scaling by the clip
// coefficient.
//
// S = sum of g^2 over every element of every tensor, each square exact in
// binary64 (bf16 and fp32 values have at most 24 significant bits), norm =
// sqrt S, coefficient = min(1, max_norm / (norm + eps)).  The tensors are cut
// into chunks of one workgroup each; a chunk leaves one partial sum, and one
// workgroup adds the partials: the last of a small list's launch, a launch of its
// own for longer lists (10 to 20 MB of traffic with the scaling: 12.6 against 15.8
// us).  Every sum runs in a fixed order.
//
// Both kernels are HBM-bound streams.  The list travels in the kernel
// arguments (kTabTensors entries per launch): no table has to be uploaded, so
// the calls can be recorded into a graph, and a list of any length is a few
// launches.
#include "exchange.h"
#include "loss_kernels.h"
#include "muon_device.h"

using muon::bf16_t;

namespace {

constexpr int kTabTensors = 128;  // two per lane: a wave finds its chunk's tensor with two ballots
constexpr int kThreads = 256;
constexpr int kGroup = 8;         // elements per thread and trip

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

struct NormTab {
  const char* data[kTabTensors];
  int64_t numel[kTabTensors];
  int32_t first[kTabTensors];   // first chunk of the tensor within this launch
  uint32_t bf16[kTabTensors / 32];
  int32_t n;
};
struct ScaleTab {
  NormTab in;
  char* out[kTabTensors];
  uint32_t out_bf16[kTabTensors / 32];
};
static_assert(sizeof(ScaleTab) + 64 <= 4096, "kernel arguments");

// The tensor that chunk b lies in: the last with first[i] <= b.
__device__ __forceinline__ int find_tensor(const NormTab& t, int b) {
  const int lane = threadIdx.x & 63;
  const int lo = lane < t.n && t.first[lane] <= b;
  const int hi = 64 + lane < t.n && t.first[64 + lane] <= b;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(lo)) + __popcll(__ballot(hi)) - 1);
}

// Groups of 8 elements start at 16-byte addresses: group q holds elements
// [8 q - lead, 8 q - lead + 8), lead = elements of the first group that lie
// before the tensor.
template <typename T> __device__ __forceinline__ int tensor_lead(const char* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

template <typename T> __device__ __forceinline__ void load_whole(const T* p, float* v) {
  if (sizeof(T) == 2) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}

template <typename T> __device__ __forceinline__ void load_group(const T* p, int64_t e0, int64_t n, float* v) {
  if (e0 >= 0 && e0 + kGroup <= n) {
    load_whole(p + e0, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i) v[i] = e0 + i >= 0 && e0 + i < n ? muon::Elem<T>::load(p + e0 + i) : 0.0f;
}

template <typename T> __device__ __forceinline__ void store_group(T* p, int64_t e0, int64_t n, const float* v) {
  if (e0 >= 0 && e0 + kGroup <= n) {
    // the output may lie at another alignment than the input
    if (sizeof(T) == 2) {
      const u32x4 w = {muon::pack_bf16x2(v[0], v[1]), muon::pack_bf16x2(v[2], v[3]), muon::pack_bf16x2(v[4], v[5]),
                       muon::pack_bf16x2(v[6], v[7])};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(p + e0));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 w = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                         __float_as_uint(v[4 * h + 3])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(p + e0 + 4 * h));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    if (e0 + i >= 0 && e0 + i < n) muon::Elem<T>::store(p + e0 + i, v[i]);
}

// Sum over the NT threads in a fixed order, in every thread.
template <int NT> __device__ __forceinline__ double block_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __shared__ double ws[NT / 64];
  __syncthreads();  // an earlier call's values have been read
  if ((threadIdx.x & 63) == 0) ws[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = ws[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) t += ws[w];
  return t;
}

// Sum of the squares of groups q0 .. q0 + groups - 1 of a tensor (this thread's
// part): at most kTrips groups a thread, all loads issued before the first use.
constexpr int kTrips = 4;
template <typename T>
__device__ __forceinline__ double chunk_squares(const char* data, int64_t numel, int64_t q0, int groups) {
  const T* p = reinterpret_cast<const T*>(data);
  const int lead = tensor_lead<T>(data), t = static_cast<int>(threadIdx.x);
  float v[kTrips][kGroup];
  const int64_t e0 = q0 * kGroup - lead;
  if (e0 >= 0 && e0 + kThreads * kTrips * kGroup <= numel && groups == kThreads * kTrips) {
    // a whole chunk inside the tensor: no bounds to look at
#pragma unroll
    for (int u = 0; u < kTrips; ++u) load_whole<T>(p + e0 + (u * kThreads + t) * kGroup, v[u]);
  } else {
#pragma unroll
    for (int u = 0; u < kTrips; ++u) {
      const int q = u * kThreads + t;
      load_group<T>(p, q < groups ? e0 + static_cast<int64_t>(q) * kGroup : numel, numel, v[u]);
    }
  }
  double acc[2] = {0.0, 0.0};
#pragma unroll
  for (int u = 0; u < kTrips; ++u)
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const double d = static_cast<double>(v[u][i]);
      acc[i & 1] = fma(d, d, acc[i & 1]);
    }
  return acc[0] + acc[1];
}

__device__ __forceinline__ void write_norm(double s, double max_norm, double eps, double* norm) {
  const double size = sqrt(s);
  double c = max_norm / (size + eps);
  if (c > 1.0) c = 1.0;  // a NaN stays
  norm[0] = s;
  norm[1] = size;
  norm[2] = c;
}

// arrived: the last workgroup adds the partials and makes the norm of them.
__global__ __launch_bounds__(kThreads) void sum_squares_kernel(NormTab t, int groups, double* __restrict__ partial,
                                                                uint64_t* arrived, double max_norm, double eps,
                                                                double* norm) {
  const int b = static_cast<int>(blockIdx.x), i = find_tensor(t, b);
  const int64_t q0 = static_cast<int64_t>(b - t.first[i]) * groups;
  const bool bf = (t.bf16[i >> 5] >> (i & 31)) & 1u;
  const double s = block_sum<kThreads>(bf ? chunk_squares<bf16_t>(t.data[i], t.numel[i], q0, groups)
                                : chunk_squares<float>(t.data[i], t.numel[i], q0, groups));
  if (arrived == nullptr) {
    if (threadIdx.x == 0) partial[b] = s;
    return;
  }
  uint64_t* words = reinterpret_cast<uint64_t*>(partial);
  if (threadIdx.x == 0) muon::publish(words + b, static_cast<uint64_t>(__double_as_longlong(s)));
  if (!muon::last_to_arrive(arrived)) return;
  constexpr int U = kArriveGroups / kThreads;
  uint64_t v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned q = u * kThreads + threadIdx.x;
    v[u] = q < gridDim.x ? muon::published(words + q) : 0;
  }
  double acc = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u) acc += __longlong_as_double(static_cast<long long>(v[u]));
  acc = block_sum<kThreads>(acc);
  if (threadIdx.x == 0) write_norm(acc, max_norm, eps, norm);
}

// Workgroup b of n adds the b-th run of the partials; the only one makes the
// norm of it, several leave their sums for another such launch.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void sum_partials_kernel(const double* __restrict__ partial, int64_t n,
                                                                    double* __restrict__ sums, double max_norm,
                                                                    double eps, double* norm) {
  const int64_t per = (n + gridDim.x - 1) / gridDim.x, lo = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t hi = lo + per < n ? lo + per : n;
  double acc = 0.0;
  constexpr int U = 8;
  for (int64_t p = lo + threadIdx.x; p < hi; p += U * kJoinThreads) {
    double v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = p + u * kJoinThreads < hi ? partial[p + u * kJoinThreads] : 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u) acc += v[u];
  }
  const double s = block_sum<kJoinThreads>(acc);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) write_norm(s, max_norm, eps, norm);
  else sums[blockIdx.x] = s;
}

__global__ void clip_coef_kernel(double max_norm, double eps, double* norm) {
  write_norm(norm[0], max_norm, eps, norm);
}

template <typename T, typename U>
__device__ __forceinline__ void chunk_scale(const char* data, char* out, int64_t numel, int64_t q0, int groups,
                                            float c) {
  const T* p = reinterpret_cast<const T*>(data);
  U* o = reinterpret_cast<U*>(out);
  const int lead = tensor_lead<T>(data);
  constexpr int N = 2;
  for (int q = threadIdx.x; q < groups; q += kThreads * N) {
    float v[N][kGroup];
#pragma unroll
    for (int u = 0; u < N; ++u)
      load_group<T>(p, q + u * kThreads < groups ? (q0 + q + u * kThreads) * kGroup - lead : numel, numel, v[u]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (q + u * kThreads >= groups) continue;
#pragma unroll
      for (int i = 0; i < kGroup; ++i) v[u][i] *= c;
      store_group<U>(o, (q0 + q + u * kThreads) * kGroup - lead, numel, v[u]);
    }
  }
}

__global__ __launch_bounds__(kThreads) void scale_kernel(ScaleTab t, int groups, const double* __restrict__ norm) {
  const int b = static_cast<int>(gridDim.x - 1 - blockIdx.x), i = find_tensor(t.in, b);
  const float c = static_cast<float>(norm[2]);
  const char* src = t.in.data[i];
  char* dst = t.out[i];
  if (src == dst && c == 1.0f) return;  // in place, and nothing changes
  const int64_t n = t.in.numel[i], q0 = static_cast<int64_t>(b - t.in.first[i]) * groups;
  const bool bi = (t.in.bf16[i >> 5] >> (i & 31)) & 1u, bo = (t.out_bf16[i >> 5] >> (i & 31)) & 1u;
  if (bi && bo) chunk_scale<bf16_t, bf16_t>(src, dst, n, q0, groups, c);
  else if (bi) chunk_scale<bf16_t, float>(src, dst, n, q0, groups, c);
  else if (bo) chunk_scale<float, bf16_t>(src, dst, n, q0, groups, c);
  else chunk_scale<float, float>(src, dst, n, q0, groups, c);
}

// Walks the list in launches of at most kTabTensors tensors and kMaxChunks
// chunks; calls launch(table, index of each entry, chunks, first chunk overall).
constexpr int64_t kMaxChunks = 1 << 23;

}  // namespace

int64_t clip_chunk(int64_t total) {
  // One group of 8 elements per thread and trip.  Four trips (16 KB of bf16 a
  // workgroup) read 2.4 GB at 6.0 TB/s where 64 KB or more a workgroup read it at
  // 5.5; lists too small to fill the device that way take one or two, as many as
  // keep them at the 1024 workgroups of a single launch (4 M fp32 scaled into
  // bf16: 16.6 us, 17.8 with up to 2048 workgroups and a second launch).
  int64_t c = kThreads * kGroup;
  while (c < kThreads * kGroup * kTrips && total / c > 1024) c *= 2;
  return c;
}

int64_t clip_chunks(const muon_tensor_t& t, int64_t chunk) {
  if (t.numel == 0) return 0;
  const int64_t e = t.dtype == MUON_BF16 ? 2 : 4;
  const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.data) & 15u) / e;
  return (t.numel + lead + chunk - 1) / chunk;
}

namespace {

// fill(slot, i) describes tensor i, launch(chunks, first chunk overall) runs
// the table of n entries.
template <typename Launch>
hipError_t walk(const muon_tensor_t* t, const muon_tensor_t* out, int64_t count, int64_t chunk, Launch launch) {
  ScaleTab tab;
  int64_t i = 0, base = 0;
  while (i < count) {
    tab.in.n = 0;
    for (int k = 0; k < kTabTensors / 32; ++k) tab.in.bf16[k] = tab.out_bf16[k] = 0;
    int64_t chunks = 0;
    for (; i < count && tab.in.n < kTabTensors; ++i) {
      const int64_t c = clip_chunks(t[i], chunk);
      if (c == 0) continue;
      if (tab.in.n > 0 && chunks + c > kMaxChunks) break;
      const int k = tab.in.n++;
      tab.in.data[k] = static_cast<const char*>(t[i].data);
      tab.in.numel[k] = t[i].numel;
      tab.in.first[k] = static_cast<int32_t>(chunks);
      if (t[i].dtype == MUON_BF16) tab.in.bf16[k >> 5] |= 1u << (k & 31);
      if (out) {
        tab.out[k] = static_cast<char*>(out[i].data);
        if (out[i].dtype == MUON_BF16) tab.out_bf16[k >> 5] |= 1u << (k & 31);
      }
      chunks += c;
    }
    if (chunks == 0) break;
    const hipError_t e = launch(tab, chunks, base);
    if (e != hipSuccess) return e;
    base += chunks;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_grad_norm(hipStream_t s, const muon_tensor_t* t, int64_t count, int64_t chunk,
                            double* partial, double max_norm, double eps, double* norm, Exchange& x) {
  int64_t total = 0, all = 0, entries = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t c = clip_chunks(t[i], chunk);
    all += c;
    entries += c > 0;
  }
  const bool one = all > 0 && all <= kArriveGroups && entries <= kTabTensors;
  const int groups = static_cast<int>(chunk / kGroup);
  hipError_t e = one ? clear_exchange(s, x) : hipSuccess;
  if (e != hipSuccess) return e;
  e = walk(t, nullptr, count, chunk, [&](const ScaleTab& tab, int64_t chunks, int64_t base) {
    sum_squares_kernel<<<static_cast<unsigned>(chunks), kThreads, 0, s>>>(
        tab.in, groups, partial + base, one ? x.words + kExchangeWords : nullptr, max_norm, eps, norm);
    total = base + chunks;
    return hipGetLastError();
  });
  if (e != hipSuccess || one) return e;
  // the sums of several workgroups follow the partials (kClipJoin of them at most)
  const int join = total > 16384 ? kClipJoin : 1;
  sum_partials_kernel<<<join, kJoinThreads, 0, s>>>(partial, total, partial + total, max_norm, eps, norm);
  if (join > 1) {
    const hipError_t j = hipGetLastError();
    if (j != hipSuccess) return j;
    sum_partials_kernel<<<1, kJoinThreads, 0, s>>>(partial + total, join, nullptr, max_norm, eps, norm);
  }
  return hipGetLastError();
}

hipError_t launch_clip_coef(hipStream_t s, double max_norm, double eps, double* norm) {
  clip_coef_kernel<<<1, 1, 0, s>>>(max_norm, eps, norm);
  return hipGetLastError();
}

hipError_t launch_scale_grads(hipStream_t s, const muon_tensor_t* t, const muon_tensor_t* out,
                              int64_t count, int64_t chunk, const double* norm) {
  const int groups = static_cast<int>(chunk / kGroup);
  return walk(t, out, count, chunk, [&](const ScaleTab& tab, int64_t chunks, int64_t) {
    scale_kernel<<<static_cast<unsigned>(chunks), kThreads, 0, s>>>(tab, groups, norm);
    return hipGetLastError();
  });
}
