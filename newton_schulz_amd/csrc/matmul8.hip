// Products of 8-bit rows: out = (a b^T) times the scales of a row and a column.
//
// Mathematics.  The integers' sum is exact in 32 bits (at most 131071 products
// of at most 2^14); it is rounded to fp32 once and multiplied by the product of
// the two scales.
#include "linear8.h"
#include "ns_mfma_common.h"
#include "tile_plan.h"

namespace {

constexpr int kTile = 64, kStep = 64, kPitch = kStep + 4;

template <typename T>
__global__ __launch_bounds__(256) void matmul8_simple_kernel(Matmul8Args a) {
  __shared__ int8_t ta[kTile * kPitch], tb[kTile * kPitch];
  const int64_t tiles_n = (a.n + kTile - 1) / kTile;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) / tiles_n * kTile, n0 = static_cast<int64_t>(blockIdx.x) % tiles_n * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.k; k0 += kStep) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      const int r = e / kStep, c = e % kStep;
      const bool in = k0 + c < a.k;
      ta[r * kPitch + c] = in && m0 + r < a.m ? a.a.p[(m0 + r) * a.a.ld + k0 + c] : 0;
      tb[r * kPitch + c] = in && n0 + r < a.n ? a.b.p[(n0 + r) * a.b.ld + k0 + c] : 0;
    }
    __syncthreads();
    for (int c = 0; c < kStep; c += 4) {
      int va[4], vb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) va[i] = *reinterpret_cast<const int*>(ta + (ty + 16 * i) * kPitch + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) vb[j] = *reinterpret_cast<const int*>(tb + (tx + 16 * j) * kPitch + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_sdot4(va[i], vb[j], acc[i][j], false);
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.m && n < a.n)
        muon::Elem<T>::store(reinterpret_cast<T*>(a.out.p) + m * a.out.ld + n,
                             static_cast<float>(acc[i][j]) * (a.a.scale[m] * a.b.scale[n]));
    }
}


// ---------------------------------------------------------------------------
// tiles of T x T outputs on the matrix cores
// ---------------------------------------------------------------------------
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBytes = 128;  // of k in a stage

// One operand's stage: T rows of 128 bytes, in LDS as rt_off lays them out.
template <int T, int NW>
struct Stage8 {
  static constexpr int NG = T / (8 * NW);  // 1 KiB loads per wave
  uint32_t base[NG];
  int kc[NG], lim[NG];
  u32x4_t rsrc;

  // Rows [row0, row0 + T) of `rows`.  A chunk that is not whole in the last
  // row would reach past the memory: finish() brings it.  From `past` on they
  // hold zeros.
  __device__ __forceinline__ void init(const Bytes& x, int64_t rows, int k, int past, int64_t row0, int wave, int lane) {
    const int here = static_cast<int>(min(rows - row0, static_cast<int64_t>(T)));
    const int ld = static_cast<int>(x.ld);
    rsrc = rsrc_words(uniform_ptr(x.p + row0 * x.ld), static_cast<uint32_t>(here - 1) * ld + (k & ~15) + (k & 15 ? 16 : 0));
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const int row = 8 * (wave + NW * q) + lane / 8;
      const int chunk = (lane % 8) ^ rt_swz<64>(row);
      kc[q] = 16 * chunk;
      lim[q] = min((row0 + row == rows - 1 || ld == 0) ? k & ~15 : k, past);
      base[q] = row < here ? static_cast<uint32_t>(row) * ld + 16 * chunk : kOOB;
    }
  }
  __device__ __forceinline__ void issue(char* lds, int k0, int wave, bool full) const {
    dma16_group<NG>(
        rsrc, static_cast<uint32_t>(k0), [&](int q) { return lds + (wave + NW * q) * 1024; },
        [&](int q) { return (full || k0 + kc[q] < lim[q]) ? base[q] : kOOB; });
  }
  // The chunk of 16 bytes that holds k, not whole: zeros behind k (what a row's
  // memory holds there meets nothing), and in the last row all of it.
  static __device__ __forceinline__ void finish(char* lds, const Bytes& x, int64_t rows, int k, int64_t row0, int k0, int tid) {
    if (tid >= T) return;
    const int64_t r = row0 + tid;
    if (r >= rows) return;
    char* at = lds + rt_off<64>(tid, ((k - 1) - k0) >> 4);
    const int n = k & 15;
    uint32_t w[4];
    if (r == rows - 1 || x.ld == 0) {
      const uint8_t* from = reinterpret_cast<const uint8_t*>(x.p) + r * x.ld + (k & ~15);
      for (int i = 0; i < 4; ++i) {
        w[i] = 0;
        for (int j = 0; j < 4; ++j)
          if (4 * i + j < n) w[i] |= static_cast<uint32_t>(from[4 * i + j]) << (8 * j);
      }
    } else {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at);
      for (int i = 0; i < 4; ++i) {
        const int keep = n - 4 * i;
        w[i] = keep >= 4 ? v[i] : keep <= 0 ? 0u : v[i] & ((1u << (8 * keep)) - 1u);
      }
    }
    *reinterpret_cast<u32x4_t*>(at) = u32x4_t{w[0], w[1], w[2], w[3]};
  }
};

// ---- staged output tile, fp32 or bf16, in two halves of T / 2 rows: element (r, c) of a
// half; 16-byte chunks swizzled by the row.
template <typename O, int T>
__device__ __forceinline__ int out_off(int r, int c) {
  constexpr int E = static_cast<int>(sizeof(O));
  const int byte = c * E;
  const int g = E == 2 ? ((r & 3) << 2) | ((r >> 2) & 3) : (r & 15);
  return r * (T * E) + ((((byte >> 4) ^ g) << 4) | (byte & 15));
}

template <typename O, int T>
__global__ __launch_bounds__(T == 256 ? 512 : 256, 1) void matmul8_tile_kernel(Matmul8Args a, TileWork work) {
  constexpr int NWN = T == 256 ? 4 : 2, NW = 2 * NWN, NT = 64 * NW;
  constexpr int WM = T / 2, WN = T / NWN, FM = WM / 32, FN = WN / 32;
  constexpr int HALF = T * kBytes, STAGE = 2 * HALF;
  __shared__ __attribute__((aligned(1024))) char st0[STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[STAGE];
  auto buf = [&](auto I) -> char* { return decltype(I)::value % 2 ? st1 : st0; };

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / NWN, wn = wave % NWN;

  const int G = static_cast<int>(gridDim.x), hw = static_cast<int>(blockIdx.x);
  const int64_t first = G % 8 == 0 ? static_cast<int64_t>(hw % 8) * (G / 8) + hw / 8 : hw;
  for (int64_t l = first; l < work.units; l += G) {
    const TileUnit unit = tile_unit(work, l);
    const int64_t m0 = unit.ti * T, n0 = unit.tj * T;

    i32x16_t acc[FM][FN];
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = (i32x16_t)(0);

    Stage8<T, NW> om, on;
    om.init(a.a, a.m, a.k, unit.past * kBytes, m0, wave, lane);
    on.init(a.b, a.n, a.k, unit.past * kBytes, n0, wave, lane);
    const int KT = work.stages, KF = min(a.k / kBytes, unit.past);
    auto issue = [&](char* st, int kt) {
      const bool full = kt < KF;
      om.issue(st, kt * kBytes, wave, full);
      on.issue(st + HALF, kt * kBytes, wave, full);
    };
    constexpr int NL = 2 * Stage8<T, NW>::NG;
    i32x4_t fa[2][FN], fb[2][FM];
    auto frags = [&](const char* sm, int kk, auto BUF) {
      constexpr int b = decltype(BUF)::value;
      const char* sn = sm + HALF;
#pragma unroll
      for (int ni = 0; ni < FN; ++ni)
        fa[b][ni] = *reinterpret_cast<const i32x4_t*>(sn + rt_off<64>(wn * WN + ni * 32 + (lane & 31), 2 * kk + (lane >> 5)));
#pragma unroll
      for (int mi = 0; mi < FM; ++mi)
        fb[b][mi] = *reinterpret_cast<const i32x4_t*>(sm + rt_off<64>(wm * WM + mi * 32 + (lane & 31), 2 * kk + (lane >> 5)));
    };
    constexpr int NMF = FM * FN, NRD = FM + FN, TAIL = NMF / 2, KK = kBytes / 32;
    auto mfmas = [&](auto BUF, auto BEGIN, auto END) {
      constexpr int b = decltype(BUF)::value;
      static_for<decltype(END)::value - decltype(BEGIN)::value>([&](auto P) {
        constexpr int p = decltype(P)::value + decltype(BEGIN)::value;
        constexpr int mi = p / FN, ni = p % FN;
        acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[b][ni], fb[b][mi], acc[mi][ni], 0, 0, 0);
      });
    };
    auto interleave = [&](auto NM) {
      static_for<decltype(NM)::value>([&](auto I) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (decltype(I)::value < NRD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      });
    };
    // stage kt has landed in st: complete its last chunk
    auto complete = [&](char* st, int kt) {
      if ((a.k & 15) && kt == KT - 1 && kt < unit.past) {
        Stage8<T, NW>::finish(st, a.a, a.m, a.k, m0, kt * kBytes, tid);
        Stage8<T, NW>::finish(st + HALF, a.b, a.n, a.k, n0, kt * kBytes, tid);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
    };
    auto stage = [&](auto S, int kt) {
      char* cur = buf(S);
      char* nxt = buf(ic<decltype(S)::value + 1>{});
      static_for<KK>([&](auto KI) {
        constexpr int kk = decltype(KI)::value;
        constexpr int b = kk & 1;
        if constexpr (kk + 1 < KK) {
          frags(cur, kk + 1, ic<b ^ 1>{});
          mfmas(ic<b>{}, ic<0>{}, ic<NMF>{});
          interleave(ic<NMF>{});
          __builtin_amdgcn_sched_barrier(0);
        } else {
          mfmas(ic<b>{}, ic<0>{}, ic<NMF - TAIL>{});
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
          complete(nxt, kt + 1);
          issue(cur, kt + 2);
          __builtin_amdgcn_sched_barrier(0);
          frags(nxt, 0, ic<0>{});
          mfmas(ic<b>{}, ic<NMF - TAIL>{}, ic<NMF>{});
          interleave(ic<TAIL>{});
          __builtin_amdgcn_sched_barrier(0);
        }
      });
    };
    // whole rounds of two stages: stages at or past K load zeros
    issue(st0, unit.first);
    issue(st1, unit.first + 1);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NL) : "memory");
    complete(st0, unit.first);
    frags(st0, 0, ic<0>{});
    for (int kt = unit.first; kt < unit.past; kt += 2) static_for<2>([&](auto S) { stage(S, kt + decltype(S)::value); });

    // ---- epilogue: scaled values through LDS, row-contiguous stores
    int el = lane;
    asm volatile("" : "+v"(el));
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    __syncthreads();
    // in rounds of the rows that the stage buffers hold: all of a tile of bf16, or
    // the rows of the waves wm == round (fp32, and integers that are not all of the sum)
    auto rounds = [&](auto Z, auto&& put, auto&& get) __attribute__((always_inline)) {
      using S = decltype(Z);
      constexpr int E = static_cast<int>(sizeof(S));
      constexpr int HROWS = E == 2 ? T / 2 : T / 4, ROUNDS = E == 2 ? 1 : 2;
      static_assert(HROWS * T * E <= STAGE, "output rows fit the stage buffers");
      static_for<ROUNDS>([&](auto R) {
        constexpr int rd = decltype(R)::value;
        if (ROUNDS == 1 || wm == rd) {
          static_for<FM>([&](auto MI) {
            constexpr int mi = decltype(MI)::value;
            const int il = wm * WM + mi * 32 + (el & 31), row = ROUNDS == 1 ? il : il - rd * WM;
            char* half = row >= HROWS ? st1 : st0;
            put(MI, il, [&](int jl) { return half + out_off<S, T>(row >= HROWS ? row - HROWS : row, jl); });
          });
        }
        __syncthreads();
        constexpr int C = 16 / E, CH = T / C;  // elements of a chunk, chunks of a row
        const int et = wave * 64 + el;
#pragma unroll 4
        for (int it = 0; it < 2 * HROWS * CH / NT; ++it) {
          const int e = et + it * NT, row = e / CH, c = e % CH;
          const char* half = row >= HROWS ? st1 : st0;
          get(rd * 2 * HROWS + row, C * c, *reinterpret_cast<const u32x4_t*>(half + out_off<S, T>(row >= HROWS ? row - HROWS : row, C * c)));
        }
        __syncthreads();
      });
    };
    if (unit.slot >= 0) {
      int* part = reinterpret_cast<int*>(work.parts) + unit.slot * (T * T);
      rounds(
          0,
          [&](auto MI, int, auto&& at) __attribute__((always_inline)) {
            constexpr int mi = decltype(MI)::value;
            static_for<FN>([&](auto NI) {
              constexpr int ni = decltype(NI)::value;
#pragma unroll
              for (int g = 0; g < 4; ++g)
                *reinterpret_cast<i32x4_t*>(at(wn * WN + ni * 32 + 8 * g + 4 * (el >> 5))) =
                    i32x4_t{acc[mi][ni][4 * g], acc[mi][ni][4 * g + 1], acc[mi][ni][4 * g + 2], acc[mi][ni][4 * g + 3]};
              __builtin_amdgcn_sched_barrier(0);
            });
          },
          [&](int row, int c, u32x4_t v) __attribute__((always_inline)) { *reinterpret_cast<u32x4_t*>(part + row * T + c) = v; });
      continue;
    }
    constexpr int E = static_cast<int>(sizeof(O)), C = 16 / E;
    float sb[FN][4][4];
#pragma unroll
    for (int ni = 0; ni < FN; ++ni)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t n = n0 + wn * WN + ni * 32 + 8 * g + 4 * (el >> 5) + q;
          sb[ni][g][q] = n < a.n ? a.b.scale[n] : 0.0f;
        }
    O* out = reinterpret_cast<O*>(a.out.p);
    const bool wide = ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(a.out.ld * E)) & 15u) == 0;
    rounds(
        O{},
        [&](auto MI, int il, auto&& at) __attribute__((always_inline)) {
          constexpr int mi = decltype(MI)::value;
          const float sa = m0 + il < a.m ? a.a.scale[m0 + il] : 0.0f;
          static_for<FN>([&](auto NI) {
            constexpr int ni = decltype(NI)::value;
            static_for<4>([&](auto GI) {
              constexpr int g = decltype(GI)::value;
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = static_cast<float>(acc[mi][ni][4 * g + q]) * (sa * sb[ni][g][q]);
              char* to = at(wn * WN + ni * 32 + 8 * g + 4 * (el >> 5));
              if constexpr (E == 2) *reinterpret_cast<uint2*>(to) = make_uint2(muon::pack_bf16x2(v[0], v[1]), muon::pack_bf16x2(v[2], v[3]));
              else *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
            });
            __builtin_amdgcn_sched_barrier(0);
          });
        },
        [&](int row, int c, u32x4_t v) __attribute__((always_inline)) {
          const int64_t m = m0 + row, n = n0 + c;
          if (m >= a.m || n >= a.n) return;
          O* to = out + m * a.out.ld + n;
          if (wide && n + C <= a.n) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(to));
          } else {
            const O* from = reinterpret_cast<const O*>(&v);
            for (int q = 0; q < C; ++q)
              if (n + q < a.n) to[q] = from[q];
          }
        });
  }
}

// The parts of the tiles that were cut, added in order: four outputs a thread.
template <typename O, int T>
__global__ __launch_bounds__(256) void matmul8_join_kernel(Matmul8Args a, TileWork work) {
  constexpr int PER = T * T / 1024;  // workgroups of a tile
  const int64_t t = blockIdx.x / PER;
  const int e = static_cast<int>(blockIdx.x % PER) * 256 + static_cast<int>(threadIdx.x), row = e / (T / 4), c = 4 * (e % (T / 4));
  const TileUnit unit = tile_unit(work, work.whole + t);
  const int* part = reinterpret_cast<const int*>(work.parts) + t * work.splits * (T * T) + row * T + c;
  const int64_t m = unit.ti * T + row, n = unit.tj * T + c;
  if (m >= a.m || n >= a.n) return;
  i32x4_t v = *reinterpret_cast<const i32x4_t*>(part);
  for (int p = 1; p < work.splits; ++p) v += *reinterpret_cast<const i32x4_t*>(part + static_cast<int64_t>(p) * (T * T));
  O* to = reinterpret_cast<O*>(a.out.p) + m * a.out.ld + n;
  const float sa = a.a.scale[m];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (n + q < a.n) muon::Elem<O>::store(to + q, static_cast<float>(v[q]) * (sa * a.b.scale[n + q]));
}

template <typename O, int T>
hipError_t go_tiles(hipStream_t s, const Matmul8Args& a, const TilePlan& p) {
  const TileWork w = tile_work(p, a.ws);
  matmul8_tile_kernel<O, T><<<static_cast<unsigned>(p.grid), T == 256 ? 512 : 256, 0, s>>>(a, w);
  if (p.splits > 1) {
    const int64_t cut = static_cast<int64_t>(p.tm) * p.tn - p.whole;
    matmul8_join_kernel<O, T><<<static_cast<unsigned>(cut * (T * T / 1024)), 256, 0, s>>>(a, w);
  }
  return hipGetLastError();
}

template <typename O>
hipError_t go(hipStream_t s, const Matmul8Args& a) {
  const int stages = (a.k + kBytes - 1) / kBytes;
  // (two small tiles on a CU take 0.6 of a large one's time for half its products)
  double large, small;
  const TilePlan l = plan_tiles(a.m, a.n, 256, 256, stages, a.cus, a.ws_bytes, &large);
  const TilePlan q = plan_tiles(a.m, a.n, 128, 128, stages, 2 * a.cus, a.ws_bytes, &small);
  return large <= 0.6 * small ? go_tiles<O, 256>(s, a, l) : go_tiles<O, 128>(s, a, q);
}

}  // namespace

hipError_t launch_matmul8(hipStream_t s, const Matmul8Args& a) {
  if (a.m == 0 || a.n == 0) return hipSuccess;
  if (a.m > 32) return a.out.bf16 ? go<bf16_t>(s, a) : go<float>(s, a);
  const unsigned grid = static_cast<unsigned>(((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile));
  if (a.out.bf16) matmul8_simple_kernel<bf16_t><<<grid, 256, 0, s>>>(a);
  else matmul8_simple_kernel<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
