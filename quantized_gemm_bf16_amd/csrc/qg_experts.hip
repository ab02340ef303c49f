// Sorting a router's choices by expert, and putting the experts' results together.
//
// Sorting: a stable counting sort of n = T K small integers. A workgroup takes
// a range of the entries, a wave a run of that range. Counts go to LDS, one
// table per wave; their prefix over the waves (and over the ranges before, from a
// table of counts that a first launch leaves where there is more than one range) says
// where a wave's entries of an expert go. Within 64 entries, the lanes that hold
// the same expert find each other by a ballot per bit of the expert's number.
// No atomic's order is visible in the results. Bound by latency: 4 bytes in
// and 8 out per entry are nothing beside two passes of dependent LDS accesses. Measured: 128 choices over 64
// experts 3.6 us, 524288 over 256 15.5 us (two launches, 4.7 and 12.4 in a trace, where each takes longer; 18.5 with 128
// ranges; 96 with the table of counts summed by a thread per two experts, a load at a time).
//
// Combination: y[t] = sum_k w[t, k] r[back[t, k]] + beta c[t], k in order, in
// fp32, rounded once. A lane takes 8 columns of one token and has eight of
// its rows' loads in flight. Bound by memory: each result is read once (8192 tokens of 8 x 7168, bf16, plus a
// shared expert's: 230 us, 5.1 TB/s).
#include "qg_experts.hpp"

#include <algorithm>

#include "qg_rows.hpp"

namespace qg {

namespace {

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64, kSortExperts = 1024;
constexpr int kMaxChunks = 256;
constexpr int kOneChunk = 2048;

__device__ __forceinline__ int lds_get(int* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT); }
__device__ __forceinline__ void lds_set(int* p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT); }

__device__ __forceinline__ int entry(const GroupArgs& a, int i) {
  const int t = i / a.K;
  const int e = a.ids[(int64_t)t * a.ldi + (i - t * a.K)];
  return e >= 0 && e < a.E ? e : -1;
}

constexpr int kHeld = 4;  // entries that a lane has loaded ahead

// f(i, e) for the entries i of the wave's run [i0, i1), 64 at a time (e < 0: nobody's, or i past the run), by whole waves
template <class F>
__device__ __forceinline__ void each64(const GroupArgs& a, int i0, int i1, F f) {
  const int l = lane_id();
  for (int i = i0; i < i1; i += 64 * kHeld) {
    int e[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) e[j] = i + 64 * j + l < i1 ? entry(a, i + 64 * j + l) : -1;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (i + 64 * j < i1) f(i + 64 * j + l, e[j]);
  }
}

// Counts of the workgroup's range, a table of E per wave.
__device__ __forceinline__ void count_range(const GroupArgs& a, int (*hist)[kSortExperts], int i0, int i1) {
  const int w = wave_id();
  for (int i = threadIdx.x; i < kSortWaves * kSortExperts; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  each64(a, i0, i1, [&](int, int e) {
    if (e >= 0) atomicAdd(&hist[w][e], 1);
  });
  __syncthreads();
}
__device__ __forceinline__ void wave_run(const GroupArgs& a, int& i0, int& i1) {
  const int c0 = blockIdx.x * a.chunk, per = a.chunk / kSortWaves;
  i0 = c0 + wave_id() * per;
  i1 = min(min(a.n, c0 + a.chunk), i0 + per);
}

__global__ __launch_bounds__(kSortThreads) void group_count_kernel(const GroupArgs a) {
  __shared__ int hist[kSortWaves][kSortExperts];
  int i0, i1;
  wave_run(a, i0, i1);
  count_range(a, hist, i0, i1);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) sum += hist[w][e];
    a.counts[(int64_t)blockIdx.x * a.E + e] = sum;
  }
}

__global__ __launch_bounds__(kSortThreads) void group_place_kernel(const GroupArgs a) {
  __shared__ int hist[kSortWaves][kSortExperts];
  __shared__ int all[kSortExperts], before[kSortExperts];
  __shared__ int wave_total[kSortWaves], grand;
  const int c = blockIdx.x, w = wave_id(), l = lane_id();
  int i0, i1;
  wave_run(a, i0, i1);
  count_range(a, hist, i0, i1);
  if (a.chunks == 1) {
    for (int e = threadIdx.x; e < kSortExperts; e += kSortThreads) {
      int sum = 0;
#pragma unroll
      for (int q = 0; q < kSortWaves; ++q) sum += hist[q][e];
      all[e] = sum;
      before[e] = 0;
    }
  } else {
    // the columns of the table of counts: `parts` threads share one where the experts are few
    for (int e = threadIdx.x; e < kSortExperts; e += kSortThreads) all[e] = before[e] = 0;
    __syncthreads();
    const int width = (a.E + 63) & ~63, parts = max(1, kSortThreads / width);
    for (int e = threadIdx.x % width, p = threadIdx.x / width; p < parts && e < a.E; e += kSortThreads) {
      int sum = 0, low = 0;
#pragma unroll 16
      for (int q = p; q < a.chunks; q += parts) {
        const int x = a.counts[(int64_t)q * a.E + e];
        sum += x;
        low += q < c ? x : 0;
      }
      atomicAdd(&all[e], sum);
      atomicAdd(&before[e], low);
    }
  }
  __syncthreads();
  // Exclusive prefix over the experts; thread t has 2 t and 2 t + 1 (kSortExperts = 2 kSortThreads).
  const int n0 = all[2 * threadIdx.x], n1 = all[2 * threadIdx.x + 1];
  int incl = n0 + n1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d, 64);
    if (l >= d) incl += y;
  }
  if (l == 63) wave_total[w] = incl;
  __syncthreads();
  int at = incl - n0 - n1;
  for (int q = 0; q < w; ++q) at += wave_total[q];
  if (threadIdx.x == kSortThreads - 1) grand = at + n0 + n1;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * threadIdx.x + j;
    if (c == 0 && e <= a.E) a.offsets[e] = at;
    int place = at + before[e];
    at += j ? n1 : n0;
#pragma unroll
    for (int q = 0; q < kSortWaves; ++q) {
      const int x = hist[q][e];
      hist[q][e] = place;
      place += x;
    }
  }
  __syncthreads();
  each64(a, i0, i1, [&](int i, int e) {
    uint64_t same = __ballot(e >= 0);
    for (int b = 1; b < a.E; b <<= 1) {
      const uint64_t set = __ballot((e & b) != 0);
      same &= e & b ? set : ~set;
    }
    int pos = -1;
    if (e >= 0) pos = lds_get(&hist[w][e]) + __popcll(same & ((uint64_t(1) << l) - 1));
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && __ffsll((unsigned long long)same) - 1 == l) lds_set(&hist[w][e], pos + __popcll(same));
    __builtin_amdgcn_wave_barrier();
    if (i < i1) a.back[i] = pos;
    if (e >= 0) a.rows[pos] = i / a.K;
  });
  // rows behind the last expert's come from nowhere
  for (int i = grand + c * kSortThreads + threadIdx.x; i < a.n; i += a.chunks * kSortThreads) a.rows[i] = -1;
}

template <int RT, int YT, class Args>
__global__ __launch_bounds__(256) void combine_kernel(const Args a) {
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int cpr = (a.H + 7) >> 3;
  const Places places(first, cpr);
  const Place at = places.at(threadIdx.x);
  if (first + threadIdx.x >= (int64_t)a.T * cpr) return;
  const int n = a.H - at.unit * 8;
  const int32_t* back = a.back + at.row * a.K;
  const float* w = a.W + at.row * a.ldw;
  float y[8] = {};
  for (int k0 = 0; k0 < a.K; k0 += 8) {
    Raw<RT> r[8];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = k0 + j < a.K ? back[k0 + j] : -1;
      const bool there = p >= 0 && p < a.N;
      f[j] = there ? w[k0 + j] : 0.f;
      r[j].template load<true>((const char*)a.R + ((int64_t)p * a.ldr + at.unit * 8) * Raw<RT>::ES, there ? n : 0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(f[j], r[j].at(i), y[i]);
  }
  if constexpr (sizeof(Args) > sizeof(CombineArgs)) {
    const auto add = [&](auto raw) {
      raw.template load<true>((const char*)a.C + (at.row * a.ldc + at.unit * 8) * raw.ES, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(a.beta, raw.at(i), y[i]);
    };
    if (a.c_type == DT_F32) add(Raw<DT_F32>());
    if (a.c_type == DT_BF16) add(Raw<DT_BF16>());
    if (a.c_type == DT_F16) add(Raw<DT_F16>());
  }
  store8<YT, false>((char*)a.Y + (at.row * a.ldy + at.unit * 8) * Raw<YT>::ES, y, n);
}

template <int RT, int YT>
hipError_t combine_ry(const CombineAddArgs& a, hipStream_t s) {
  // a dispatch counts its threads in 32 bits: rows go out in parts of fewer
  const int64_t cpr = (a.H + 7) / 8, most = (int64_t)(UINT32_MAX / 256) * 256 / cpr;
  for (int64_t t = 0; t < a.T; t += most) {
    CombineAddArgs p = a;
    p.T = (int32_t)std::min<int64_t>(most, a.T - t);
    p.back = a.back + t * a.K;
    p.W = a.W + t * a.ldw;
    p.Y = (char*)a.Y + t * a.ldy * Raw<YT>::ES;
    const dim3 blocks((unsigned)(((int64_t)p.T * cpr + 255) / 256));
    if (a.beta != 0.f) {
      p.C = (const char*)a.C + t * a.ldc * (a.c_type == DT_F32 ? 4 : 2);
      hipLaunchKernelGGL((combine_kernel<RT, YT, CombineAddArgs>), blocks, dim3(256), 0, s, p);
    } else {
      hipLaunchKernelGGL((combine_kernel<RT, YT, CombineArgs>), blocks, dim3(256), 0, s, (const CombineArgs&)p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <int RT>
hipError_t combine_r(const CombineAddArgs& a, int y_type, hipStream_t s) {
  switch (y_type) {
    case DT_F32: return combine_ry<RT, DT_F32>(a, s);
    case DT_F16: return combine_ry<RT, DT_F16>(a, s);
    case DT_BF16: return combine_ry<RT, DT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// One workgroup sorts 2048 choices in 7 us and 8192 in 18, two launches take 10 for either; from Python the calls of one
// launch are let through 0.5 us sooner.
void group_chunks(int64_t n, bool workspace, int* chunk, int* chunks) {
  const int64_t ranges = n <= (workspace ? kOneChunk : kGroupAlone) ? 1 : kMaxChunks;
  *chunk = (int)(std::max<int64_t>(1, ((n + ranges - 1) / ranges + kSortThreads - 1) / kSortThreads) * kSortThreads);
  *chunks = (int)std::max<int64_t>(1, (n + *chunk - 1) / *chunk);
}

hipError_t launch_group(const GroupArgs& a, hipStream_t s) {
  if (a.chunks > 1) {
    hipLaunchKernelGGL(group_count_kernel, dim3(a.chunks), dim3(kSortThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_place_kernel, dim3(a.chunks), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineAddArgs& a, int r_type, int y_type, hipStream_t s) {
  switch (r_type) {
    case DT_F32: return combine_r<DT_F32>(a, y_type, s);
    case DT_F16: return combine_r<DT_F16>(a, y_type, s);
    case DT_BF16: return combine_r<DT_BF16>(a, y_type, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
