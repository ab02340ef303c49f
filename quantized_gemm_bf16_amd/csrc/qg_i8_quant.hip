// Int8 quantise and dequantise kernels: one scale per row.
//
// A row of y (the row itself, or silu(gate) * up) with largest magnitude amax
// has the scale s = fp32(amax / 127) and the codes rne(y / s), both as 64-bit
// arithmetic gives them: a row's maximum has to be known before its first
// code, so a row is read once into registers (up to 16384 elements, 65536 with
// four times the waves) and its codes leave from there; longer ones are read twice.
//
// fp32 decides what it can. With t = v * (1 / s), where v is the fp32 value,
// the code is rint(t) unless t is within its error of a half: then that
// element alone is done again in 64 bits, from memory (the caches have it).
// The error of t: identity 2^-23 t. SwiGLU: v = (g u) rcp(1 + exp2(-g log2 e)):
// the argument of exp2 is off by 2.25 * 2^-24 of itself (the constant's rounding, the
// product's), so e by |g| 2.25 * 2^-24 of itself, the other steps by 8 * 2^-24 (exp2 and rcp
// one step each, the sum, three products): within 2^-19 for g >= -8 and 2^-17 for
// g >= -32 (below that exp2 may overflow: always in 64 bits). The maximum of a gated row is taken in 64 bits
// too, over the elements whose v is within 2^-16 of the largest v. Rows whose
// largest v is not finite, or so small that v or the scale may have lost bits
// (below 2^-60), go through 64 bits as a whole.
#include "qg_i8_quant.hpp"

#include <algorithm>

#include "qg_rows.hpp"

namespace qg {

namespace {

// Element k of y in 64 bits, from memory.
template <int DT, bool GATED>
__device__ __attribute__((noinline)) double value64(const char* row, int K, int k) {
  const auto get = [&](int64_t i) -> double {
    if constexpr (DT == DT_F32) return ((const float*)row)[i];
    const uint16_t h = ((const uint16_t*)row)[i];
    return DT == DT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
  };
  if constexpr (!GATED) return get(k);
  const double g = get(k), u = get((int64_t)K + k);
  return g / (1.0 + exp(-g)) * u;
}

// Maximum over aligned groups of L lanes, in every lane of them.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
  return x;
}
template <int L>
__device__ __forceinline__ double lanes_max(double x) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) x = fmax(x, __shfl_xor(x, d, 64));
  return x;
}

// L lanes (a part of a wave, or whole waves: the workgroup) take one row,
// U units of 8 elements each.
template <int DT, bool GATED, int L, int U>
__global__ __launch_bounds__(L < 256 ? 256 : L) void i8_quantize_kernel(const I8QuantArgs a) {
  constexpr int NT = L < 256 ? 256 : L, RPB = NT / L, LW = L < 64 ? L : 64, NW = L / 64;
  __shared__ uint32_t wave_top[L > 64 ? NW : 1];
  __shared__ double wave_top64[L > 64 ? NW : 1];
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / L;
  const int l = threadIdx.x % L;
  const bool live = row < a.R;
  int64_t src = row;
  if (a.rows && live) src = a.rows[row];
  const bool there = live && src >= 0 && src < a.T;
  const char* x = (const char*)a.X + (there ? src : 0) * (int64_t)a.ldx * Raw<DT>::ES;
  float v[U][8];
  uint32_t deep[U];  // elements that need 64 bits whatever their neighbours (bit per element)
  uint32_t top = 0;
  {
    Raw<DT> in[U], up[GATED ? U : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = (i * L + l) * 8, n = there ? a.K - k : 0;
      in[i].template load<true>(x + (int64_t)k * Raw<DT>::ES, n);
      if constexpr (GATED) up[i].template load<false>(x + ((int64_t)a.K + k) * Raw<DT>::ES, n);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      deep[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = in[i].at(j);
        if constexpr (GATED) {
          const float g = v[i][j];
          v[i][j] = g * up[i].at(j) * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
          deep[i] |= (g < -32.f ? 1u : 0u) << j | (g < -8.f ? 1u : 0u) << (8 + j);
        }
        top = max(top, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7FFFFFFFu);
      }
    }
  }
  // the row's largest |v|, as bits (a NaN is more than everything)
  top = lanes_max<LW>(top);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) top = max(top, wave_top[w]);
  }
  const bool slow = top >= 0x7F800000u || (top != 0 && top < 0x21800000u);  // not finite, or under 2^-60
  double amax = __builtin_bit_cast(float, top);
  if constexpr (GATED) {
    // in 64 bits over the candidates
    const float near = slow ? 0.f : __builtin_bit_cast(float, top) * (1.f - 0x1p-16f);
    double m = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      uint32_t todo = deep[i] & 0xFF;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (slow || (top != 0 && fabsf(v[i][j]) >= near)) todo |= 1u << j;
      const int k = (i * L + l) * 8, n = there ? a.K - k : 0;
      if (n < 8) todo &= n > 0 ? (1u << n) - 1 : 0;
      while (todo) {
        const int j = __builtin_ctz(todo);
        todo &= todo - 1;
        const double y = fabs(value64<DT, GATED>(x, a.K, k + j));
        bad |= !(y <= 1.7976931348623157e308);
        m = fmax(m, y);
      }
    }
    if (bad) m = __builtin_bit_cast(double, (uint64_t)0x7FF << 52);
    m = lanes_max<LW>(m);
    if constexpr (L > 64) {
      if ((threadIdx.x & 63) == 0) wave_top64[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmax(m, wave_top64[w]);
    }
    amax = m;
  }
  // (a bound on amax first: fp32 infinity is a row that cannot be scaled either)
  float s = (float)(amax / 127.0);
  const bool none = !(amax <= 1.7976931348623157e308) || !(s <= 3.4028234663852886e38f);
  if (none) s = __builtin_bit_cast(float, 0x7FC00000u);
  const bool zero = none || s == 0.f;
  const float inv = zero ? 0.f : (float)(1.0 / (double)s);
  if (live && l == 0) a.S[row * a.lds] = s;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int k = (i * L + l) * 8, n = live ? a.K - k : 0;
    uint32_t lo = 0, hi = 0, todo = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = v[i][j] * inv, q = rintf(t);
      const float off = !GATED ? 0x1p-22f : (deep[i] >> (8 + j) & 1) ? 0x1p-17f : 0x1p-19f;
      if (__builtin_fmaf(fabsf(t), off, fabsf(t - q)) >= 0.5f) todo |= 1u << j;
      const uint32_t c = (uint32_t)(int)q & 0xFF;
      (j < 4 ? lo : hi) |= c << (8 * (j & 3));
    }
    todo |= slow ? 0xFF : deep[i] & 0xFF;
    if (zero || !there) todo = lo = hi = 0;
    if (n < 8) todo &= n > 0 ? (1u << n) - 1 : 0;
    while (todo) {
      const int j = __builtin_ctz(todo);
      todo &= todo - 1;
      const double q = fmin(fmax(rint(value64<DT, GATED>(x, a.K, k + j) / (double)s), -127.0), 127.0);
      const uint32_t c = (uint32_t)(int)q & 0xFF, at = 8 * (j & 3), keep = ~(0xFFu << at);
      if (j < 4)
        lo = (lo & keep) | c << at;
      else
        hi = (hi & keep) | c << at;
    }
    char* q = a.Q + row * a.ldq + k;
    if (n >= 8) {
      *(uint64_t*)q = (uint64_t)hi << 32 | lo;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = (char)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
  }
}

template <int DT, int U>
__global__ __launch_bounds__(256) void i8_dequantize_kernel(const I8QuantArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (256 * U);
  const Places places(first, a.cpr);
  uint64_t q[U];
  float s[U];
  Place at[U];
  int n[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t off = i * 256 + threadIdx.x;
    at[i] = places.at(off);
    n[i] = first + off < (int64_t)a.R * a.cpr ? a.K - at[i].unit * 8 : 0;
    q[i] = 0;
    s[i] = 0.f;
    if (n[i] > 0) {
      q[i] = *(const uint64_t*)(a.Q + at[i].row * a.ldq + at[i].unit * 8);  // inside the pitch
      s[i] = a.S[at[i].row * a.lds];
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)(q[i] >> (8 * j)) * s[i];
    store8<DT, true>((char*)a.X + (at[i].row * a.ldx + at[i].unit * 8) * Raw<DT>::ES, v, n[i]);
  }
}

// A dispatch counts its threads in 32 bits, and a launch of more loses the rest without an error: rows go
// out in parts of fewer.
template <class Kernel>
hipError_t launch_parts(Kernel kernel, const I8QuantArgs& a, int64_t most, int64_t pitch, int threads, int64_t per_block,
                        int64_t units_per_row, hipStream_t s) {
  for (int64_t r = 0; r < a.R; r += most) {
    I8QuantArgs p = a;
    p.R = (int32_t)std::min<int64_t>(most, a.R - r);
    p.Q = a.Q + r * a.ldq;
    p.S = a.S + r * a.lds;
    if (a.rows) {
      p.rows = a.rows + r;
    } else {
      p.X = (char*)a.X + r * pitch;
      p.T = p.R;
    }
    const int64_t blocks = ((int64_t)p.R * units_per_row + per_block - 1) / per_block;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, bool GATED, int L, int U>
hipError_t quantize_lu(const I8QuantArgs& a, hipStream_t s) {
  constexpr int NT = L < 256 ? 256 : L, RPB = NT / L;
  const int64_t most = (int64_t)(UINT32_MAX / NT) * RPB;
  return launch_parts(i8_quantize_kernel<DT, GATED, L, U>, a, most, (int64_t)a.ldx * Raw<DT>::ES, NT, RPB, 1, s);
}

template <int DT, bool GATED>
hipError_t quantize_t(const I8QuantArgs& a, hipStream_t s) {
  if (a.cpr <= 8) return quantize_lu<DT, GATED, 8, 1>(a, s);
  if (a.cpr <= 16) return quantize_lu<DT, GATED, 16, 1>(a, s);
  if (a.cpr <= 32) return quantize_lu<DT, GATED, 32, 1>(a, s);
  if (a.cpr <= 64) return quantize_lu<DT, GATED, 64, 1>(a, s);
  if (a.cpr <= 128) return quantize_lu<DT, GATED, 64, 2>(a, s);
  if (a.cpr <= 256) return quantize_lu<DT, GATED, 64, 4>(a, s);
  if (a.cpr <= 512) return quantize_lu<DT, GATED, 256, 2>(a, s);
  if (a.cpr <= 1024) return quantize_lu<DT, GATED, 256, 4>(a, s);
  if (a.cpr <= 2048) return quantize_lu<DT, GATED, 256, 8>(a, s);
  return quantize_lu<DT, GATED, 1024, 8>(a, s);
}

template <int DT, int U>
hipError_t dequantize_u(const I8QuantArgs& a, hipStream_t s) {
  const int64_t most = (int64_t)(UINT32_MAX / 256) * 256 * U / a.cpr;
  return launch_parts(i8_dequantize_kernel<DT, U>, a, most, (int64_t)a.ldx * Raw<DT>::ES, 256, 256 * U, a.cpr, s);
}
template <int DT>
hipError_t dequantize_t(const I8QuantArgs& a, int cus, hipStream_t s) {
  const bool many = (int64_t)a.R * a.cpr >= (int64_t)cus * 8 * 4 * 256;
  return many ? dequantize_u<DT, 4>(a, s) : dequantize_u<DT, 1>(a, s);
}

}  // namespace

hipError_t launch_i8_quantize(const I8QuantArgs& a, int x_type, bool swiglu, hipStream_t s) {
  switch (x_type) {
    case DT_F32: return swiglu ? quantize_t<DT_F32, true>(a, s) : quantize_t<DT_F32, false>(a, s);
    case DT_F16: return swiglu ? quantize_t<DT_F16, true>(a, s) : quantize_t<DT_F16, false>(a, s);
    case DT_BF16: return swiglu ? quantize_t<DT_BF16, true>(a, s) : quantize_t<DT_BF16, false>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_i8_dequantize(const I8QuantArgs& a, int x_type, int cus, hipStream_t s) {
  switch (x_type) {
    case DT_F32: return dequantize_t<DT_F32>(a, cus, s);
    case DT_F16: return dequantize_t<DT_F16>(a, cus, s);
    case DT_BF16: return dequantize_t<DT_BF16>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
