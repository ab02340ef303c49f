// Int8 quantise and dequantise kernels: one scale per row.
//
// A row of y (the row itself, or silu(gate) * up) with largest magnitude amax
// has the scale s = fp32(amax / 127) and the codes rne(y / s), both as 64-bit
// arithmetic gives them: a row's maximum has to be known before its first
// code, so a row is read once into registers (up to 65536 elements: 1024 lanes
// of 64) and its codes leave from there.
//
// fp32 decides what it can. With t = v * (1 / s), where v is the fp32 value,
// the code is rint(t) unless t is within its error of a half: then that
// element alone is done again in 64 bits, from memory (the caches have it), and
// stored over the first code. The error of t: identity 2^-23 t. SwiGLU: v = (g u) rcp(1 +
// exp2(-g log2 e)): the argument of exp2 is off by 1.25 * 2^-24 of itself (the product's rounding,
// the constant's), so e by |g| 1.25 * 2^-24 of itself, the other steps by 8 * 2^-24 (exp2 and rcp
// 2^-23 each, the sum, three products), 1 / s and its product by 2^-23: within 2^-19 for
// g >= -8 and 2^-17 for g >= -32 (below that exp2 may overflow: always in 64 bits). The maximum of a
// gated row is taken in 64 bits too, over the elements whose v is within 2^-16 of the largest v. Rows whose
// largest v is not finite, or so small that v or the scale may have lost bits (below 2^-60), go
// through 64 bits as a whole.
//
// Bound by memory. Measured, bf16: 8192 x 14336 gated 124 to 128 us (587 MB, 4.7 TB/s; a copy of 1 GiB reaches 5.15), 8192 x
// 7168 gated 56 (5.2), 8192 x 14336 63 (5.6), 4096 rows gathered to 32768 x 7168 97 to 102 (each row read eight times, 705 MB
// through the memory-side cache; its own 294 MB would take 63), the same codes back to values 117 to 125 (5.7 to 6.0 TB/s;
// the 470 MB written alone would take 107 at the rate that a copy's writes reach), one row of 4096 2.2 to 2.6 us and 1.7 to 1.9 back.
#include "qg_i8_quant.hpp"

#include <algorithm>

#include "qg_rows.hpp"

namespace qg {

namespace {

// Element k of y in 64 bits, from memory.
template <int DT, bool GATED>
__device__ __forceinline__ double value64(const char* row, int K, int k) {
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
// U units of 8 elements each. (512 gated lanes: registers for two workgroups per CU, which load in turn.)
template <int DT, bool GATED, int L, int U>
__global__ __launch_bounds__(L < 256 ? 256 : L, GATED && L == 512 ? 4 : 1) void i8_quantize_kernel(const I8QuantArgs a) {
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
  // what is held of a row: its elements as loaded, or y in fp32 with each unit's lowest gate
  Raw<DT> in[U];
  float v[GATED ? U : 1][8], low[GATED ? U : 1];
  uint32_t most[U], top = 0;  // largest |y| of a unit, of the row (as bits: a NaN is more than everything)
  static_assert(U <= 8, "a bit per element");
  // the element of the lowest bit of `todo`, which is cleared: bit 8 i + j is the lane's unit i, element j
  const auto element = [&](uint64_t& todo) {
    const int b = __builtin_ctzll(todo);
    todo &= todo - 1;
    return ((b >> 3) * L + l) * 8 + (b & 7);
  };
  const auto val = [&](int i, int j) { return GATED ? v[GATED ? i : 0][j] : in[i].at(j); };
  {
    Raw<DT> up[GATED ? U : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = (i * L + l) * 8, n = there ? a.K - k : 0;
      in[i].template load<true>(x + (int64_t)k * Raw<DT>::ES, n);
      if constexpr (GATED) up[i].template load<false>(x + ((int64_t)a.K + k) * Raw<DT>::ES, n);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if constexpr (GATED) {
        low[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float g = in[i].at(j);
          v[i][j] = g * up[i].at(j) * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
          low[i] = fminf(low[i], g);
        }
      }
      most[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) most[i] = max(most[i], __builtin_bit_cast(uint32_t, val(i, j)) & 0x7FFFFFFFu);
      top = max(top, most[i]);
    }
  }
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
    // in 64 bits over the elements that may be the largest
    const uint32_t near = slow ? 0u : top == 0 ? ~0u : __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, top) * (1.f - 0x1p-16f));
    uint64_t todo = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      uint32_t bits = low[i] < -32.f ? 0xFF : 0;
      if (most[i] >= near) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((__builtin_bit_cast(uint32_t, v[i][j]) & 0x7FFFFFFFu) >= near) bits |= 1u << j;
      }
      todo |= (uint64_t)bits << (8 * i);
    }
    double m = 0;
    bool bad = false;
    while (todo) {
      const int k = element(todo);
      if (!there || k >= a.K) continue;
      const double y = fabs(value64<DT, GATED>(x, a.K, k));
      bad |= !(y <= 1.7976931348623157e308);
      m = fmax(m, y);
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
  uint64_t todo = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int k = (i * L + l) * 8, n = live ? a.K - k : 0;
    // a code is the low byte of v / s + 1.5 * 2^23, which rounds to an integer (ties to even)
    constexpr float kRound = 12582912.f;
    const float off = !GATED ? 0x1p-22f : low[GATED ? i : 0] < -8.f ? 0x1p-17f : 0x1p-19f;
    uint32_t c[8], q[2];
    float worst = 0.f;
    const auto doubt = [&](int j, uint32_t& code) {
      // (fmas spelled out: both evaluations of an element are the same)
      const float x = val(i, j), r = __builtin_fmaf(x, inv, kRound);
      code = __builtin_bit_cast(uint32_t, r);
      return __builtin_fmaf(fabsf(x * inv), off, fabsf(__builtin_fmaf(x, inv, kRound - r)));
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) worst = fmaxf(worst, doubt(j, c[j]));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      q[h] = zero ? 0
                  : __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x0C0C0400u),
                                          __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0C0C0400u), 0x05040100u);
    uint32_t bits = slow || (GATED && low[GATED ? i : 0] < -32.f) ? 0xFF : 0;
    if (worst >= 0.5f) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (doubt(j, c[j]) >= 0.5f) bits |= 1u << j;
    }
    todo |= (uint64_t)bits << (8 * i);
    char* p = a.Q + row * a.ldq + k;
    if (n >= 8) {
      *(uint64_t*)p = (uint64_t)q[1] << 32 | q[0];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = (char)(q[j / 4] >> (8 * (j & 3)));
    }
  }
  // the codes in doubt again, over those that just went out
  if (zero || !there) todo = 0;
  while (todo) {
    const int k = element(todo);
    if (k < a.K) a.Q[row * a.ldq + k] = (char)(int)fmin(fmax(rint(value64<DT, GATED>(x, a.K, k) / (double)s), -127.0), 127.0);
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

// Lanes per row and units per lane, so that a row just fits: a lane of one wave has up to four units, of several up to four
// too, of 1024 lanes eight. bf16, 8192 rows gated, K 14336: 124 us with 512 lanes of four units (two such workgroups per CU;
// 176 with the registers that one takes), 168 with 256 of eight, 193 with 1024 of two. 32768 rows gathered, K 7168, one after the
// other: 107 to 116 with 256 of four, 133 with one wave of 16, 112 with two of eight; 125 with the next row's loads ahead of this one's work.
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
  if (a.cpr <= 2048) return quantize_lu<DT, GATED, 512, 4>(a, s);
  if (a.cpr <= 4096) return quantize_lu<DT, GATED, 1024, 4>(a, s);
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
