// MXFP4 quantise and dequantise kernels.
//
// A block of 32 values along K shares the scale 2^(floor(log2 amax) - 2) (E8M0
// byte: amax's exponent field less 2); a value over the scale is rounded to
// the nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to even, past 6 to
// 6. Scaling by a power of two is exact, so a code is one rounding of the
// value, done by v_cvt_scalef32_pk_fp4_f32.
//
// Both kernels are bound by memory: an element costs its own 2 or 4 bytes
// and 17/32 byte of MXFP4. One lane takes a unit of 8 consecutive elements
// (one 16-byte access of 16-bit values, one dword of codes), the four lanes
// of a quad take one block, so the block maximum is two DPP exchanges and
// nothing goes through LDS. Units are numbered row after row, whatever K is, so
// that a wave is full at any width; a workgroup does one division to find its
// first row and its lanes one multiplication each. Measured, bf16: 8192 x 14336
// gated 99 us (532 MB, 5.4 TB/s; a copy of 1 GiB reaches 5.15), 4096 rows
// gathered to 32768 x 7168 91 us (each row read eight times, mostly from the
// caches; its own 184 MB would take 36; gated 162), the same codes back to
// values 84 us (594 MB, 7 TB/s: the codes come from the memory-side cache), one
// row of 4096 2 us each way.
//
// SwiGLU: the codes are those of silu(g) * u without rounding before them, so
// fp32 arithmetic alone would put values next to a rounding border on its
// wrong side (about one in 10^6). The fp32 value v = (g u) rcp(1 + e), where
// it is normal, is within 2^-18 of the exact one (for g >= -32: the argument of
// exp2 is off by at most 48 * 2^-24, the other steps by a few 2^-23; g u, no
// smaller than v, is normal too, where g rcp(1 + e) need not be). Each lane
// rounds v (1 - 2^-17) and v (1 + 2^-17)
// instead of v: equal codes are the exact value's code. Where they differ, or
// the block maximum is as near a power of two, or fp32's range or the bound
// does not hold, the wave redoes its units in 64 bits. (A v below fp32's normal
// range is a zero code in any block that is not redone: those reach 2^-60.)
// Normal values ask for it so seldom that it does not show beside the memory;
// with one gate in 10^4 below -32 (a wave in 20) 8192 x 14336 takes 106 us,
// with one in 1000 175 and once every wave is redone 290.
#include "qg_mx_quant.hpp"

#include <algorithm>

#include "qg_args.hpp"
#include "qg_device.hpp"

namespace qg {

namespace {

constexpr int kThreads = 256;

typedef i32x4 __attribute__((aligned(2))) i32x4_u2;

// Rounds two values (already over their scale) to E2M1 codes in byte SEL of a dword.
template <int SEL>
__device__ __forceinline__ uint32_t cvt_fp4(uint32_t old, float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, 1.0f, SEL);
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float m) {
  uint32_t q = 0;
  q = cvt_fp4<0>(q, v[0] * m, v[1] * m);
  q = cvt_fp4<1>(q, v[2] * m, v[3] * m);
  q = cvt_fp4<2>(q, v[4] * m, v[5] * m);
  q = cvt_fp4<3>(q, v[6] * m, v[7] * m);
  return q;
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return x;
}

// Eight elements as loaded: one 16-byte chunk of 16-bit values or two of fp32.
template <int DT>
struct Raw {
  static constexpr int ES = DT == DT_F32 ? 4 : 2;
  i32x4 d[DT == DT_F32 ? 2 : 1];
  // n of the eight exist (the rest read as zero); p is aligned to 16 bytes
  // where AL, else to the element
  template <bool AL>
  __device__ __forceinline__ void load(const char* p, int n) {
    if (n >= 8) {
#pragma unroll
      for (int i = 0; i < ES / 2; ++i) d[i] = AL ? ((const i32x4*)p)[i] : ((const i32x4_u2*)p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < ES / 2; ++i) d[i] = i32x4{};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          if constexpr (ES == 4)
            d[j / 4][j % 4] = ((const int*)p)[j];
          else
            d[0][j / 2] |= (int)((uint32_t)((const uint16_t*)p)[j] << (16 * (j & 1)));
        }
    }
  }
  __device__ __forceinline__ float at(int j) const {
    // (a copy: a bit cast of a vector's element itself would take element 0)
    const uint32_t w = (uint32_t)(DT == DT_F32 ? d[j / 4][j % 4] : d[0][j / 2]);
    if constexpr (DT == DT_F32) return __builtin_bit_cast(float, w);
    if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, j & 1 ? w & 0xFFFF0000u : w << 16);
    return f16_bits_to_f32((uint16_t)(j & 1 ? w >> 16 : w));
  }
};

// Row and unit-in-row of unit `first + off` (off < 2^16): `first` is
// workgroup-uniform, so its division is done once.
struct Place {
  int64_t row;
  int unit;
};
struct Places {
  int64_t row0;
  uint32_t u0, cpr, magic;
  __device__ __forceinline__ Places(int64_t first, int cpr_) : cpr((uint32_t)cpr_) {
    row0 = first < (int64_t(1) << 32) ? (int64_t)((uint32_t)first / cpr) : first / cpr_;
    u0 = (uint32_t)(first - row0 * cpr_);
    // n / cpr = (n * magic) >> 32 is exact for n * cpr < 2^32; a workgroup
    // crosses at most one row's end where rows have 2^15 units or more
    magic = cpr > 1 ? 0xFFFFFFFFu / cpr + 1 : 0;
  }
  __device__ __forceinline__ Place at(uint32_t off) const {
    uint32_t n = u0 + off, q;
    if (cpr >= (1u << 15)) {
      q = n >= cpr;
    } else {
      q = cpr == 1 ? n : __umulhi(n, magic);
    }
    return Place{row0 + q, (int)(n - q * cpr)};
  }
};

// Codes (low half) and scale byte (high half) of eight values silu(g) u, in 64
// bits. Called by whole waves: the block's maximum is taken over the quad.
template <int DT>
__device__ __attribute__((noinline)) uint64_t swiglu_codes64(Raw<DT> g, Raw<DT> u) {
  double v[8], top = 0;
  int bad = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double x = g.at(j);
    v[j] = x / (1.0 + exp(-x)) * (double)u.at(j);
    const double m = fabs(v[j]);
    bad |= !(m <= 1.7976931348623157e308);
    top = m > top ? m : top;
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const double o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
    bad |= __shfl_xor(bad, d, 64);
  }
  if (bad) return (uint64_t)255 << 32;
  const int e = (int)((__builtin_bit_cast(uint64_t, top) >> 52) & 0x7FF) - 1023 - 2 + 127;
  const int byte = max(0, min(254, e));
  const double inv = __builtin_bit_cast(double, (uint64_t)(127 - byte + 1023) << 52);
  uint32_t q = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double t = fabs(v[j]) * inv;
    // even codes take the ties: <= below them, < above
    const uint32_t c = (t > 0.25) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0);
    // (the sign bit, as the 32-bit path has it: a -0 keeps its sign too)
    q |= (c | (uint32_t)(__builtin_bit_cast(uint64_t, v[j]) >> 63) << 3) << (4 * j);
  }
  return q | (uint64_t)byte << 32;
}

template <int DT, bool GATED, int U>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const MxQuantArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * U);
  const Places places(first, a.cpr);
  Raw<DT> x[U], up[GATED ? U : 1];
  Place at[U];
  bool live[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t off = i * kThreads + threadIdx.x;
    live[i] = first + off < (int64_t)a.R * a.cpr;  // the same for a whole quad: units come in fours
    at[i] = places.at(off);
    int64_t src = at[i].row;
    if (a.rows && live[i]) src = a.rows[at[i].row];
    const int k = at[i].unit * 8;
    const int n = live[i] && src >= 0 && src < a.T ? a.K - k : 0;
    const char* p = (const char*)a.X + (src * (int64_t)a.ldx + k) * Raw<DT>::ES;
    x[i].template load<true>(p, n);
    if constexpr (GATED) up[i].template load<false>(p + (int64_t)a.K * Raw<DT>::ES, n);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float v[8];
    uint32_t top = 0, q;
    int byte;
    bool redo = false;
    float low = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = x[i].at(j);
      if constexpr (GATED) {
        low = fminf(low, v[j]);
        const float e = __builtin_amdgcn_exp2f(v[j] * -1.44269504f);
        v[j] = v[j] * up[i].at(j) * __builtin_amdgcn_rcpf(1.f + e);
      }
      top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
    }
    top = quad_max(top);
    byte = max((int)(top >> 23) - 2, 0);
    const float inv = __builtin_bit_cast(float, (uint32_t)(254 - min(byte, 252)) << 23);
    if constexpr (GATED) {
      constexpr float kOff = 0x1p-17f;
      q = codes8(v, inv * (1.f - kOff));
      const float t = __builtin_bit_cast(float, top);
      redo = codes8(v, inv * (1.f + kOff)) != q || top >= 0x7F000000u || (top != 0 && t < 0x1p-60f) || low < -32.f ||
             (__builtin_bit_cast(uint32_t, t * (1.f - kOff)) ^ __builtin_bit_cast(uint32_t, t * (1.f + kOff))) >> 23;
      if (__any(redo)) {
        const uint64_t r = swiglu_codes64<DT>(x[i], up[i]);
        q = (uint32_t)r;
        byte = (int)(r >> 32);
      }
    } else {
      q = codes8(v, inv);
      if (top >= 0x7F800000u) q = 0, byte = 255;
    }
    if (live[i]) {
      *(uint32_t*)(a.Q + at[i].row * a.ldq + at[i].unit * 4) = q;
      if ((threadIdx.x & 3) == 0) a.S[at[i].row * a.lds + (at[i].unit >> 2)] = (char)byte;
    }
  }
}

// 16-bit values go out past the L2 (non-temporal): they are many times what it
// holds, and it keeps the codes that are still to be read instead.
template <int DT, int U>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const MxQuantArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * U);
  const Places places(first, a.cpr);
  uint32_t q[U], s[U];
  Place at[U];
  bool live[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t off = i * kThreads + threadIdx.x;
    live[i] = first + off < (int64_t)a.R * a.cpr;
    at[i] = places.at(off);
    q[i] = s[i] = 0;
    if (live[i]) {
      q[i] = *(const uint32_t*)(a.Q + at[i].row * a.ldq + at[i].unit * 4);
      s[i] = (uint8_t)a.S[at[i].row * a.lds + (at[i].unit >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (!live[i]) continue;
    // 2^(s - 127): byte 0 is fp32's subnormal 2^-127, byte 255 NaN
    const float scale = __builtin_bit_cast(float, s[i] == 255 ? 0x7FC00000u : s[i] ? s[i] << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 y = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i] >> (8 * h), 1.0f, 0);
      v[2 * h] = y[0] * scale;
      v[2 * h + 1] = y[1] * scale;
    }
    const int k = at[i].unit * 8;
    const int64_t base = at[i].row * a.ldx + k;
    if constexpr (DT == DT_F32) {
      float* y = (float*)a.X + base;
      if (k + 8 <= a.K) {
        // two accesses that each fill half of every line: merged in the L2
        ((f32x4*)y)[0] = f32x4{v[0], v[1], v[2], v[3]};
        ((f32x4*)y)[1] = f32x4{v[4], v[5], v[6], v[7]};
      } else {
        for (int j = 0; j < 8; ++j)
          if (k + j < a.K) y[j] = v[j];
      }
    } else {
      uint16_t* y = (uint16_t*)a.X + base;
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = DT == DT_BF16 ? f32_to_bf16_bits(v[j]) : f32_to_f16_bits(v[j]);
      if (k + 8 <= a.K) {
        const i32x4 p = {(int)(h[0] | h[1] << 16), (int)(h[2] | h[3] << 16), (int)(h[4] | h[5] << 16),
                         (int)(h[6] | h[7] << 16)};
        __builtin_nontemporal_store(p, (i32x4*)y);
      } else {
        for (int j = 0; j < 8; ++j)
          if (k + j < a.K) y[j] = (uint16_t)h[j];
      }
    }
  }
}

// A dispatch counts its threads in 32 bits, and a launch of more loses the rest without an error: rows go
// out in parts of fewer (a row always fits).
template <class Kernel>
hipError_t launch_parts(Kernel kernel, const MxQuantArgs& a, int per_lane, int64_t value_pitch, hipStream_t s) {
  const int64_t most = (int64_t)(UINT32_MAX / kThreads) * kThreads * per_lane / a.cpr;
  for (int64_t r = 0; r < a.R; r += most) {
    MxQuantArgs p = a;
    p.R = (int32_t)std::min<int64_t>(most, a.R - r);
    p.Q = a.Q + r * a.ldq;
    p.S = a.S + r * a.lds;
    if (a.rows) {
      p.rows = a.rows + r;
    } else {
      p.X = (char*)a.X + r * value_pitch;
      p.T = p.R;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)mx_quant_blocks((int64_t)p.R * a.cpr, per_lane)), dim3(kThreads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, bool GATED, int U>
hipError_t quantize_u(const MxQuantArgs& a, hipStream_t s) {
  return launch_parts(mx_quantize_kernel<DT, GATED, U>, a, U, (int64_t)a.ldx * Raw<DT>::ES, s);
}
// Several units per lane, for more loads in flight, once that still leaves
// every CU eight workgroups; one below, so that few rows spread wide. 4096 rows
// gathered to 32768 x 7168 and back: 178 us with four units both ways, 183 with
// two, 209 with one; 8192 x 14336 gated and back: 149 us with two, 151 to 155 with one.
bool several(const MxQuantArgs& a, int cus, int per_lane) { return (int64_t)a.R * a.cpr >= (int64_t)cus * 8 * per_lane * kThreads; }

template <int DT>
hipError_t quantize_t(const MxQuantArgs& a, bool swiglu, int cus, hipStream_t s) {
  if (swiglu) return several(a, cus, 2) ? quantize_u<DT, true, 2>(a, s) : quantize_u<DT, true, 1>(a, s);
  return several(a, cus, 4) ? quantize_u<DT, false, 4>(a, s) : quantize_u<DT, false, 1>(a, s);
}
template <int DT, int U>
hipError_t dequantize_u(const MxQuantArgs& a, hipStream_t s) {
  return launch_parts(mx_dequantize_kernel<DT, U>, a, U, (int64_t)a.ldx * Raw<DT>::ES, s);
}
template <int DT>
hipError_t dequantize_t(const MxQuantArgs& a, int cus, hipStream_t s) {
  return several(a, cus, 4) ? dequantize_u<DT, 4>(a, s) : dequantize_u<DT, 1>(a, s);
}

}  // namespace

int64_t mx_quant_blocks(int64_t units, int per_lane) { return (units + kThreads * per_lane - 1) / (kThreads * per_lane); }

hipError_t launch_mx_quantize(const MxQuantArgs& a, int x_type, bool swiglu, int cus, hipStream_t s) {
  switch (x_type) {
    case DT_F32: return quantize_t<DT_F32>(a, swiglu, cus, s);
    case DT_F16: return quantize_t<DT_F16>(a, swiglu, cus, s);
    case DT_BF16: return quantize_t<DT_BF16>(a, swiglu, cus, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, int x_type, int cus, hipStream_t s) {
  switch (x_type) {
    case DT_F32: return dequantize_t<DT_F32>(a, cus, s);
    case DT_F16: return dequantize_t<DT_F16>(a, cus, s);
    case DT_BF16: return dequantize_t<DT_BF16>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
