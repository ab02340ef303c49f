// Rows of values taken in units of eight elements, as the quantise kernels and the experts' combination read them.
#pragma once
#include "qg_args.hpp"
#include "qg_device.hpp"

namespace qg {

typedef i32x4 __attribute__((aligned(2))) i32x4_u2;

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

// Stores the first n of eight values, each rounded once (RNE) to the type; p is aligned to 16 bytes.
// 16-bit values past the L2 where NT (a result many times what it holds); fp32 values through it: each of the
// two accesses fills half of every line, and it merges them.
template <int DT, bool NT>
__device__ __forceinline__ void store8(char* p, const float (&v)[8], int n) {
  if constexpr (DT == DT_F32) {
    float* y = (float*)p;
    if (n >= 8) {
      ((f32x4*)y)[0] = f32x4{v[0], v[1], v[2], v[3]};
      ((f32x4*)y)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) y[j] = v[j];
    }
  } else {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = DT == DT_BF16 ? f32_to_bf16_bits(v[j]) : f32_to_f16_bits(v[j]);
    if (n >= 8) {
      const i32x4 q = {(int)(h[0] | h[1] << 16), (int)(h[2] | h[3] << 16), (int)(h[4] | h[5] << 16),
                       (int)(h[6] | h[7] << 16)};
      if constexpr (NT)
        __builtin_nontemporal_store(q, (i32x4*)p);
      else
        *(i32x4*)p = q;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) ((uint16_t*)p)[j] = (uint16_t)h[j];
    }
  }
}

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

}  // namespace qg
