// Choice of experts: a wave per token, or four tokens per wave where they are many.
//
// Score p = softmax(x) or sigmoid(x); key = p + bias, or x itself where there is
// no bias (the same order, and exact). A group's standing is its best key or
// the sum of its two best; the best groups keep their experts; the K best
// keys are chosen, ties to the lowest index.
//
// A lane holds NV consecutive experts of one group, so that lane order is
// index order, a group is an aligned run of lanes, and the lowest lane of a
// ballot is the lowest index. A round of the choice is a maximum of the
// keys as ordered integers over the token's lanes (DPP), a ballot for its place, and the removal of that key.
// 16384 tokens over 256 experts read 17 MB (2.7 us), and take 8.3 us where the logits alone decide, 14 to 16 with a
// bias, 18 to 20 with groups too, tokens in doubt included (about 5 us for each, among others). Of the 18 us each SIMD's
// vector instructions (5500 of four cycles) take half; the rest is latency that its four waves do not cover.
//
// Keys are those of 64-bit arithmetic: fp32 decides where two neighbours in the
// order (or the groups on both sides of the cut) are further apart than the
// errors of their keys, or have the same key (equal logit, equal bias); a
// token where they are not is done again in 64 bits, by its wave. At the cut
// the last one chosen has to stand above everything that is left out, whose
// errors may be larger than that of the first of them; where that one has the same
// logit and bias, above the best of those that have not. Errors of an
// fp32 score, relative, in 2^-23, exp2 and rcp being good to 1 each: e^x is off
// by 0.61 |x| (the product's rounding, the constant's) + 1. Sigmoid: (1 - s) of that (what
// e does to 1 / (1 + e)), 0.5 for the sum, 1 for rcp: at most 4 + |x| (1 - s). Softmax: its
// own e^x and the sum's (weighted, so less than the largest |x| e^x, under 0.4), 11 for the
// sum's 22 roundings (16 serially, then a tree), 2 for rcp and the product: at most 16 + 1.5 |x|.
#include "qg_experts.hpp"

#include <algorithm>

#include "qg_args.hpp"
#include "qg_device.hpp"

namespace qg {

namespace {

constexpr float kLog2e = 1.44269504f;
constexpr float kMinusInf = -__builtin_inff();

// x of the lanes that DPP control CTRL shifts in, `none` where there is none
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, 0xF, 0xF, false);
}
// Row shifts by 1, 2, 4, 8, then the broadcasts of lane 15 and lane 31: lane 63 has seen every lane.
template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t none, uint32_t x, F f) {
  x = f(x, dpp<0x111>(none, x));
  x = f(x, dpp<0x112>(none, x));
  x = f(x, dpp<0x114>(none, x));
  x = f(x, dpp<0x118>(none, x));
  x = f(x, dpp<0x142>(none, x));
  x = f(x, dpp<0x143>(none, x));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return wave_reduce(0, x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
  const uint32_t high = wave_max((uint32_t)(x >> 32));
  return (uint64_t)high << 32 | wave_max((uint32_t)(x >> 32) == high ? (uint32_t)x : 0u);
}
// (row_bcast sums rows 0 and 1 into row 1, and so on: every lane's value is in lane 63's sum once)
__device__ __forceinline__ float wave_sum(float x) {
  return __builtin_bit_cast(float, wave_reduce(0, __builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
                              return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                            }));
}
__device__ __forceinline__ double wave_sum(double x) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// Integers in the order of the floating values (0 is below all of them; -0 and +0 are one).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

template <int DT>
__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
  if constexpr (DT == DT_F32) return ((const float*)a.X)[t * a.ldx + e];
  const uint16_t h = ((const uint16_t*)a.X)[t * a.ldx + e];
  return DT == DT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
}

// The `rounds` best keys (0: not there): lane r gets the expert of the r-th, -1 where fewer are there; the others stay in
// `key`. Few keys per lane are put in order first (`tag` holds a byte for each, its place in the lane), so that a round looks
// at the lanes' first keys only and the winner's others move up.
template <class Key, int NV>
__device__ __forceinline__ int choose(Key (&key)[NV], uint32_t& tag, int e0, int rounds, int& found) {
  constexpr bool kSorted = NV <= 4;
  const int lane = lane_id();
  tag = 0;
  if constexpr (kSorted) {
    uint32_t at[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) at[j] = j;
    const auto order = [&](int i, int j) {  // equal keys stay as they are: i is before j
      const bool swap = key[j] > key[i];
      const Key k = swap ? key[j] : key[i];
      key[j] = swap ? key[i] : key[j];
      key[i] = k;
      const uint32_t t = swap ? at[j] : at[i];
      at[j] = swap ? at[i] : at[j];
      at[i] = t;
    };
    // (neighbours only, so that no key passes an equal one)
#pragma unroll
    for (int n = NV - 1; n > 0; --n)
#pragma unroll
      for (int j = 0; j < n; ++j) order(j, j + 1);
#pragma unroll
    for (int j = 0; j < NV; ++j) tag |= at[j] << (8 * j);
  }
  int mine = -1;
  found = 0;
  for (int r = 0; r < rounds; ++r) {
    Key top = key[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int j = 1; j < NV; ++j) top = max(top, key[j]);
    }
    top = wave_max(top);
    if (top == 0) break;
    int w, e;
    if constexpr (kSorted) {
      w = __builtin_ctzll(__ballot(key[0] == top));
      e = __builtin_amdgcn_readlane(e0, w) + (__builtin_amdgcn_readlane((int)tag, w) & 0xFF);
      if (lane == w) {
#pragma unroll
        for (int j = 0; j + 1 < NV; ++j) key[j] = key[j + 1];
        key[NV - 1] = 0;
        tag >>= 8;
      }
    } else {
      uint64_t at[NV], any = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) any |= at[j] = __ballot(key[j] == top);
      w = __builtin_ctzll(any);
      int first = NV - 1;
#pragma unroll
      for (int j = NV - 2; j >= 0; --j)
        if (at[j] >> w & 1) first = j;
      e = __builtin_amdgcn_readlane(e0, w) + first;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane == w && j == first) key[j] = 0;
    }
    if (lane == r) mine = e;
    ++found;
  }
  return mine;
}

// A lane's group standing from its own keys' two best, over the run of lanes that holds the group.
template <class F>
__device__ __forceinline__ F standing(F b1, F b2, int shift, bool best2) {
  for (int d = 1; d < 1 << shift; d <<= 1) {
    const F o1 = __shfl_xor(b1, d, 64), o2 = __shfl_xor(b2, d, 64);
    const F low = b1 < o1 ? b1 : o1;
    b1 = b1 < o1 ? o1 : b1;
    b2 = b2 < o2 ? o2 : b2;
    b2 = b2 < low ? low : b2;
  }
  return best2 && b2 > (F)kMinusInf ? b1 + b2 : b1;
}

// The choice in 64 bits. Logits are read again where they are needed: this seldom runs, and its registers are the kernel's.
template <int DT, int NV>
__device__ __attribute__((noinline)) int choose64(const RouteArgs a, int shift, int64_t t, int e0, int count, int& found) {
  const auto get = [&](int j) -> double {
    const double x = j < count ? logit<DT>(a, t, e0 + j) : kMinusInf;
    return x > kMinusInf ? x : (double)kMinusInf;
  };
  double m = kMinusInf, sum = 1;
  if (!(a.flags & ROUTE_SIGMOID)) {
    for (int j = 0; j < count; ++j) m = fmax(m, get(j));
    for (int d = 1; d < 64; d <<= 1) m = fmax(m, __shfl_xor(m, d, 64));
  }
  const auto score = [&](double x) -> double {
    if (a.flags & ROUTE_SIGMOID) return 1.0 / (1.0 + exp(-x));
    return !(x > kMinusInf) ? 0.0 : x == m ? 1.0 : exp(x - m);
  };
  if (!(a.flags & ROUTE_SIGMOID)) {
    sum = 0;
    for (int j = 0; j < count; ++j) sum += score(get(j));
    sum = wave_sum(sum);
  }
  uint64_t key[NV];
  double b1 = kMinusInf, b2 = kMinusInf;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const double x = get(j);
    double s = score(x) / sum, k = x;
    if (a.bias && j < count) k = s += a.bias[e0 + j];
    const bool there = x > kMinusInf && k > kMinusInf;
    key[j] = there ? ordered(k) : 0;
    if (!(a.flags & ROUTE_BEST2)) s = k;
    if (!there) s = kMinusInf;
    b2 = s > b1 ? b1 : s > b2 ? s : b2;
    b1 = s > b1 ? s : b1;
  }
  if (a.groups > 1) {
    const double st = standing(b1, b2, shift, (a.flags & ROUTE_BEST2) != 0);
    const int mine = lane_id() >> shift;
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(st, g << shift, 64);
      before += o > st || (o == st && g < mine);
    }
    if (before >= a.kept) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = 0;
    }
  }
  uint32_t tag;
  return choose(key, tag, e0, a.K, found);
}

// What the fp32 path knows of a token's scores.
struct Scores {
  bool sigmoid;
  float m = kMinusInf, total = 1.f;  // softmax: largest logit, 1 / sum
  // (without the softmax's 1 / sum)
  __device__ __forceinline__ float raw(float x) const {
    if (sigmoid) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -kLog2e));
    return x == m ? 1.f : __builtin_amdgcn_exp2f((x - m) * kLog2e);
  }
  // how far score s of logit x plus a bias, together k, may be off
  __device__ __forceinline__ float error(float x, float s, float k) const {
    const float rel = sigmoid ? 4.f + fminf(fabsf(x), 128.f) * (1.f - s) : 16.f + (x == m ? 0.f : 1.5f * fminf(m - x, 128.f));
    return (s * rel + fabsf(k)) * 0x1p-23f + 0x1p-120f;
  }
  // The same for every key of up to k, whatever its score: s rel is at most 4.3 for a sigmoid and 16 of the largest
  // score for a softmax, and k + |k| 2^-23 grows with k.
  __device__ __forceinline__ float error_up_to(float k) const {
    return ((sigmoid ? 5.f : 17.f * total) + fabsf(k)) * 0x1p-23f + 0x1p-120f;
  }
};
// How far the standings of two groups may be off together. With a bias: two scores each (at most 5, or 16, times
// 2^-23), and the roundings of four keys of up to `most` and two sums. Without: scores of up to e^-88 (smaller
// ones are zero), relative to standing st.
__device__ __forceinline__ float standing_error(bool bias, bool sigmoid, float st, float most) {
  return bias ? (sigmoid ? 0x1p-18f : 0x1p-17f) + most * 0x1p-21f : st * 0x1p-14f + 0x1p-120f;
}
// The magnitude of a key, as bits.
__device__ __forceinline__ uint32_t size_of(uint32_t key) {
  return key ? __builtin_bit_cast(uint32_t, unordered(key)) & 0x7FFFFFFFu : 0;
}

template <int DT, int NV>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs a) {
  const int lane = lane_id();
  const int run = 1 << a.shift, g = lane >> a.shift, e0 = g * a.per + (lane & (run - 1)) * NV;
  const int count = g < a.groups ? max(0, min(NV, a.per - (lane & (run - 1)) * NV)) : 0;
  const bool sigmoid = a.flags & ROUTE_SIGMOID, best2 = a.flags & ROUTE_BEST2, renorm = a.flags & ROUTE_RENORM;
  const bool scores = a.bias || best2;  // the choice looks at the scores, not the logits alone
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave_id(); t < a.T; t += (int64_t)gridDim.x * 4) {
    float x[NV];
    Scores sc{sigmoid};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = kMinusInf;
      if (j < count) x[j] = logit<DT>(a, t, e0 + j);
      if (!(x[j] > kMinusInf)) x[j] = kMinusInf;  // NaN too
      sc.m = fmaxf(sc.m, x[j]);
    }
    float p[NV];
    if (!sigmoid && (scores || !renorm)) {
      const uint32_t k = wave_max(sc.m > kMinusInf ? ordered(sc.m) : 0);
      sc.m = k ? unordered(k) : kMinusInf;
      float sum = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) sum += p[j] = x[j] > kMinusInf ? sc.raw(x[j]) : 0.f;
      sc.total = __builtin_amdgcn_rcpf(wave_sum(sum));
    }
    uint32_t key[NV];
    float b1 = kMinusInf, b2 = kMinusInf;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float s = 0.f, k = x[j];
      if (scores) s = sigmoid ? sc.raw(x[j]) : p[j] * sc.total;
      if (a.bias && j < count) k = s += a.bias[e0 + j];
      const bool there = x[j] > kMinusInf && k > kMinusInf;
      key[j] = there ? ordered(k) : 0;
      if (!best2) s = k;
      if (!there) s = kMinusInf;
      b2 = s > b1 ? b1 : fmaxf(s, b2);
      b1 = fmaxf(s, b1);
    }
    bool unsure = false;
    if (a.groups > 1) {
      const float st = standing(b1, b2, a.shift, best2);
      uint32_t most = 0;
      if (a.bias) {
#pragma unroll
        for (int j = 0; j < NV; ++j) most = max(most, size_of(key[j]));
        most = wave_max(most);
      }
      const float tol = standing_error(a.bias, sigmoid, st, __builtin_bit_cast(float, most));
      int sure = 0, maybe = 0;
      for (int o = 0; o < a.groups; ++o) {
        const float other = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, st), o << a.shift));
        const bool first = o < g;
        if (scores && st > kMinusInf) {
          sure += other > st + tol;
          maybe += o != g && !(other < st - tol);
        } else {
          const bool before = other > st || (other == st && first);
          sure += before;
          maybe += before;
        }
      }
      unsure = g < a.groups && maybe >= a.kept && sure < a.kept;
      if (maybe >= a.kept) {
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = 0;
      }
    }
    int found = 0, mine = -1;
    float l = 0.f;
    bool redo = __any(unsure);
    if (!redo) {
      uint32_t tag;
      mine = choose(key, tag, e0, a.bias ? a.K + 1 : a.K, found);
      if (mine >= 0) l = logit<DT>(a, t, mine);
      if (a.bias) {
        // every key against the next one (the last one chosen: against all that are left out): too near to call, and not
        // the same expert twice?
        const float b = mine >= 0 ? a.bias[mine] : 0.f, s = sc.raw(l) * sc.total, k = s + b, err = sc.error(l, s, k);
        const float ln = __shfl_down(l, 1, 64), bn = __shfl_down(b, 1, 64), kn = __shfl_down(k, 1, 64);
        const float ek = __shfl_down(err, 1, 64), en = lane == a.K - 1 ? sc.error_up_to(kn) : ek;
        const bool near = lane + 1 < found && !(k - kn > err + en), same = l == ln && b == bn;
        redo = __any(near && !same);
        // (a token's logits again, 0.5 us; without the look at which keys are equal experts' every such token would be redone:
        // 1024 x 256 in bf16 without biases 5.3 us, 8.5)
        if (__any(near && same && lane == a.K - 1)) {
          const float lk = __shfl(l, a.K - 1, 64), bk = __shfl(b, a.K - 1, 64);
          uint32_t left = 0;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int e = e0 + (NV <= 4 ? tag >> (8 * j) & 0xFF : j);
            if (key[j] != 0 && !(logit<DT>(a, t, e) == lk && a.bias[e] == bk)) left = max(left, key[j]);
          }
          left = wave_max(left);
          const float kl = unordered(left);
          redo |= __any(lane == a.K - 1 && left != 0 && !(k - kl > err + sc.error_up_to(kl)));
        }
      }
    }
    if (redo) {
      mine = choose64<DT, NV>(a, a.shift, t, e0, count, found);
      if (mine >= 0) l = logit<DT>(a, t, mine);
    }
    const bool have = mine >= 0 && lane < a.K;
    float w = have ? sc.raw(l) * sc.total : 0.f;
    if (renorm) {
      float sum = wave_sum(sigmoid ? w : 0.f);
      if (!sigmoid || sum < 0x1p-80f) {
        // relative to the best of the chosen: softmax by its definition, sigmoids as small as that within 2^-80 of it
        const uint32_t k = wave_max(have ? ordered(l) : 0);
        const float best = k ? unordered(k) : 0.f;
        w = !have ? 0.f : l == best ? 1.f : __builtin_amdgcn_exp2f((l - best) * kLog2e);
        sum = wave_sum(w);
      }
      w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < a.K) {
      a.ids[t * a.ldi + lane] = have ? mine : -1;
      a.W[t * a.ldw + lane] = have ? w * a.scale : 0.f;
    }
  }
}

// Maximum and sum over a row of 16 lanes, in every lane of it.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, dpp<0x128>(0, x));
  x = max(x, dpp<0x124>(0, x));
  x = max(x, dpp<0x122>(0, x));
  return max(x, dpp<0x121>(0, x));
}
__device__ __forceinline__ float row_sum(float x) {
  const auto add = [](float v, uint32_t o) { return v + __builtin_bit_cast(float, o); };
  x = add(x, dpp<0x128>(0, __builtin_bit_cast(uint32_t, x)));
  x = add(x, dpp<0x124>(0, __builtin_bit_cast(uint32_t, x)));
  x = add(x, dpp<0x122>(0, __builtin_bit_cast(uint32_t, x)));
  return add(x, dpp<0x121>(0, __builtin_bit_cast(uint32_t, x)));
}

// Many tokens: four per wave, a row of 16 lanes each, so that a round of the choice serves four tokens and its
// reductions are four row rotations. A lane's NV keys are lists of four, each in order; a round looks at their heads. Fewer
// than 16 choices, groups that fit into 16 lanes (a.shift is the row's: log2 of a group's lanes among 16).
template <int DT, int NV>
__global__ __launch_bounds__(256) void route_rows_kernel(const RouteArgs a) {
  constexpr int NL = NV / 4;
  __shared__ int16_t chosen[16][16];  // by token of the workgroup and rank
  const int lane = lane_id(), l = lane & 15, at = threadIdx.x >> 4;
  const int run = 1 << a.shift, g = l >> a.shift, e0 = g * a.per + (l & (run - 1)) * NV;
  const int64_t t = (int64_t)blockIdx.x * 16 + at;
  const int count = g < a.groups && t < a.T ? max(0, min(NV, a.per - (l & (run - 1)) * NV)) : 0;
  const bool sigmoid = a.flags & ROUTE_SIGMOID, best2 = a.flags & ROUTE_BEST2, renorm = a.flags & ROUTE_RENORM;
  const bool scores = a.bias || best2;
  uint32_t key[NV];
  Scores sc{sigmoid};
  float b1 = kMinusInf, b2 = kMinusInf;
  {
    float x[NV], p[NV], add[NV];
    const char* row = (const char*)a.X + (t * a.ldx + e0) * (DT == DT_F32 ? 4 : 2);
    // whole lanes of aligned experts: 16-byte loads
    const bool wide = count == NV && ((a.per * (DT == DT_F32 ? 4 : 2)) & 15) == 0 && NV * (DT == DT_F32 ? 4 : 2) >= 16;
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = kMinusInf;
    if (wide) {
      if constexpr (DT == DT_F32) {
#pragma unroll
        for (int j = 0; j < NV; j += 4) {
          const f32x4 v = ((const f32x4*)row)[j / 4];
          x[j] = v[0], x[j + 1] = v[1], x[j + 2] = v[2], x[j + 3] = v[3];
        }
      } else if constexpr (NV >= 8) {
#pragma unroll
        for (int j = 0; j < NV; j += 8) {
          const i32x4 v = ((const i32x4*)row)[j / 8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t d = (uint32_t)v[i / 2];
            const uint16_t h = (uint16_t)(i & 1 ? d >> 16 : d);
            x[j + i] = DT == DT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j < count) x[j] = logit<DT>(a, t, e0 + j);
    }
    if (a.bias) {
      typedef f32x4 __attribute__((aligned(4))) f32x4_u4;
      if (count == NV) {
#pragma unroll
        for (int j = 0; j < NV; j += 4) {
          const f32x4 v = ((const f32x4_u4*)(a.bias + e0))[j / 4];
          add[j] = v[0], add[j + 1] = v[1], add[j + 2] = v[2], add[j + 3] = v[3];
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) add[j] = j < count ? a.bias[e0 + j] : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!(x[j] > kMinusInf)) x[j] = kMinusInf;  // NaN too
      sc.m = fmaxf(sc.m, x[j]);
    }
    if (!sigmoid && (scores || !renorm)) {
      const uint32_t k = row_max(sc.m > kMinusInf ? ordered(sc.m) : 0);
      sc.m = k ? unordered(k) : kMinusInf;
      float sum = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) sum += p[j] = x[j] > kMinusInf ? sc.raw(x[j]) : 0.f;
      sc.total = __builtin_amdgcn_rcpf(row_sum(sum));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float s = 0.f, k = x[j];
      if (scores) s = sigmoid ? sc.raw(x[j]) : p[j] * sc.total;
      if (a.bias) k = s += add[j];
      const bool there = x[j] > kMinusInf && k > kMinusInf;
      key[j] = there ? ordered(k) : 0;
      if (a.groups > 1) {
        if (!best2) s = k;
        if (!there) s = kMinusInf;
        b2 = s > b1 ? b1 : fmaxf(s, b2);
        b1 = fmaxf(s, b1);
      }
    }
  }
  bool unsure = false;
  if (a.groups > 1) {
    const float st = standing(b1, b2, a.shift, best2);
    uint32_t most = 0;
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < NV; ++j) most = max(most, size_of(key[j]));
      most = row_max(most);
    }
    const float tol = scores && st > kMinusInf ? standing_error(a.bias, sigmoid, st, __builtin_bit_cast(float, most)) : 0.f;
    int sure = 0, maybe = 0;
    for (int o = 0; o < a.groups; ++o) {
      const float other = __shfl(st, (lane & 48) | o << a.shift, 64);
      const bool tie = other == st && o < g;  // decides where the standings are exact
      sure += other > st + tol || (tol == 0.f && tie);
      maybe += tol == 0.f ? other > st || tie : o != g && !(other < st - tol);
    }
    unsure = g < a.groups && maybe >= a.kept && sure < a.kept;
    if (maybe >= a.kept) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = 0;
    }
  }
  // each list of four in order, equal keys as they are
  uint32_t tag[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    uint32_t* k = key + 4 * i;
    uint32_t p[4] = {0, 1, 2, 3};
    const auto order = [&](int u, int v) {
      const bool swap = k[v] > k[u];
      const uint32_t x = swap ? k[v] : k[u], y = swap ? p[v] : p[u];
      k[v] = swap ? k[u] : k[v];
      p[v] = swap ? p[u] : p[v];
      k[u] = x;
      p[u] = y;
    };
    order(0, 1), order(1, 2), order(2, 3), order(0, 1), order(1, 2), order(0, 1);
    tag[i] = p[0] | p[1] << 8 | p[2] << 16 | p[3] << 24;
  }
  const int rounds = a.bias ? a.K + 1 : a.K;
  int found = 0;
  for (int r = 0; r < rounds; ++r) {
    uint32_t mine = key[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) mine = max(mine, key[4 * i]);
    const uint32_t top = row_max(mine);
    // the lowest lane of the row that has it
    const uint32_t who = (uint32_t)(__ballot(mine == top) >> (lane & 48)) & 0xFFFF;
    bool win = top != 0 && mine == top && (who & ((1u << l) - 1)) == 0;
    found += top != 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint32_t* k = key + 4 * i;
      if (win && k[0] == top) {
        chosen[at][r] = (int16_t)(e0 + 4 * i + (tag[i] & 0xFF));
        k[0] = k[1], k[1] = k[2], k[2] = k[3], k[3] = 0;
        tag[i] >>= 8;
        win = false;
      }
    }
  }
  __builtin_amdgcn_wave_barrier();  // (a token's ranks are written and read by its own wave, whose LDS accesses stay in order)
  int mine = l < found ? chosen[at][l] : -1;
  float x = mine >= 0 ? logit<DT>(a, t, mine) : 0.f;
  if (a.bias) {
    const float b = mine >= 0 ? a.bias[mine] : 0.f, s = sc.raw(x) * sc.total, k = s + b, err = sc.error(x, s, k);
    const float xn = __shfl_down(x, 1, 64), bn = __shfl_down(b, 1, 64), kn = __shfl_down(k, 1, 64);
    const float ek = __shfl_down(err, 1, 64), en = l == a.K - 1 ? sc.error_up_to(kn) : ek;
    const bool near = l + 1 < found && !(k - kn > err + en), same = x == xn && b == bn;
    unsure |= near && !same;
    if (__any(near && same && l == a.K - 1)) {
      const int cut = (lane & 48) | (a.K - 1);
      const float xk = __shfl(x, cut, 64), bk = __shfl(b, cut, 64);
      uint32_t left = 0;
      if (__shfl(near && same, cut, 64)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = e0 + (i & ~3) + (tag[i / 4] >> (8 * (i & 3)) & 0xFF);
          if (key[i] != 0 && !(logit<DT>(a, t, e) == xk && a.bias[e] == bk)) left = max(left, key[i]);
        }
      }
      left = row_max(left);
      const float kl = unordered(left);
      unsure |= near && same && l == a.K - 1 && left != 0 && !(k - kl > err + sc.error_up_to(kl));
    }
  }
  uint64_t redo = __ballot(unsure);
  while (redo) {
    // a token at a time, by the whole wave
    constexpr int NV64 = NL;
    const int q = __builtin_ctzll(redo) >> 4, run64 = 4 << a.shift, g64 = lane >> (a.shift + 2);
    const int first = (lane & (run64 - 1)) * NV64, count64 = g64 < a.groups ? max(0, min(NV64, a.per - first)) : 0;
    int n;
    const int m = choose64<DT, NV64>(a, a.shift + 2, (int64_t)blockIdx.x * 16 + wave_id() * 4 + q, g64 * a.per + first, count64, n);
    const int got = __shfl(m, l, 64);
    if (lane >> 4 == q) {
      mine = got;
      if (mine >= 0) x = logit<DT>(a, t, mine);
    }
    redo &= ~(uint64_t(0xFFFF) << (16 * q));
  }
  const bool have = mine >= 0 && l < a.K;
  float w = have ? sc.raw(x) * sc.total : 0.f;
  if (renorm) {
    float sum = row_sum(sigmoid ? w : 0.f);
    // (as in the kernel for few tokens)
    const uint32_t k = row_max(have ? ordered(x) : 0);
    const float best = k ? unordered(k) : 0.f;
    const float v = !have ? 0.f : x == best ? 1.f : __builtin_amdgcn_exp2f((x - best) * kLog2e);
    const float vs = row_sum(v);
    const bool relative = !sigmoid || sum < 0x1p-80f;
    w = relative ? v : w;
    sum = relative ? vs : sum;
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (l < a.K && t < a.T) {
    a.ids[t * a.ldi + l] = have ? mine : -1;
    a.W[t * a.ldw + l] = have ? w * a.scale : 0.f;
  }
}

template <int DT, int NV>
hipError_t route_nv(const RouteArgs& a, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>(((int64_t)a.T + 3) / 4, 1 << 20);
  hipLaunchKernelGGL((route_kernel<DT, NV>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DT, int NV>
hipError_t route_rows(const RouteArgs& a, hipStream_t s) {
  // a dispatch counts its threads in 32 bits: tokens go out in parts of fewer
  constexpr int64_t kMost = int64_t(1) << 27;
  for (int64_t t = 0; t < a.T; t += kMost) {
    RouteArgs p = a;
    p.T = (int32_t)std::min<int64_t>(kMost, a.T - t);
    p.X = (const char*)a.X + t * a.ldx * (DT == DT_F32 ? 4 : 2);
    p.ids = a.ids + t * a.ldi;
    p.W = a.W + t * a.ldw;
    p.shift = (int8_t)(a.shift - 2);  // a group's lanes among 16
    hipLaunchKernelGGL((route_rows_kernel<DT, NV>), dim3((unsigned)(((int64_t)p.T + 15) / 16)), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t route_t(const RouteArgs& a, int cus, hipStream_t s) {
  const int nv = (a.per + (1 << a.shift) - 1) >> a.shift;  // experts per lane of 64
  // Four tokens per wave once that still gives every SIMD one (softmax over 64: 8192 tokens 3.6 us, 6.5 with a token per
  // wave; 256 experts in 8 groups with a bias: 16384 tokens 19 us, 30; 1024 tokens 12.9, 10.5)
  if (a.T >= cus * 16 && a.K < 16 && a.shift >= 2 && nv <= 8) {
    if (nv <= 1) return route_rows<DT, 4>(a, s);
    if (nv <= 2) return route_rows<DT, 8>(a, s);
    if (nv <= 4) return route_rows<DT, 16>(a, s);
    return route_rows<DT, 32>(a, s);
  }
  if (nv <= 1) return route_nv<DT, 1>(a, s);
  if (nv <= 2) return route_nv<DT, 2>(a, s);
  if (nv <= 4) return route_nv<DT, 4>(a, s);
  if (nv <= 8) return route_nv<DT, 8>(a, s);
  return route_nv<DT, 16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int x_type, int cus, hipStream_t s) {
  switch (x_type) {
    case DT_F32: return route_t<DT_F32>(a, cus, s);
    case DT_F16: return route_t<DT_F16>(a, cus, s);
    case DT_BF16: return route_t<DT_BF16>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
