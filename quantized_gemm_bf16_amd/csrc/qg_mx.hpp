// MXFP4 GEMM cores for gfx950: A and B hold E2M1 codes (two to a byte) with
// one E8M0 scale per row and 32 elements of K,
//     a(i, k) = qa(i, k) * 2^(U[i, k / 32] - 127),   b(j, k) likewise with V
// (the U, V scale operands of the page "InternLM Lmdeploy Gemm Interface",
// I/O Contract; one step of the scales per group along K as in the page
// "InternLM Lmdeploy Gemm MainloopSm80V2").
//
// The matrix instructions take the scales themselves: in
// v_mfma_scale_f32_32x32x64_f8f6f4 (16x16x128) with 4-bit operands a lane
// supplies 32 consecutive codes of one row, 16 bytes, which is exactly one
// scale block, and one scale byte for them, picked by an immediate from a
// VGPR. Products are exact and sums fp32, so nothing is left to do per block.
//
// Which blocks of a k-tile meet in one instruction is free as long as A and B
// agree. Lane half h (quarter, for 16x16) takes the h-th half (quarter) of
// the tile's blocks, one per k-step: its scales for the whole k-tile then
// are consecutive bytes of the row's scales, one LDS dword read, and the
// k-step is the immediate that picks the byte.
#pragma once
#include <type_traits>

#include "qg_tile.hpp"

namespace qg {

template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (N > 0) {
    static_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// 4-bit operands fill the first four of the eight dwords of the operand type.
__device__ __forceinline__ i32x8 widen(i32x4 x) { return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1); }
// c + a b with 2^(scale - 127) of byte OP of sa and of sb
template <int OP>
__device__ __forceinline__ f32x16 mfma_mx(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, 4, 4, OP, sa, OP, sb);
}
template <int OP>
__device__ __forceinline__ f32x4 mfma16_mx(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, 4, 4, OP, sa, OP, sb);
}

// Zeroes, in LDS, the codes of a 16-byte chunk (32 codes) from `keep` on, 0 < keep < 32.
__device__ __forceinline__ void lds_chunk_trim_codes(char* p, int keep) {
  asm volatile("" ::: "memory");
  i32x4 x = *(const i32x4*)p;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int n = keep - 8 * d;  // codes of dword d that lie before K
    const uint32_t m = n >= 8 ? ~0u : (n <= 0 ? 0u : (1u << (4 * n)) - 1u);
    x[d] = (int)((uint32_t)x[d] & m);
  }
  *(i32x4*)p = x;
  asm volatile("" ::: "memory");
}
// Zeroes the bytes of a dword of scales from `keep` on, 0 < keep < 4: scales
// past K's last block are the caller's padding, and a 255 there is a NaN even
// beside zero codes.
__device__ __forceinline__ void lds_dword_trim(char* p, int keep) {
  asm volatile("" ::: "memory");
  *(uint32_t*)p &= (1u << (8 * keep)) - 1u;
  asm volatile("" ::: "memory");
}

// ---- tiles ------------------------------------------------------------------
// The LDS ring, swizzle, load issue and epilogue of the tile core, with
// ROWB bytes (2 ROWB codes) of each row and their ROWB / 16 scales per stage.
// The scales follow the operand tiles in a stage as planes of one dword per row
// (A's rows, then B's): plane h holds the dword of lane half h, or, where a
// k-tile has only 4 scales (64 bytes of codes), one plane serves both halves.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int ROWB_>
struct MxCfg : TileCfg<El::E4M3, BM_, BN_, WM_, WN_, STAGES_, ROWB_> {
  using Base = TileCfg<El::E4M3, BM_, BN_, WM_, WN_, STAGES_, ROWB_>;
  static constexpr int BK = 2 * ROWB_;          // codes per k-tile
  static constexpr int KS = ROWB_ / 32;         // MFMAs along k per k-tile
  static constexpr int PLANES = ROWB_ / 64;     // scale dwords per row and k-tile
  static constexpr int HALF = Base::NW / 2;     // waves that issue the loads
  static constexpr int SL = PLANES * (BM_ + BN_) / 64;  // 64-lane scale loads per stage
  static constexpr int LSA = PLANES * BM_ / 64 / HALF, LSB = PLANES * BN_ / 64 / HALF;  // ... of one issuing wave
  static constexpr int LS = LSA + LSB;
  static constexpr int STAGE = Base::STAGE_BYTES + SL * 256;
  static constexpr int LPH = 2 * Base::LPW + LS;        // loads of an issuing wave per stage
  static_assert(LS * HALF == SL && BM_ % 64 == 0 && BN_ % 64 == 0, "scale rows must split evenly over the issuing waves");
  static_assert(STAGES_ * STAGE <= 160 * 1024 - 1024, "LDS budget");
  static_assert(LPH * (STAGES_ - 1) < 64, "vmcnt range");
};

template <class Cfg>
struct Mx : Tile<Cfg> {
  using Base = Tile<Cfg>;
  using Acc = typename Base::Acc;
  static constexpr int TM = Cfg::TM, TN = Cfg::TN, BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT;
  static constexpr int SMEM_BYTES = Cfg::STAGES * Cfg::STAGE;

  __device__ __forceinline__ static void mainloop(const Args& a, const Unit& u, char* smem, Acc& acc) {
    const int w = wave_id(), l = lane_id();
    const int wm = w / Cfg::WAVES_N, wn = w % Cfg::WAVES_N;
    const int64_t lda_b = a.lda / 2, ldb_b = a.ldb / 2;
    const uint32_t K = (uint32_t)a.K, nb = (K + 31) / 32;
    const int a_rows = max(0, min(BM, u.m_end - u.m0));
    const int b_rows = max(0, min(BN, a.N - u.n0));
    const i32x4 rA = make_rsrc_words((const char*)a.A + (int64_t)u.m0 * lda_b, (uint32_t)(a_rows * lda_b));
    const i32x4 rB = make_rsrc_words((const char*)a.B + (int64_t)u.expert * (a.b_batch / 2) + (int64_t)u.n0 * ldb_b,
                                     (uint32_t)(b_rows * ldb_b));
    const i32x4 rU = make_rsrc_words((const char*)a.U + (int64_t)u.m0 * a.ldu, (uint32_t)(a_rows * a.ldu));
    const i32x4 rV = make_rsrc_words((const char*)a.V + (int64_t)u.expert * a.v_batch + (int64_t)u.n0 * a.ldv,
                                     (uint32_t)(b_rows * a.ldv));

    // As in the tile core: the first half of the waves issues every load of a
    // stage, wave w filling its own row slots and those of wave w + HALF.
    constexpr int CPR = Cfg::CPR, RPI = Cfg::RPI, ROWB = Cfg::ROWB, HALF = Cfg::HALF, LA = Cfg::LA, LB = Cfg::LB;
    static_assert((HALF * LA * RPI) % 16 == 0 && (HALF * LB * RPI) % 16 == 0,
                  "the second half's rows keep the swizzle key (period 16 rows)");
    uint32_t offA[LA], offB[LB], chA[LA], chB[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int row = (w * LA + i) * RPI + l / CPR;
      chA[i] = (uint32_t)(((l % CPR) ^ swz<CPR>(row)) * 16);
      offA[i] = (uint32_t)(row * lda_b) + chA[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = (w * LB + i) * RPI + l / CPR;
      chB[i] = (uint32_t)(((l % CPR) ^ swz<CPR>(row)) * 16);
      offB[i] = (uint32_t)(row * ldb_b) + chB[i];
    }
    const uint32_t stepA = (uint32_t)(HALF * LA * RPI * lda_b), stepB = (uint32_t)(HALF * LB * RPI * ldb_b);
    // A wave's scale load i: of A for i < LSA, else of B; 64 rows of a plane.
    constexpr int LSA = Cfg::LSA, LS = Cfg::LS, GA = BM / 64, GB = BN / 64;
    uint32_t offS[LS], plS[LS], ldsS[LS];  // row offset, plane, place in the stage
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      const int j = i < LSA ? w * LSA + i : w * Cfg::LSB + i - LSA;
      const int g = i < LSA ? j % GA : j % GB;
      plS[i] = (uint32_t)(i < LSA ? j / GA : j / GB);
      offS[i] = (uint32_t)((g * 64 + l) * (i < LSA ? a.ldu : a.ldv));
      ldsS[i] = Cfg::STAGE_BYTES + (plS[i] * (BM + BN) + (i < LSA ? 0 : BM) + g * 64) * 4;
    }

    auto issue = [&](int stage, int kt) {
      if (w >= HALF) return;
      char* sbase = smem + stage * Cfg::STAGE;
      const uint32_t kk = (uint32_t)kt * ROWB;
      const bool live = kt < u.ke;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ws = w + h * HALF;
        if (live && 2 * (kk + ROWB) <= K) {
#pragma unroll
          for (int i = 0; i < LA; ++i) load_lds_x4(rA, sbase + (ws * LA + i) * 1024, offA[i] + h * stepA + kk);
#pragma unroll
          for (int i = 0; i < LB; ++i)
            load_lds_x4(rB, sbase + Cfg::A_BYTES + (ws * LB + i) * 1024, offB[i] + h * stepB + kk);
        } else {
#pragma unroll
          for (int i = 0; i < LA; ++i)
            load_lds_x4(rA, sbase + (ws * LA + i) * 1024,
                        live && 2 * (kk + chA[i]) < K ? offA[i] + h * stepA + kk : kOOB);
#pragma unroll
          for (int i = 0; i < LB; ++i)
            load_lds_x4(rB, sbase + Cfg::A_BYTES + (ws * LB + i) * 1024,
                        live && 2 * (kk + chB[i]) < K ? offB[i] + h * stepB + kk : kOOB);
        }
      }
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        const uint32_t block = (uint32_t)kt * CPR + plS[i] * 4;
        load_lds_x1a(i < LSA ? rU : rV, sbase + ldsS[i], live && block < nb ? offS[i] + block : kOOB);
      }
    };

    // The k-tile that holds K's end, where that is not on whole scale dwords:
    // the lane that loaded a chunk zeroes the codes past K in it, and the
    // scales past the last block, before the barrier that publishes the stage.
    const int ktail = (K & 127) ? (int)((K - 1) / (2 * ROWB)) : -1;
    auto trim = [&](int stage, int kt) {
      if (w >= HALF) return;
      const uint32_t ke = pinned(K);  // keeps this work inside the branch
      char* sbase = smem + stage * Cfg::STAGE;
      const uint32_t kk = (uint32_t)kt * ROWB;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ws = w + h * HALF;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
          const int keep = (int)(ke - 2 * (kk + chA[i]));
          if (keep > 0 && keep < 32) lds_chunk_trim_codes(sbase + (ws * LA + i) * 1024 + l * 16, keep);
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
          const int keep = (int)(ke - 2 * (kk + chB[i]));
          if (keep > 0 && keep < 32) lds_chunk_trim_codes(sbase + Cfg::A_BYTES + (ws * LB + i) * 1024 + l * 16, keep);
        }
      }
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        const int keep = (int)((ke + 31) / 32) - (kt * CPR + (int)plS[i] * 4);
        if (keep > 0 && keep < 4) lds_dword_trim(sbase + ldsS[i] + l * 4, keep);
      }
    };

    // Fragments of k-step ks: lane l takes row l % 32 and chunk KS h + ks of
    // its half h; the scales of all its chunks are one dword (PLANES 2) or
    // the h-th half of one.
    constexpr int KS = Cfg::KS;
    const int orow = l & 31, ohalf = l >> 5;
    struct Frags {
      i32x4 a[TM], b[TN];
    };
    struct Scales {
      int a[TM], b[TN];
    };
    auto read_frags = [&](int stage, int ks, Frags& f) {
      const char* sA = smem + stage * Cfg::STAGE;
      const char* sB = sA + Cfg::A_BYTES;
      const int c = ohalf * KS + ks;
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        const int row = wm * Cfg::WTM + tm * 32 + orow;
        f.a[tm] = *(const i32x4*)(sA + row * ROWB + ((c ^ swz<CPR>(row)) << 4));
      }
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int row = wn * Cfg::WTN + tn * 32 + orow;
        f.b[tn] = *(const i32x4*)(sB + row * ROWB + ((c ^ swz<CPR>(row)) << 4));
      }
    };
    auto read_scales = [&](int stage, Scales& s) {
      const int* p = (const int*)(smem + stage * Cfg::STAGE + Cfg::STAGE_BYTES);
      if constexpr (Cfg::PLANES == 2) p += ohalf * (BM + BN);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) s.a[tm] = p[wm * Cfg::WTM + tm * 32 + orow];
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) s.b[tn] = p[BM + wn * Cfg::WTN + tn * 32 + orow];
      if constexpr (Cfg::PLANES == 1) {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) s.a[tm] = (int)((uint32_t)s.a[tm] >> (16 * ohalf));
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) s.b[tn] = (int)((uint32_t)s.b[tn] >> (16 * ohalf));
      }
    };
    // MFMAs of k-step KI over the n-tiles [tn0, tn1) of the wave tile.
    auto mma = [&](auto KI, const Frags& f, const Scales& s, int tn0, int tn1) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          if (tn < tn0 || tn >= tn1) continue;
          acc.v[tn][tm] = mfma_mx<decltype(KI)::value>(f.b[tn], f.a[tm], acc.v[tn][tm], s.b[tn], s.a[tm]);
        }
    };

#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc.v[tn][tm] = f32x16{};

    const int nk = u.ke - u.kb;
    constexpr int S = Cfg::STAGES;
#pragma unroll
    for (int st = 0; st < S; ++st) issue(st, u.kb + st);
    wait_vmcnt<Cfg::LPH*(S - 1)>();
    if (u.kb == ktail) trim(0, ktail);
    lds_barrier();
    Frags cur;
    Scales sc;
    read_frags(0, 0, cur);
    read_scales(0, sc);
    for (int it = 0; it < nk; ++it) {
      const int st = it % S;
      static_for<KS>([&](auto KI) {
        constexpr int ks = decltype(KI)::value;
        Frags nxt;
        if constexpr (ks + 1 < KS) {
          read_frags(st, ks + 1, nxt);
          mma(KI, cur, sc, 0, TN);
          interleave_reads<TM + TN, TM * TN>();
        } else {
          // Last k-step of this stage, as in the tile core: half of its MFMAs
          // cover the wait for the next stage, the rest the next stage's
          // first fragments and scales.
          Scales ns;
          mma(KI, cur, sc, 0, TN / 2);
          wait_vmcnt<Cfg::LPH*(S - 2)>();
          if (u.kb + it + 1 == ktail) trim((it + 1) % S, ktail);
          lds_barrier();
          issue(st, u.kb + it + S);
          read_frags((it + 1) % S, 0, nxt);
          read_scales((it + 1) % S, ns);
          mma(KI, cur, sc, TN / 2, TN);
          interleave_reads<2 * (TM + TN), TM*(TN - TN / 2)>();
          sc = ns;
        }
        cur = nxt;
      });
    }
    // the ring still receives the zeros of k-tiles past the unit (see the tile core)
    wait_vmcnt<0>();
    __syncthreads();
  }
};

template <class Cfg>
hipError_t launch_mx(const Args& a, int grid, hipStream_t s) {
  return launch_sched<Mx<Cfg>>(a, grid, s);
}

}  // namespace qg
