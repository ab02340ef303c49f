// MXFP4 core for few rows (decode; experts with a row or two): M <= 16 MT.
//
// Such a product reads every weight once for a handful of rows, so what
// bounds it is the stream of B from HBM. As in the skinny core for 16-bit
// operands a wave streams its own k-blocks of B, 256 contiguous bytes (512
// codes) and 16 scale bytes per row and block, into a private ring of LDS
// slots and waits only for its own loads. Two ways to share the work:
//   k-interleaved (SHARED_A false): the waves of a workgroup cover the same
//     BN columns and take every NW-th block, each with its own copy of A's
//     rows; their sums meet in LDS in wave order.
//   N-split (SHARED_A true): each wave owns BN / NW columns over the whole
//     k-range; A's rows of a block are loaded once per workgroup, and the waves
//     meet at a barrier per block.
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies row l % 16 and the 32
// codes of one scale block; quarter l / 16 takes chunks 4 (l / 16) + s of the
// block's 16 in step s, so that its four scales are one dword. B's rows are the
// first operand: a lane ends up with 4 consecutive columns of one row of D.
//
// Measured: 1 x 4096 x 14336 k-interleaved in 8.3 us (31 MB: 3.8 TB/s with the
// launch; the mainloops take 6.0), 64 experts of 2048 x 7168 with 128 rows
// N-split in 84 us (477 MB: 5.7 TB/s, a plain streaming read 5.9). Four waves
// and two blocks each: eight waves 9.4 us, 32 columns per workgroup 9.7. The
// shared ring takes two blocks too, so that three workgroups fit on a CU: with
// three blocks and two workgroups the same at K = 7168, but 33 instead of 30 us
// at K = 2048 and 50 instead of 37 at K = 468 (128 experts, 95 rows, N 5120).
#pragma once
#include "qg_mx.hpp"
#include "qg_skinny.hpp"

namespace qg {

template <int BN_, int NW_, int MT_, int DEPTH_, bool SHARED_>
struct MxSkinnyCfg {
  static constexpr bool SHARED_A = SHARED_;
  static constexpr int BN = BN_, NW = NW_, MT = MT_, DEPTH = DEPTH_;
  static constexpr int BNW = SHARED_A ? BN / NW : BN;  // columns per wave
  static constexpr int NT = NW * 64, BM = 16 * MT, TN = BNW / 16;
  static constexpr int BLKB = 256, BK = 2 * BLKB;      // bytes and codes of k per row and block
  static constexpr int ROWS = BLKB + 16;               // LDS bytes of a row's codes and scales
  static constexpr int SLOT = (BNW + (SHARED_A ? 0 : BM)) * ROWS;  // one wave's ring slot
  static constexpr int ASLOT = SHARED_A ? BM * ROWS : 0;           // one slot of the shared A ring
  static constexpr int LB = BNW / 4, LA = SHARED_A ? (BM / 4 + NW - 1) / NW : BM / 4;  // 1 KB loads per wave and block
  static constexpr int LSB = BNW / 16, LSA = SHARED_A ? 1 : MT;                        // scale loads (16 rows)
  static constexpr int LPS = LB + LA + LSB + LSA;
  static constexpr int RING = NW * DEPTH * SLOT + DEPTH * ASLOT;
  static constexpr int RED = SHARED_A ? 0 : NW * TN * MT * 1024;  // the cross-wave sum reuses the ring
  static constexpr int LDS_BYTES = RING > RED ? RING : RED;
  static_assert(BNW % 16 == 0 && BNW * (SHARED_A ? NW : 1) == BN, "skinny tile");
  static_assert(LDS_BYTES <= 160 * 1024 - 4352, "LDS budget");
  static_assert(LPS * DEPTH < 64 && (!SHARED_A || DEPTH >= 2), "ring depth");
};

template <class Cfg>
struct MxSkinny {
  using S4 = f32x4;
  static constexpr int TN = Cfg::TN, MT = Cfg::MT, NW = Cfg::NW, DEPTH = Cfg::DEPTH, BNW = Cfg::BNW, BLKB = Cfg::BLKB;
  static constexpr int BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT;
  static constexpr int SMEM_BYTES = Cfg::LDS_BYTES;
  static constexpr bool SH = Cfg::SHARED_A;
  struct Acc {
    f32x4 v[TN][MT];
    f32x4 c[TN][MT];  // this lane's C values, loaded when the unit starts
  };

  __device__ __forceinline__ static void prefetch_c(const Args& a, const Unit& u, Acc& acc) {
    const int w = wave_id(), l = lane_id();
    const bool need = a.c_type >= 0 && a.beta != 0.f && (SH || w == 0);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int m = u.m0 + mt * 16 + (l & 15);
        const int n = u.n0 + (SH ? w * BNW : 0) + tn * 16 + 4 * (l >> 4);
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        if (need && m < u.m_end && n < a.N) load_c4(a, m, n, c);
        acc.c[tn][mt] = f32x4{c[0], c[1], c[2], c[3]};
      }
  }

  __device__ __forceinline__ static void mainloop(const Args& a, const Unit& u, char* smem, Acc& acc) {
    const int w = wave_id(), l = lane_id();
    const int64_t lda_b = a.lda / 2, ldb_b = a.ldb / 2;
    const uint32_t K = (uint32_t)a.K, nb = (K + 31) / 32;
    const int a_rows = max(0, min(BM, u.m_end - u.m0));
    const int n0 = u.n0 + (SH ? w * BNW : 0);
    const int b_rows = max(0, min(BNW, a.N - n0));
    const i32x4 rA = make_rsrc_words((const char*)a.A + (int64_t)u.m0 * lda_b, (uint32_t)(a_rows * lda_b));
    const i32x4 rU = make_rsrc_words((const char*)a.U + (int64_t)u.m0 * a.ldu, (uint32_t)(a_rows * a.ldu));
    const i32x4 rB = make_rsrc_words((const char*)a.B + (int64_t)u.expert * (a.b_batch / 2) + (int64_t)n0 * ldb_b,
                                     (uint32_t)(b_rows * ldb_b));
    const i32x4 rV = make_rsrc_words((const char*)a.V + (int64_t)u.expert * a.v_batch + (int64_t)n0 * a.ldv,
                                     (uint32_t)(b_rows * a.ldv));
    // One 64-lane load fills 4 rows x 256 bytes of a slot: lane l -> row l / 16,
    // physical chunk l % 16, which holds logical chunk (l % 16) ^ (row & 15).
    // A scale load fills 16 rows x 16 bytes: lane l -> row l / 4, dword l % 4.
    constexpr int LB = Cfg::LB, LA = Cfg::LA, LSB = Cfg::LSB, LSA = Cfg::LSA, KSTRIDE = SH ? 1 : NW;
    char* bring = smem + w * DEPTH * Cfg::SLOT;
    char* aring = SH ? smem + NW * DEPTH * Cfg::SLOT : bring + BNW * Cfg::ROWS;
    constexpr int ASTEP = SH ? Cfg::ASLOT : Cfg::SLOT;  // from one slot of A's ring to the next
    uint32_t offB[LB], chB[LB], offA[LA], chA[LA], offV[LSB], offU[LSA];
    int ia[LA], isa[LSA];  // which of the block's A loads are this wave's (shared A: repeats where there are fewer than waves)
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = i * 4 + (l >> 4);
      chB[i] = (uint32_t)(((l & 15) ^ (row & 15)) * 16);
      offB[i] = (uint32_t)(row * ldb_b) + chB[i];
    }
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      ia[i] = SH ? (w * LA + i) % (BM / 4) : i;
      const int row = ia[i] * 4 + (l >> 4);
      chA[i] = (uint32_t)(((l & 15) ^ (row & 15)) * 16);
      offA[i] = (uint32_t)(row * lda_b) + chA[i];
    }
#pragma unroll
    for (int i = 0; i < LSB; ++i) offV[i] = (uint32_t)((i * 16 + (l >> 2)) * a.ldv) + (l & 3) * 4;
#pragma unroll
    for (int i = 0; i < LSA; ++i) {
      isa[i] = SH ? w % MT : i;
      offU[i] = (uint32_t)((isa[i] * 16 + (l >> 2)) * a.ldu) + (l & 3) * 4;
    }
    // Loads k-block blk into ring slot d; blocks past the unit read nothing.
    auto issue = [&](int d, int blk) {
      char* b = bring + d * Cfg::SLOT;
      char* sa = aring + d * ASTEP;
      const bool live = blk < u.ke;
      const uint32_t kk = (uint32_t)blk * BLKB, ks = (uint32_t)blk * 16;
#pragma unroll
      for (int i = 0; i < LB; ++i) load_lds_x4(rB, b + i * 1024, live && 2 * (kk + chB[i]) < K ? offB[i] + kk : kOOB);
#pragma unroll
      for (int i = 0; i < LA; ++i) load_lds_x4(rA, sa + ia[i] * 1024, live && 2 * (kk + chA[i]) < K ? offA[i] + kk : kOOB);
      const bool s_in = live && ks + (l & 3) * 4 < nb;
#pragma unroll
      for (int i = 0; i < LSB; ++i) load_lds_x1a(rV, b + BNW * BLKB + i * 256, s_in ? offV[i] + ks : kOOB);
#pragma unroll
      for (int i = 0; i < LSA; ++i) load_lds_x1a(rU, sa + BM * BLKB + isa[i] * 256, s_in ? offU[i] + ks : kOOB);
    };
    // The block that holds K's end: the lane that loaded a chunk zeroes the
    // codes past K in it, and the scales past the last one (waves that load
    // the same A chunk each trim it after their own copy has landed).
    const int ktail = (K & 127) ? (int)((K - 1) / Cfg::BK) : -1;
    auto trim = [&](int d, int blk) {
      const uint32_t ke = pinned(K);  // keeps this work inside the branch
      char* b = bring + d * Cfg::SLOT;
      char* sa = aring + d * ASTEP;
      const uint32_t kk = (uint32_t)blk * BLKB;
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        const int keep = (int)(ke - 2 * (kk + chB[i]));
        if (keep > 0 && keep < 32) lds_chunk_trim_codes(b + i * 1024 + l * 16, keep);
      }
#pragma unroll
      for (int i = 0; i < LA; ++i) {
        const int keep = (int)(ke - 2 * (kk + chA[i]));
        if (keep > 0 && keep < 32) lds_chunk_trim_codes(sa + ia[i] * 1024 + l * 16, keep);
      }
      const int keep = (int)((ke + 31) / 32) - (blk * 16 + (l & 3) * 4);
      if (keep > 0 && keep < 4) {
#pragma unroll
        for (int i = 0; i < LSB; ++i) lds_dword_trim(b + BNW * BLKB + i * 256 + l * 4, keep);
#pragma unroll
        for (int i = 0; i < LSA; ++i) lds_dword_trim(sa + BM * BLKB + isa[i] * 256 + l * 4, keep);
      }
    };
    i32x4 fb[4][TN], fa[4][MT];
    int sb[TN], sa[MT];
    const int r16 = l & 15, q = l >> 4;
    auto read = [&](int d) {
      const char* b = bring + d * Cfg::SLOT;
      const char* pa = aring + d * ASTEP;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int c = ((4 * q + s) ^ r16) << 4;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) fb[s][tn] = *(const i32x4*)(b + (tn * 16 + r16) * BLKB + c);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) fa[s][mt] = *(const i32x4*)(pa + (mt * 16 + r16) * BLKB + c);
      }
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) sb[tn] = *(const int*)(b + BNW * BLKB + (tn * 16 + r16) * 16 + q * 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) sa[mt] = *(const int*)(pa + BM * BLKB + (mt * 16 + r16) * 16 + q * 4);
    };
    auto compute = [&]() {
      static_for<4>([&](auto S) {
        constexpr int s = decltype(S)::value;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc.v[tn][mt] = mfma16_mx<s>(fb[s][tn], fa[s][mt], acc.v[tn][mt], sb[tn], sa[mt]);
      });
    };

#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc.v[tn][mt] = f32x4{};
    prefetch_c(a, u, acc);

    const int nk = u.ke - u.kb;
    if constexpr (SH) {
      // Per block: wait for this wave's loads of block b, meet (every wave's
      // part of A(b) has landed, every wave is done reading block b - 1), refill block
      // b - 1's slots with block b + DEPTH - 1, read block b, compute. The count is
      // rounded up to whole rounds: blocks past the unit read nothing and add zeros.
      const int rounds = (nk + DEPTH - 1) / DEPTH;
#pragma unroll
      for (int d = 0; d < DEPTH - 1; ++d) issue(d, u.kb + d);
      for (int r = 0; r < rounds; ++r) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          wait_vmcnt<Cfg::LPS*(DEPTH - 2)>();
          if (u.kb + r * DEPTH + d == ktail) trim(d, ktail);
          lds_barrier();
          issue((d + DEPTH - 1) % DEPTH, u.kb + r * DEPTH + d + DEPTH - 1);
          read(d);
          compute();
        }
      }
      wait_vmcnt<0>();
      __syncthreads();  // the rings are reused by the next unit
    } else {
      // This wave's blocks are kb + w, kb + w + NW, ...
      const int count = nk > w ? (nk - w + KSTRIDE - 1) / KSTRIDE : 0;
      const int rounds = (count + DEPTH - 1) / DEPTH;
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) issue(d, u.kb + w + d * KSTRIDE);
      for (int r = 0; r < rounds; ++r) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          wait_vmcnt<Cfg::LPS*(DEPTH - 1)>();
          asm volatile("" ::: "memory");
          const int blk = u.kb + w + (r * DEPTH + d) * KSTRIDE;
          if (blk == ktail) trim(d, blk);
          read(d);
          // refill the slot as soon as its fragments are in registers
          __builtin_amdgcn_s_waitcnt(0xc07f);
          asm volatile("" ::: "memory");
          issue(d, blk + DEPTH * KSTRIDE);
          compute();
        }
      }
      wait_vmcnt<0>();
      __syncthreads();  // every wave is done with its ring before it is reused below
      // Sum the waves' partial sums in wave order into wave 0.
      S4* red = (S4*)smem;
      if (w > 0) {
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) red[((w * TN + tn) * MT + mt) * 64 + l] = acc.v[tn][mt];
      }
      __syncthreads();
      if (w == 0) {
        for (int w2 = 1; w2 < NW; ++w2)
#pragma unroll
          for (int tn = 0; tn < TN; ++tn)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc.v[tn][mt] += red[((w2 * TN + tn) * MT + mt) * 64 + l];
      }
      __syncthreads();
    }
  }

  // Epilogue: wave 0 holds the tile (k-interleaved) or each wave its columns (N-split).
  __device__ __forceinline__ static void store(const Args& a, const Unit& u, Acc& acc, char* /*smem*/) {
    if (!holds_partial()) return;
    const int l = lane_id();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = u.m0 + mt * 16 + (l & 15);
      if (m >= u.m_end) continue;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int n = u.n0 + (SH ? wave_id() * BNW : 0) + tn * 16 + 4 * (l >> 4);
        if (n < a.N) epi_store4c(a, m, n, acc.v[tn][mt], acc.c[tn][mt]);
      }
    }
  }

  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t slot_rsrc(const Args& a, int slot) {
    return make_rsrc((const char*)a.partials + (size_t)slot * (BM * BN * 4), BM * BN * 4);
  }
  // Partial tile layout: [wave (N-split)][tn][mt][lane] x 16 bytes; chunk c = tn * MT + mt of a lane.
  static constexpr int NCH = TN * MT;
  __device__ __forceinline__ static bool holds_partial() { return SH || wave_id() == 0; }
  __device__ __forceinline__ static uint32_t chunk_off(int c) {
    return (uint32_t)((((SH ? wave_id() : 0) * NCH + c) * 64 + lane_id()) * 16);
  }
  __device__ __forceinline__ static S4 get4(const Acc& acc, int c) { return acc.v[c / MT][c % MT]; }
  __device__ __forceinline__ static void set4(Acc& acc, int c, const S4& x) { acc.v[c / MT][c % MT] = x; }
  __device__ __forceinline__ static void write_partial(const Args& a, int slot, Acc& acc) {
    if (!holds_partial()) return;
    const auto r = slot_rsrc(a, slot);
#pragma unroll
    for (int c = 0; c < NCH; ++c) store_sc1_x4(r, chunk_off(c), __builtin_bit_cast(i32x4, get4(acc, c)));
  }
};

template <class Cfg>
hipError_t launch_mx_skinny(const Args& a, int grid, hipStream_t s) {
  return launch_sched<MxSkinny<Cfg>>(a, grid, s);
}

}  // namespace qg
