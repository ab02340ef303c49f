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

// Byte address in LDS of a shared array, for load_lds_x4s. Taken once: each
// conversion of a generic pointer costs a 64-bit add, a compare and a select.
__device__ __forceinline__ uint32_t lds_address(void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)p);
}
// As load_lds_x4 (qg_device.hpp), to an LDS address and with a scalar offset.
// The hardware checks voff against the resource's size less soff, which must
// not exceed that size.
__device__ __forceinline__ void load_lds_x4s(const i32x4& rsrc, uint32_t lds_wave_base, uint32_t voff, uint32_t soff) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds_wave_base);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(m0v), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}
// A copy of a lane's value that the compiler cannot move out of the branch it
// is taken in (as pinned(), for values that differ between lanes).
__device__ __forceinline__ int pinned_lane(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// ---- tiles ------------------------------------------------------------------
// The LDS ring, swizzle and epilogue of the tile core, with ROWB bytes (2 ROWB
// codes) of each row per stage. Large products are bound by power: 4096^3
// takes 42 to 46 us (up to 3.27 PFLOP/s) at a shader clock of 1.8 GHz, of which an MFMA-only
// copy of the loop takes 25 and a launch and the stores 8, and a grouped prompt
// (64 experts, 65536 x 2048 x 7168) 660 us; small ones by the latency of
// their few k-tiles. What the loop does about both:
//  - every wave issues its own loads one by one between its MFMAs, for the
//    k-tile STAGES - 1 ahead, whose stage the last barrier freed: a wave that
//    issues a stage's loads in a row stands still while they pass the address
//    unit at 64 bytes a cycle (4096^3: 3860 instead of 4160 shader cycles per
//    256 of k);
//  - scales have a ring of their own, SPANS spans of 16 bytes (512 codes) per
//    row, A's rows and then B's, two of them loaded together: what the L2 can
//    serve is a number of requests, and a k-tile's 4 or 8 bytes of scales of a
//    row would cost it as much as the row's 64 or 128 bytes of codes (5180
//    cycles);
//  - a wave alone on its SIMD issues an instruction every four cycles or more,
//    and a small tile has one wave per SIMD and few tiles: WAVES_K groups of
//    waves, each with rings of its own, share the tile's k-tiles in contiguous
//    halves, and their sums meet in LDS at the end, in order (64 x 8192 x 8192:
//    10.3 us, 12.7 with one group).
// The 256 x 256 tile takes 64-byte rows and four stages: with 128-byte rows only
// two fit in LDS and the loop spills.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int ROWB_, int WK_>
struct MxCfg : TileCfg<El::E4M3, BM_, BN_, WM_, WN_, 2, ROWB_> {
  using Base = TileCfg<El::E4M3, BM_, BN_, WM_, WN_, 2, ROWB_>;
  static constexpr int STAGES = STAGES_;         // (the base's bounds are those of its own load issue)
  static constexpr int WAVES_K = WK_, NT = Base::NW * WK_ * 64;
  static constexpr int BK = 2 * ROWB_;           // codes per k-tile
  static constexpr int KS = ROWB_ / 32;          // MFMAs along k per k-tile
  static constexpr int KPS = 256 / ROWB_;        // k-tiles per span of scales
  static constexpr int GA = BM_ / 64, GT = GA + (BN_ + 63) / 64;  // 64-row scale loads per span: of A, in all
  static constexpr int SPAN = GT * 1024;
  static constexpr int RING = STAGES_ * Base::STAGE_BYTES;
  static_assert(BM_ % 64 == 0 && GT <= Base::NW, "a wave loads the scales of 64 rows");
  // Spans in the ring, and how many before their own two are loaded: a wave's
  // loads are known to have landed STAGES - 2 k-tiles after the one that they went out in.
  static constexpr int LEAD = (STAGES_ - 1 + KPS - 1) / KPS, SPANS = LEAD + 2;
  static_assert(STAGES_ >= 2 && Base::LPW * (STAGES_ - 1) + SPANS < 64, "vmcnt range");
  static constexpr int GROUP_BYTES = RING + SPANS * SPAN;  // LDS of one group of waves
  static_assert(WK_ * GROUP_BYTES <= 160 * 1024 - 4352 && BM_ * BN_ * 4 * (WK_ - 1) <= WK_ * GROUP_BYTES, "LDS budget");
};

template <class Cfg>
struct Mx : Tile<Cfg> {
  using Base = Tile<Cfg>;
  using Acc = typename Base::Acc;
  static constexpr int TM = Cfg::TM, TN = Cfg::TN, BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT;
  static constexpr int SMEM_BYTES = Cfg::WAVES_K * Cfg::GROUP_BYTES;
  static constexpr int WK = Cfg::WAVES_K;
  // Grouped, 256 x 256 tiles: an XCD's tiles share their rows of A and B in its
  // L2 (64 experts, 16384 rows, N 2048, K 7168: 227 us, 237 without; 128 x 128
  // tiles, bound by other things than the L2's misses, 272 and 250).
  static constexpr bool GROUPED_XCD = BM == 256;

  // Waves of the first group hold the tile once the mainloop has ended.
  __device__ __forceinline__ static bool holds_partial() { return WK == 1 || wave_id() < Cfg::NW; }

  __device__ __forceinline__ static void mainloop(const Args& a, const Unit& unit, char* smem0, Acc& acc) {
    const int group = WK == 1 ? 0 : wave_id() / Cfg::NW;
    const int share = (unit.ke - unit.kb + WK - 1) / WK;  // k-tiles of a group; the last ones may have fewer
    Unit u = unit;
    u.kb = min(unit.ke, unit.kb + group * share);
    u.ke = min(unit.ke, u.kb + share);
    char* smem = smem0 + group * Cfg::GROUP_BYTES;
    const int w = WK == 1 ? wave_id() : wave_id() % Cfg::NW, l = lane_id();
    const int wm = w / Cfg::WAVES_N, wn = w % Cfg::WAVES_N;
    const int64_t lda_b = a.lda / 2, ldb_b = a.ldb / 2;
    const uint32_t K = (uint32_t)a.K;
    const int a_rows = max(0, min(BM, u.m_end - u.m0));
    const int b_rows = max(0, min(BN, a.N - u.n0));
    const i32x4 rA = make_rsrc_words((const char*)a.A + (int64_t)u.m0 * lda_b, (uint32_t)(a_rows * lda_b));
    const i32x4 rB = make_rsrc_words((const char*)a.B + (int64_t)u.expert * (a.b_batch / 2) + (int64_t)u.n0 * ldb_b,
                                     (uint32_t)(b_rows * ldb_b));
    // this wave's scales: 64 rows of A or of B (where there are fewer such
    // groups than waves, some waves repeat one: the same bytes to the same place)
    const int grp = w % Cfg::GT;
    const bool of_a = grp < Cfg::GA;
    const int64_t ld_s = of_a ? a.ldu : a.ldv;
    const i32x4 rS = make_rsrc_words(of_a ? (const char*)a.U + (int64_t)u.m0 * a.ldu
                                          : (const char*)a.V + (int64_t)u.expert * a.v_batch + (int64_t)u.n0 * a.ldv,
                                     (uint32_t)((of_a ? a_rows : b_rows) * ld_s));
    const uint32_t offS = (uint32_t)(((of_a ? grp : grp - Cfg::GA) * 64 + l) * ld_s);

    constexpr int CPR = Cfg::CPR, RPI = Cfg::RPI, ROWB = Cfg::ROWB, LA = Cfg::LA, LPW = Cfg::LPW, KPS = Cfg::KPS;
    // Load i < LA of a wave fills RPI rows of A's part of a stage, the others of
    // B's: lane l -> row l / CPR, physical chunk l % CPR, whose logical chunk
    // begins at byte chunk(i, l) of the row's k-tile.
    auto row_of = [&](int i, int ll) { return (i < LA ? w * LA + i : w * Cfg::LB + i - LA) * RPI + ll / CPR; };
    auto chunk = [&](int i, int ll) { return (uint32_t)(((ll % CPR) ^ swz<CPR>(row_of(i, ll))) * 16); };
    uint32_t off[LPW];
#pragma unroll
    for (int i = 0; i < LPW; ++i) off[i] = (uint32_t)(row_of(i, l) * (i < LA ? lda_b : ldb_b)) + chunk(i, l);
    char* spans = smem + Cfg::RING;
    const uint32_t lds = lds_address(smem);
    const uint32_t dstA = lds + w * LA * 1024, dstB = lds + Cfg::A_BYTES + w * Cfg::LB * 1024;
    const uint32_t dstS = lds + Cfg::RING + grp * 1024;

    // Load i of k-tile kt into ring stage `stage`. FULL: the k-tile lies wholly
    // before K; otherwise chunks past K read as zero (lane: the lane's number).
    auto load = [&](auto FULL, int i, int stage, int kt, int lane) {
      const uint32_t kk = (uint32_t)kt * ROWB;
      const bool in = decltype(FULL)::value || 2 * (kk + chunk(i, lane)) < K;
      const uint32_t dst = (i < LA ? dstA + i * 1024 : dstB + (i - LA) * 1024) + stage * Cfg::STAGE_BYTES;
      load_lds_x4s(i < LA ? rA : rB, dst, in ? off[i] : kOOB, kk);
    };
    // Scales of spans [j, end); those past K do not exist.
    const int spans_k = (int)((K + 511) / 512);
    auto load_spans = [&](int j, int end) {
      for (; j < min(end, spans_k); ++j) load_lds_x4s(rS, dstS + j % Cfg::SPANS * Cfg::SPAN, offS, (uint32_t)j * 16);
    };
    // Spans 2 i and 2 i + 1 are loaded at the first k-tile of span 2 i - LEAD:
    // every wave has read the scales of all spans before that one by then, and
    // the two that they replace, SPANS before them, are such.
    constexpr int LEAD = Cfg::LEAD;
    auto load_next_spans = [&](int kt) {
      if (kt % (2 * KPS) == LEAD % 2 * KPS && kt != u.kb) load_spans(kt / KPS + LEAD, kt / KPS + LEAD + 2);
    };
    auto load_tile = [&](int stage, int kt) {
      const int ll = pinned_lane(l);  // keeps this rare work out of the loops' registers
#pragma unroll
      for (int i = 0; i < LPW; ++i) load(std::false_type{}, i, stage, kt, ll);
    };

    // Before the barrier that publishes them, the lanes that loaded them zero
    // what lies past K: codes in the last chunk of a row (K not a multiple of
    // 32), in the k-tile that holds it, and scales in the last span (their
    // number not a multiple of 16: past it is the caller's padding, and a 255
    // there is a NaN even beside zero codes), once its first k-tile is resident.
    const int nb = (int)((K + 31) / 32);
    const int tail_codes = (K & 31) ? (int)((K - 1) / (2 * ROWB)) : -1;
    const int tail_scales = (nb & 15) ? max(u.kb, (nb - 1) / 16 * KPS) : -1;
    auto trim = [&](int stage, int kt) {
      const int ll = pinned_lane(l);
      const uint32_t ke = pinned(K);
      if (kt == tail_codes) {
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
          const int keep = (int)(ke - 2 * ((uint32_t)kt * ROWB + chunk(i, ll)));
          char* p = smem + stage * Cfg::STAGE_BYTES + (i < LA ? (w * LA + i) * 1024 : Cfg::A_BYTES + (w * Cfg::LB + i - LA) * 1024);
          if (keep > 0 && keep < 32) lds_chunk_trim_codes(p + ll * 16, keep);
        }
      }
      if (kt == tail_scales)
        lds_chunk_trim(spans + kt / KPS % Cfg::SPANS * Cfg::SPAN + grp * 1024 + ll * 16, (int)((ke + 31) / 32) & 15);
    };

    // Fragments of k-step ks: lane l takes row l % 32 and chunk KS h + ks of
    // its half h; the scales of its KS chunks are consecutive bytes.
    constexpr int KS = Cfg::KS;
    const int orow = l & 31, ohalf = l >> 5;
    struct Frags {
      i32x4 a[TM], b[TN];
    };
    struct Scales {
      int a[TM], b[TN];
    };
    auto read_frags = [&](int stage, int ks, Frags& f) {
      const char* sA = smem + stage * Cfg::STAGE_BYTES;
      const char* sB = sA + Cfg::A_BYTES;
      const int c = ohalf * KS + ks;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int row = wn * Cfg::WTN + tn * 32 + orow;
        f.b[tn] = *(const i32x4*)(sB + row * ROWB + ((c ^ swz<CPR>(row)) << 4));
      }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        const int row = wm * Cfg::WTM + tm * 32 + orow;
        f.a[tm] = *(const i32x4*)(sA + row * ROWB + ((c ^ swz<CPR>(row)) << 4));
      }
    };
    auto read_scales = [&](int kt, Scales& s) {
      // KS 4: the k-tile's 8 scales are a dword per half; KS 2: one dword, two bytes per half
      const char* p = spans + kt / KPS % Cfg::SPANS * Cfg::SPAN + kt % KPS * (ROWB / 16) + (KS == 4 ? ohalf * 4 : 0);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) s.a[tm] = *(const int*)(p + (wm * Cfg::WTM + tm * 32 + orow) * 16);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) s.b[tn] = *(const int*)(p + (BM + wn * Cfg::WTN + tn * 32 + orow) * 16);
    };
    auto half_scales = [&](Scales& s) {
      if constexpr (KS == 2) {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) s.a[tm] = (int)((uint32_t)s.a[tm] >> (16 * ohalf));
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) s.b[tn] = (int)((uint32_t)s.b[tn] >> (16 * ohalf));
      }
    };

#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc.v[tn][tm] = f32x16{};

    // The k-tiles before `fast` prefetch a whole k-tile and find nothing to
    // trim in the next one.
    constexpr int S = Cfg::STAGES, P = S - 1;  // k-tiles under way
    const int whole = min(u.ke, (int)(K / (2 * ROWB)));  // k-tiles [kb, whole) are whole
    int fast = whole - P;
    if (tail_scales >= 0) fast = min(fast, tail_scales - 1);
    fast = max(fast, u.kb);
    // Waits until at most the code loads of the last n k-tiles are under way
    // (scales loaded among them make it wait for a load or two more).
    auto wait_tiles = [&](int n) {
      static_for<P>([&](auto N) {
        if (n == decltype(N)::value) wait_vmcnt<LPW * decltype(N)::value>();
      });
    };
    load_spans(u.kb / KPS, ((u.kb / KPS + LEAD) & ~1) + 2);  // all that no later k-tile of the unit loads
#pragma unroll
    for (int st = 0; st < P; ++st)
      if (u.kb + st < u.ke) load_tile(st, u.kb + st);
    wait_tiles(max(0, min(u.ke - u.kb, P) - 1));
    if (u.kb == tail_codes || u.kb == tail_scales) trim(0, u.kb);
    lds_barrier();
    constexpr int NM = TM * TN;  // MFMAs of a k-step
    int kt = u.kb, st = 0;       // the k-tile and its stage
    // Meets the other waves once k-tile kt + 1 has landed.
    auto publish = [&](auto FAST, int kt, int next) {
      if constexpr (decltype(FAST)::value) {
        wait_vmcnt<LPW*(S - 2)>();
      } else {
        wait_tiles(max(0, min(u.ke, kt + S) - (kt + 2)));
        if (kt + 1 == tail_codes || kt + 1 == tail_scales) trim(next, kt + 1);
      }
      lds_barrier();
    };

    constexpr int EARLY = NM / 2;  // MFMAs of the last k-step before the barrier
    Frags cur;
    Scales sc;
    read_frags(0, 0, cur);
    read_scales(kt, sc);
    half_scales(sc);
    int ahead = S - 1;  // stage of the k-tile being loaded
    auto step = [&](auto FAST) {
      constexpr bool F = decltype(FAST)::value;
      const int next = st + 1 == S ? 0 : st + 1;
      load_next_spans(kt);
      if constexpr (!F)
        if (kt + P < u.ke) load_tile(ahead, kt + P);
      static_for<KS>([&](auto KI) {
        constexpr int ks = decltype(KI)::value;
        constexpr bool last = ks + 1 == KS;
        Frags nxt;
        Scales ns;
        if constexpr (!last) read_frags(st, ks + 1, nxt);
        // loads [l0, l1) go out in this k-step, in the last one before the barrier
        constexpr int l0 = LPW * ks / KS, l1 = LPW * (ks + 1) / KS, room = last ? EARLY : NM;
        static_for<NM>([&](auto MI) {
          constexpr int m = decltype(MI)::value, tn = m / TM, tm = m % TM;
          if constexpr (F) {
            static_for<l1 - l0>([&](auto LI) {
              constexpr int j = decltype(LI)::value;
              if constexpr (j * room / (l1 - l0) == m) {
                load(std::true_type{}, l0 + j, ahead, kt + P, l);
                __builtin_amdgcn_sched_barrier(0);
              }
            });
          }
          if constexpr (last && m == EARLY) {
            publish(FAST, kt, next);
            read_frags(next, 0, nxt);
            read_scales(kt + 1, ns);
          }
          acc.v[tn][tm] = mfma_mx<ks>(cur.b[tn], cur.a[tm], acc.v[tn][tm], sc.b[tn], sc.a[tm]);
        });
        if constexpr (last) {
          half_scales(ns);
          sc = ns;
        }
        cur = nxt;
      });
      ahead = st;
      st = next;
      ++kt;
    };
    while (kt < fast) step(std::true_type{});
    while (kt < u.ke) step(std::false_type{});
    for (int i = u.ke - u.kb; i < share; ++i) lds_barrier();  // the barriers of a group with more k-tiles
    __syncthreads();
    if constexpr (WK > 1) {
      // the groups' sums, in k order, to the first group
      f32x4* red = (f32x4*)smem0;
      if (group > 0) {
#pragma unroll
        for (int c = 0; c < Base::NCH; ++c) red[(((group - 1) * Base::NCH + c) * Cfg::NW + w) * 64 + l] = Base::get4(acc, c);
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int g = 0; g < WK - 1; ++g)
#pragma unroll
          for (int c = 0; c < Base::NCH; ++c)
            Base::set4(acc, c, Base::get4(acc, c) + red[((g * Base::NCH + c) * Cfg::NW + w) * 64 + l]);
      }
      __syncthreads();
    }
  }

  __device__ __forceinline__ static void write_partial(const Args& a, int slot, Acc& acc) {
    if (holds_partial()) Base::write_partial(a, slot, acc);
  }

  __device__ __forceinline__ static void store(const Args& a, const Unit& u, Acc& acc, char* smem) {
    if constexpr (Base::STAGED) {
      if (Base::plain16(a)) {
        if (holds_partial())
          Base::template store_staged<false>(a, u, acc, smem);
        else
          lds_barrier();  // the one that ends it
        return;
      }
    }
    if (holds_partial()) Base::store(a, u, acc, smem);
  }
};

template <class Cfg>
hipError_t launch_mx(const Args& a, int grid, hipStream_t s) {
  return launch_sched<Mx<Cfg>>(a, grid, s);
}

}  // namespace qg
