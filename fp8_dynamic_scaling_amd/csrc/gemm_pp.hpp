// gemm_pp.hpp -- the ping-pong FP8 GEMM kernel of the dense and grouped products
// (gemm_fp8_fast.hip) and of the gated products (gemm_gated.hip).
#pragma once

#include <type_traits>

#include "gated.hpp"
#include "gemm_common.hpp"

namespace fp8dyn {

// Epilogue of a gated tile of 64 MI rows x 128 features. A wave has 32 MI rows x 32 features: element 4 q + u of
// block i is row 32 i + lane % 32, feature 8 q + 4 (lane / 32) + u; block column 0 holds g, column 1 u. Lanes l
// and l + 32 exchange halves of two neighbouring q, after which each has 8 features of its row. Every 32 rows of
// a group's four waves then go through LDS (the ring is idle), so that a store writes whole lines, 256 bytes of
// each of four rows: CHANGE_ME. F % 8 != 0 or outputs off 16 bytes: single values.
constexpr int kGatedEpilogueLds = 2 * 2 * 3 * 32 * 256 + 8 * 64 * 4;

template <bool GELU, bool ROW, int MI>
__device__ __forceinline__ void gated_epilogue(const GemmParams& p, const TileInfo& ti, int64_t F,
                                               const float __attribute__((ext_vector_type(16))) (&acc)[MI][2],
                                               uint8_t* lds, int wave, int lane) {
  constexpr int ARRAY = 32 * 256, GROUP = 3 * ARRAY, BUF = 2 * GROUP;  // 32 rows of out, g and u; two groups
  // opaque: offsets formed before the K loop would hold registers through it
  asm volatile("" : "+v"(lane));
  const int lrow = lane & 31, lg = lane >> 5, grp = wave >> 2, wn = wave & 3;
  const int row0 = grp * 32 * MI, f0 = wn * 32;
  const float* SA = reinterpret_cast<const float*>(p.sa);
  const float* SB = reinterpret_cast<const float*>(p.sb);
  static_assert(2 * BUF + 8 * 64 * 4 == kGatedEpilogueLds, "epilogue buffers");
  float* s_cs = reinterpret_cast<float*>(lds + (MI == 1 ? 1 : 2) * BUF) + wave * 64;
  float st = 1.0f, rs[MI];
  if constexpr (ROW) {  // lanes 0-31: the gate rows' scales, 32-63 the up rows'
    int64_t f = ti.n0 + f0 + lrow;
    f = f < F ? f : F - 1;
    s_cs[lane] = SB[(int64_t)ti.e * 2 * F + lg * F + f];
  } else {
    st = SA[0] * SB[0];
  }
  const int32_t m_lim = (int32_t)(ti.m_end - ti.m0) - row0, f_lim = (int32_t)(F - ti.n0);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int64_t m = ti.m0 + row0 + 32 * i + lrow;
    m = m < ti.m_end ? m : ti.m_end - 1;
    rs[i] = ROW ? SA[m] : 1.0f;
  }
  __builtin_amdgcn_s_waitcnt(0);
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + (ti.m0 + row0) * F + ti.n0;
  uint16_t* gu = p.gu ? p.gu + (ti.m0 + row0) * 2 * F + ti.n0 : nullptr;
  const bool wide = F % 8 == 0 && (((uintptr_t)p.out | (uintptr_t)p.gu) & 15) == 0;
  int32_t F32 = (int32_t)F;
  asm volatile("" : "+s"(F32));
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    uint8_t* buf = lds + (i & 1) * BUF + grp * GROUP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 features: q = 2 h and 2 h + 1
      uint32_t w[3][2][2];         // out, g, u; q; pairs of features
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float cg[4], cu[4];
        if constexpr (ROW) {
          const float4 a = *reinterpret_cast<const float4*>(s_cs + 16 * h + 8 * q + 4 * lg);
          const float4 b = *reinterpret_cast<const float4*>(s_cs + 32 + 16 * h + 8 * q + 4 * lg);
          cg[0] = a.x, cg[1] = a.y, cg[2] = a.z, cg[3] = a.w;
          cu[0] = b.x, cu[1] = b.y, cu[2] = b.z, cu[3] = b.w;
        }
        float g[4], u[4], o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = acc[i][0][8 * h + 4 * q + e] * (ROW ? rs[i] * cg[e] : st);
          u[e] = acc[i][1][8 * h + 4 * q + e] * (ROW ? rs[i] * cu[e] : st);
          o[e] = gate_act<GELU>(g[e]) * u[e];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[0][q][e] = pack_bf16(o[2 * e], o[2 * e + 1]);
          w[1][q][e] = pack_bf16(g[2 * e], g[2 * e + 1]);
          w[2][q][e] = pack_bf16(u[2 * e], u[2 * e + 1]);
        }
      }
      // upper lanes' q = 0 against lower lanes' q = 1: features 16 h + 8 lg .. + 7 of the row
#pragma unroll
      for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const auto s = __builtin_amdgcn_permlane32_swap(w[c][0][e], w[c][1][e], false, false);
          w[c][0][e] = s[0], w[c][1][e] = s[1];
        }
      if (wide) {
        // a row's 16 pieces of 16 bytes swizzled by the row, so that 16 rows' stores hit all banks
        const int at = lrow * 256 + (((wn * 4 + 2 * h + lg) ^ (lrow & 15)) * 16);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c == 0 || gu)
            *reinterpret_cast<uint4*>(buf + c * ARRAY + at) =
                make_uint4(w[c][0][0], w[c][0][1], w[c][1][0], w[c][1][1]);
        continue;
      }
      const int32_t ml = 32 * i + lrow, fl = f0 + 16 * h + 8 * lg;
      if (ml >= m_lim) continue;
      const uint32_t off = (uint32_t)(ml * F32 + fl), off2 = off + (uint32_t)(ml * F32);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (fl + e >= f_lim) continue;
        const int sh = 16 * (e & 1);
        out[off + e] = (uint16_t)(w[0][e >> 2][(e >> 1) & 1] >> sh);
        if (gu) {
          gu[off2 + e] = (uint16_t)(w[1][e >> 2][(e >> 1) & 1] >> sh);
          gu[off2 + F32 + e] = (uint16_t)(w[2][e >> 2][(e >> 1) & 1] >> sh);
        }
      }
    }
    if (wide) {
      // the four waves' 32 rows are in LDS; the last step's reads of the other buffer are done as well
      wait_lgkm_and_barrier();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = 16 * s + wn * 4 + (lane >> 4), piece = lane & 15;
        const int32_t ml = 32 * i + row, fl = 8 * piece;
        const int at = row * 256 + ((piece ^ (row & 15)) * 16);
        const uint32_t off = (uint32_t)(ml * F32 + fl), off2 = off + (uint32_t)(ml * F32);
        if (ml < m_lim && fl < f_lim) {
          st_nt16(out + off, *reinterpret_cast<const uint4*>(buf + at));
          if (gu) {
            st_nt16(gu + off2, *reinterpret_cast<const uint4*>(buf + ARRAY + at));
            st_nt16(gu + off2 + F32, *reinterpret_cast<const uint4*>(buf + 2 * ARRAY + at));
          }
        }
      }
    }
  }
  // the next tile's first loads refill the ring
  wait_lgkm_and_barrier();
}

// ---------------------------------------------------------------------------
// Ping-pong kernel (tensorwise, rowwise and MX scales): 256 x 256 tile, 8 waves
// of 128 x 64 in two groups of four, one wave of each group per SIMD. The
// groups alternate between a memory phase (fragment reads of one 64-deep stage
// from LDS, LDS DMA of a later stage) and a compute phase (the 8 MFMAs of the
// stage read before), one s_barrier per phase, so each SIMD's matrix core is
// fed by one wave while the other waits on LDS and HBM. With one wave per
// SIMD doing both in turn (4 waves of 128 x 128), the in-order issue left the
// matrix cores idle whenever that wave waited on LDS: on the Llama3-8B and
// DeepSeek-V3-shaped GEMMs this kernel is 5-17% faster.
//  - v_mfma_scale_f32_32x32x64_f8f6f4, 64-deep K per instruction; measured
//    lane layout: lane l feeds row l % 32, its low 16 bytes are
//    K [16g, 16g + 16) and its high 16 bytes K [32 + 16g, 32 + 16g + 16),
//    g = l / 32, so the instruction's K order is memory order; the scale
//    operand of lane l covers row l % 32, K block g.
//  - LDS stage: 256 rows of A then 256 rows of B, 64 bytes each, 16-byte
//    chunks XOR-swizzled by (row / 4) % 4 so a wave's reads hit distinct
//    banks; the loads are global_load_lds_dwordx4 issued from inline assembly
//    with explicit vmcnt waits (the compiler cannot tell those LDS writes from
//    the fragment reads).
//  - group 0: output rows 0-127, loads the A half of every stage;
//    group 1: rows 128-255, loads the B half; wave w % 4 = column block.
//  - phase 2u: group 0 reads stage u, group 1 computes stage u - 1;
//    phase 2u + 1: group 0 computes stage u, group 1 reads stage u.
//  - ring of 4 stages; in its memory phase for stage u a wave issues its part
//    of stage u + 3 into the slot of stage u - 1 (free once group 1 read it at
//    the end of phase 2u - 1); stage u + 1 has landed (each wave waits for its
//    own loads before the barrier that ends phase 2u + 1).
//  - MX: when K % 512 == 0 and the scale pointers are 16-byte aligned, a row's
//    E8M0 bytes for four stage pairs (512-deep K) come in one 16-byte load per
//    lane with one stage in eight, into an LDS ring of two such blocks;
//    otherwise a stage pair's bytes (one dword per row, 128-deep K) ride in a
//    ring of 4 pairs with each even stage's loads. In an even stage's memory
//    phase each lane reads its rows' dwords of the pair (bytes: K blocks
//    4 p .. 4 p + 3) and shifts them right by 8 g, so byte 0 is its K block
//    of the even stage and byte 2 that of the odd one; the instruction's byte
//    select picks it. A per-stage byte read and mask cost about a sixth of
//    the MX GEMM's time on the Llama-4-style MoE shape.
//  - EX (tensorwise and rowwise scales): full-precision accumulation. The
//    compute phase decodes each 32-byte fragment to bf16 once and runs four
//    v_mfma_f32_32x32x16_bf16 per pair instead of one FP8 instruction: bytes
//    [8 q, 8 q + 8) of every lane feed instruction q, on both operands, so
//    the four instructions together take each K of the stage exactly once.
//  - GATE (kGateNone, or the activation of a gated product): N = 2F, the gate's
//    rows of B before the up projection's, and the output is act(g) u, [M][F].
//    A tile is 256 x 128 features: the 64 B rows of a wave in LDS are the 32
//    gate rows of its features, then their 32 up rows, so that a lane holds g
//    and u of the same elements in its two column blocks and the epilogue needs
//    no exchange; the main loop does not know of it. The products are transposed
//    (B rows as the instruction's rows), so that a lane has one row of the output
//    and groups of four neighbouring features. p.gu, if given, gets g and u as
//    bf16, [M][2F].
//  - BMT (gated products): rows of a tile, 256, 128 or 64, for shapes of few tiles and experts of few rows. A
//    group's waves then have half as many rows each and load half as much of A.
template <bool AE5, bool BE5, int SK, bool OF32, bool GR, bool PKB, bool EX = false, int GATE = kGateNone,
          int BMT = 256>
__global__ __launch_bounds__(512, 1) void k_gemm_fp8_pp(GemmParams p) {
  constexpr int BM = BMT, BN = 256, BK = 64, NS = 4;
  constexpr bool GT = GATE != kGateNone;
  constexpr int FN = GT ? BN / 2 : BN;  // output columns of a tile
  constexpr int TM = BM / 2, TN = 64, MI = TM / 32, NI = TN / 32;
  constexpr int SA_BYTES = BM * BK, STAGE = SA_BYTES + BN * BK;
  // wave-wide loads per wave per stage: its group's operand over 4 waves
  constexpr int DA = BM / 64, DH = BN / 64;
  typedef float v16f __attribute__((ext_vector_type(16)));
  constexpr bool MXS = SK == kScaleMX;
  constexpr int X = MXS ? 1 : 0;  // scale loads of an even stage
  static_assert(SK == kScaleTensor || SK == kScaleRow || MXS, "tensorwise, rowwise or MX");
  static_assert(!(EX && MXS), "full-precision accumulation: tensorwise or rowwise scales");
  static_assert(!GT || (!MXS && !OF32), "gated products: tensorwise or rowwise scales, bf16");
  static_assert(BM == 256 || (GT && (BM == 128 || BM == 64)), "smaller tiles: gated products");

  // the gated epilogue's two buffers and scales take the ring's place, and are larger than that of 128 rows
  constexpr int LDS = GT && BM == 128 ? kGatedEpilogueLds : NS * STAGE;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  __shared__ int32_t s_off[GR ? kMaxExperts + 1 : 2];
  __shared__ int64_t s_pref[GR ? kMaxExperts + 1 : 2];
  // MX: E8M0 scales, A rows then B rows. Either a ring of 4 stage pairs, one
  // dword per row each, or (K % 512 == 0, 16-byte aligned scales) a ring of 2
  // blocks of 4 pairs, 16 bytes per row each
  __shared__ __attribute__((aligned(16))) uint32_t s_scl[MXS ? 4 * (BM + BN) * 2 : 1];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2, wn = wave & 3, wm = grp;
  const int lrow = lane & 31, lg = lane >> 5;
  const int64_t N = p.N, K = p.K;
  const int64_t F = GT ? N / 2 : N;  // output columns
  const int64_t nt = (F + FN - 1) / FN;
  // gated, row-major: K a multiple of 16, the last stage then partly zeros
  const int64_t nk = GT ? (K + BK - 1) / BK : K / BK;
  const int32_t tail = GT && !PKB ? (int32_t)(K % BK) : 0;
  const uint32_t lds0 = lds_addr(lds);
  // MX scales 16 bytes per row at a time: a dword per row touches a cache
  // line per lane, and the DMA pays per line touched
  const bool scl16 = MXS && nk % 8 == 0 && ((uintptr_t)p.sa % 16) == 0 && ((uintptr_t)p.sb % 16) == 0;

  int64_t total;
  if constexpr (GR) {
    total = build_tile_prefix<BM, 512>(p, nt, s_off, s_pref);
  } else {
    total = ((p.M + BM - 1) / BM) * nt;
  }
  int64_t t_begin, t_end, t_step;
  xcd_range(total, t_begin, t_end, t_step);

  const int ld_row = lane >> 2, ld_pch = lane & 3;
  uint32_t fa_lo[MI], fa_hi[MI], fb_lo[NI], fb_hi[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = wm * TM + 32 * i + lrow, sw = (r >> 2) & 3;
    fa_lo[i] = (uint32_t)(r * BK + 16 * (lg ^ sw));
    fa_hi[i] = (uint32_t)(r * BK + 16 * ((lg + 2) ^ sw));
  }
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int r = wn * TN + 32 * j + lrow, sw = (r >> 2) & 3;
    fb_lo[j] = (uint32_t)(SA_BYTES + r * BK + 16 * (lg ^ sw));
    fb_hi[j] = (uint32_t)(SA_BYTES + r * BK + 16 * ((lg + 2) ^ sw));
  }

  for (int64_t t = t_begin; t < t_end; t += t_step) {
    TileInfo ti;
    // the column-tile count opaque per tile: the divisions below then form
    // their reciprocal per tile instead of holding it in a register across the
    // K loop (the MX form spilled it, and the reload waited for the previous
    // tile's stores)
    int64_t nt_t = nt;
    asm volatile("" : "+s"(nt_t));
    if constexpr (GR) {
      tile_of<BM, FN>(t, s_off, s_pref, p.E, nt_t, ti);
    } else {
      const int64_t mt = (p.M + BM - 1) / BM;
      const int64_t g = t / (kGroupM * nt_t), rem = t % (kGroupM * nt_t);
      const int64_t gm = (mt - g * kGroupM) < kGroupM ? (mt - g * kGroupM) : kGroupM;
      ti.e = 0;
      ti.m0 = (g * kGroupM + rem % gm) * BM;
      ti.m_end = p.M;
      ti.n0 = (rem / gm) * FN;
    }
    ti.m0 = uniform64(ti.m0);
    ti.m_end = uniform64(ti.m_end);
    ti.n0 = uniform64(ti.n0);
    ti.e = __builtin_amdgcn_readfirstlane(ti.e);
    const int32_t K32 = (int32_t)K;
    const int32_t a_rows = (int32_t)(ti.m_end - ti.m0);
    const int32_t b_rows = (int32_t)(F - ti.n0 < FN ? F - ti.n0 : FN);
    // B k-packed: the expert's (or the dense) [N][K] codes as 1 KB chunks of
    // 16 rows x 64 K, chunk (n / 16, k / 64) at ((n / 16) * (K / 64) + k / 64)
    // * 1024, so one
    // stage's load of 16 rows is one contiguous KB (whole cache lines) and the
    // next stage is 1 KB further
    // Grouped k-packed: A pair-interleaved, rows 2i and 2i + 1 sharing a
    // 128-byte line per 64-deep K block (row m, block s at (m / 2) * 2K +
    // s * 128 + (m % 2) * 64), so a 16-row load touches 8 or 9 whole lines
    // however the expert's rows start
    const bool pk = PKB && grp == 1;
    const bool pa = PKB && GR && grp == 0;
    const int64_t m0e = ti.m0 & ~(int64_t)1;
    const uint8_t* base = pa ? p.a + m0e * K
                          : grp == 0 ? p.a + ti.m0 * K
                          : pk       ? p.b + (int64_t)ti.e * N * K
                                     : p.b + ((int64_t)ti.e * N + ti.n0) * K;
    const int64_t sstride = pk ? 1024 : pa ? 128 : BK;
    const int32_t rows = grp == 0 ? a_rows : b_rows;
    uint32_t off[DH];
#pragma unroll
    for (int d = 0; d < DH; ++d) {
      if (grp == 0 && d >= DA) continue;
      const int r = (grp == 0 ? 16 * DA : 16 * DH) * wn + 16 * d + ld_row;
      const int c = ld_pch ^ ((r >> 2) & 3);
      if (GT && grp == 1) {
        // rows past F fetch the last; never stored
        const int fr = 32 * wn + 16 * (d & 1) + ld_row;
        if (PKB) {
          int64_t gi = ti.n0 / 16 + 2 * wn + (d & 1);
          gi = (gi < F / 16 ? gi : F / 16 - 1) + (d >> 1) * (F / 16);
          off[d] = (uint32_t)(gi * (K / 64) * 1024 + ld_row * 64 + 16 * c);
        } else {
          off[d] = (uint32_t)(((fr < rows ? fr : rows - 1) + (d >> 1) * F) * K + 16 * c);
        }
      } else if (pk) {
        // groups past N (N % 16 == 0) fetch the last group; never stored
        int64_t gi = ti.n0 / 16 + 4 * wn + d;
        gi = gi < N / 16 ? gi : N / 16 - 1;
        off[d] = (uint32_t)(gi * (K / 64) * 1024 + ld_row * 64 + 16 * c);
      } else if (pa) {
        const int32_t rr = r < rows ? r : rows - 1;
        const int64_t m = ti.m0 + rr;
        off[d] = (uint32_t)(((m >> 1) - (m0e >> 1)) * 2 * K + (m & 1) * 64 + 16 * c);
      } else {
        const int32_t rr = r < rows ? r : rows - 1;
        off[d] = (uint32_t)(rr * K32 + 16 * c);
      }
    }
    const uint32_t part_lds = grp == 0 ? (uint32_t)(wn * DA * 1024) : (uint32_t)(SA_BYTES + wn * DH * 1024);
    // the lane's 16 bytes of the last stage lie past K: it loads the stage's first ones, and zeroes them
    const int32_t ld_c = 16 * (ld_pch ^ ((ld_row >> 2) & 3));
    const bool past = tail != 0 && ld_c >= tail;
    // MX: this wave's 64 rows (those of its stage loads) of its operand's
    // E8M0 bytes, 4 per row per stage pair (rows past the expert / N fetch a
    // valid row)
    const uint8_t* sc_base = nullptr;
    uint32_t sc_off = 0u, sc_lds = 0u;
    if constexpr (MXS) {
      const int64_t kb32 = K / 32;
      const int r = 64 * wn + lane;
      const int32_t rr = r < rows ? r : rows - 1;
      sc_base = grp == 0 ? reinterpret_cast<const uint8_t*>(p.sa) + ti.m0 * kb32
                         : reinterpret_cast<const uint8_t*>(p.sb) + ((int64_t)ti.e * N + ti.n0) * kb32;
      sc_off = (uint32_t)(rr * (int32_t)kb32);
      sc_lds = (uint32_t)(4 * ((grp == 0 ? 0 : BM) + 64 * wn));
    }

    // the loads of stage s (and, s even, the scales of its pair)
    auto issue = [&](int64_t s) {
      const uint32_t slot = lds0 + (uint32_t)((s & (NS - 1)) * STAGE) + part_lds;
      const uint8_t* bk = base + s * sstride;
      const uint32_t back = GT && !PKB && past && s == nk - 1 ? (uint32_t)ld_c : 0u;
#pragma unroll
      for (int d = 0; d < DH; ++d)
        if (d < DA || grp != 0) dma16(bk, off[d] - back, slot + (uint32_t)(d * 1024));
      if constexpr (MXS) {
        const uint32_t o = sc_off + (uint32_t)(2 * s);  // byte 4 (s / 2) of the row
        if (scl16) {
          if ((s & 7) == 0) {  // pairs s / 2 .. s / 2 + 3
            const uint32_t l = lds_addr(&s_scl[((s >> 3) & 1) * 4 * (BM + BN)]) + 4 * sc_lds;
            asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(o), "s"(sc_base), "{m0}"(l) : "memory");
          }
        } else if ((s & 1) == 0) {
          const uint32_t l = lds_addr(&s_scl[((s >> 1) & 3) * (BM + BN)]) + sc_lds;
          asm volatile("global_load_lds_dword %0, %1" ::"v"(o), "s"(sc_base), "{m0}"(l) : "memory");
        }
      }
    };
    v8i fa[MI], fb[NI];
    int sa[MI], sb[NI];
    // P: the stage's parity where MX reads scales (even stages only), else 0
    auto read = [&](int64_t s, auto par) {
      constexpr int P = decltype(par)::value;
      // slot offset opaque per call: the 12 addresses are formed per read, not
      // precomputed for all 4 slots (48 registers)
      uint32_t so = (uint32_t)((s & (NS - 1)) * STAGE);
      asm volatile("" : "+s"(so));
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const uint4 lo = *reinterpret_cast<const uint4*>(lds + so + fa_lo[i]);
        const uint4 hi = *reinterpret_cast<const uint4*>(lds + so + fa_hi[i]);
        fa[i] = (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const uint4 lo = *reinterpret_cast<const uint4*>(lds + so + fb_lo[j]);
        const uint4 hi = *reinterpret_cast<const uint4*>(lds + so + fb_hi[j]);
        fb[j] = (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
      }
      if constexpr (MXS && P == 0) {
        // the row's dword of the pair s / 2 (16-byte rows: dword (s / 2) % 4),
        // shifted so this lane's K block 2 s + g sits in byte 0 and 2 s + 2 + g
        // in byte 2
        const uint32_t* dp;
        int rs;  // dwords per row
        if (scl16) {
          dp = &s_scl[((s >> 3) & 1) * 4 * (BM + BN) + (int)((s >> 1) & 3)];
          rs = 4;
        } else {
          dp = &s_scl[((s >> 1) & 3) * (BM + BN)];
          rs = 1;
        }
        const int sh = 8 * lg;
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = (int)(dp[rs * (wm * TM + 32 * i + lrow)] >> sh);
#pragma unroll
        for (int j = 0; j < NI; ++j) sb[j] = (int)(dp[rs * (BM + wn * TN + 32 * j + lrow)] >> sh);
      }
    };
    // MX: the scale operands take their final values here, in the memory
    // phase, so no VALU op on one can sit right before its MFMA. Called after
    // the fragment reads and the DMA issue: the wait these pins imply then
    // costs one LDS round trip for all reads of the phase.
    auto pin_scales = [&]() {
      if constexpr (MXS) {
#pragma unroll
        for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(sa[i]));
#pragma unroll
        for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(sb[j]));
      }
    };
    v16f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    // EX: the stage's B fragments and first A row block decoded to bf16 in
    // the memory phase, where the converts overlap the other group's
    // products; pinned there (converts have no side effects and would
    // otherwise sink past the barrier into the compute phase)
    v8bf bd[NI][4], ad[2][4];
    auto predecode = [&]() {
      if constexpr (EX) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) bd[j][q] = bf16x8<BE5>(fb[j], q);
#pragma unroll
        for (int q = 0; q < 4; ++q) ad[0][q] = bf16x8<AE5>(fa[0], q);
        asm volatile("" : "+v"(ad[0][0]), "+v"(ad[0][1]), "+v"(ad[0][2]), "+v"(ad[0][3]));
#pragma unroll
        for (int j = 0; j < NI; ++j)
          asm volatile("" : "+v"(bd[j][0]), "+v"(bd[j][1]), "+v"(bd[j][2]), "+v"(bd[j][3]));
      }
    };
    auto mma = [&](auto par) {
      constexpr int SEL = decltype(par)::value ? 2 : 0;  // MX: byte of the scale operands
      __builtin_amdgcn_s_setprio(1);
      if constexpr (EX) {
        // Each fragment decoded once per stage: both B column blocks and the
        // first A row block in the memory phase (predecode), then every
        // further A row block between the previous one's eight instructions
        // (two converts after each), into the other of two buffers, so the
        // matrix core runs while the converts issue. Every decoded fragment
        // stays live to the end of the phase, so no decode reuses a register
        // an issued instruction may still read.
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const int b = i & 1;
#pragma unroll
          for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[i][j] = GT ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(bd[j][q], ad[b][q], acc[i][j], 0, 0, 0)
                             : __builtin_amdgcn_mfma_f32_32x32x16_bf16(ad[b][q], bd[j][q], acc[i][j], 0, 0, 0);
          if (i + 1 < MI) {
#pragma unroll
            for (int q = 0; q < 4; ++q) ad[b ^ 1][q] = bf16x8<AE5>(fa[i + 1], q);
            // 4 NI instructions, 16 converts
#pragma unroll
            for (int k = 0; k < 4 * NI; ++k) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" ::"v"(ad[0][0]), "v"(ad[0][1]), "v"(ad[0][2]), "v"(ad[0][3]));
        if constexpr (MI > 1) asm volatile("" ::"v"(ad[1][0]), "v"(ad[1][1]), "v"(ad[1][2]), "v"(ad[1][3]));
#pragma unroll
        for (int j = 0; j < NI; ++j)
          asm volatile("" ::"v"(bd[j][0]), "v"(bd[j][1]), "v"(bd[j][2]), "v"(bd[j][3]));
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
        return;
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if constexpr (MXS)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], AE5 ? 1 : 0,
                                                                        BE5 ? 1 : 0, SEL, sa[i], SEL, sb[j]);
          else if constexpr (GT)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], BE5 ? 1 : 0,
                                                                        AE5 ? 1 : 0, 0, 127, 0, 127);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], AE5 ? 1 : 0,
                                                                        BE5 ? 1 : 0, 0, 127, 0, 127);
      if constexpr (SEL == 0 && MXS) {
        // an even stage's products stay before the barrier that follows: they
        // have no side effects, and the compiler would otherwise sink them
        // into the odd stage's compute phase (their first use)
        asm volatile(""
                     : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[1][0]), "+v"(acc[1][1]), "+v"(acc[2][0]),
                       "+v"(acc[2][1]), "+v"(acc[3][0]), "+v"(acc[3][1]));
      }
      __builtin_amdgcn_s_setprio(0);
    };
    // this wave's loads of stage u + 1 have landed: those issued after it
    // (stages u + 2 .. min(u + 3, nk - 1); one of two consecutive stages is
    // even and carries a scale load) may stay in flight
    // (16-byte scale rows: a scale load rides with the stages s, s % 8 == 0,
    // so it is among the later ones when u % 8 is 5 or 6; counting it there
    // keeps the wait from taking one of stage u + 2's loads early, which cost
    // about a tenth of the MX GEMM's time on the Llama-4-style MoE shape)
    auto wait_next = [&](int64_t u) {
      if (DA != DH && grp == 0 && u + 2 < nk) {
        if (u + 3 < nk) wait_vm_lgkm_and_barrier<2 * DA>();
        else wait_vm_lgkm_and_barrier<DA>();
      } else if (u + 3 < nk) {
        if (scl16) {
          if ((u & 7) == 5 || (u & 7) == 6) wait_vm_lgkm_and_barrier<2 * DH + 1>();
          else wait_vm_lgkm_and_barrier<2 * DH>();
        } else {
          wait_vm_lgkm_and_barrier<2 * DH + X>();
        }
      } else if (u + 2 < nk) {
        wait_vm_lgkm_and_barrier<DH>();  // MX: stage nk - 1 is odd
      } else {
        if (GT && !PKB && tail != 0 && u + 2 == nk) {
          // this wave's loads of the last stage have landed, and nobody reads it before the barrier
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          if (past) {
            uint8_t* at = lds + (int)((nk - 1) & (NS - 1)) * STAGE + part_lds + 16 * lane;
#pragma unroll
            for (int d = 0; d < DH; ++d)
              if (d < DA || grp != 0) *reinterpret_cast<uint4*>(at + d * 1024) = make_uint4(0, 0, 0, 0);
          }
        }
        wait_vm_lgkm_and_barrier<0>();
      }
    };

    // prologue: stages 0 .. min(nk, 3) - 1; then stage 0 has landed
    issue(0);
    issue(1);
    if (nk >= 3) {
      issue(2);
      if (DA != DH && grp == 0) wait_vm_lgkm_and_barrier<2 * DA>();
      else if (scl16) wait_vm_lgkm_and_barrier<2 * DH>();
      else wait_vm_lgkm_and_barrier<2 * DH + X>();
    } else {
      if (DA != DH && grp == 0) wait_vm_lgkm_and_barrier<DA>();
      else wait_vm_lgkm_and_barrier<DH>();
    }
    // both groups run the same loop, group 1 one phase behind: memory phase
    // (reads of stage u, loads of stage u + 3, own loads of stage u + 1
    // landed), barrier, compute phase (MFMAs of stage u), barrier
    if (grp == 1) wait_vm_lgkm_and_barrier<63>();
    auto phase = [&](int64_t u, auto par) {
      read(u, par);
      if (u + 3 < nk) issue(u + 3);
      pin_scales();
      predecode();
      wait_next(u);
      __builtin_amdgcn_sched_barrier(0);
      mma(par);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
    };
    if constexpr (MXS) {
      // stage pairs (nk is even): the odd stage reuses the pair's scale dwords
      for (int64_t u = 0; u < nk; u += 2) {
        phase(u, std::integral_constant<int, 0>{});
        phase(u + 1, std::integral_constant<int, 1>{});
      }
    } else {
      for (int64_t u = 0; u < nk; ++u) phase(u, std::integral_constant<int, 0>{});
    }
    if (grp == 0) asm volatile("s_barrier" ::: "memory");

    // ---- epilogue (the ring is idle: every wave passed the last barrier) ----
    const float* SA = reinterpret_cast<const float*>(p.sa);
    const float* SB = reinterpret_cast<const float*>(p.sb);
    if constexpr (GT) {
      gated_epilogue<GATE == kGateGelu, SK == kScaleRow, MI>(p, ti, F, acc, lds, wave, lane);
      continue;
    }
    float cs[NI];
    float st = 1.0f;
    if constexpr (SK == kScaleTensor || MXS) {
      if constexpr (!MXS) st = SA[0] * SB[0];
#pragma unroll
      for (int j = 0; j < NI; ++j) cs[j] = 1.0f;
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        int64_t n = ti.n0 + wn * TN + 32 * j + lrow;
        n = n < N ? n : N - 1;
        cs[j] = SB[(int64_t)ti.e * N + n];
      }
    }
    const int32_t m_lim = (int32_t)(ti.m_end - ti.m0);
    const int32_t n_lim = (int32_t)(F - ti.n0);
    float* s_rs = reinterpret_cast<float*>(lds) + wave * TM;
    if constexpr (SK == kScaleRow) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int64_t m = ti.m0 + wm * TM + 64 * h + lane;
        m = m < ti.m_end ? m : ti.m_end - 1;
        s_rs[64 * h + lane] = SA[m];
      }
    }
    __builtin_amdgcn_s_waitcnt(0);
    int32_t N32 = (int32_t)F;
    asm volatile("" : "+s"(N32));
    int32_t ml0 = wm * TM + 4 * lg, nl0 = wn * TN + lrow;
    asm volatile("" : "+v"(ml0), "+v"(nl0));
    const int64_t corner = ti.m0 * F + ti.n0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float4 rs4 = make_float4(st, st, st, st);
        if constexpr (SK == kScaleRow) rs4 = *reinterpret_cast<const float4*>(&s_rs[32 * i + 8 * q + 4 * lg]);
        const float rsv[4] = {rs4.x, rs4.y, rs4.z, rs4.w};
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int32_t nl = nl0 + 32 * j;
          if (nl >= n_lim) continue;
#pragma unroll
          for (int t2 = 0; t2 < 4; ++t2) {
            const int32_t ml = ml0 + 32 * i + 8 * q + t2;
            if (ml >= m_lim) continue;
            const uint32_t o = (uint32_t)(ml * N32 + nl);
            const float v = acc[i][j][4 * q + t2] * rsv[t2] * cs[j];
            if constexpr (OF32)
              (reinterpret_cast<float*>(p.out) + corner)[o] = v;
            else
              (reinterpret_cast<uint16_t*>(p.out) + corner)[o] = f32_to_bf16_rne(v);
          }
        }
      }
    }
    // the next tile's first loads refill slot 0, which holds the row scales
    if constexpr (SK == kScaleRow) __syncthreads();
  }
}

}  // namespace fp8dyn
