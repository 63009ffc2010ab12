// gemm_gated_pp.hpp -- the gated product's kernel for many rows, and its epilogue.
#pragma once

#include "gated.hpp"
#include "gemm_common.hpp"

namespace fp8dyn {

// LDS of the epilogue: 32 rows of out, g and u of two groups of waves, and the waves' 64 column scales.
constexpr int kGatedBuf = 2 * 3 * 32 * 256, kGatedEpilogueLds = kGatedBuf + 8 * 64 * 4;

// Epilogue of a gated tile of 64 MI rows x 128 features. A wave has 32 MI rows x 32 features: element 4 q + u of
// block i is row 32 i + lane % 32, feature 8 q + 4 (lane / 32) + u; block column 0 holds g, column 1 u. Lanes l
// and l + 32 exchange halves of two neighbouring q, after which each has 8 features of its row. Every 32 rows of
// a group's four waves then go through LDS, so that a store writes whole lines, 256 bytes of each of four rows.
// Measured, 8192 x 14336 x 4096 with both projections: single values 796 us (without the projections 757), 16 bytes
// of 32 rows 838 (732), whole lines 782 (715): lines that are written in parts leave the caches half full.
// F % 8 != 0 or outputs off 16 bytes: single values. rs: the lane's row scales; cs: its column scale (lanes 0-31 of
// the gate rows, 32-63 of the up rows); both with the one scale of a tensorwise product where ROW is false.
template <bool GELU, bool ROW, int MI>
__device__ __forceinline__ void gated_epilogue(const GemmParams& p, const TileInfo& ti, int64_t F,
                                               const float __attribute__((ext_vector_type(16))) (&acc)[MI][2],
                                               const float (&rs)[MI], float cs, bool wide, uint8_t* lds, int wave,
                                               int lane) {
  constexpr int ARRAY = 32 * 256, GROUP = 3 * ARRAY;
  // opaque: offsets formed before the K loop would hold registers through it
  asm volatile("" : "+v"(lane));
  const int lrow = lane & 31, lg = lane >> 5, grp = wave >> 2, wn = wave & 3;
  const int row0 = grp * 32 * MI, f0 = wn * 32;
  float* s_cs = reinterpret_cast<float*>(lds + kGatedBuf) + wave * 64;
  if constexpr (ROW) {
    s_cs[lane] = cs;  // read by this wave alone
    wave_lds_fence();
  }
  const int32_t m_lim = (int32_t)(ti.m_end - ti.m0) - row0, f_lim = (int32_t)(F - ti.n0);
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + (ti.m0 + row0) * F + ti.n0;
  uint16_t* gu = p.gu ? p.gu + (ti.m0 + row0) * 2 * F + ti.n0 : nullptr;
  int32_t F32 = (int32_t)F;
  asm volatile("" : "+s"(F32));
  uint8_t* buf = lds + grp * GROUP;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
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
          g[e] = acc[i][0][8 * h + 4 * q + e] * (ROW ? rs[i] * cg[e] : cs);
          u[e] = acc[i][1][8 * h + 4 * q + e] * (ROW ? rs[i] * cu[e] : cs);
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
      wait_lgkm_and_barrier();  // the four waves' 32 rows are in LDS
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
      wait_lgkm_and_barrier();  // and have been read
    }
  }
}

// ---------------------------------------------------------------------------
// Ping-pong kernel of the gated product: the tiles, the ring, the phases and the operands' layouts are those of
// k_gemm_fp8_pp (gemm_fp8_fast.hip), which says why; tensorwise and rowwise scales. What differs:
//  - N = 2F, the gate's rows of B before the up projection's. A tile is BM rows x 128 features: the 64 B rows of a
//    wave in LDS are the 32 gate rows of its features, then their 32 up rows, so that a lane holds g and u of the
//    same elements in its two column blocks and forms act(g) u without an exchange.
//  - The products are transposed (B rows as the instruction's rows), so that a lane has one row of the output and
//    groups of four neighbouring features.
//  - BM = 256, 128 or 64 rows, for shapes of few tiles and experts of few rows: a group's waves then have half as
//    many rows each and load half as much of A.
//  - The loop's last three phases, which load nothing and wait in steps, are a loop of their own: with the shorter
//    tiles a phase has few products, and its branches showed (512 x 2048 x 4096 26.7 -> 20.1 us, 1024 x 2048 x 2048
//    17.6 -> 14.4; a ring of five or six stages was no faster: 21.7 and 15.6). With 256 rows and full precision it
//    gains 3% where B is packed and costs 2% where it is not (8192 x 4096 x 4096 374 -> 361, 370 -> 377).
//  - K is any multiple of 16 above 64 where B is row-major: the lanes whose 16 bytes of the last stage lie past K
//    load the stage's first ones instead, and zero them once they have landed.
//  - The lane's scales are loaded at a tile's start, and the next tile's first stages are under way during a
//    tile's epilogue, whose buffer is the ring's last slot and what lies behind it. (Its first phases wait for the
//    epilogue's stores, which the counter of outstanding accesses holds with the loads. Waits that left the known
//    number of a whole tile's stores outstanding gained 0.5 to 1%, and cost the loop its registers.)
template <int SK, bool GR, bool PKB, bool EX, int GATE, int BM>
__global__ __launch_bounds__(512, 1) void k_gated_pp(GemmParams p) {
  constexpr int BN = 256, BK = 64, NS = 4, FN = BN / 2;
  constexpr int TM = BM / 2, TN = 64, MI = TM / 32, NI = TN / 32;
  constexpr int SA_BYTES = BM * BK, STAGE = SA_BYTES + BN * BK;
  constexpr int DA = BM / 64, DB = BN / 64;  // wave-wide loads per wave per stage, of A (group 0) and B (group 1)
  constexpr bool ROW = SK == kScaleRow;
  typedef float v16f __attribute__((ext_vector_type(16)));
  static_assert(SK == kScaleTensor || SK == kScaleRow, "tensorwise or rowwise scales");
  static_assert(BM == 256 || BM == 128 || BM == 64, "rows of a tile");

  constexpr int LDS = (NS - 1) * STAGE + (STAGE > kGatedEpilogueLds ? STAGE : kGatedEpilogueLds);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  __shared__ int32_t s_off[GR ? kMaxExperts + 1 : 2];
  __shared__ int64_t s_pref[GR ? kMaxExperts + 1 : 2];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2, wn = wave & 3, wm = grp;
  const int lrow = lane & 31, lg = lane >> 5;
  const int64_t N = p.N, K = p.K, F = N / 2;
  const int64_t nt = (F + FN - 1) / FN;
  const int64_t nk = (K + BK - 1) / BK;
  const int32_t tail = PKB ? 0 : (int32_t)(K % BK);
  const uint32_t lds0 = lds_addr(lds);
  const float* SA = reinterpret_cast<const float*>(p.sa);
  const float* SB = reinterpret_cast<const float*>(p.sb);
  const bool wide = F % 8 == 0 && (((uintptr_t)p.out | (uintptr_t)p.gu) & 15) == 0;

  int64_t total;
  if constexpr (GR)
    total = build_tile_prefix<BM, 512>(p, nt, s_off, s_pref);
  else
    total = ((p.M + BM - 1) / BM) * nt;
  int64_t t_begin, t_end, t_step;
  xcd_range(total, t_begin, t_end, t_step);
  if (t_begin >= t_end) return;

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
  // the chunk of a row that this lane fetches: the swizzle goes by the row's place in 16, the same for all loads
  const int32_t ld_c = 16 * (ld_pch ^ ((ld_row >> 2) & 3));
  const bool past = tail != 0 && ld_c >= tail;  // past K in the last stage
  const uint32_t part_lds = grp == 0 ? (uint32_t)(wn * DA * 1024) : (uint32_t)(SA_BYTES + wn * DB * 1024);
  const bool pk = PKB && grp == 1, pa = PKB && GR && grp == 0;
  const int64_t sstride = pk ? 1024 : pa ? 128 : BK;

  // the tile whose stages are loaded: set by aim(), one tile ahead of the products during an epilogue
  TileInfo ti;
  const uint8_t* base;
  uint32_t off[DB];
  auto aim = [&](int64_t t) {
    int64_t nt_t = nt;
    asm volatile("" : "+s"(nt_t));  // the divisions' reciprocal formed per tile, not held through the K loop
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
    const int64_t m0e = ti.m0 & ~(int64_t)1;
    base = pa         ? p.a + m0e * K
           : grp == 0 ? p.a + ti.m0 * K
           : pk       ? p.b + (int64_t)ti.e * N * K
                      : p.b + ((int64_t)ti.e * N + ti.n0) * K;
    // rows past the expert's end and features past F fetch the last one; never stored
    const int32_t rows = grp == 0 ? (int32_t)(ti.m_end - ti.m0) : (int32_t)(F - ti.n0 < FN ? F - ti.n0 : FN);
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      if (grp == 0) {
        const int r = 16 * DA * wn + 16 * d + ld_row;
        const int32_t rr = r < rows ? r : rows - 1;
        const int64_t m = ti.m0 + rr;
        if (pa)
          off[d] = (uint32_t)(((m >> 1) - (m0e >> 1)) * 2 * K + (m & 1) * 64 + ld_c);
        else
          off[d] = (uint32_t)(rr * (int32_t)K + ld_c);
      } else if (PKB) {
        int64_t gi = ti.n0 / 16 + 2 * wn + (d & 1);
        gi = (gi < F / 16 ? gi : F / 16 - 1) + (d >> 1) * (F / 16);
        off[d] = (uint32_t)(gi * (K / 64) * 1024 + ld_row * 64 + ld_c);
      } else {
        const int fr = 32 * wn + 16 * (d & 1) + ld_row;
        off[d] = (uint32_t)(((fr < rows ? fr : rows - 1) + (d >> 1) * F) * K + ld_c);
      }
    }
  };
  // the loads of stage s into a slot of the ring
  auto issue = [&](int64_t s, int at) {
    const uint32_t slot = lds0 + (uint32_t)(at * STAGE) + part_lds;
    const uint8_t* bk = base + s * sstride;
    const uint32_t back = !PKB && past && s == nk - 1 ? (uint32_t)ld_c : 0u;
#pragma unroll
    for (int d = 0; d < DB; ++d)
      if (d < DA || grp != 0) dma16(bk, off[d] - back, slot + (uint32_t)(d * 1024));
  };
  auto prologue = [&]() {
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      if (s < 2 || s < nk) issue(s, s);
  };
  v8i fa[MI], fb[NI];
  auto read = [&](int at) {
    // slot offset opaque per call: the addresses are formed per read, not precomputed for all slots
    uint32_t so = (uint32_t)(at * STAGE);
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
  };
  v16f acc[MI][NI];
  // EX: B and the first A row block decoded in the memory phase, further row blocks between products
  v8bf bd[NI][4], ad[2][4];
  auto predecode = [&]() {
    if constexpr (EX) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) bd[j][q] = bf16x8<false>(fb[j], q);
#pragma unroll
      for (int q = 0; q < 4; ++q) ad[0][q] = bf16x8<false>(fa[0], q);
      asm volatile("" : "+v"(ad[0][0]), "+v"(ad[0][1]), "+v"(ad[0][2]), "+v"(ad[0][3]));
#pragma unroll
      for (int j = 0; j < NI; ++j)
        asm volatile("" : "+v"(bd[j][0]), "+v"(bd[j][1]), "+v"(bd[j][2]), "+v"(bd[j][3]));
    }
  };
  auto mma = [&]() {
    __builtin_amdgcn_s_setprio(1);
    if constexpr (EX) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int b = i & 1;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bd[j][q], ad[b][q], acc[i][j], 0, 0, 0);
        if (i + 1 < MI) {
#pragma unroll
          for (int q = 0; q < 4; ++q) ad[b ^ 1][q] = bf16x8<false>(fa[i + 1], q);
#pragma unroll
          for (int k = 0; k < 4 * NI; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // live to the end of the phase: no decode reuses a register that an issued instruction may still read
      asm volatile("" ::"v"(ad[0][0]), "v"(ad[0][1]), "v"(ad[0][2]), "v"(ad[0][3]));
      if constexpr (MI > 1) asm volatile("" ::"v"(ad[1][0]), "v"(ad[1][1]), "v"(ad[1][2]), "v"(ad[1][3]));
#pragma unroll
      for (int j = 0; j < NI; ++j)
        asm volatile("" ::"v"(bd[j][0]), "v"(bd[j][1]), "v"(bd[j][2]), "v"(bd[j][3]));
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 0, 0, 0, 127, 0, 127);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // waits until at most `stages` stages of this wave's loads are outstanding, then for the barrier
  auto wait_but = [&](int64_t stages) {
    if (stages >= 2) {
      if (DA != DB && grp == 0) wait_vm_lgkm_and_barrier<2 * DA>();
      else wait_vm_lgkm_and_barrier<2 * DB>();
    } else if (stages == 1) {
      if (DA != DB && grp == 0) wait_vm_lgkm_and_barrier<DA>();
      else wait_vm_lgkm_and_barrier<DB>();
    } else {
      wait_vm_lgkm_and_barrier<0>();
    }
  };
  // this wave's loads of stage u + 1 have landed: later ones, up to stage u + NS - 1, may stay in flight
  auto wait_next = [&](int64_t u, int last) {
    if (!PKB && tail != 0 && u + 2 == nk) {
      // this wave's loads of the last stage have landed, and nobody reads it before the barrier
      wait_vm<0>();
      if (past) {
        uint8_t* at = lds + last * STAGE + part_lds + 16 * lane;
#pragma unroll
        for (int d = 0; d < DB; ++d)
          if (d < DA || grp != 0) *reinterpret_cast<uint4*>(at + d * 1024) = make_uint4(0, 0, 0, 0);
      }
    }
    wait_but(nk - 2 - u);
  };

  aim(t_begin);
  prologue();
  for (int64_t t = t_begin; t < t_end; t += t_step) {
    const TileInfo cur = ti;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    // opaque: a first phase with a constant 0 for the accumulator may get a destination that overlaps its sources,
    // and this compiler does not keep multi-pass instructions from that
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    // stage 0 has landed
    wait_but(nk - 1);
    // the lane's scales, for the epilogue (the next two waits take them for loads of a stage: stricter, by
    // loads that have long landed)
    float rs[MI], cs;
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t m = cur.m0 + wm * TM + 32 * i + lrow;
        rs[i] = SA[m < cur.m_end ? m : cur.m_end - 1];
      }
      const int64_t f = cur.n0 + wn * 32 + lrow;
      cs = SB[(int64_t)cur.e * N + lg * F + (f < F ? f : F - 1)];
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i) rs[i] = 1.0f;
      cs = SA[0] * SB[0];
    }
    // two wait states between the address arithmetic above and the products, however the blocks are laid out
    asm volatile("s_nop 1" ::: "memory");
    // both groups run the same loop, group 1 one phase behind
    if (grp == 1) wait_vm_lgkm_and_barrier<63>();
    // slots of stage u and of the last one issued
    int rd = 0, last = (int)(nk < NS ? nk - 1 : NS - 2);
    auto products = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      // no vector instruction right before the products, in any order of the blocks
      asm volatile("s_nop 1" ::: "memory");
      mma();
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
      rd = rd + 1 == NS ? 0 : rd + 1;
    };
    int64_t u = 0;
    for (; u + NS - 1 < nk; ++u) {  // loads under way all the time
      read(rd);
      last = rd == 0 ? NS - 1 : rd - 1;
      issue(u + NS - 1, last);
      predecode();
      wait_but(NS - 2);
      products();
    }
    for (; u < nk; ++u) {
      read(rd);
      predecode();
      wait_next(u, last);
      products();
    }
    if (grp == 0) asm volatile("s_barrier" ::: "memory");
    // the ring is idle: every wave passed the last barrier. The scales are waited for here, with nothing else
    // outstanding.
#pragma unroll
    for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(rs[i]));
    asm volatile("" : "+v"(cs));
    const bool more = t + t_step < t_end;
    if (more) {
      aim(t + t_step);
      prologue();
    }
    gated_epilogue<GATE == kGateGelu, ROW, MI>(p, cur, F, acc, rs, cs, wide, lds + (NS - 1) * STAGE, wave, lane);
  }
}

}  // namespace fp8dyn
