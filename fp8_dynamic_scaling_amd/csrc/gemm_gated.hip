// gemm_gated.hip -- the gated product of a feed-forward block, act(a Wg^T) (a Wu^T), as one FP8 GEMM:
// dense, and grouped over a device offset tensor.
//
// Both projections are one product with N = 2F. A tile holds the gate and up rows of the same features, so that
// both end up in the same lane, and the epilogue forms act(g) u in fp32 and rounds it once. The projections
// themselves are written only for a backward: without them F values a row leave the kernel instead of 2F, and no
// pass reads them again.
//  - k_gated_pp (gemm_gated_pp.hpp): many rows, bound by the matrix cores. Measured, 8192 x 14336 x 4096: 717 to
//    744 us (2.59 to 2.68 PFLOP/s; the library's plain FP8 product of the same size reaches 2.75), with both
//    projections, 0.7 GB of stores in all, 758 to 816; full precision 1261 to 1302 and 1303 to 1350 us.
//  - k_gated_few (below): few rows, bound by reading the weights. One token of 14336 x 4096: 20.5 to 22 us (5.3 to
//    5.7 TB/s), 16 tokens 25.
//  - k_gemm_fp8 (gemm_generic.hpp): grouped products of K up to 64 or weights past 32-bit offsets.
// gated_tiles.hpp has the rule that chooses.
#include <algorithm>

#include "gated_tiles.hpp"
#include "gemm_gated_pp.hpp"
#include "gemm_generic.hpp"

namespace fp8dyn {

namespace {

// ---------------------------------------------------------------------------
// Few rows (and small products): one pass over the weights, straight from memory to registers.
//  - A workgroup has 16 features, their 16 gate and 16 up rows of B, and 16 MT rows of A; its waves share K in
//    units of 128, so that a short K too has its loads under way at once. Their sums meet in LDS, in order.
//  - Loads go along the rows, eight lanes a line of 128 bytes (k-packed: a chunk's contiguous KB), and are turned
//    in the wave's own piece of LDS into what the instruction's lanes want: row lane % 16, K [16 g, 16 g + 16) and
//    [64 + 16 g, 64 + 16 g + 16) of the unit, g = lane / 16. Loaded as the lanes want it, a load touches 16 rows
//    and takes up to four times as long.
//  - The codes are decoded to bf16 and multiplied by v_mfma_f32_16x16x32_bf16, features as the instruction's
//    rows: full-precision sums, with either use_fast_accum (the products are a small part), and a lane ends with
//    4 neighbouring features of a row.
//  - D units are in flight a wave.
template <int MT, int WV, int GATE, bool PKB, bool ROW>
__global__ __launch_bounds__(64 * WV) void k_gated_few(GemmParams p) {
  constexpr int D = 2;
  constexpr int ROWS = 32 + 16 * MT, STRIDE = 144;  // rows of a unit in LDS; 16 rows' pieces hit all banks
  constexpr int WAVE_BYTES = ROWS * STRIDE;
  constexpr int RED = WV * 8 * MT * 64 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[WV * WAVE_BYTES > RED ? WV * WAVE_BYTES : RED];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t F = p.N / 2, K = p.K, M = p.M;
  const int64_t units = (K + 127) / 128;
  const int64_t u0 = wave * units / WV, u1 = (wave + 1) * units / WV;
  uint8_t* mine = lds + wave * WAVE_BYTES;
  const int64_t f0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  // a unit's loads: 4 of B (row-major: 8 rows each, gate rows first; k-packed: gate chunks, then up chunks),
  // 2 MT of A (8 rows each). Rows past F or M read the last one, and are never stored.
  const int lr = lane >> 3, lp = lane & 7;
  const uint8_t* wp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (PKB) {
      wp[j] = p.b + (((j >> 1) * F + f0) / 16 * (K / 64) + (j & 1)) * 1024 + lane * 16;
    } else {
      const int64_t f = f0 + 8 * (j & 1) + lr;
      wp[j] = p.b + ((j >> 1) * F + (f < F ? f : F - 1)) * K;
    }
  }
  const uint8_t* ap[2 * MT];
#pragma unroll
  for (int j = 0; j < 2 * MT; ++j) {
    const int64_t m = m0 + 8 * j + lr;
    ap[j] = p.a + (m < M ? m : M - 1) * K;
  }
  struct Unit {
    u32x4 w[4], a[2 * MT];
  } buf[D];
  auto load = [&](Unit& b, int64_t u) {
    // the last unit may be shorter: its pieces past K read the row's last one instead
    int64_t o = 128 * u + 16 * lp;
    o = o < K - 16 ? o : K - 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b.w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[j] + (PKB ? u * 2048 : o)));
#pragma unroll
    for (int j = 0; j < 2 * MT; ++j) b.a[j] = *reinterpret_cast<const u32x4*>(ap[j] + o);
  };
  v4f acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  auto frag = [&](int row0) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(mine + (row0 + r) * STRIDE + 16 * g);
    const u32x4 y = *reinterpret_cast<const u32x4*>(mine + (row0 + r) * STRIDE + 64 + 16 * g);
    return (v8i){(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };
  auto compute = [&](Unit& b, int64_t u) {
    if (!PKB && 128 * u + 128 > K) {  // pieces past K are codes of 0 on both sides
      const uint32_t in = 128 * u + 16 * lp < K ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) b.w[j] &= in;
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) b.a[j] &= in;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = PKB ? 16 * (j >> 1) + (lane >> 2) : 8 * j + lr;
      const int piece = PKB ? 4 * (j & 1) + (lane & 3) : lp;
      *reinterpret_cast<u32x4*>(mine + row * STRIDE + 16 * piece) = b.w[j];
    }
#pragma unroll
    for (int j = 0; j < 2 * MT; ++j) *reinterpret_cast<u32x4*>(mine + (32 + 8 * j + lr) * STRIDE + 16 * lp) = b.a[j];
    wave_lds_fence();
    v8bf wb[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v8i f = frag(16 * h);
#pragma unroll
      for (int q = 0; q < 4; ++q) wb[h][q] = bf16x8<false>(f, q);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const v8i f = frag(32 + 16 * i);
      v8bf ab[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) ab[q] = bf16x8<false>(f, q);
      // two wait states between a decode and the instruction that reads it
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_nop 1" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[h][q], ab[q], acc[i][h], 0, 0, 0);
      asm volatile("" ::"v"(ab[0]), "v"(ab[1]), "v"(ab[2]), "v"(ab[3]));
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) asm volatile("" ::"v"(wb[h][0]), "v"(wb[h][1]), "v"(wb[h][2]), "v"(wb[h][3]));
    wave_lds_fence();  // the next unit's stores come behind these reads
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (u0 + d < u1) load(buf[d], u0 + d);
  int64_t u = u0;
  for (; u + 2 * D <= u1; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(buf[d], u + d);
      load(buf[d], u + D + d);
    }
  }
  for (; u < u1; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (u + d < u1) compute(buf[d], u + d);
      if (u + D + d < u1) load(buf[d], u + D + d);
    }
  }
  __syncthreads();  // the sums take the units' place
  float(*red)[8 * MT][64] = reinterpret_cast<float(*)[8 * MT][64]>(lds);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][8 * i + 4 * h + e][lane] = acc[i][h][e];
  __syncthreads();
  // wave i: the rows 16 i + lane % 16, features 4 (lane / 16) + e
  const int64_t m = m0 + 16 * wave + r;
  const int64_t f = f0 + 4 * g;
  if (wave >= MT || m >= M || f >= F) return;
  const float* SA = reinterpret_cast<const float*>(p.sa);
  const float* SB = reinterpret_cast<const float*>(p.sb);
  const float sm = ROW ? SA[m] : SA[0];
  float gt[4], up[4], h[4];
  const int left = F - f < 4 ? (int)(F - f) : 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float s[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int v = 8 * wave + 4 * c + e;
      s[c] = red[0][v][lane];
#pragma unroll
      for (int x = 1; x < WV; ++x) s[c] += red[x][v][lane];
    }
    const int64_t fe = e < left ? f + e : f;
    gt[e] = s[0] * sm * (ROW ? SB[fe] : SB[0]);
    up[e] = s[1] * sm * (ROW ? SB[F + fe] : SB[0]);
    h[e] = gate_act<GATE == kGateGelu>(gt[e]) * up[e];
  }
  auto put = [&](uint16_t* o, const float* x) {
    if (left == 4 && ((uintptr_t)o & 7) == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) o[e] = (uint16_t)pack_bf16(x[e], 0.0f);
  };
  put(reinterpret_cast<uint16_t*>(p.out) + m * F + f, h);
  if (p.gu) {
    put(p.gu + m * p.N + f, gt);
    put(p.gu + m * p.N + F + f, up);
  }
}

template <int GATE, int SK>
hipError_t launch_few(const GatedMmArgs& g) {
  constexpr bool ROW = SK == kScaleRow;
  const int64_t nf = (g.F + 15) / 16;
  auto fits = [&](int m) { return nf * ((g.M + 16 * m - 1) / (16 * m)) <= 256; };
  // fewer rows a workgroup where that many still run at once (40 x 512 x 4096: 64 rows 11.0 us, 32 7.8, 16 6.4;
  // 333 x 1040 x 720, more than run at once, 8.3, 8.2 and 10.7)
  const int mt = g.M <= 16 || fits(1) ? 1 : g.M <= 32 || fits(2) ? 2 : 4;
  const int64_t nm = (g.M + 16 * mt - 1) / (16 * mt);
  // eight waves for K where few registers or few workgroups let them all run
  const bool eight = mt == 1 || nf * nm <= 256;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(65535, ((int64_t)1 << 22) / nf));  // of one grid
  for (int64_t y = 0; y < nm; y += most) {
    const int64_t m0 = y * 16 * mt;
    GemmParams p{g.a + m0 * g.K, g.b, g.sa + (ROW ? m0 : 0), g.sb, nullptr, 1, g.M - m0, 2 * g.F, g.K,
                 g.out + m0 * g.F, g.gu ? g.gu + m0 * 2 * g.F : nullptr};
    const dim3 grid((unsigned)nf, (unsigned)std::min<int64_t>(most, nm - y));
    auto run = [&](auto m) {
      constexpr int MT = decltype(m)::value;
      if (eight) {
        if (g.packed) hipLaunchKernelGGL((k_gated_few<MT, 8, GATE, true, ROW>), grid, dim3(512), 0, g.stream, p);
        else hipLaunchKernelGGL((k_gated_few<MT, 8, GATE, false, ROW>), grid, dim3(512), 0, g.stream, p);
      } else {
        if (g.packed) hipLaunchKernelGGL((k_gated_few<MT, 4, GATE, true, ROW>), grid, dim3(256), 0, g.stream, p);
        else hipLaunchKernelGGL((k_gated_few<MT, 4, GATE, false, ROW>), grid, dim3(256), 0, g.stream, p);
      }
    };
    if (mt == 1) run(std::integral_constant<int, 1>{});
    else if (mt == 2) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 4>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int GATE, int SK, bool GR, bool PKB, bool EX, int BM>
hipError_t launch_pp_rows(const GatedMmArgs& g) {
  GemmParams p{g.a, g.b, g.sa, g.sb, g.offsets, g.E, g.M, 2 * g.F, g.K, g.out, g.gu};
  const int64_t nt = (g.F + 127) / 128;
  const int64_t tiles = ((g.M + BM - 1) / BM + (GR ? g.E : 0)) * nt;
  int64_t grid = device_cus();
  if (tiles < grid) grid = tiles;
  if (grid >= kNumXcd) grid -= grid % kNumXcd;
  hipLaunchKernelGGL((k_gated_pp<SK, GR, PKB, EX, GATE, BM>), dim3((unsigned)grid), dim3(512),
                     0, g.stream, p);
  return hipGetLastError();
}

template <int GATE, int SK, bool GR, bool PKB, bool EX>
hipError_t launch_pp(const GatedMmArgs& g, int rows) {
  return rows == 64    ? launch_pp_rows<GATE, SK, GR, PKB, EX, 64>(g)
         : rows == 128 ? launch_pp_rows<GATE, SK, GR, PKB, EX, 128>(g)
                       : launch_pp_rows<GATE, SK, GR, PKB, EX, 256>(g);
}

// Grouped products of K below two stages, or of weights past 32-bit offsets.
template <int GATE, bool EX>
hipError_t launch_generic(const GatedMmArgs& g) {
  GemmParams p{g.a, g.b, g.sa, g.sb, g.offsets, g.E, g.M, 2 * g.F, g.K, g.out, g.gu};
  const int64_t tiles = ((g.M + 127) / 128 + g.E) * ((g.F + 63) / 64);
  int64_t grid = device_cus();
  if (tiles < grid)
    grid = tiles;
  else if (grid >= kNumXcd)
    grid -= grid % kNumXcd;
  hipLaunchKernelGGL((k_gemm_fp8<128, 128, 2, 2, false, false, kScaleRow, false, EX, GATE>), dim3((unsigned)grid),
                     dim3(256), 0, g.stream, p);
  return hipGetLastError();
}

// Grouped products of K = 0: act(0) * 0 in the experts' rows; those behind stay. end: offsets[E].
__global__ void k_gated_zero(const int32_t* end, int64_t M, int64_t F, uint16_t* out, uint16_t* gu) {
  const int64_t last = *end, n = (last < 0 ? 0 : last < M ? last : M) * F;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    out[i] = 0;
    if (gu) gu[2 * i] = gu[2 * i + 1] = 0;
  }
}

template <int GATE, int SK, bool EX>
hipError_t launch_form(const GatedMmArgs& g) {
  const int rows = gated_tile_rows(g.M, g.F, g.K, g.offsets ? g.E : 0, g.packed, g.exact, device_cus());
  if (rows == kGatedFew) return launch_few<GATE, SK>(g);
  if constexpr (SK == kScaleRow) {
    if (rows == kGatedGeneric) return launch_generic<GATE, EX>(g);
    if (g.offsets)
      return g.packed ? launch_pp<GATE, SK, true, true, EX>(g, rows) : launch_pp<GATE, SK, true, false, EX>(g, rows);
  }
  return g.packed ? launch_pp<GATE, SK, false, true, EX>(g, rows) : launch_pp<GATE, SK, false, false, EX>(g, rows);
}

template <int GATE>
hipError_t launch_act(const GatedMmArgs& g) {
  if (g.row_scales) return g.exact ? launch_form<GATE, kScaleRow, true>(g) : launch_form<GATE, kScaleRow, false>(g);
  return g.exact ? launch_form<GATE, kScaleTensor, true>(g) : launch_form<GATE, kScaleTensor, false>(g);
}

}  // namespace

bool gated_mm_packed_ok(const GatedMmArgs& g) { return gated_fast_eligible(g.F, g.K); }

hipError_t launch_gated_mm(const GatedMmArgs& g) {
  if (g.K == 0) {
    const int64_t grid = std::min<int64_t>((g.M * g.F + 255) / 256, 8 * (int64_t)device_cus());
    hipLaunchKernelGGL(k_gated_zero, dim3((unsigned)grid), dim3(256), 0, g.stream, g.offsets + g.E, g.M, g.F, g.out,
                       g.gu);
    return hipGetLastError();
  }
  return g.gelu ? launch_act<kGateGelu>(g) : launch_act<kGateSilu>(g);
}

}  // namespace fp8dyn
