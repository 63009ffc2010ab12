// gemm_gated.hip -- the gated product of a feed-forward block, act(a Wg^T) (a Wu^T), as one FP8 GEMM:
// dense, and grouped over a device offset tensor.
//
// Both projections are one product with N = 2F; the tile walk, the main loops, the scales and the packed
// layouts are those of the plain products (gemm_pp.hpp, gemm_generic.hpp). What differs is which rows of B
// a tile holds, the gate and up rows of the same features, so that both end up in the same lane, and the
// epilogue, which forms act(g) u in fp32 and rounds it once. The projections themselves are written only
// for a backward: without them F values a row leave the kernel instead of 2F, and no pass reads them again.
#include "gemm_generic.hpp"
#include "gemm_pp.hpp"

namespace fp8dyn {

namespace {

// as the plain products' conditions: 32-bit offsets within a tile of A, in B and in the output
bool fast_eligible(const GatedMmArgs& g) {
  return g.K % 128 == 0 && 2 * g.F <= (1 << 22) && g.K <= (1 << 22) && 2 * g.F * g.K < ((int64_t)1 << 31);
}

template <int GATE, int SK, bool GR, bool PKB, bool EX>
hipError_t launch_pp(const GatedMmArgs& g) {
  GemmParams p{g.a, g.b, g.sa, g.sb, g.offsets, g.E, g.M, 2 * g.F, g.K, g.out, g.gu};
  const int64_t nt = (g.F + 127) / 128;
  const int64_t tiles = ((g.M + 255) / 256 + (GR ? g.E : 0)) * nt;
  int64_t grid = device_cus();
  if (tiles < grid) grid = tiles;
  if (grid >= kNumXcd) grid -= grid % kNumXcd;
  hipLaunchKernelGGL((k_gemm_fp8_pp<false, false, SK, false, GR, PKB, EX, GATE>), dim3((unsigned)grid), dim3(512), 0,
                     g.stream, p);
  return hipGetLastError();
}

template <int B, int GATE, int SK, bool EX>
hipError_t launch_generic(const GatedMmArgs& g) {
  GemmParams p{g.a, g.b, g.sa, g.sb, g.offsets, g.E, g.M, 2 * g.F, g.K, g.out, g.gu};
  const int64_t nt = (g.F + B / 2 - 1) / (B / 2);
  const int64_t tiles = ((g.M + B - 1) / B + (g.offsets ? g.E : 0)) * nt;
  int64_t grid = device_cus();
  if (tiles < grid)
    grid = tiles;
  else if (grid >= kNumXcd)
    grid -= grid % kNumXcd;
  hipLaunchKernelGGL((k_gemm_fp8<B, B, 2, 2, false, false, SK, false, EX, GATE>), dim3((unsigned)grid), dim3(256), 0,
                     g.stream, p);
  return hipGetLastError();
}

template <int GATE, int SK, bool EX>
hipError_t launch_form(const GatedMmArgs& g) {
  if (g.packed) {
    if constexpr (SK == kScaleRow)
      if (g.offsets) return launch_pp<GATE, SK, true, true, EX>(g);
    return launch_pp<GATE, SK, false, true, EX>(g);
  }
  if (!g.offsets && gemm_fp8_small_dense(g.M, 2 * g.F)) return launch_generic<64, GATE, SK, EX>(g);
  if (fast_eligible(g)) {
    if constexpr (SK == kScaleRow)
      if (g.offsets) return launch_pp<GATE, SK, true, false, EX>(g);
    return launch_pp<GATE, SK, false, false, EX>(g);
  }
  return launch_generic<128, GATE, SK, EX>(g);
}

template <int GATE>
hipError_t launch_act(const GatedMmArgs& g) {
  if (g.row_scales) return g.exact ? launch_form<GATE, kScaleRow, true>(g) : launch_form<GATE, kScaleRow, false>(g);
  return g.exact ? launch_form<GATE, kScaleTensor, true>(g) : launch_form<GATE, kScaleTensor, false>(g);
}

}  // namespace

bool gated_mm_packed_ok(const GatedMmArgs& g) { return fast_eligible(g); }

hipError_t launch_gated_mm(const GatedMmArgs& g) {
  return g.gelu ? launch_act<kGateGelu>(g) : launch_act<kGateSilu>(g);
}

}  // namespace fp8dyn
