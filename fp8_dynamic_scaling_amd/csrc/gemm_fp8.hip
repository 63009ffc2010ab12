// gemm_fp8.hip -- scaled FP8 GEMMs on gfx950 matrix cores: dense, and the MoE
// grouped form driven by a device offset tensor, with tensorwise, rowwise
// (per-row A x per-expert-column B), 128-blockwise and MX (E8M0) scales.
//
// Contract ("FP8 Training: Quantization, Autograd, Torchao", section 4
// "_scaled_mm layout requirements"): A is [M][K] row-major, B is the
// column-major K x N operand stored as [N][K]; the fp32 accumulation is
// multiplied by the inverse scales. Grouped form ("FP8 training on AMD GPUs
// with TorchTitan and TorchAO", section "Scaling FP8 to MoE Architectures",
// Figure 3): an offset tensor routes row ranges of A to experts and one
// launch covers all experts.
//
// Design for MI355X:
//  - v_mfma_scale_f32_16x16x128_f8f6f4. Operand layout, measured on MI355X: lane
//    l feeds row l % 16; its low 16 bytes are K [16g, 16g + 16) and its high 16
//    bytes are K [64 + 16g, 64 + 16g + 16) of the 128-deep step, g = l / 16;
//    the E8M0 scale of lane l covers row l % 16 and K [32g, 32g + 32). Loading
//    16-byte chunks g and g + 4 of each 128-byte row therefore keeps the
//    instruction's K order equal to memory order, so each lane's scale is the
//    scale of one 32-element group of the tensor. Operand formats (e4m3 / e5m2)
//    are immediates. For the non-MX scalings the hardware scale is 2^0 and the
//    scales are applied in the epilogue (tensor, row) or per 128-K step
//    (blockwise).
//  - Block tile BM x BN x 128 with a wave grid WM x WN; LDS double buffer,
//    16-byte chunks XOR-swizzled by row so fragment reads avoid bank
//    conflicts; one barrier per K step.
//  - Persistent grid of one workgroup per CU. Tiles are numbered expert by
//    expert, and inside an expert in groups of GM m-tiles with n running
//    fastest, so that the 32 workgroups of one XCD (workgroups are dealt to
//    the 8 XCDs round robin) work on a GM x (32/GM) patch of tiles that
//    shares A rows and B columns in that XCD's L2. Each XCD takes a contiguous
//    eighth of the tile list.
//  - Offsets stay on the device: every workgroup reads them into LDS and
//    builds the per-expert tile prefix itself; empty experts own no tiles.
#include "gemm_generic.hpp"

namespace fp8dyn {

// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, bool AE5, bool BE5, int SK, bool OF32, bool EX>
static hipError_t launch_cfg(const GemmArgs& g) {
  GemmParams p{g.a, g.b, g.sa, g.sb, g.offsets, g.E, g.M, g.N, g.K, g.out};
  const int64_t nt = (g.N + BN - 1) / BN;
  const int64_t tiles_ub = g.offsets ? ((g.M + BM - 1) / BM + g.E) * nt : ((g.M + BM - 1) / BM) * nt;
  // fewer tiles than CUs: one workgroup per tile (the kernel then deals tiles
  // by workgroup index); else a persistent grid, a multiple of the XCD count
  int64_t grid = device_cus();
  if (tiles_ub < grid)
    grid = tiles_ub;
  else if (grid >= kNumXcd)
    grid -= grid % kNumXcd;
  if (grid < 1) grid = 1;
  hipLaunchKernelGGL((k_gemm_fp8<BM, BN, WM, WN, AE5, BE5, SK, OF32, EX>), dim3((unsigned)grid),
                     dim3(WM * WN * 64), 0, g.stream, p);
  return hipGetLastError();
}

template <bool AE5, bool BE5, int SK, bool OF32>
static hipError_t launch_sk(const GemmArgs& g) {
  if constexpr (SK == kScaleTensor || SK == kScaleRow) {
    if (g.offsets == nullptr && gemm_fp8_small_dense(g.M, g.N)) {
      if (g.exact) return launch_cfg<64, 64, 2, 2, AE5, BE5, SK, OF32, true>(g);
      return launch_cfg<64, 64, 2, 2, AE5, BE5, SK, OF32, false>(g);
    }
  }
  // 64 x 64 per wave: the accumulators, a blockwise step's partial product
  // and the decoded operands of full precision all fit in registers (with
  // 128 x 128 per wave they spilled)
  if (g.exact) return launch_cfg<128, 128, 2, 2, AE5, BE5, SK, OF32, true>(g);
  return launch_cfg<128, 128, 2, 2, AE5, BE5, SK, OF32, false>(g);
}

template <bool AE5, bool BE5>
static hipError_t launch_fmt(const GemmArgs& g) {
  switch (g.scale_kind) {
    case kScaleTensor:
      return g.out_f32 ? launch_sk<AE5, BE5, kScaleTensor, true>(g) : launch_sk<AE5, BE5, kScaleTensor, false>(g);
    case kScaleRow:
      return g.out_f32 ? launch_sk<AE5, BE5, kScaleRow, true>(g) : launch_sk<AE5, BE5, kScaleRow, false>(g);
    case kScaleBlock:
      return g.out_f32 ? launch_sk<AE5, BE5, kScaleBlock, true>(g) : launch_sk<AE5, BE5, kScaleBlock, false>(g);
    default:
      return g.out_f32 ? launch_sk<AE5, BE5, kScaleMX, true>(g) : launch_sk<AE5, BE5, kScaleMX, false>(g);
  }
}

// Small dense outputs: when the 64 x 64 tiles number at most one per CU, the
// 256 x 256 ping-pong kernel would run on a handful of CUs, each streaming a
// whole 256-row panel of A and B; 64 x 64 tiles of four 32 x 32 waves spread
// the same work over up to a CU each. Measured on MI355X with cold caches
// (tensorwise, fp32 out): 256 x 512 x 512 in 9.5 us instead of 17.8 us,
// 1024 x 1024 x 1024 in 13.4 instead of 23.4, 256 x 4096 x 4096 in 34
// instead of 55; from 512 such tiles on the ping-pong kernel is as fast or
// faster (1024 x 2048 x 2048: 34 us either way).
bool gemm_fp8_small_dense(int64_t M, int64_t N) {
  return ((M + 63) / 64) * ((N + 63) / 64) <= (int64_t)device_cus();
}

hipError_t launch_gemm_fp8(const GemmArgs& g) {
  if (g.M == 0 || g.N == 0) return hipSuccess;
  const bool small = g.offsets == nullptr && !g.b_kpacked &&
                     (g.scale_kind == kScaleTensor || g.scale_kind == kScaleRow) && gemm_fp8_small_dense(g.M, g.N);
  if (!small && gemm_fp8_fast_eligible(g)) return launch_gemm_fp8_fast(g);
  // B is always the e4m3 variant (the API rejects e5m2 B)
  if (g.b_e5) return hipErrorInvalidValue;
  return g.a_e5 ? launch_fmt<true, false>(g) : launch_fmt<false, false>(g);
}

}  // namespace fp8dyn
