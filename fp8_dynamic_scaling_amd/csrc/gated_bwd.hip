// gated_bwd.hip -- gradient through a gated product h = act(g) u, with the rowwise FP8
// quantization of the gradient that the grad-input GEMM takes.
//
//   dg = dh u act'(g), du = dh act(g); d = [dg | du], a row of 2F values in fp32
//   amax = max |d| of the row; q = encode(d scale) as the rowwise quantizer scales;
//   dgu = bf16(d), the operand of the weight gradient; h = bf16(act(g) u) if wanted.
// The amax is that of the fp32 values, not of their bf16 copies: one rounding, not two.
//
// One pass: a row's gradient stays in registers from the loads to the codes. The kernel is
// bound by HBM: 2 + 4 B read and 4 + 2 B written for each element of h. Measured, 8192 x 14336
// SiLU with e5m2 codes (1.41 GB): 235 us, 6.0 TB/s, where a large torch copy reaches 5.3. dgu
// leaves by streaming stores, the codes by plain ones: the next GEMM reads them, and with both
// streaming 255 us, with streaming loads as well; with both plain 252. Two pieces a lane:
// four 251 us; a persistent grid of two workgroups a CU 254.
#include "gated.hpp"
#include "internal.hpp"

namespace fp8dyn {

namespace {

// A lane holds J pieces of 8 features (8 gate and 8 up values each). WAVE: a row is a wavefront's, four
// rows a workgroup of 256; otherwise a workgroup's, of as many threads as its pieces need.
template <int J, bool E5, bool GELU, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_gated_bwd(const GatedBwdArgs a) {
  __shared__ uint32_t red[16];
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int threads = WAVE ? 64 : blockDim.x;
  const int64_t F = a.F;
  const int64_t rows_step = (int64_t)gridDim.x * (WAVE ? 4 : 1);
  for (int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x; row < a.M; row += rows_step) {
    const uint16_t* gu = a.gu + row * 2 * F;
    const uint16_t* dh = a.dh + row * F;
    uint4 vd[J], vg[J], vu[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t c = 8 * (t + (int64_t)threads * j);
      const bool in = c < F;
      vd[j] = in ? *reinterpret_cast<const uint4*>(dh + c) : make_uint4(0, 0, 0, 0);
      vg[j] = in ? *reinterpret_cast<const uint4*>(gu + c) : make_uint4(0, 0, 0, 0);
      vu[j] = in ? *reinterpret_cast<const uint4*>(gu + F + c) : make_uint4(0, 0, 0, 0);
    }
    float dg[J][8], du[J][8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t c = 8 * (t + (int64_t)threads * j);
      const uint32_t wd[4] = {vd[j].x, vd[j].y, vd[j].z, vd[j].w}, wg[4] = {vg[j].x, vg[j].y, vg[j].z, vg[j].w},
                     wu[4] = {vu[j].x, vu[j].y, vu[j].z, vu[j].w};
      float h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = k & 1 ? bf16_hi(wd[k >> 1]) : bf16_lo(wd[k >> 1]);
        const float g = k & 1 ? bf16_hi(wg[k >> 1]) : bf16_lo(wg[k >> 1]);
        const float u = k & 1 ? bf16_hi(wu[k >> 1]) : bf16_lo(wu[k >> 1]);
        float act, der;
        gate_act_d<GELU>(g, act, der);
        dg[j][k] = d * u * der;
        du[j][k] = d * act;
        h[k] = act * u;
        // magnitudes ordered by their bits, those of a NaN above all
        const uint32_t x = __float_as_uint(dg[j][k]) & 0x7fffffffu, y = __float_as_uint(du[j][k]) & 0x7fffffffu;
        top = max(top, max(x, y));
      }
      if (c < F) {
        if (a.dgu) {
          uint16_t* o = a.dgu + row * 2 * F + c;
          st_nt16(o, make_uint4(pack_bf16(dg[j][0], dg[j][1]), pack_bf16(dg[j][2], dg[j][3]),
                                pack_bf16(dg[j][4], dg[j][5]), pack_bf16(dg[j][6], dg[j][7])));
          st_nt16(o + F, make_uint4(pack_bf16(du[j][0], du[j][1]), pack_bf16(du[j][2], du[j][3]),
                                    pack_bf16(du[j][4], du[j][5]), pack_bf16(du[j][6], du[j][7])));
        }
        if (a.h)
          st_nt16(a.h + row * F + c, make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]),
                                                pack_bf16(h[6], h[7])));
      }
    }
    if (!a.q) continue;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if constexpr (!WAVE) {
      const int waves = blockDim.x >> 6;
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
      __syncthreads();
      top = red[0];
      for (int w = 1; w < waves; ++w) top = max(top, red[w]);
      __syncthreads();  // before the next row's maxima
    }
    float scale, inv;
    scale_from_amax(__uint_as_float(top), a.fmax, a.eps, scale, inv);
    // a row that is not finite has NaN scales, and so codes that stand for NaN
    if (top >= 0x7f800000u) scale = inv = __uint_as_float(0x7fc00000u);
    if (t == 0) {
      a.scale[row] = scale;
      if (a.inv) a.inv[row] = inv;
    }
    const float fm = (float)a.fmax;
    auto codes = [&](const float* x) {
      return make_uint2(cvt4<E5>(clampf(x[0] * scale, fm), clampf(x[1] * scale, fm), clampf(x[2] * scale, fm),
                                 clampf(x[3] * scale, fm)),
                        cvt4<E5>(clampf(x[4] * scale, fm), clampf(x[5] * scale, fm), clampf(x[6] * scale, fm),
                                 clampf(x[7] * scale, fm)));
    };
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t c = 8 * (t + (int64_t)threads * j);
      if (c < F) {
        uint8_t* o = a.q + row * 2 * F + c;
        *reinterpret_cast<uint2*>(o) = codes(dg[j]);
        *reinterpret_cast<uint2*>(o + F) = codes(du[j]);
      }
    }
  }
}

template <int J, bool WAVE>
hipError_t launch_bwd(const GatedBwdArgs& a, int threads) {
  const int64_t groups = WAVE ? (a.M + 3) / 4 : a.M;
  const int64_t most = WAVE ? kMaxGrid256 : kMaxGrid256 / 4;
  const dim3 grid((unsigned)(groups < most ? groups : most)), block(threads);
  if (a.gelu) {
    if (a.e5) hipLaunchKernelGGL((k_gated_bwd<J, true, true, WAVE>), grid, block, 0, a.stream, a);
    else hipLaunchKernelGGL((k_gated_bwd<J, false, true, WAVE>), grid, block, 0, a.stream, a);
  } else {
    if (a.e5) hipLaunchKernelGGL((k_gated_bwd<J, true, false, WAVE>), grid, block, 0, a.stream, a);
    else hipLaunchKernelGGL((k_gated_bwd<J, false, false, WAVE>), grid, block, 0, a.stream, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_bwd(const GatedBwdArgs& a) {
  const int64_t pieces = a.F / 8;
  if (pieces <= 64) return launch_bwd<1, true>(a, 256);
  if (pieces <= 128) return launch_bwd<2, true>(a, 256);
  const int j = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
  const int threads = (int)((pieces + j * 64 - 1) / (j * 64)) * 64;
  return j == 1 ? launch_bwd<1, false>(a, threads)
         : j == 2 ? launch_bwd<2, false>(a, threads)
                  : launch_bwd<4, false>(a, threads);
}

}  // namespace fp8dyn
