// norm_bwd.hip -- backward of the row normalization (RMSNorm, LayerNorm) with
// the gradient of the residual stream added.
//
// With xh = (h - mean) rstd and g = dy gamma of a row of n elements:
//   c2 = sum(g xh) / n, c1 = sum(g) / n (LayerNorm; 0 for RMSNorm)
//   dx = dh + rstd (g - c1 - xh c2)
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy.
// dx is the gradient of both addends of h = x + res. mean and rstd are the
// forward's fp32 values. All sums are fp32: a row's over its lanes' at most 16
// terms and a tree, a column's over the rows of one workgroup, then over the
// workgroups in a fixed order, so the same inputs give the same bits. dx,
// dgamma and dbeta are rounded once, to bf16.
//
// The kernel is bound by HBM: it reads dy, h and dh and writes dx once, 8 B an
// element. TPR threads hold a row in J pieces of 8 elements each, so that a lane
// keeps its columns of gamma and of the dgamma and dbeta sums in registers over
// all the rows of its workgroup; the next row is loaded while the present one
// is reduced. Measured, rows and then column sums: 8192 x 4096 RMSNorm 46 + 4.6 us
// (268 MB, 5.8 TB/s), 4000 x 7168 41 + 4.6 (229 MB), 16384 x 1024 24 + 4.2, 2000 x 16384
// 51 + 4.8 (262 MB; LayerNorm 69: its sums leave 1024 threads no registers to spare),
// 301 x 5120 LayerNorm 8.5 + 3.9, where latency counts.
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace fp8dyn {

typedef __bf16 nb_bf16x2 __attribute__((ext_vector_type(2)));

namespace {
constexpr int kMaxBwdBlocks = 512;  // workgroups, each with one row of partial column sums

// Threads a row: as few pieces a lane as there are threads for, and no more than two,
// so that the column sums and the row ahead stay in registers.
int bwd_tpr(int64_t cols) { return cols <= 1024 ? 64 : cols <= 4096 ? 256 : cols <= 8192 ? 512 : 1024; }

// Workgroups: at most kMaxBwdBlocks (two of 256 threads a CU, or one of 512), and two
// rows to a row slot where there are that many, so that the partial sums stay below the
// rows read. One of 256 threads a CU: LayerNorm of 8192 x 2048 37 us instead of 27; two
// of 512: 4000 x 7168 45 instead of 41. One row a slot: 64 x 4096 5.8 + 2.5 -> 4.9 + 3.0 us
// and no difference at 301 x 5120; four: 7.9 + 2.6 us, 9.4 + 3.4 instead of 8.5 + 3.9.
int64_t bwd_blocks(int64_t rows, int64_t cols) {
  const int tpr = bwd_tpr(cols);
  const int64_t slots = tpr == 64 ? 4 : 1, most = tpr >= 512 ? kMaxBwdBlocks / 2 : kMaxBwdBlocks;
  const int64_t groups = (rows + slots - 1) / slots;
  const int64_t b = (groups + 1) / 2;
  return b < 1 ? 1 : b > most ? most : b;
}
}  // namespace

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// AHEAD: the next row is loaded ahead; 1024 threads a row leave no registers for that.
template <int TPR, int J, bool LAYER, bool AHEAD>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void k_norm_bwd(
    const uint16_t* dy, const uint16_t* dh, const uint16_t* __restrict__ h, const uint16_t* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows, int64_t cols, uint16_t* dx,
    float* __restrict__ part, int want_cols) {
  constexpr int NT = TPR == 64 ? 256 : TPR;
  constexpr int SLOTS = NT / TPR;
  constexpr int WAVES = TPR / 64;  // wavefronts that share a row
  __shared__ float red[2][2][WAVES];
  __shared__ float comb[SLOTS > 1 ? SLOTS * 64 * 8 * J : 1];
  const int t = threadIdx.x % TPR;
  const int slot = threadIdx.x / TPR;
  const int64_t stride = (int64_t)gridDim.x * SLOTS;
  const float inv_n = 1.0f / (float)cols;
  bool in[J];
  uint4 ga[J];
  float sg[J][8], sb[J][8];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t c = 8 * (t + TPR * j);
    in[j] = c < cols;
    ga[j] = in[j] ? *reinterpret_cast<const uint4*>(gamma + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) sg[j][k] = sb[j][k] = 0.0f;
  }
  struct Row {
    uint4 y[J], h[J], d[J];
    float mu, rs;
  } next;
  auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t o = row * cols + 8 * (t + TPR * j);
      next.y[j] = in[j] ? ld_nt16(dy + o) : make_uint4(0, 0, 0, 0);
      next.h[j] = in[j] ? ld_nt16(h + o) : make_uint4(0, 0, 0, 0);
      next.d[j] = dh && in[j] ? ld_nt16(dh + o) : make_uint4(0, 0, 0, 0);
    }
    next.rs = rstd[row];
    next.mu = LAYER ? mean[row] : 0.0f;
  };
  int64_t row = (int64_t)blockIdx.x * SLOTS + slot;
  if (AHEAD && row < rows) load(row);
  int buf = 0;
  // rows of a workgroup with several waves a row are the same for all of them,
  // so every wave reaches every barrier
  for (; row < rows; row += stride) {
    if (!AHEAD) load(row);
    Row cur = next;
    if (AHEAD && row + stride < rows) load(row + stride);
    // element k of piece j: dy, xh and g; zeros in lanes past the row's end
    auto element = [&](int j, int k, float& y, float& xh, float& g) {
      const uint32_t a[4] = {cur.y[j].x, cur.y[j].y, cur.y[j].z, cur.y[j].w};
      const uint32_t b[4] = {cur.h[j].x, cur.h[j].y, cur.h[j].z, cur.h[j].w};
      const uint32_t c[4] = {ga[j].x, ga[j].y, ga[j].z, ga[j].w};
      y = k & 1 ? bf16_hi(a[k >> 1]) : bf16_lo(a[k >> 1]);
      const float x = k & 1 ? bf16_hi(b[k >> 1]) : bf16_lo(b[k >> 1]);
      xh = LAYER ? (in[j] ? (x - cur.mu) * cur.rs : 0.0f) : x * cur.rs;
      g = y * (k & 1 ? bf16_hi(c[k >> 1]) : bf16_lo(c[k >> 1]));
    };
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float y, xh, g;
        element(j, k, y, xh, g);
        c2 += g * xh;
        if constexpr (LAYER) {
          c1 += g;
          sb[j][k] += y;
        }
        sg[j][k] += y * xh;
      }
    }
    c2 = wave_sum(c2);
    if constexpr (LAYER) c1 = wave_sum(c1);
    if constexpr (WAVES > 1) {
      // two buffers: a wave writes the next row's sums while a slower one
      // still reads this row's; the barrier between holds it back after that
      if ((t & 63) == 0) {
        red[buf][0][t >> 6] = c2;
        if constexpr (LAYER) red[buf][1][t >> 6] = c1;
      }
      __syncthreads();
      c2 = c1 = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        c2 += red[buf][0][i];
        if constexpr (LAYER) c1 += red[buf][1][i];
      }
      buf ^= 1;
    }
    c2 *= inv_n;
    c1 *= inv_n;
    if constexpr (!AHEAD && LAYER) {
      // as if the packed row were new: else the compiler keeps g and xh of the
      // first pass and spills
#pragma unroll
      for (int j = 0; j < J; ++j)
        asm volatile("" : "+v"(cur.y[j].x), "+v"(cur.y[j].y), "+v"(cur.y[j].z), "+v"(cur.y[j].w), "+v"(cur.h[j].x),
                     "+v"(cur.h[j].y), "+v"(cur.h[j].z), "+v"(cur.h[j].w));
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!in[j]) continue;
      const uint32_t e[4] = {cur.d[j].x, cur.d[j].y, cur.d[j].z, cur.d[j].w};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float y, x0, g0, x1, g1;
        element(j, 2 * k, y, x0, g0);
        element(j, 2 * k + 1, y, x1, g1);
        const float lo = bf16_lo(e[k]) + cur.rs * (g0 - c1 - x0 * c2);
        const float hi = bf16_hi(e[k]) + cur.rs * (g1 - c1 - x1 * c2);
        const nb_bf16x2 p = {(__bf16)lo, (__bf16)hi};
        o[k] = __builtin_bit_cast(uint32_t, p);
      }
      st_nt16(dx + row * cols + 8 * (t + TPR * j), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  if (!want_cols) return;
  // the workgroup's column sums: part[0][block][cols] (gamma), part[1][...] (beta)
#pragma unroll
  for (int z = 0; z < (LAYER ? 2 : 1); ++z) {
    float* dst = part + ((int64_t)z * gridDim.x + blockIdx.x) * cols;
    if constexpr (SLOTS > 1) {
      if (z) __syncthreads();
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          comb[slot * (64 * 8 * J) + 8 * (t + TPR * j) + k] = z ? sb[j][k] : sg[j][k];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += NT) {
        float a = comb[c];
#pragma unroll
        for (int i = 1; i < SLOTS; ++i) a += comb[i * (64 * 8 * J) + c];
        dst[c] = a;
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (!in[j]) continue;
        float4* o = reinterpret_cast<float4*>(dst + 8 * (t + TPR * j));
        const float* v = z ? sb[j] : sg[j];
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}

// Column sums over the workgroups' partial rows: 32 columns a workgroup (8
// lanes of 4), its 32 row slices summed in order through LDS.
__global__ __launch_bounds__(256) void k_norm_bwd_cols(const float* __restrict__ part, int64_t blocks, int64_t cols,
                                                       uint16_t* __restrict__ dgamma, uint16_t* __restrict__ dbeta) {
  __shared__ float4 sum[32][8];
  const int lane = threadIdx.x & 7, slice = threadIdx.x >> 3;
  uint16_t* dst = blockIdx.y ? dbeta : dgamma;
  if (!dst) return;
  const int64_t c = (int64_t)blockIdx.x * 32 + 4 * lane;
  const float* p = part + (int64_t)blockIdx.y * blocks * cols;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < cols) {
#pragma unroll 8
    for (int64_t b = slice; b < blocks; b += 32) {
      const float4 v = *reinterpret_cast<const float4*>(p + b * cols + c);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
  sum[slice][lane] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    if (col >= cols) return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += reinterpret_cast<const float*>(&sum[i][0])[threadIdx.x];
    const __bf16 v = (__bf16)s;
    dst[col] = __builtin_bit_cast(uint16_t, v);
  }
}

int64_t norm_bwd_ws_floats(int64_t rows, int64_t cols, bool layer) {
  return bwd_blocks(rows, cols) * cols * (layer ? 2 : 1);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a) {
  const int64_t blocks = bwd_blocks(a.rows, a.cols);
  const int want = a.dgamma || a.dbeta;
  auto go = [&](auto kern, int threads) {
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(threads), 0, a.stream, a.dy, a.dh, a.h, a.gamma, a.mean,
                       a.rstd, a.rows, a.cols, a.dx, a.ws, want);
  };
  auto by_kind = [&](auto T, auto P) {
    const int threads = T.value == 64 ? 256 : T.value;
    if (a.layer)
      go(k_norm_bwd<T.value, P.value, true, T.value <= 512>, threads);
    else
      go(k_norm_bwd<T.value, P.value, false, T.value <= 512>, threads);
  };
  const std::integral_constant<int, 2> two;
  const int tpr = bwd_tpr(a.cols);
  if (tpr == 64)
    by_kind(std::integral_constant<int, 64>{}, two);
  else if (tpr == 256)
    by_kind(std::integral_constant<int, 256>{}, two);
  else if (tpr == 512)
    by_kind(std::integral_constant<int, 512>{}, two);
  else
    by_kind(std::integral_constant<int, 1024>{}, two);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !want) return e;
  hipLaunchKernelGGL(k_norm_bwd_cols, dim3((unsigned)((a.cols + 31) / 32), a.layer ? 2 : 1), dim3(256), 0, a.stream,
                     a.ws, blocks, a.cols, a.dgamma, a.dbeta);
  return hipGetLastError();
}

}  // namespace fp8dyn
