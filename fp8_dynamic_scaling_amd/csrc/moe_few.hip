// moe_few.hip -- a mixture-of-experts layer for a few tokens (at most 64), in
// two launches:
//   a[t, j] = w[t][j] silu(Wg_e x_t) * (Wu_e x_t)   e = ids[t][j]  (k_moe_up)
//   out[t]  = sum_j W2_e a[t, j]                                  (k_moe_down)
// with the experts' weights in e4m3, one inverse scale a row.
//
// With few tokens the layer is bound by reading the chosen experts' codes once
// (3 F D bytes each) from HBM; the products are a small part. So the codes go
// straight from HBM to registers, 16 bytes a lane, are decoded to bf16 (exact)
// and multiplied by 16 tokens at a time with the BF16 matrix-core instruction,
// which sums at fp32 precision; x and a are bf16 and come from the caches.
//  - k_moe_up: a workgroup has one expert and 16 gate and 16 up rows; its waves
//    share D among them, so that thousands of waves each read some 20 KB and all
//    of their loads are in flight at once. The waves' partial sums meet in LDS,
//    in a fixed order.
//  - k_moe_down: a workgroup has 16 rows of D for all experts; its waves share
//    the (expert, piece of F) units. A token's sum over its experts stays in
//    fp32 registers, so no partial output is written and no atomics are needed:
//    the same inputs give the same bits.
// The rounding of a to bf16 (with its gate weight, half a step: 2^-9 relative)
// is that of the activations the grouped GEMMs take; everything else is fp32
// up to the one rounding of the output.
//
// A token may name an expert twice: its first slot carries the sum of the
// weights. Ids outside [0, E) name none.
#include "gemm_common.hpp"

namespace fp8dyn {

namespace {
constexpr int kUpWaves = 8;
constexpr int kDownWaves = 8;
constexpr int kFewT = 64;
constexpr int kFewK = 32;
}  // namespace

// Eight e4m3 codes -> eight bf16 (every e4m3 value is a bf16 value).
__device__ __forceinline__ v8bf decode8(uint32_t d0, uint32_t d1) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, true);
  return (v8bf){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Byte offset of the 16 codes (row, kc .. kc + 15) of an [N][K] matrix.
template <bool PACKED>
__device__ __forceinline__ int64_t code_at(int64_t row, int64_t kc, int64_t K) {
  if constexpr (PACKED)
    return ((row >> 4) * (K >> 6) + (kc >> 6)) * 1024 + (row & 15) * 64 + (kc & 63);
  else
    return row * K + kc;
}

// The ids in LDS and a bit for each expert that some token names.
__device__ __forceinline__ void few_ids(const int32_t* __restrict__ ids, int n, int E, int32_t* sid, uint32_t* bits) {
  if (threadIdx.x < 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = ids[i];
    const bool ok = e >= 0 && e < E;
    sid[i] = ok ? e : -1;
    if (ok) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The s-th named expert in order, or -1 past the last (the same in every lane).
__device__ __forceinline__ int few_expert(const uint32_t* bits, int s) {
  const int lane = threadIdx.x & 63;
  const uint32_t w = lane < 32 ? bits[lane] : 0;
  int upto = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up(upto, o, 64);
    if (lane >= o) upto += u;
  }
  const int before = upto - __popc(w);
  const uint64_t hit = __ballot(lane < 32 && s >= before && s < upto);
  if (!hit) return -1;
  const int word = __ffsll((unsigned long long)hit) - 1;
  uint32_t v = __shfl(w, word, 64);
  for (int r = s - __shfl(before, word, 64); r > 0; --r) v &= v - 1;
  return 32 * word + __ffs(v) - 1;
}

// One wave's products of 16 weight rows with NT tiles of 16 tokens over a unit of
// 128 values of the contraction: w holds two 16-byte pieces a lane (64 values
// apart), x the same values of the lane's tokens.
template <int NT>
__device__ __forceinline__ void unit_products(const uint4 (&w)[2], const uint4 (&x)[NT][4], v4f (&acc)[NT]) {
  v8bf a[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    a[2 * h] = decode8(w[h].x, w[h].y);
    a[2 * h + 1] = decode8(w[h].z, w[h].w);
  }
  // two wait states between the converts and the matrix instructions
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 1" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const v8bf b = __builtin_bit_cast(v8bf, x[n][q]);
      acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b, acc[n], 0, 0, 0);
      keep_live(b);
    }
  }
  asm volatile("" ::"v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]));
}

template <int NT, bool PACKED>
__device__ __forceinline__ void moe_up_tile(const MoeFewArgs& p, int e, int m, const int32_t* list, int64_t f0,
                                            const int32_t* sid, float4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, kg = lane >> 4;
  const uint8_t* wb = p.w13 + (int64_t)e * 2 * p.F * p.D;
  const uint16_t* xp[NT];
  bool has[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = 16 * n + lr;
    has[n] = i < m;
    xp[n] = p.x + (int64_t)(has[n] ? list[i] / p.k : 0) * p.D;
  }
  v4f ag[NT], au[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) ag[n] = au[n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t units = (p.D + 127) / 128;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t u = wave; u < units; u += kUpWaves) {
    uint4 wg[2], wu[2], xv[NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t kc = 128 * u + 64 * h + 16 * kg;
      const bool in = kc < p.D;
      wg[h] = in ? ld_nt16(wb + code_at<PACKED>(f0 + lr, kc, p.D)) : zero;
      wu[h] = in ? ld_nt16(wb + code_at<PACKED>(p.F + f0 + lr, kc, p.D)) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4* xs = reinterpret_cast<const uint4*>(xp[n] + kc);
        xv[n][2 * h] = in && has[n] ? xs[0] : zero;
        xv[n][2 * h + 1] = in && has[n] ? xs[1] : zero;
      }
    }
    unit_products<NT>(wg, xv, ag);
    unit_products<NT>(wu, xv, au);
  }
  // partial sums of the waves
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[((2 * n) * kUpWaves + wave) * 64 + lane] = make_float4(ag[n][0], ag[n][1], ag[n][2], ag[n][3]);
    red[((2 * n + 1) * kUpWaves + wave) * 64 + lane] = make_float4(au[n][0], au[n][1], au[n][2], au[n][3]);
  }
  __syncthreads();
  if (wave >= NT) return;
  const int item = 16 * wave + lr;  // this wave finishes tile `wave`
  if (item >= m) return;
  float g[4] = {0, 0, 0, 0}, uu[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kUpWaves; ++w) {
    const float4 a = red[((2 * wave) * kUpWaves + w) * 64 + lane];
    const float4 b = red[((2 * wave + 1) * kUpWaves + w) * 64 + lane];
    g[0] += a.x;
    g[1] += a.y;
    g[2] += a.z;
    g[3] += a.w;
    uu[0] += b.x;
    uu[1] += b.y;
    uu[2] += b.z;
    uu[3] += b.w;
  }
  const int64_t f = f0 + 4 * kg;
  const float* sc = p.inv13 + (int64_t)e * 2 * p.F;
  const int it = list[item];
  const int t = it / p.k;
  float gate = 0.0f;  // the weights of all the token's slots that name e
  for (int j = it % p.k; j < p.k; ++j) gate += sid[t * p.k + j] == e ? p.weights[t * p.k + j] : 0.0f;
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float gv = g[i] * sc[f + i], uv = uu[i] * sc[p.F + f + i];
    r[i] = gate * (gv / (1.0f + expf(-gv)) * uv);
  }
  const v2bf lo = {(__bf16)r[0], (__bf16)r[1]}, hi = {(__bf16)r[2], (__bf16)r[3]};
  *reinterpret_cast<uint2*>(p.act + (int64_t)it * p.F + f) =
      make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

template <int NTM, bool PACKED>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(MoeFewArgs p) {
  __shared__ float4 red[NTM * 2 * kUpWaves * 64];
  __shared__ int32_t sid[kFewT * kFewK];
  __shared__ int32_t list[kFewT];
  __shared__ uint32_t bits[32];
  __shared__ int count;
  const int n = (int)p.T * p.k;
  few_ids(p.ids, n, p.E, sid, bits);
  const int e = few_expert(bits, blockIdx.y);
  if (e < 0) return;
  // the expert's pairs in order, the first of each token's only
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int m = 0;
    for (int i0 = 0; i0 < n; i0 += 64) {
      const int i = i0 + lane;
      bool mine = i < n && sid[i] == e;
      for (int j = i - i % p.k; mine && j < i; ++j) mine = sid[j] != e;
      const uint64_t b = __ballot(mine);
      if (mine) list[m + __popcll(b & ((1ull << lane) - 1))] = i;
      m += __popcll(b);
    }
    if (lane == 0) count = m;
  }
  __syncthreads();
  const int m = count;
  const int64_t f0 = 16 * (int64_t)blockIdx.x;
  if constexpr (NTM >= 4) {
    if (m > 32) return moe_up_tile<4, PACKED>(p, e, m, list, f0, sid, red);
  }
  if constexpr (NTM >= 2) {
    if (m > 16) return moe_up_tile<2, PACKED>(p, e, m, list, f0, sid, red);
  }
  moe_up_tile<1, PACKED>(p, e, m, list, f0, sid, red);
}

template <int NT, bool PACKED>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeFewArgs p) {
  __shared__ float4 red[NT * kDownWaves * 64];
  __shared__ int32_t sid[kFewT * kFewK];
  __shared__ int32_t act_e[kMaxExperts];
  __shared__ uint32_t bits[32];
  __shared__ int count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, kg = lane >> 4;
  const int T = (int)p.T, k = p.k;
  few_ids(p.ids, T * k, p.E, sid, bits);
  // the named experts in order
  if (threadIdx.x < 64) {
    const uint32_t w = lane < 32 ? bits[lane] : 0;
    int upto = __popc(w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up(upto, o, 64);
      if (lane >= o) upto += u;
    }
    int at = upto - __popc(w);
    for (uint32_t v = w; v; v &= v - 1) act_e[at++] = 32 * lane + __ffs(v) - 1;
    if (lane == 31) count = upto;
  }
  __syncthreads();
  const int nact = count;
  const int64_t d0 = 16 * (int64_t)blockIdx.x;
  const int units = (int)((p.F + 127) / 128);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  v4f sum[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) sum[n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  for (int a = 0; a < nact; ++a) {
    // the waves take the units in turn; where an expert has no unit left for
    // this wave there is nothing to scale
    int u = (wave - a * units) % kDownWaves;
    u = u < 0 ? u + kDownWaves : u;
    if (u >= units) continue;
    const int e = act_e[a];
    const uint8_t* wb = p.w2 + (int64_t)e * p.D * p.F;
    const uint16_t* ap[NT];
    bool has[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = 16 * n + lr;
      int at = -1;
      for (int j = k - 1; t < T && j >= 0; --j) at = sid[t * k + j] == e ? j : at;
      has[n] = at >= 0;
      ap[n] = p.act + (int64_t)(has[n] ? t * k + at : 0) * p.F;
    }
    v4f acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    for (; u < units; u += kDownWaves) {
      uint4 w[2], xv[NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t kc = 128 * (int64_t)u + 64 * h + 16 * kg;
        const bool in = kc < p.F;
        w[h] = in ? ld_nt16(wb + code_at<PACKED>(d0 + lr, kc, p.F)) : zero;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4* xs = reinterpret_cast<const uint4*>(ap[n] + kc);
          xv[n][2 * h] = in && has[n] ? xs[0] : zero;
          xv[n][2 * h + 1] = in && has[n] ? xs[1] : zero;
        }
      }
      unit_products<NT>(w, xv, acc);
    }
    // a lane's products are all of the one token of its column, so only the
    // tokens that named the expert take its sums (a NaN code stays with them)
    const float* sc = p.inv2 + (int64_t)e * p.D + d0 + 4 * kg;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] += has[n] ? acc[n][i] * sc[i] : 0.0f;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
    red[(n * kDownWaves + wave) * 64 + lane] = make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
  __syncthreads();
  if (wave >= NT) return;
  const int t = 16 * wave + lr;
  if (t >= T) return;
  float r[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kDownWaves; ++w) {
    const float4 a = red[(wave * kDownWaves + w) * 64 + lane];
    r[0] += a.x;
    r[1] += a.y;
    r[2] += a.z;
    r[3] += a.w;
  }
  const v2bf lo = {(__bf16)r[0], (__bf16)r[1]}, hi = {(__bf16)r[2], (__bf16)r[3]};
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.D + d0 + 4 * kg) =
      make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

template <bool PACKED>
static hipError_t launch_few_t(const MoeFewArgs& a) {
  const int64_t pairs = a.T * a.k;
  const dim3 gu((unsigned)(a.F / 16), (unsigned)(pairs < a.E ? pairs : a.E)), gd((unsigned)(a.D / 16));
  const dim3 bu(64 * kUpWaves), bd(64 * kDownWaves);
  auto go = [&](auto up, auto down) {
    if (a.F > 0) hipLaunchKernelGGL(up, gu, bu, 0, a.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(down, gd, bd, 0, a.stream, a);
    return hipGetLastError();
  };
  if (a.T <= 16) return go(k_moe_up<1, PACKED>, k_moe_down<1, PACKED>);
  if (a.T <= 32) return go(k_moe_up<2, PACKED>, k_moe_down<2, PACKED>);
  return go(k_moe_up<4, PACKED>, k_moe_down<4, PACKED>);
}

hipError_t launch_moe_few(const MoeFewArgs& a) {
  if (a.T == 0 || a.D == 0) return hipSuccess;
  return a.packed ? launch_few_t<true>(a) : launch_few_t<false>(a);
}

}  // namespace fp8dyn
