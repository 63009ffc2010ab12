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
//    share D among them. The waves' partial sums meet in LDS, in a fixed order.
//  - k_moe_down: a workgroup has 16 rows of D for all experts; its waves share
//    the (expert, piece of F) units. A wave adds what it has of a token to its
//    own fp32 sums in LDS, and the waves' sums are added in order at the end: no
//    partial output in memory and no atomics, so the same inputs give the same
//    bits.
// A wave's unit of work is 16 rows (k_moe_up: twice 16) x 128 values of the
// contraction and the same 128 values of its tokens; the loads of the next
// units are in flight while one is multiplied. An expert's tokens are compacted
// into tiles of 16.
// The rounding of a to bf16 (with its gate weight, half a step: 2^-8 relative)
// is that of the activations the grouped GEMMs take; everything else is fp32
// up to the one rounding of the output.
//
// A token may name an expert twice: its first slot carries the sum of the
// weights. Ids outside [0, E) name none.
#include "gemm_common.hpp"

namespace fp8dyn {

namespace {
constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kFewT = 64;
constexpr int kFewK = 32;

// What k_moe_up leaves in the workspace for k_moe_down, behind a: the number of
// named experts, each one's id and number of tokens, and its pairs (t * k + j).
struct FewMeta {
  int32_t* head;   // [0] the number of experts
  int32_t* expert;  // [T * k]
  int32_t* count;   // [T * k]
  uint16_t* pairs;  // [T * k][kFewT]
};
__host__ __device__ inline FewMeta few_meta(uint16_t* act, int64_t T, int k, int64_t F) {
  FewMeta m;
  m.head = reinterpret_cast<int32_t*>(act + T * k * F);
  m.expert = m.head + 4;
  m.count = m.expert + T * k;
  m.pairs = reinterpret_cast<uint16_t*>(m.count + T * k);
  return m;
}
}  // namespace

size_t moe_few_ws_bytes(int64_t T, int k, int64_t F) {
  return (size_t)(T * k) * (2 * F + 8 + 2 * kFewT) + 16;
}

// Eight e4m3 codes -> eight bf16 (every e4m3 value is a bf16 value).
__device__ __forceinline__ v8bf decode8(uint32_t d0, uint32_t d1) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, true);
  return (v8bf){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// 16-byte pieces of a row-major or k-packed [N][K] matrix of codes: where the
// lane's piece of rows [16 i, 16 i + 16) begins, and the bytes from one 64-value
// step of the contraction to the next (the packed 1 KB chunks of 16 x 64 follow
// each other).
template <bool PACKED>
__device__ __forceinline__ const uint8_t* code_ptr(const uint8_t* w, int64_t row0, int64_t K) {
  const int lane = threadIdx.x & 63, lr = lane & 15, kg = lane >> 4;
  return PACKED ? w + row0 * K + lr * 64 + kg * 16 : w + (row0 + lr) * K + kg * 16;
}
template <bool PACKED>
constexpr int kStep = PACKED ? 1024 : 64;

// The operands of one unit, 128 values of the contraction: R tiles of 16 weight
// rows (lane: row l & 15, values 16 (l >> 4) .. + 15 of each 64) and NT tiles of
// 16 tokens (lane: token l & 15, the same values).
template <int R, int NT>
struct Unit {
  uint4 w[R][2];
  uint4 x[NT][4];
};

template <int R, int NT, bool PACKED>
__device__ __forceinline__ void load_unit(Unit<R, NT>& s, const uint8_t* const (&wp)[R],
                                          const uint16_t* const (&xp)[NT], int u, int K) {
  const int kg = (threadIdx.x & 63) >> 4;
  const bool full = 128 * (u + 1) <= K;  // else lanes past K hold zeros
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = full || 128 * u + 64 * h + 16 * kg < K;
#pragma unroll
    for (int r = 0; r < R; ++r)
      s.w[r][h] = in ? ld_nt16(wp[r] + (int64_t)(2 * u + h) * kStep<PACKED>) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4* q = reinterpret_cast<const uint4*>(xp[n] + 128 * u + 64 * h);
      s.x[n][2 * h] = in ? q[0] : make_uint4(0, 0, 0, 0);
      s.x[n][2 * h + 1] = in ? q[1] : make_uint4(0, 0, 0, 0);
    }
  }
}

template <int R, int NT>
__device__ __forceinline__ void multiply_unit(const Unit<R, NT>& s, v4f (&acc)[R][NT]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v8bf a[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[2 * h] = decode8(s.w[r][h].x, s.w[r][h].y);
      a[2 * h + 1] = decode8(s.w[r][h].z, s.w[r][h].w);
    }
    // two wait states between the converts and the matrix instructions
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 1" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v8bf b = __builtin_bit_cast(v8bf, s.x[n][q]);
        acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b, acc[r][n], 0, 0, 0);
        keep_live(b);
      }
    }
    asm volatile("" ::"v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]));
  }
}

// acc += the products of units [u0, u1), P of them in flight.
template <int R, int NT, int P, bool PACKED>
__device__ __forceinline__ void stream_units(const uint8_t* const (&wp)[R], const uint16_t* const (&xp)[NT], int u0,
                                             int u1, int K, v4f (&acc)[R][NT]) {
  Unit<R, NT> s[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (u0 + i < u1) load_unit<R, NT, PACKED>(s[i], wp, xp, u0 + i, K);
  for (int u = u0; u < u1; u += P) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (u + i >= u1) break;
      multiply_unit<R, NT>(s[i], acc);
      if (u + i + P < u1) load_unit<R, NT, PACKED>(s[i], wp, xp, u + i + P, K);
    }
  }
}

// Units in flight by the tiles of tokens: the registers of P units, 16 R + 16 NT
// each, stay near 128.
template <int NT>
constexpr int kInFlight = NT == 1 ? 4 : NT == 2 ? 3 : 2;

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

template <int NT, bool PACKED>
__device__ __forceinline__ void moe_up_tile(const MoeFewArgs& p, int e, int m, const int32_t* list, int64_t f0,
                                            const int32_t* sid, float4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, kg = lane >> 4;
  const uint8_t* wb = p.w13 + (int64_t)e * 2 * p.F * p.D;
  const uint8_t* const wp[2] = {code_ptr<PACKED>(wb, f0, p.D), code_ptr<PACKED>(wb, p.F + f0, p.D)};
  const uint16_t* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // a lane past the last token takes the first one's values: a column of the
    // product that nobody reads
    const int i = 16 * n + lr < m ? 16 * n + lr : 0;
    xp[n] = p.x + (int64_t)(list[i] / p.k) * p.D + 16 * kg;
  }
  v4f acc[2][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  const int units = (int)((p.D + 127) / 128);
  stream_units<2, NT, kInFlight<NT>, PACKED>(wp, xp, units * wave / kUpWaves, units * (wave + 1) / kUpWaves, (int)p.D,
                                             acc);
  // partial sums of the waves
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      red[((2 * n + r) * kUpWaves + wave) * 64 + lane] =
          make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
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
  const FewMeta meta = few_meta(p.act, p.T, p.k, p.F);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    int c = 0;
    for (int i = 0; i < 32; ++i) c += __popc(bits[i]);
    meta.head[0] = c;
  }
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
  if (blockIdx.x == 0) {
    if (threadIdx.x < m) meta.pairs[blockIdx.y * kFewT + threadIdx.x] = (uint16_t)list[threadIdx.x];
    if (threadIdx.x == 0) {
      meta.expert[blockIdx.y] = e;
      meta.count[blockIdx.y] = m;
    }
  }
  const int64_t f0 = 16 * (int64_t)blockIdx.x;
  if constexpr (NTM >= 4) {
    if (m > 32) return moe_up_tile<4, PACKED>(p, e, m, list, f0, sid, red);
  }
  if constexpr (NTM >= 2) {
    if (m > 16) return moe_up_tile<2, PACKED>(p, e, m, list, f0, sid, red);
  }
  moe_up_tile<1, PACKED>(p, e, m, list, f0, sid, red);
}

// Units [u0, u1) of one expert for 16 rows, added to the wave's sums [T][16].
template <int NT, bool PACKED>
__device__ __forceinline__ void moe_down_run(const MoeFewArgs& p, int e, int m, const uint16_t* pairs, int64_t d0,
                                             int u0, int u1, float* sum) {
  const int lane = threadIdx.x & 63, lr = lane & 15, kg = lane >> 4;
  const uint8_t* const wp[1] = {code_ptr<PACKED>(p.w2 + (int64_t)e * p.D * p.F, d0, p.F)};
  const uint16_t* xp[NT];
  int tok[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int pair = pairs[16 * n + lr < m ? 16 * n + lr : 0];
    tok[n] = pair / p.k;
    xp[n] = p.act + (int64_t)pair * p.F + 16 * kg;
  }
  v4f acc[1][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  stream_units<1, NT, kInFlight<NT>, PACKED>(wp, xp, u0, u1, (int)p.F, acc);
  const float* sc = p.inv2 + (int64_t)e * p.D + d0 + 4 * kg;
  const float s0 = sc[0], s1 = sc[1], s2 = sc[2], s3 = sc[3];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // an expert's tokens differ, so no two lanes meet
    if (16 * n + lr >= m) continue;
    float4* d = reinterpret_cast<float4*>(sum + tok[n] * 16 + 4 * kg);
    float4 v = *d;
    v.x += acc[0][n][0] * s0;
    v.y += acc[0][n][1] * s1;
    v.z += acc[0][n][2] * s2;
    v.w += acc[0][n][3] * s3;
    *d = v;
  }
}

template <int NTM, bool PACKED>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeFewArgs p) {
  constexpr int kTok = 16 * NTM;
  __shared__ float4 sums[kDownWaves * kTok * 4];  // [wave][token][16]
  const int wave = threadIdx.x >> 6;
  const FewMeta meta = few_meta(p.act, p.T, p.k, p.F);
  for (int i = threadIdx.x; i < kDownWaves * kTok * 4; i += 64 * kDownWaves) sums[i] = make_float4(0, 0, 0, 0);
  __syncthreads();
  const int64_t d0 = 16 * (int64_t)blockIdx.x;
  const int units = (int)((p.F + 127) / 128);
  const int64_t all = (int64_t)meta.head[0] * units;
  int64_t i = all * wave / kDownWaves;
  const int64_t end = all * (wave + 1) / kDownWaves;
  float* sum = reinterpret_cast<float*>(&sums[wave * kTok * 4]);
  while (i < end) {
    const int a = (int)(i / units), u0 = (int)(i % units);
    const int u1 = (int)(end - i < units - u0 ? u0 + (end - i) : units);
    const int e = meta.expert[a], m = meta.count[a];
    const uint16_t* pairs = meta.pairs + a * kFewT;
    bool done = false;
    if constexpr (NTM >= 4) {
      if (m > 32) {
        moe_down_run<4, PACKED>(p, e, m, pairs, d0, u0, u1, sum);
        done = true;
      }
    }
    if constexpr (NTM >= 2) {
      if (!done && m > 16) {
        moe_down_run<2, PACKED>(p, e, m, pairs, d0, u0, u1, sum);
        done = true;
      }
    }
    if (!done) moe_down_run<1, PACKED>(p, e, m, pairs, d0, u0, u1, sum);
    i += u1 - u0;
  }
  __syncthreads();
  const int t = threadIdx.x >> 2, q = threadIdx.x & 3;
  if (t >= (int)p.T) return;
  float r[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kDownWaves; ++w) {
    const float4 a = sums[(w * kTok + t) * 4 + q];
    r[0] += a.x;
    r[1] += a.y;
    r[2] += a.z;
    r[3] += a.w;
  }
  const v2bf lo = {(__bf16)r[0], (__bf16)r[1]}, hi = {(__bf16)r[2], (__bf16)r[3]};
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.D + d0 + 4 * q) =
      make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

template <bool PACKED>
static hipError_t launch_few_t(const MoeFewArgs& a) {
  const int64_t pairs = a.T * a.k;
  const dim3 gu((unsigned)(a.F / 16), (unsigned)(pairs < a.E ? pairs : a.E)), gd((unsigned)(a.D / 16));
  const dim3 bu(64 * kUpWaves), bd(64 * kDownWaves);
  auto go = [&](auto up, auto down) {
    hipLaunchKernelGGL(up, gu, bu, 0, a.stream, a);
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
  if (a.T == 0 || a.D == 0 || a.F == 0) return hipSuccess;
  return a.packed ? launch_few_t<true>(a) : launch_few_t<false>(a);
}

}  // namespace fp8dyn
