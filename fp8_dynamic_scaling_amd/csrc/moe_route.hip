// moe_route.hip -- the expert router: for each token the k largest logits and
// their gate weights, and the (token, choice) pairs sorted by expert, with the
// offsets that the grouped GEMMs take; and the gate weights' gradient.
//
// Choosing compares and never computes, so it is exact: a logit's 32-bit
// pattern is mapped to an unsigned integer of the same order, with the
// complement of the expert's index below it, and the largest 64-bit key is
// taken k times (equal logits: the lowest index first). -inf and NaN have key
// 0, below every other, and are never chosen; a token with fewer than k other
// logits gets id -1 and weight 0 in the slots left.
//
// Sorting is by counting. A block of tokens counts its pairs an expert and
// numbers each pair among its block's (in token order); a second launch adds,
// for every block, the counts of the blocks before it and of the experts before
// it. No atomics: the order is that of a stable sort, whatever the schedule.
// With one block (up to 64 tokens) a single launch does all.
//
// G lanes share a token and hold its E logits in registers (V each, element v
// of lane g being expert g + G v), so that a wavefront works on 64 / G tokens
// at once: a maximum is V - 1 comparisons and log2 G exchanges.
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace fp8dyn {

namespace {
constexpr int kChunk = 64;         // tokens a workgroup chooses for at a time
constexpr int kMaxRouteK = 32;
constexpr int kMaxRouteE = 1024;
constexpr int kMaxRouteBlocks = 256;

// Tokens a block: a multiple of kChunk, so that at most kMaxRouteBlocks
// (one a CU) count; the second launch reads all their counts in every block.
int64_t route_block_tokens(int64_t T) {
  const int64_t per = (T + kMaxRouteBlocks - 1) / kMaxRouteBlocks;
  return (per + kChunk - 1) / kChunk * kChunk;
}
}  // namespace

template <bool F32>
__device__ __forceinline__ float ld_logit(const void* p, int64_t i) {
  if constexpr (F32)
    return static_cast<const float*>(p)[i];
  else
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// Order-preserving key of a logit and its expert; 0 for -inf and NaN.
__device__ __forceinline__ uint64_t logit_key(float f, int e) {
  if (!(f > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 as +0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((uint64_t)o << 32) | (uint32_t)~e;
}
__device__ __forceinline__ int key_expert(uint64_t key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

template <int G>
__device__ __forceinline__ uint64_t group_max(uint64_t v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) {
    const uint64_t w = __shfl_xor((unsigned long long)v, o, 64);
    v = w > v ? w : v;
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The pair's place among the earlier pairs of its block with the same expert,
// for 64 pairs of a wavefront in their order; cnt holds the counts so far and
// is brought up to date. e: the pair's expert, -1 for none.
__device__ __forceinline__ int wave_rank(int e, int bits, uint32_t* cnt) {
  uint64_t same = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? set : ~set;
  }
  const int lane = threadIdx.x & 63;
  const int before = __popcll(same & ((1ull << lane) - 1));
  const uint32_t c = e >= 0 ? cnt[e] : 0;
  // the first of an expert's pairs writes, after all of them have read
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (e >= 0 && before == 0) cnt[e] = c + (uint32_t)__popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return (int)c + before;
}

template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void k_moe_route(const void* __restrict__ logits, int64_t T, int E, int k, int gate,
                                                   int bits, int64_t block_tokens, int32_t* __restrict__ ids,
                                                   float* __restrict__ weights, int32_t* __restrict__ offsets,
                                                   int32_t* __restrict__ order, int32_t* __restrict__ slot,
                                                   uint32_t* __restrict__ counts) {
  extern __shared__ uint32_t lds[];
  uint32_t* cnt = lds;                                         // [E]
  int32_t* cid = reinterpret_cast<int32_t*>(lds + E);          // [kChunk * k]
  float* cval = reinterpret_cast<float*>(lds + E + kChunk * k);  // [kChunk * k]
  constexpr int PER = 64 / G;  // tokens a wavefront works on at once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane % G;
  const int64_t first = (int64_t)blockIdx.x * block_tokens;
  const int64_t last = first + block_tokens < T ? first + block_tokens : T;
  const bool sorted = offsets != nullptr;
  if (sorted)
    for (int e = threadIdx.x; e < E; e += 256) cnt[e] = 0;
  for (int64_t chunk = first; chunk < last; chunk += kChunk) {
    for (int base = wave * PER; base < kChunk; base += 4 * PER) {
      const int ct = base + lane / G;
      const int64_t t = chunk + ct;
      const bool live = t < last && ct < kChunk;
      float l[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = g + G * v;
        l[v] = live && e < E ? ld_logit<F32>(logits, t * E + e) : -INFINITY;
      }
      uint64_t key[V];
      float bad = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        key[v] = logit_key(l[v], g + G * v);
        if (l[v] != l[v]) bad = l[v];
      }
      bad = group_sum<G>(bad);  // 0, or NaN where a logit of the token is
      float top = 0.0f, zk = 0.0f;
      for (int j = 0; j < k; ++j) {
        uint64_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
        m = group_max<G>(m);
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == m ? 0 : key[v];
        const float val = m ? key_logit(m) : -INFINITY;
        if (j == 0) top = val;
        zk += m ? expf(val - top) : 0.0f;
        if (g == 0 && live) {
          cid[ct * k + j] = m ? key_expert(m) : -1;
          cval[ct * k + j] = val;
        }
      }
      float z = zk;
      if (gate == kGateSoftmax) {
        z = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) z += l[v] > -INFINITY ? expf(l[v] - top) : 0.0f;
        z = group_sum<G>(z);
      }
      // the group's own writes to LDS, read back by its other lanes
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (live) {
        for (int j = g; j < k; j += G) {
          const int e = cid[ct * k + j];
          const float val = cval[ct * k + j];
          const float w = gate == kGateSigmoid ? 1.0f / (1.0f + expf(-val)) : expf(val - top) / z;
          ids[t * k + j] = e;
          weights[t * k + j] = e >= 0 ? w + bad : 0.0f;
        }
      }
    }
    if (!sorted) continue;
    __syncthreads();
    if (wave == 0) {
      const int64_t left = last - chunk;
      const int n = (int)(left < kChunk ? left : kChunk) * k;
      for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + lane;
        const int e = i < n ? cid[i] : -1;
        const int r = wave_rank(e, bits, cnt);
        if (i < n) slot[chunk * k + i] = e >= 0 ? r : -1;
      }
    }
    __syncthreads();
  }
  if (!sorted) return;
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < E; e += 256) counts[(int64_t)blockIdx.x * E + e] = cnt[e];
    return;
  }
  // one block: its counts are the totals, and the last chunk's ids are at hand
  // (block_tokens == kChunk)
  uint32_t run = 0;
  if (wave == 0) {
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t c = e < E ? cnt[e] : 0;
      uint32_t s = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
      }
      if (e < E) {
        cnt[e] = run + s - c;
        offsets[e] = (int32_t)(run + s - c);
      }
      run += __shfl(s, 63, 64);
    }
    if (lane == 0) {
      offsets[E] = (int32_t)run;
      cval[0] = __uint_as_float(run);  // the gate values are no longer needed
    }
  }
  __syncthreads();
  const int total = (int)__float_as_uint(cval[0]);
  for (int i = threadIdx.x; i < (int)(last - first) * k; i += 256) {
    const int e = cid[i];
    if (e >= 0) {
      const int at = (int)cnt[e] + slot[i];
      slot[i] = at;
      order[at] = i;
    }
    if (i >= total) order[i] = -1;
  }
}

// Second launch, for more than one block: block b's pairs of expert e begin at
// offsets[e] + (the counts of e in the blocks before b).
__global__ __launch_bounds__(256) void k_moe_route_place(const uint32_t* __restrict__ counts, int64_t T, int E, int k,
                                                         int64_t block_tokens, const int32_t* __restrict__ ids,
                                                         int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                         int32_t* __restrict__ slot) {
  extern __shared__ uint32_t lds[];
  uint32_t* base = lds;       // [E] counts of the blocks before this one
  uint32_t* total = lds + E;  // [E] of all blocks, then the offsets
  __shared__ uint32_t all;
  const int b = blockIdx.x, nb = gridDim.x;
  for (int e = threadIdx.x; e < 2 * E; e += 256) lds[e] = 0;
  __syncthreads();
  // threads share an expert's column of counts where there are fewer experts
  // than threads: integer additions, whose order changes nothing
  const int parts = E < 256 ? 256 / E : 1;
  const int part = E < 256 ? threadIdx.x / E : 0;
  if (part < parts) {
    for (int e = E < 256 ? threadIdx.x % E : threadIdx.x; e < E; e += 256) {
      uint32_t before = 0, sum = 0;
#pragma unroll 8
      for (int i = part; i < nb; i += parts) {
        const uint32_t c = counts[(int64_t)i * E + e];
        sum += c;
        before += i < b ? c : 0;
      }
      atomicAdd(&total[e], sum);
      atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    uint32_t run = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t c = e < E ? total[e] : 0;
      uint32_t s = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
      }
      if (e < E) {
        base[e] += run + s - c;
        if (b == 0) offsets[e] = (int32_t)(run + s - c);
      }
      run += __shfl(s, 63, 64);
    }
    if (lane == 0) {
      all = run;
      if (b == 0) offsets[E] = (int32_t)run;
    }
  }
  __syncthreads();
  const int64_t first = (int64_t)b * block_tokens * k;
  const int64_t last = first + block_tokens * k < T * k ? first + block_tokens * k : T * k;
  for (int64_t i = first + threadIdx.x; i < last; i += 256) {
    const int e = ids[i];
    if (e >= 0) {
      const int32_t at = (int32_t)base[e] + slot[i];
      slot[i] = at;
      order[at] = (int32_t)i;
    }
    if (i >= (int64_t)all) order[i] = -1;
  }
}

int64_t route_ws_words(int64_t T, int32_t E) {
  if (T <= kChunk) return 0;
  const int64_t bt = route_block_tokens(T);
  return (T + bt - 1) / bt * E;
}

// Lanes a token and logits a lane: the smallest group whose lanes hold at most
// 8 logits each up to 128 experts, then 16.
template <class F>
static void by_experts(int E, F&& go) {
  if (E <= 16)
    go(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  else if (E <= 32)
    go(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else if (E <= 64)
    go(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  else if (E <= 128)
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  else if (E <= 256)
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
  else
    go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

hipError_t launch_moe_route(const RouteArgs& a) {
  if (a.T == 0) return hipSuccess;
  const int64_t bt = route_block_tokens(a.T);
  const int64_t blocks = (a.T + bt - 1) / bt;
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  const size_t lds = 4 * ((size_t)a.E + 2 * kChunk * a.k);
  by_experts(a.E, [&](auto G, auto V) {
    auto kern = a.f32 ? k_moe_route<G.value, V.value, true> : k_moe_route<G.value, V.value, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), lds, a.stream, a.logits, a.T, a.E, a.k, a.gate, bits,
                       bt, a.ids, a.weights, a.offsets, a.order, a.slot, a.ws);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1 || !a.offsets) return e;
  hipLaunchKernelGGL(k_moe_route_place, dim3((unsigned)blocks), dim3(256), 8 * (size_t)a.E, a.stream, a.ws, a.T, a.E,
                     a.k, bt, a.ids, a.offsets, a.order, a.slot);
  return hipGetLastError();
}

// Gradient of the gate weights. With S the chosen experts, w their weights
// and dw the weights' gradients:
//   SOFTMAX       dl_e = p_e ([e in S] dw_e - sum_S p_s dw_s), p over all experts
//   SOFTMAX_TOPK  the same over the chosen experts (p = w, 0 elsewhere)
//   SIGMOID       dl_s = w_s (1 - w_s) dw_s, 0 elsewhere
// p is computed again from the logits; -inf and a token of -inf alone get 0.
template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void k_moe_route_bwd(const void* logits, int64_t T, int E, int k, int gate,
                                                       const int32_t* __restrict__ ids,
                                                       const float* __restrict__ weights,
                                                       const float* __restrict__ dweights, void* dlogits) {
  constexpr int PER = 256 / G;
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / G;
  const bool live = t < T;
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  float dot = 0.0f;
  for (int j = g; live && j < k; j += G)
    dot += ids[t * k + j] >= 0 ? weights[t * k + j] * dweights[t * k + j] : 0.0f;
  dot = group_sum<G>(dot);
  if (gate == kGateSoftmax) {
    float l[V], top = -INFINITY, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = g + G * v;
      l[v] = live && e < E ? ld_logit<F32>(logits, t * E + e) : -INFINITY;
      top = fmaxf(top, l[v]);
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // a NaN logit stays one, so the token's gradients are NaN as its weights were
      l[v] = l[v] == -INFINITY ? 0.0f : expf(l[v] - top);
      z += l[v];
    }
    z = group_sum<G>(z);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = z == 0.0f ? 0.0f : -l[v] / z * dot;
  }
  if (!live) return;
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    const float w = weights[t * k + j], dw = dweights[t * k + j];
    const float c = gate == kGateSigmoid ? w * (1.0f - w) * dw : gate == kGateSoftmaxTopk ? w * (dw - dot) : w * dw;
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] += e == g + G * v ? c : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = g + G * v;
    if (e >= E) continue;
    if constexpr (F32) {
      static_cast<float*>(dlogits)[t * E + e] = d[v];
    } else {
      const __bf16 b = (__bf16)d[v];
      static_cast<uint16_t*>(dlogits)[t * E + e] = __builtin_bit_cast(uint16_t, b);
    }
  }
}

hipError_t launch_moe_route_bwd(const RouteBwdArgs& a) {
  if (a.T == 0) return hipSuccess;
  by_experts(a.E, [&](auto G, auto V) {
    auto kern = a.f32 ? k_moe_route_bwd<G.value, V.value, true> : k_moe_route_bwd<G.value, V.value, false>;
    const int64_t per = 256 / G.value;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, a.stream, a.logits, a.T, a.E, a.k,
                       a.gate, a.ids, a.weights, a.dweights, a.dlogits);
  });
  return hipGetLastError();
}

}  // namespace fp8dyn
