// moe_route.hip -- the expert router: for each token the k largest logits and
// their gate weights, and the (token, choice) pairs sorted by expert, with the
// offsets that the grouped GEMMs take; and the gate weights' gradient.
//
// Choosing compares and never computes, so it is exact: a logit's 32-bit
// pattern is mapped to an unsigned integer of the same order, and k times the
// largest is found, then the lowest expert that has it, which is taken out (bf16
// logits leave room for the expert in the integer, so that one search finds both).
// -inf and NaN have key 0, below every other, and are never chosen; a token with
// fewer than k other logits gets id -1 and weight 0 in the slots left.
//
// Sorting is by counting. 64 tokens at a time mark themselves in a 64-bit word of
// each expert they chose: the bits below a token's own are the earlier pairs of
// that expert, all of them its count. A second launch adds, for every block of
// tokens, the counts of the blocks before it and of the experts before it. No
// order but the tokens' enters: it is that of a stable sort, whatever the
// schedule. With one block (up to 64 tokens) a single launch does all.
//
// G lanes share a token and hold its E logits in registers (V each, by fours:
// element v of lane g is expert 4 (g + G (v / 4)) + v % 4), so that a wavefront
// works on 64 / G tokens at once: a maximum is V - 1 comparisons and log2 G
// exchanges between lanes, up to 16 lanes within the vector unit. What remains is
// latency: the exchanges, k rounds of them, and two to three trips to memory.
// Measured, choosing + placing: 64 tokens x 32 experts, k 8: 4.3 us; 16384 x 32, k 8:
// 5.9 + 6.0 us (2 MB of logits); 4096 x 256: 7.9 + 8.1; 65536 x 128, k 8: 25 + 9 us with bf16
// logits, 29 + 9 with fp32, bound by the vector instructions of the choices.
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace fp8dyn {

namespace {
constexpr int kChunk = 64;         // tokens a workgroup chooses for at a time
constexpr int kMaxRouteBlocks = 256;

// Tokens a block: all of them up to kChunk; else so that at most kMaxRouteBlocks
// (one a CU) count, for the second launch reads all their counts in every block
// (4096 x 256, 64 tokens a block: 13 + 5 us, 16 tokens: 7.9 + 8.1, 8 tokens: 13 + 23).
int64_t route_block_tokens(int64_t T) {
  if (T <= kChunk) return kChunk;
  const int64_t per = (T + kMaxRouteBlocks - 1) / kMaxRouteBlocks;
  return per <= kChunk ? (per + 7) / 8 * 8 : (per + kChunk - 1) / kChunk * kChunk;
}
}  // namespace

// Threads of a block: what counts is the number of rounds over a chunk (65536 x 128
// experts with 512: 30 us, with 1024: 25), and in the second launch over the counts
// (4096 x 256 with 256: 12 us, with 1024: 8.1); small blocks take the same time with either.
constexpr int kRouteThreads = 1024;
constexpr int kPlaceThreads = 1024;

template <int G>
__device__ __forceinline__ int expert_of(int g, int v) {
  return 4 * (g + G * (v >> 2)) + (v & 3);
}

// A token's logits in its lanes; -inf behind E and where the token is not live.
// vec: rows are 16-byte (bf16: 8-byte) aligned and E % 4 == 0. Else element by element: 65536
// tokens, 126 instead of 128 experts: 31 and 28 us with fp32 logits, 26 and 24 with bf16; the
// backward, whose stores are single too, 27 and 19, 20 and 18.
template <int G, int V, bool F32>
__device__ __forceinline__ void load_logits(const void* p, int64_t t, int E, int g, bool live, bool vec,
                                            float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    const int e = expert_of<G>(g, v);
    const int64_t at = t * E + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) l[v + i] = -INFINITY;
    if (!live || e >= E) continue;
    if (vec) {
      if constexpr (F32) {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        l[v] = f.x;
        l[v + 1] = f.y;
        l[v + 2] = f.z;
        l[v + 3] = f.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
        l[v] = bf16_lo(w.x);
        l[v + 1] = bf16_hi(w.x);
        l[v + 2] = bf16_lo(w.y);
        l[v + 3] = bf16_hi(w.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= E) continue;
        if constexpr (F32)
          l[v + i] = static_cast<const float*>(p)[at + i];
        else
          l[v + i] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[at + i] << 16);
      }
    }
  }
}

// The value of the lane that a group's reduction step S pairs this one with:
// lanes 1, 2 apart, then mirrored in 8 and in 16 (the lanes of a half are equal by
// then), then 16 and 32 apart.
template <int S>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (S == 0) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);
  if constexpr (S == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);
  if constexpr (S == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);
  if constexpr (S == 3) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);
  return (uint32_t)__shfl_xor((int)v, S == 4 ? 16 : 32, 64);
}
// Reduction over the G lanes of a group by op(a, b), symmetric; every lane gets it.
template <int G, int S = 0, class T, class Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
  if constexpr ((1 << S) >= G) {
    return v;
  } else {
    const T w = __builtin_bit_cast(T, partner<S>(__builtin_bit_cast(uint32_t, v)));
    return group_reduce<G, S + 1>(op(v, w), op);
  }
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<G>(v, [](float a, float b) { return a + b; });
}

// Order-preserving key of a logit; 0 for -inf and NaN.
__device__ __forceinline__ uint32_t logit_key(float f) {
  if (!(f > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// A bf16 logit's order is in the upper half of its key. The lower half holds how far
// the expert is from the last one, so that one maximum gives the largest logit and
// the lowest expert that has it, and no two experts' keys are equal.
__device__ __forceinline__ uint32_t expert_key(uint32_t key, int e) {
  return key ? (key & 0xffff0000u) | (0xffffu - (uint32_t)e) : 0;
}
template <bool F32>
__device__ __forceinline__ float key_logit(uint32_t o) {
  const uint32_t u = o & 0x80000000u ? o & 0x7fffffffu : ~o;
  return o ? __uint_as_float(F32 ? u : u & 0xffff0000u) : -INFINITY;
}

// Exclusive sums of n words in LDS, by the first wavefront; returns the total.
__device__ __forceinline__ uint32_t wave_scan(uint32_t* x, int n) {
  const int lane = threadIdx.x & 63;
  uint32_t run = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int e = e0 + lane;
    const uint32_t c = e < n ? x[e] : 0;
    uint32_t s = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t u = __shfl_up(s, o, 64);
      if (lane >= o) s += u;
    }
    if (e < n) x[e] = run + s - c;
    run += __shfl(s, 63, 64);
  }
  return run;
}

template <int G, int V, bool F32>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(const void* __restrict__ logits, int64_t T, int E, int k,
                                                             int gate, int vec, int64_t block_tokens,
                                                             int32_t* __restrict__ ids, float* __restrict__ weights,
                                                             int32_t* __restrict__ offsets,
                                                             int32_t* __restrict__ order, int32_t* __restrict__ slot,
                                                             uint32_t* __restrict__ counts) {
  extern __shared__ uint64_t lds64[];
  uint64_t* mark = lds64;                                      // [E] the tokens of the chunk that chose e
  uint32_t* cnt = reinterpret_cast<uint32_t*>(lds64 + E);      // [E] the pairs of the chunks before
  int32_t* cid = reinterpret_cast<int32_t*>(cnt + E);          // [kChunk * k]
  uint32_t* ckey = reinterpret_cast<uint32_t*>(cid + kChunk * k);  // [kChunk * k]
  __shared__ uint32_t total;
  constexpr int PER = 64 / G;  // tokens a wavefront works on at once
  constexpr int NT = kRouteThreads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane % G;
  const int64_t first = (int64_t)blockIdx.x * block_tokens;
  const int64_t last = first + block_tokens < T ? first + block_tokens : T;
  const bool sorted = offsets != nullptr;
  if (sorted) {
    for (int e = threadIdx.x; e < E; e += NT) {
      cnt[e] = 0;
      mark[e] = 0;
    }
    __syncthreads();
  }
  // the logits of the wavefront's next tokens, on their way while the present ones are chosen for
  float ahead[V];
  auto load = [&](int64_t chunk, int base) {
    const int64_t t = chunk + base + lane / G;
    load_logits<G, V, F32>(logits, t, E, g, base + lane / G < kChunk && t < last, vec != 0, ahead);
  };
  load(first, wave * PER);
  for (int64_t chunk = first; chunk < last; chunk += kChunk) {
    const int here = (int)(last - chunk < kChunk ? last - chunk : kChunk);  // tokens
    for (int base = wave * PER; base < here; base += NT / 64 * PER) {
      const int ct = base + lane / G;
      const int64_t t = chunk + ct;
      const bool live = ct < here;
      float l[V];
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = ahead[v];
      if (base + NT / 64 * PER < kChunk)
        load(chunk, base + NT / 64 * PER);
      else
        load(chunk + kChunk, wave * PER);
      uint32_t key[V];
      float bad = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        key[v] = logit_key(l[v]);
        if constexpr (!F32) key[v] = expert_key(key[v], expert_of<G>(g, v));
        if (l[v] != l[v]) bad = l[v];
      }
      bad = group_sum<G>(bad);  // 0, or NaN where a logit of the token is
      float top = 0.0f;
      for (int j = 0; j < k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
        m = group_max<G>(m);
        uint32_t best;  // m = 0: none, not used
        if constexpr (F32) {
          best = ~0u;  // the lowest expert with that key
#pragma unroll
          for (int v = V - 1; v >= 0; --v) best = key[v] == m ? (uint32_t)expert_of<G>(g, v) : best;
          best = group_min<G>(best);
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = best == (uint32_t)expert_of<G>(g, v) ? 0 : key[v];
        } else {
          best = 0xffffu - (m & 0xffffu);
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = key[v] == m ? 0 : key[v];
        }
        if (j == 0) top = key_logit<F32>(m);
        if (g == 0 && live) {
          const int e = m ? (int)best : -1;
          cid[ct * k + j] = e;
          ckey[ct * k + j] = m;
          if (sorted && e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mark[e]), 1ull << ct);
        }
      }
      // the group's own writes to LDS, read back by its other lanes
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      float z = 0.0f;
      if (gate == kGateSoftmax) {
#pragma unroll
        for (int v = 0; v < V; ++v) z += l[v] > -INFINITY ? expf(l[v] - top) : 0.0f;
        z = group_sum<G>(z);
      } else if (gate == kGateSoftmaxTopk) {
        for (int j = g; live && j < k; j += G) {
          const uint32_t m = ckey[ct * k + j];
          z += m ? expf(key_logit<F32>(m) - top) : 0.0f;
        }
        z = group_sum<G>(z);
      }
      if (live) {
        for (int j = g; j < k; j += G) {
          const int e = cid[ct * k + j];
          const float val = key_logit<F32>(ckey[ct * k + j]);
          const float w = gate == kGateSigmoid ? 1.0f / (1.0f + expf(-val)) : expf(val - top) / z;
          ids[t * k + j] = e;
          weights[t * k + j] = e >= 0 ? w + bad : 0.0f;
        }
      }
    }
    if (!sorted) continue;
    __syncthreads();
    const int n = here * k;
    if (gridDim.x == 1) {
      // the only block, and its only chunk (block_tokens == kChunk)
      for (int e = threadIdx.x; e < E; e += NT) cnt[e] = __popcll(mark[e]);
      __syncthreads();
      if (wave == 0) {
        const uint32_t sum = wave_scan(cnt, E);
        if (lane == 0) total = sum;
      }
      __syncthreads();
      for (int e = threadIdx.x; e <= E; e += NT) offsets[e] = (int32_t)(e < E ? cnt[e] : total);
    }
    for (int i = threadIdx.x; i < n; i += NT) {
      const int e = cid[i];
      const int at = e >= 0 ? (int)cnt[e] + __popcll(mark[e] & ((1ull << (i / k)) - 1)) : -1;
      slot[chunk * k + i] = at;
      if (gridDim.x == 1) {
        if (at >= 0) order[at] = i;
        if (i >= (int)total) order[i] = -1;
      }
    }
    if (gridDim.x == 1) return;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += NT) {
      cnt[e] += __popcll(mark[e]);
      mark[e] = 0;
    }
    __syncthreads();
  }
  if (sorted)
    for (int e = threadIdx.x; e < E; e += NT) counts[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// Second launch, for more than one block: block b's pairs of expert e begin at
// offsets[e] + (the counts of e in the blocks before b).
__global__ __launch_bounds__(kPlaceThreads) void k_moe_route_place(const uint32_t* __restrict__ counts, int64_t T, int E, int k,
                                                         int64_t block_tokens, const int32_t* __restrict__ ids,
                                                         int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                         int32_t* __restrict__ slot) {
  extern __shared__ uint32_t lds[];
  uint32_t* base = lds;       // [E] counts of the blocks before this one
  uint32_t* total = lds + E;  // [E] of all blocks, then the offsets
  __shared__ uint32_t all;
  const int b = blockIdx.x, nb = gridDim.x;
  for (int e = threadIdx.x; e < 2 * E; e += kPlaceThreads) lds[e] = 0;
  __syncthreads();
  // threads share an expert's column of counts where there are fewer experts
  // than threads: integer additions, whose order changes nothing
  const int parts = E < kPlaceThreads ? kPlaceThreads / E : 1;
  const int part = E < kPlaceThreads ? threadIdx.x / E : 0;
  if (part < parts) {
    for (int e = threadIdx.x % E; e < E; e += kPlaceThreads) {
      uint32_t before = 0, sum = 0;
#pragma unroll 16
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
    const uint32_t sum = wave_scan(total, E);
    if (threadIdx.x == 0) all = sum;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlaceThreads) base[e] += total[e];
  if (b == 0)
    for (int e = threadIdx.x; e <= E; e += kPlaceThreads) offsets[e] = (int32_t)(e < E ? total[e] : all);
  __syncthreads();
  const int64_t first = (int64_t)b * block_tokens * k;
  const int64_t last = first + block_tokens * k < T * k ? first + block_tokens * k : T * k;
  for (int64_t i = first + threadIdx.x; i < last; i += kPlaceThreads) {
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
// 8 logits each up to 128 experts, then 16 (32768 x 512: 34 us with 32 lanes a
// token, 60 with 64, half of them without experts).
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
  else if (E <= 512)
    go(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
  else
    go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

// Whether every row of logits can be loaded by fours.
static int rows_aligned(const void* logits, int E, bool f32) {
  return E % 4 == 0 && (uintptr_t)logits % (f32 ? 16 : 8) == 0;
}

hipError_t launch_moe_route(const RouteArgs& a) {
  if (a.T == 0) return hipSuccess;
  const int64_t bt = route_block_tokens(a.T);
  const int64_t blocks = (a.T + bt - 1) / bt;
  const size_t lds = 12 * (size_t)a.E + 8 * kChunk * a.k;
  const int vec = rows_aligned(a.logits, a.E, a.f32);
  by_experts(a.E, [&](auto G, auto V) {
    auto kern = a.f32 ? k_moe_route<G.value, V.value, true> : k_moe_route<G.value, V.value, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kRouteThreads), lds, a.stream, a.logits, a.T, a.E, a.k,
                       a.gate, vec, bt, a.ids, a.weights, a.offsets, a.order, a.slot, a.ws);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1 || !a.offsets) return e;
  hipLaunchKernelGGL(k_moe_route_place, dim3((unsigned)blocks), dim3(kPlaceThreads), 8 * (size_t)a.E, a.stream,
                     a.ws, a.T, a.E,
                     a.k, bt, a.ids, a.offsets, a.order, a.slot);
  return hipGetLastError();
}

// Gradient of the gate weights. With S the chosen experts, w their weights
// and dw the weights' gradients:
//   SOFTMAX       dl_e = p_e ([e in S] dw_e - sum_S p_s dw_s), p over all experts
//   SOFTMAX_TOPK  the same over the chosen experts (p = w, 0 elsewhere)
//   SIGMOID       dl_s = w_s (1 - w_s) dw_s, 0 elsewhere
// p is computed again from the logits; -inf and a token of -inf alone get 0. Reads and
// writes a logit once; measured 8.3 us for 8192 x 256 fp32 logits, k 8 (17 MB), of which
// an empty launch is 3.5: one trip to memory, the exchanges, the stores.
template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void k_moe_route_bwd(const void* logits, int64_t T, int E, int k, int gate, int vec,
                                                       const int32_t* __restrict__ ids,
                                                       const float* __restrict__ weights,
                                                       const float* __restrict__ dweights, void* dlogits) {
  constexpr int PER = 256 / G;
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / G;
  const bool live = t < T;
  float l[V], d[V];
  if (gate == kGateSoftmax) load_logits<G, V, F32>(logits, t, E, g, live, (vec & 1) != 0, l);
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  // the pairs are shared by the group's lanes
  float dot = 0.0f;
  for (int j = g; live && j < k; j += G) {
    const float wd = weights[t * k + j] * dweights[t * k + j];
    dot += ids[t * k + j] >= 0 ? wd : 0.0f;
  }
  dot = group_sum<G>(dot);
  if (gate == kGateSoftmax) {
    float top = -INFINITY, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
    top = group_max<G>(top);
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
  const int base = (threadIdx.x & 63) - g;  // the group's first lane
  for (int j0 = 0; j0 < k; j0 += G) {
    int e = -1;
    float c = 0.0f;
    if (live && j0 + g < k) {
      e = ids[t * k + j0 + g];
      const float w = weights[t * k + j0 + g], dw = dweights[t * k + j0 + g];
      c = gate == kGateSigmoid ? w * (1.0f - w) * dw : gate == kGateSoftmaxTopk ? w * (dw - dot) : w * dw;
    }
    for (int i = 0; i < G && j0 + i < k; ++i) {
      const int ei = __shfl(e, base + i, 64);
      const float ci = __shfl(c, base + i, 64);
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] += ei == expert_of<G>(g, v) ? ci : 0.0f;
    }
  }
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    const int e = expert_of<G>(g, v);
    const int64_t at = t * E + e;
    if (e >= E) continue;
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 b01 = {(__bf16)d[v], (__bf16)d[v + 1]}, b23 = {(__bf16)d[v + 2], (__bf16)d[v + 3]};
    const uint2 w = make_uint2(__builtin_bit_cast(uint32_t, b01), __builtin_bit_cast(uint32_t, b23));
    if (vec & 2) {
      if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(dlogits) + at) =
            make_float4(d[v], d[v + 1], d[v + 2], d[v + 3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + at) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= E) continue;
        if constexpr (F32)
          static_cast<float*>(dlogits)[at + i] = d[v + i];
        else
          static_cast<uint16_t*>(dlogits)[at + i] = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
      }
    }
  }
}

hipError_t launch_moe_route_bwd(const RouteBwdArgs& a) {
  if (a.T == 0) return hipSuccess;
  const int vec = rows_aligned(a.logits, a.E, a.f32) | rows_aligned(a.dlogits, a.E, a.f32) << 1;
  by_experts(a.E, [&](auto G, auto V) {
    auto kern = a.f32 ? k_moe_route_bwd<G.value, V.value, true> : k_moe_route_bwd<G.value, V.value, false>;
    const int64_t per = 256 / G.value;
    // one launch unless the tokens pass what a grid holds; a later one's rows are as aligned
    // as the first's, for their number is a multiple of 16
    for (int64_t t = 0; t < a.T; t += kMaxGrid256 * per) {
      const int64_t n = a.T - t < kMaxGrid256 * per ? a.T - t : kMaxGrid256 * per;
      const int64_t at = t * a.E * (a.f32 ? 4 : 2);
      hipLaunchKernelGGL(kern, dim3((unsigned)((n + per - 1) / per)), dim3(256), 0, a.stream,
                         static_cast<const uint8_t*>(a.logits) + at, n, a.E, a.k, a.gate, vec, a.ids + t * a.k,
                         a.weights + t * a.k, a.dweights + t * a.k, static_cast<uint8_t*>(a.dlogits) + at);
    }
  });
  return hipGetLastError();
}

}  // namespace fp8dyn
