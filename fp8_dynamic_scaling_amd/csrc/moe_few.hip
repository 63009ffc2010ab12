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
//  - k_moe_up: four workgroups a CU share the named experts' tiles of 16 gate and
//    16 up rows evenly; a workgroup's waves share D among them. The waves'
//    partial sums meet in LDS, in a fixed order.
//  - k_moe_down: the workgroups share the tiles of rows of D, each for all
//    experts, evenly; the waves share a tile's (expert, piece of F) units. A wave
//    adds what it has of a token to its own fp32 sums in LDS, the waves' sums are
//    added in order, and so are those of workgroups that share a tile: the same
//    inputs give the same bits. How tiles are shared goes by the experts that the
//    batch names, so a token's sums may be taken in another order in another batch.
// A wave's unit of work is twice 16 rows x 128 values of the
// contraction and the same 128 values of its tokens. An expert's tokens are
// compacted into tiles of 16.
//
// After HBM the loads' own rate is the next bound: measured, a 16-byte load of
// a wavefront takes 17 clocks of its CU's load path where each four neighbouring
// lanes read an aligned 64 bytes, 33 where they read 64-byte steps (a packed
// chunk as the matrix instruction's lanes want it) and 65 where they read four
// rows. So codes and rows of x are loaded with neighbouring lanes along the row
// and turned in a wave's own piece of LDS, a is written in the order in which
// k_moe_down reads it, and tokens are loaded by fours: one load of a unit
// for up to 4 tokens of an expert, two up to 8.
//
// a is kept as the sum of two bf16 values (some 16 bits of its fp32 value), each
// multiplied by the codes: one bf16 value alone would add as large an error to the
// output as the output's own rounding. The second one costs 2 to 3% of the call with
// few tokens (63.2 -> 64.5 us with one, 333 -> 343 with 64 that take one of 16 experts
// each) and up to 14% where an expert has many (293 -> 334 us, 64 tokens that take 8 of
// 32). Some of the outputs are therefore rounded to the other neighbour than with an fp32 a
// (1e-4 of the norm); their error against 64 bits is the same. Everything else is fp32 up to
// the one rounding of the output.
//
// Measured, both launches, bytes of codes read: one token, 8 of 32 experts of D 7168 and
// F 2048, packed: 352 MB in 63.5 us (5.5 TB/s); 16 tokens of the same, 31 experts named:
// 1.38 GB in 225 us (6.1 TB/s); 64 tokens, 16 experts of D 5120, F 8192, row-major: 2.0 GB
// in 343 us (5.9 TB/s), packed 340. A kernel that only reads such an amount reaches 5.7
// to 6.3 TB/s with these loads.
//
// A token may name an expert twice: its first slot carries the sum of the
// weights. Ids outside [0, E) name none.
#include <type_traits>

#include "gemm_common.hpp"

namespace fp8dyn {

namespace {
// Medians of launches back to back, one token (8 of 32 experts, D 7168, F 2048), 16 tokens of
// the same and 64 tokens (1 of 16 experts, D 5120, F 8192): with 512 workgroups k_moe_up
// takes 59, 240 and 350 us, with 1024 40, 154 and 237, with 2048, which take turns on the
// CUs, 40, 183 and 282. k_moe_down with one tile of 16 rows a unit takes 37, 128 and 189 us,
// with two, which share a load of the tokens, 24, 84 and 129.
constexpr int kUpWaves = 2;
constexpr int kUpBlocks = 1024;  // four a CU
constexpr int kDownWaves = 8;
constexpr int kDownBlocks = 256;  // one a CU
constexpr int kDownTiles = 2;     // tiles of 16 rows a unit has at most
constexpr int kDownRows = 16 * kDownTiles;

// What k_moe_up leaves in the workspace for k_moe_down: a, in units of 128 values
// of F, the last one with room for as many; an expert's units are at pair 4 start
// (room for m tokens, rounded up to a multiple mp of four), in a unit the first
// parts [16 groups of 8 values][mp tokens][8], then the second parts alike; the
// number of named experts; each one's id, in order, where its pairs begin,
// and the tokens of the pairs. k_moe_down joins split sums by `done` (counters
// that k_moe_up clears) and `part` ([workgroup][first or last tile][T][rows]).
struct FewMeta {
  float* part;       // [kDownBlocks][2][T][kDownRows]
  uint32_t* done;    // [kDownBlocks]
  int32_t* head;     // [0]: the number of experts
  uint16_t* expert;  // [T * k]
  uint16_t* start;   // [T * k + 1]
  uint16_t* token;   // [T * k]
};
__host__ __device__ inline int64_t act_pair(int64_t F) { return (F + 127) / 128 * 256; }  // bf16 values a pair
__host__ __device__ inline FewMeta few_meta(uint16_t* act, int64_t T, int k, int64_t F) {
  FewMeta m;
  m.part = reinterpret_cast<float*>(act + 4 * T * k * act_pair(F));
  m.done = reinterpret_cast<uint32_t*>(m.part + kDownBlocks * 2 * T * kDownRows);
  m.head = reinterpret_cast<int32_t*>(m.done + kDownBlocks);
  m.expert = reinterpret_cast<uint16_t*>(m.head + 1);
  m.start = m.expert + T * k;
  m.token = m.start + T * k + 1;
  return m;
}
}  // namespace

size_t moe_few_ws_bytes(int64_t T, int k, int64_t F) {
  return (size_t)(T * k) * (8 * act_pair(F) + 6) + 8 + kDownBlocks * (size_t)(4 + 8 * T * kDownRows);
}

// Eight e4m3 codes -> eight bf16 (every e4m3 value is a bf16 value).
__device__ __forceinline__ v8bf decode8(uint32_t d0, uint32_t d1) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, true);
  return (v8bf){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The wavefront's number, known to be the same in all of its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Orders a wavefront's LDS reads behind its writes (LDS serves a wavefront in order).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- one unit's operands --------------------------------------------------------
//
// A unit is the values [128 u, 128 u + 128) of the contraction, of length K; the
// last one may hold fewer, a multiple of 16. Every load is unconditional, so that
// the compiler knows how many are in flight and waits for the oldest unit alone:
// a lane whose piece would lie behind K loads the unit's first piece, and
// mask_unit takes its values out.
//
// A tile of codes, 16 rows x 128 values, as two 16-byte loads a lane. Packed:
// load h is the 1 KB chunk of 64 values, row l >> 2, 16 bytes l & 3 (the chunks
// follow each other along the contraction). Row-major: load i has rows
// 8 i + (l >> 3), 16 bytes l & 7.
template <bool PACKED>
struct Codes {
  uint32_t off, last;  // the lane's offset, and in the last unit
  __device__ __forceinline__ explicit Codes(int K) {
    const int l = threadIdx.x & 63, c = l & 7, rest = K - (K - 1) / 128 * 128;
    off = PACKED ? l * 16 : (l >> 3) * (uint32_t)K + c * 16;
    last = PACKED || 16 * c < rest ? off : off - 16 * c;
  }
  // tile: the first of the 16 rows
  __device__ __forceinline__ void load(uint4 (&w)[2], const uint8_t* tile, int u, int K) const {
    if constexpr (PACKED) {
      const uint8_t* p = tile + (int64_t)u * 2048;
      w[0] = ld_nt16(p + off);
      w[1] = ld_nt16(p + (128 * u + 64 < K ? 1024 : 0) + off);  // K % 64 == 0: the last unit may be half
    } else {
      const uint8_t* p = tile + 128 * u;
      const uint32_t o = 128 * (u + 1) <= K ? off : last;
      w[0] = ld_nt16(p + o);
      w[1] = ld_nt16(p + 8 * (int64_t)K + o);
    }
  }
};
// The lanes' operands of a loaded tile, row l & 15 and values 16 (l >> 4) .. + 15
// of each 64, through 2 KB of LDS. Pieces of 16 bytes are placed so that the 16
// rows of a column of pieces fall on all banks: packed, row r's piece c of a
// chunk at r * 64 + 16 (c ^ (r / 4)); row-major, at r * 128 + 16 (c ^ (r / 2 % 8)).
template <bool PACKED>
__device__ __forceinline__ void turn_codes(uint4 (&w)[2], uint8_t* lds) {
  const int l = threadIdx.x & 63, lr = l & 15, kg = l >> 4;
  if constexpr (PACKED) {
    const int r = l >> 2, c = l & 3;
    uint8_t* d = lds + r * 64 + 16 * (c ^ (r >> 2));
    *reinterpret_cast<uint4*>(d) = w[0];
    *reinterpret_cast<uint4*>(d + 1024) = w[1];
    wave_lds_fence();
    const uint8_t* q = lds + lr * 64 + 16 * (kg ^ (lr >> 2));
    w[0] = *reinterpret_cast<const uint4*>(q);
    w[1] = *reinterpret_cast<const uint4*>(q + 1024);
  } else {
    const int r = l >> 3, c = l & 7;
    *reinterpret_cast<uint4*>(lds + r * 128 + 16 * (c ^ (r >> 1))) = w[0];
    *reinterpret_cast<uint4*>(lds + (r + 8) * 128 + 16 * (c ^ ((r >> 1) + 4))) = w[1];
    wave_lds_fence();
    w[0] = *reinterpret_cast<const uint4*>(lds + lr * 128 + 16 * (kg ^ (lr >> 1)));
    w[1] = *reinterpret_cast<const uint4*>(lds + lr * 128 + 16 * ((4 + kg) ^ (lr >> 1)));
  }
  wave_lds_fence();
}

// The operands of a tile of 16 tokens: of matrix instruction q, the values
// 64 (q / 2) + 16 (l >> 4) + 8 (q % 2) .. + 7 of token l & 15, those of the codes'
// bytes 8 (q % 2) .. + 7 of load q / 2.
struct Tokens {
  v8bf v[4];
};

// Rows of x: load i has tokens 4 i + (l >> 4), 16 bytes l & 15, and goes through
// 4 KB of LDS for 16 tokens: token r's piece c lies at r * 256 + 16 (c ^ r).
// G loads for 4 G tokens.
template <int G>
__device__ __forceinline__ void load_rows(v8bf (&x)[G], const uint16_t* base, const uint32_t (&off)[G], uint32_t back,
                                          int u, int K) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base + 128 * u);
  const uint32_t o = 128 * (u + 1) <= K ? 0 : back;
#pragma unroll
  for (int i = 0; i < G; ++i) x[i] = *reinterpret_cast<const v8bf*>(p + (off[i] - o));
}
template <int G, int NT>
__device__ __forceinline__ void turn_rows(const v8bf (&x)[G], Tokens (&t)[NT], uint8_t* lds) {
  const int l = threadIdx.x & 63, lr = l & 15, kg = l >> 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < (G < 4 ? G : 4); ++i) {
      const int r = 4 * i + kg;
      *reinterpret_cast<v8bf*>(lds + r * 256 + 16 * (lr ^ r)) = x[4 * n + i];
    }
    wave_lds_fence();
    // lanes without a token read what LDS holds: a column that nobody reads
#pragma unroll
    for (int q = 0; q < 4; ++q)
      t[n].v[q] = *reinterpret_cast<const v8bf*>(lds + lr * 256 + 16 * ((8 * (q >> 1) + 2 * kg + (q & 1)) ^ lr));
    wave_lds_fence();
  }
}

// Zeros for the values of the last unit that lie behind K.
template <int R, int NT, int S>
__device__ __forceinline__ void mask_unit(uint4 (&w)[R][2], Tokens (&x)[S][NT], int u, int K) {
  if (128 * (u + 1) <= K) return;
  const int kg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (128 * u + 64 * h + 16 * kg < K) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) w[r][h] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int z = 0; z < S; ++z)
#pragma unroll
      for (int n = 0; n < NT; ++n) x[z][n].v[2 * h] = x[z][n].v[2 * h + 1] = (v8bf){};
  }
}

// The products of R tiles of codes with NT tiles of tokens, whose values are the sums of S
// parts.
template <int R, int NT, int S>
__device__ __forceinline__ void multiply(const uint4 (&w)[R][2], const Tokens (&x)[S][NT], v4f (&acc)[R][NT]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v8bf a[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[2 * h] = decode8(w[r][h].x, w[r][h].y);
      a[2 * h + 1] = decode8(w[r][h].z, w[r][h].w);
    }
    // two wait states between the converts and the matrix instructions
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 1" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int z = 0; z < S; ++z) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], x[z][n].v[q], acc[r][n], 0, 0, 0);
      }
    }
    // the operands stay live past the matrix instructions, which nothing may
    // move behind this point: no destination shares a source's registers
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      keep_live(a[q]);
#pragma unroll
      for (int z = 0; z < S; ++z)
#pragma unroll
        for (int n = 0; n < NT; ++n) keep_live(x[z][n].v[q]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
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

// Inclusive count of the bits up to each of the 32 words, in lanes 0 to 31.
__device__ __forceinline__ int few_count(uint32_t w) {
  const int lane = threadIdx.x & 63;
  int upto = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up(upto, o, 64);
    if (lane >= o) upto += u;
  }
  return upto;
}

// The s-th named expert in order, s below their number (the same in every lane);
// w and upto: the bits and their counts in lanes 0 to 31.
__device__ __forceinline__ int few_expert(uint32_t w, int upto, int s) {
  const int lane = threadIdx.x & 63;
  const int before = upto - __popc(w);
  const uint64_t hit = __ballot(lane < 32 && s >= before && s < upto);
  const int word = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
  uint32_t v = __builtin_amdgcn_readlane(w, word);
  for (int r = s - __builtin_amdgcn_readlane(before, word); r > 0; --r) v &= v - 1;
  return 32 * word + __ffs(v) - 1;
}

// Calls go with the loads of four tokens for m tokens, at most 16 NTM.
template <int NTM, class F>
__device__ __forceinline__ void by_tokens(int m, F&& go) {
  if (NTM >= 4 && m > 32)
    go(std::integral_constant<int, NTM >= 4 ? 16 : 4>{});
  else if (NTM >= 2 && m > 16)
    go(std::integral_constant<int, NTM >= 2 ? 8 : 4>{});
  else if (m > 8)
    go(std::integral_constant<int, 4>{});
  else if (m > 4)
    go(std::integral_constant<int, 2>{});
  else
    go(std::integral_constant<int, 1>{});
}

struct UpShared {
  int32_t sid[kFewT * kMaxMoeK];
  int32_t list[kFewT];
  float gate[kFewT];
  float scale[2][32];
  uint32_t bits[kMaxMoeE / 32];
  int count[2];
};

template <int G, bool PACKED>
__device__ __forceinline__ void moe_up_tiles(const MoeFewArgs& p, int e, int m, int64_t act0, int64_t f0, int nt,
                                             UpShared& sh, float4* red, uint8_t* turn) {
  constexpr int NT = (G + 3) / 4;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int lr = lane & 15, kg = lane >> 4;
  const uint8_t* wb = p.w13 + (int64_t)e * 2 * p.F * p.D;
  const float* sc = p.inv13 + (int64_t)e * 2 * p.F + (lane & 16 ? p.F : 0) + f0 + lr;
  const int D = (int)p.D;
  const Codes<PACKED> codes(D);
  // past the last token the first one's values: a column that nobody reads
  uint32_t xoff[G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int it = 4 * i + kg < m ? 4 * i + kg : 0;
    xoff[i] = 2 * ((uint32_t)(sh.list[it] / p.k) * (uint32_t)D + 8 * lr);
  }
  const int mp = (m + 3) & ~3;
  const uint32_t back = 8 * lr < D - (D - 1) / 128 * 128 ? 0 : 16 * lr;
  const int units = (D + 127) / 128;
  const int u0 = units * wave / kUpWaves, nu = units * (wave + 1) / kUpWaves - u0;
  uint4 w[2][2];
  v8bf x[G];
  auto load = [&](int tile, int u) {
    codes.load(w[0], wb + (f0 + 16 * tile) * p.D, u0 + u, D);
    codes.load(w[1], wb + (p.F + f0 + 16 * tile) * p.D, u0 + u, D);
    load_rows<G>(x, p.x, xoff, back, u0 + u, D);
  };
  float scale = sc[0];
  uint8_t* mine = turn + wave * 4096;
  v4f acc[2][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  int tile = 0;
  auto finish = [&]() {
    // The waves' partial sums (and the rows' scales), in one of two buffers: a
    // wave writes it again two tiles on, behind a barrier that the reader
    // reaches after reading. Four token tiles have one buffer, which lets
    // four workgroups share a CU's LDS, and a barrier before it is written again.
    if (NT == 4 && tile > 0) __syncthreads();
    float4* r = red + (NT < 4 ? tile & 1 : 0) * (NT * 2 * kUpWaves * 64);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        r[((2 * n + z) * kUpWaves + wave) * 64 + lane] =
            make_float4(acc[z][n][0], acc[z][n][1], acc[z][n][2], acc[z][n][3]);
        acc[z][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    if (wave == 0 && lane < 32) sh.scale[tile & 1][lane] = scale;
    scale = sc[16 * (tile + 1 < nt ? tile + 1 : tile)];
    __syncthreads();
    // the waves finish the token tiles in turn
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kUpWaves) {
      const int n = n0 + (wave + tile) % kUpWaves;
      const int item = 16 * n + lr;
      if (n >= NT || item >= m) continue;
      float g[4] = {0, 0, 0, 0}, uu[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kUpWaves; ++i) {
        const float4 a = r[((2 * n) * kUpWaves + i) * 64 + lane];
        const float4 b = r[((2 * n + 1) * kUpWaves + i) * 64 + lane];
        g[0] += a.x;
        g[1] += a.y;
        g[2] += a.z;
        g[3] += a.w;
        uu[0] += b.x;
        uu[1] += b.y;
        uu[2] += b.z;
        uu[3] += b.w;
      }
      const float gate = sh.gate[item];
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gv = g[i] * sh.scale[tile & 1][4 * kg + i], uv = uu[i] * sh.scale[tile & 1][16 + 4 * kg + i];
        v[i] = gate * (gv / (1.0f + expf(-gv)) * uv);
      }
      // v as a bf16 value and the bf16 value of what is left, nothing beside an infinity
      v2bf hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __bf16 h = (__bf16)v[i];
        hi[i >> 1][i & 1] = h;
        lo[i >> 1][i & 1] = (__bf16)(isinf((float)h) ? 0.0f : v[i] - (float)h);
      }
      const int f = (int)f0 + 16 * tile + 4 * kg;
      uint16_t* d = p.act + 4 * act0 * act_pair(p.F) + (int64_t)(f >> 7) * 256 * mp +
                    ((f >> 3 & 15) * mp + item) * 8 + (f & 7);
      *reinterpret_cast<uint2*>(d) =
          make_uint2(__builtin_bit_cast(uint32_t, hi[0]), __builtin_bit_cast(uint32_t, hi[1]));
      *reinterpret_cast<uint2*>(d + 128 * mp) =
          make_uint2(__builtin_bit_cast(uint32_t, lo[0]), __builtin_bit_cast(uint32_t, lo[1]));
    }
    ++tile;
  };
  if (nu == 0) {  // fewer units than waves: this wave has zeros to add
    while (tile < nt) finish();
    return;
  }
  load(0, 0);
  while (tile < nt) {
    for (int u = 0; u < nu; ++u) {
      turn_codes<PACKED>(w[0], mine);
      turn_codes<PACKED>(w[1], mine);
      Tokens t[1][NT];
      turn_rows<G, NT>(x, t[0], mine);
      mask_unit<2, NT, 1>(w, t, u0 + u, D);
      multiply<2, NT, 1>(w, t, acc);
      const bool here = u + 1 < nu;
      load(here || tile + 1 == nt ? tile : tile + 1, here ? u + 1 : 0);  // behind the last unit one that nobody uses
    }
    finish();
  }
}

// The workgroups share the named experts' tiles of 16 columns of F evenly, each
// a run of neighbours: an expert's tokens are looked up once or twice a
// workgroup, and its codes are read in long runs.
template <int NTM, bool PACKED>
__global__ __launch_bounds__(64 * kUpWaves, 2) void k_moe_up(MoeFewArgs p) {
  __shared__ float4 red[(NTM < 4 ? 2 : 1) * NTM * 2 * kUpWaves * 64];
  __shared__ __align__(16) uint8_t turn[kUpWaves * 4096];
  __shared__ UpShared sh;
  const int lane = threadIdx.x & 63;
  const int n = (int)p.T * p.k;
  // the first pairs' weights, under way while the ids are looked at
  const float weight0 = threadIdx.x < 64 && lane < n ? p.weights[lane] : 0.0f;
  few_ids(p.ids, n, p.E, sh.sid, sh.bits);
  const uint32_t named = lane < 32 ? sh.bits[lane] : 0;
  const int upto = few_count(named), nact = __builtin_amdgcn_readlane(upto, 31);
  const FewMeta meta = few_meta(p.act, p.T, p.k, p.F);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) meta.head[0] = nact;
    for (int i = threadIdx.x; i < kDownBlocks; i += 64 * kUpWaves) meta.done[i] = 0;
  }
  // at most 2^10 experts of 2^16 tiles
  const uint32_t per = (uint32_t)(p.F / 16), all = nact * per, each = all / gridDim.x, rest = all % gridDim.x;
  uint32_t tile = each * blockIdx.x + (blockIdx.x < rest ? blockIdx.x : rest);
  const uint32_t end = tile + each + (blockIdx.x < rest);
  while (tile < end) {
    const int a = (int)(tile / per), first = (int)(tile % per);
    const int nt = (int)(end - tile < per - first ? end - tile : per - first);
    const int e = few_expert(named, upto, a);
    // the expert's pairs in order, the first of each token's only, with the
    // weights of all the token's slots that name e, and the number of pairs of
    // the experts before it
    __syncthreads();
    if (threadIdx.x < 64) {
      int m = 0, below = 0;
      for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + lane;
        const int id = i < n ? sh.sid[i] : -1;
        bool head = id >= 0 && id <= e;
        for (int j = i - i % p.k; head && j < i; ++j) head = sh.sid[j] != id;
        const uint64_t b = __ballot(head && id == e);
        if (head && id == e) {
          const int at = m + __popcll(b & ((1ull << lane) - 1));
          float gate = i0 == 0 ? weight0 : p.weights[i];
          for (int j = i + 1; j < i - i % p.k + p.k; ++j)
            if (sh.sid[j] == e) gate += p.weights[j];
          sh.list[at] = i;
          sh.gate[at] = gate;
        }
        m += __popcll(b);
        below += __popcll(__ballot(head && id < e));
      }
      if (lane == 0) {
        sh.count[0] = m;
        sh.count[1] = below;
      }
    }
    __syncthreads();
    const int m = __builtin_amdgcn_readfirstlane(sh.count[0]), act0 = __builtin_amdgcn_readfirstlane(sh.count[1]);
    if (first == 0) {  // one workgroup of the expert's says who its tokens are
      if (threadIdx.x < m) meta.token[act0 + threadIdx.x] = (uint16_t)(sh.list[threadIdx.x] / p.k);
      if (threadIdx.x == 0) {
        meta.expert[a] = (uint16_t)e;
        meta.start[a] = (uint16_t)act0;
        if (a == nact - 1) meta.start[nact] = (uint16_t)(act0 + m);
      }
    }
    const int64_t f0 = 16 * (int64_t)first;
    auto run = [&](auto loads) { moe_up_tiles<loads.value, PACKED>(p, e, m, act0, f0, nt, sh, red, turn); };
    by_tokens<NTM>(m, run);
    tile += nt;
  }
}

struct DownShared {
  uint16_t expert[kMaxMoeE], start[kMaxMoeE + 1], token[kFewT * kMaxMoeK];
  int count;
};

// A wave's run [i, end) of the (expert, unit) pairs of R tiles of 16 rows, the next one
// loaded as soon as one has been multiplied. At an expert's last unit its sums,
// times the rows' scales, are added to the wave's sums [token][row].
template <int G, bool PACKED, int R>
__device__ __forceinline__ void moe_down_run(const MoeFewArgs& p, const DownShared& sh, int64_t d0, int units, int i,
                                             int end, float* sum, uint8_t* turn) {
  constexpr int NT = (G + 3) / 4;
  const int lane = threadIdx.x & 63, lr = lane & 15, kg = lane >> 4, F = (int)p.F;
  uint4 w[R][2];
  v8bf x[2][G];
  const Codes<PACKED> codes(F);
  // the first row of tile r; behind D the first tile again, whose sums are not written
  auto row_of = [&](int r) { return d0 + 16 * r < p.D ? d0 + 16 * r : d0; };
  // the unit that the registers hold, or that is on its way to them
  int a = i / units, u = i % units, mp = 0;
  const uint8_t* wp[R];
  const uint8_t* ap = nullptr;
  // Up to 8 tokens: a part's 256 mp bytes in a row, mp / 4 loads (with fewer than
  // G, the first again), turned in LDS. More: the lanes' own operands.
  uint32_t aoff[G];
  auto point = [&]() {
    const int64_t e = __builtin_amdgcn_readfirstlane(sh.expert[a]);
    const int b = __builtin_amdgcn_readfirstlane(sh.start[a]);
    const int m = __builtin_amdgcn_readfirstlane(sh.start[a + 1]) - b;
    mp = (m + 3) & ~3;
#pragma unroll
    for (int r = 0; r < R; ++r) wp[r] = p.w2 + (e * p.D + row_of(r)) * p.F;
    ap = reinterpret_cast<const uint8_t*>(p.act + 4 * (int64_t)b * act_pair(p.F));
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if constexpr (G <= 2) {
        aoff[j] = 16 * lane + (4 * j < mp ? 1024 * j : 0);
      } else {
        // past the last token its value: a column that nobody reads
        const int item = 16 * (j / 4) + lr < m ? 16 * (j / 4) + lr : m - 1, q = j % 4;
        aoff[j] = 16 * ((8 * (q >> 1) + 2 * kg + (q & 1)) * mp + item);
      }
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) codes.load(w[r], wp[r], u, F);
    const uint8_t* at = ap + (int64_t)u * 512 * mp;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
      for (int j = 0; j < G; ++j) x[z][j] = *reinterpret_cast<const v8bf*>(at + 256 * z * mp + aoff[j]);
    }
  };
  auto operands = [&](const v8bf (&x)[G], Tokens (&t)[NT]) {
    if constexpr (G <= 2) {
#pragma unroll
      for (int j = 0; j < G; ++j) *reinterpret_cast<v8bf*>(turn + 1024 * j + 16 * lane) = x[j];
      wave_lds_fence();
      const int item = lr < mp ? lr : mp - 1;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        t[0].v[q] = *reinterpret_cast<const v8bf*>(turn + 16 * ((8 * (q >> 1) + 2 * kg + (q & 1)) * mp + item));
      wave_lds_fence();
    } else {
#pragma unroll
      for (int j = 0; j < G; ++j) t[j / 4].v[j % 4] = x[j];
    }
  };
  v4f acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  point();
  load();
  for (; i < end; ++i) {
#pragma unroll
    for (int r = 0; r < R; ++r) turn_codes<PACKED>(w[r], turn);
    Tokens t[2][NT];
    operands(x[0], t[0]);
    operands(x[1], t[1]);
    mask_unit<R, NT, 2>(w, t, u, F);
    multiply<R, NT, 2>(w, t, acc);
    const int of = a;
    if (i + 1 < end) {
      if (++u == units) {
        u = 0;
        ++a;
        point();
      }
    }
    load();  // behind the last unit it again, and nobody uses it
    if (a == of && i + 1 < end) continue;
    // the rows' scales through the scalar cache, past the loads in flight
    typedef const __attribute__((address_space(4))) float* ScalarPtr;
    const float* inv = p.inv2 + (int64_t)__builtin_amdgcn_readfirstlane(sh.expert[of]) * p.D;
    const int b = sh.start[of], mc = sh.start[of + 1] - b;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const ScalarPtr sp = (ScalarPtr)(uintptr_t)(inv + row_of(r));
      float c[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        float v[4] = {sp[z], sp[4 + z], sp[8 + z], sp[12 + z]};
        asm("" : "+s"(v[0]), "+s"(v[1]), "+s"(v[2]), "+s"(v[3]));  // loaded as scalars, then chosen by lane
        c[z] = kg < 2 ? (kg == 0 ? v[0] : v[1]) : (kg == 2 ? v[2] : v[3]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // an expert's tokens differ, so no two lanes meet
        if (16 * n + lr < mc) {
          float4* d = reinterpret_cast<float4*>(sum + sh.token[b + 16 * n + lr] * (16 * R) + 16 * r + 4 * kg);
          float4 v = *d;
          v.x += acc[r][n][0] * c[0];
          v.y += acc[r][n][1] * c[1];
          v.z += acc[r][n][2] * c[2];
          v.w += acc[r][n][3] * c[3];
          *d = v;
        }
        acc[r][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  }
}

// The workgroups share the (16 rows, expert, unit) triples evenly, so a
// workgroup has an end of a tile of rows, whole ones, and a beginning. The sums
// of a tile that several share meet in memory, and the one that comes last adds
// them, in the workgroups' order. Where a tile has few units it is not split.
template <int NTM, bool PACKED, int R>
__global__ __launch_bounds__(64 * kDownWaves, 2) void k_moe_down(MoeFewArgs p) {
  constexpr int kRows = 16 * R, kQuads = 16 * NTM * kRows / 4;  // a tile's rows; a wave's sums, by fours
  __shared__ float4 sums[kDownWaves * kQuads];  // [wave][token][row]
  __shared__ __align__(16) uint8_t turn[kDownWaves * 2048];
  __shared__ DownShared sh;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const FewMeta meta = few_meta(p.act, p.T, p.k, p.F);
  const int n = (int)p.T * p.k, slots = n < p.E ? n : p.E;
  // all that the workspace may hold of the lists; k_moe_up wrote the parts that are used
  for (int i = threadIdx.x; i < n; i += 64 * kDownWaves) {
    sh.token[i] = meta.token[i];
    if (i < slots) sh.expert[i] = meta.expert[i];
  }
  for (int i = threadIdx.x; i <= slots; i += 64 * kDownWaves) sh.start[i] = meta.start[i];
  if (threadIdx.x == 0) sh.count = meta.head[0];
  __syncthreads();
  const int nact = __builtin_amdgcn_readfirstlane(sh.count);
  int most = 0;  // the largest number of tokens of an expert
  for (int a = lane; a < nact; a += 64) most = max(most, sh.start[a + 1] - sh.start[a]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o, 64));
  most = __builtin_amdgcn_readfirstlane(most);
  const int units = (int)((p.F + 127) / 128);
  const int64_t tiles = (p.D + kRows - 1) / kRows, per = (int64_t)nact * units, all = tiles * per;
  if (nact == 0) {  // no token has an expert: zeros
    for (int64_t i = (int64_t)blockIdx.x * 64 * kDownWaves + threadIdx.x; i < p.T * p.D / 8;
         i += (int64_t)gridDim.x * 64 * kDownWaves)
      reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  int64_t share = (all + kDownBlocks - 1) / kDownBlocks;
  if (share < per) {
    // a joined tile costs some 2 us, so none with less than 32 units a wave is split
    // (128 units a tile: 22.9 us unsplit, 25.9 split; 1024 units: 155 us unsplit, 115
    // split), and no part has less than 4
    if (per <= kDownWaves * 32)
      share = per;
    else if (share < kDownWaves * 4)
      share = kDownWaves * 4;
  }
  int64_t i = share * blockIdx.x;
  const int64_t end = i + share < all ? i + share : all;
  while (i < end) {
    const int64_t tile = i / per, d0 = kRows * tile;
    const int from = (int)(i - tile * per);
    const int to = (int)(end - tile * per < per ? end - tile * per : per);
    float* sum = reinterpret_cast<float*>(&sums[wave * kQuads]);
    for (int z = lane; z < kQuads; z += 64) sums[wave * kQuads + z] = make_float4(0, 0, 0, 0);
    wave_lds_fence();
    const int i0 = from + (int)((int64_t)(to - from) * wave / kDownWaves);
    const int i1 = from + (int)((int64_t)(to - from) * (wave + 1) / kDownWaves);
    uint8_t* mine = turn + wave * 2048;
    if (i0 < i1) {
      auto run = [&](auto loads) { moe_down_run<loads.value, PACKED, R>(p, sh, d0, units, i0, i1, sum, mine); };
      by_tokens<NTM>(most, run);
    }
    __syncthreads();
    // each thread adds up the waves' sums of up to two fours of rows of a token
    constexpr int kMine = (kQuads + 64 * kDownWaves - 1) / (64 * kDownWaves);
    const int quads = (int)p.T * (kRows / 4);
    float r[kMine][4];
#pragma unroll
    for (int y = 0; y < kMine; ++y) {
      const int z = threadIdx.x + y * 64 * kDownWaves;
      r[y][0] = r[y][1] = r[y][2] = r[y][3] = 0.0f;
      if (z >= quads) continue;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) {
        const float4 a = sums[w * kQuads + z];
        r[y][0] += a.x;
        r[y][1] += a.y;
        r[y][2] += a.z;
        r[y][3] += a.w;
      }
    }
    bool write = true;
    if (to - from < per) {
      // the workgroups that share this tile, from b0 to b1; b0 has its counter
      const int64_t b0 = tile * per / share, b1 = ((tile + 1) * per - 1) / share;
      auto slot = [&](int64_t b) {
        const int64_t first = share * b / per;  // a workgroup's first tile
        return meta.part + (2 * b + (tile != first)) * p.T * kDownRows;
      };
      // Every value that crosses workgroups is stored and loaded by an atomic of
      // agent scope, which reaches the memory that all XCDs share, so no cache
      // has to be written back or emptied; the wait has the stores there before
      // the barrier, and the count goes up behind it.
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        const int z = threadIdx.x + y * 64 * kDownWaves;
        if (z >= quads) continue;
        float* d = slot(blockIdx.x) + 4 * z;
#pragma unroll
        for (int c = 0; c < 4; ++c) __hip_atomic_store(d + c, r[y][c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (threadIdx.x == 0)
        sh.count = (int)__hip_atomic_fetch_add(&meta.done[b0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      write = sh.count == (int)(b1 - b0);
      if (write) {
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
          const int z = threadIdx.x + y * 64 * kDownWaves;
          if (z >= quads) continue;
          r[y][0] = r[y][1] = r[y][2] = r[y][3] = 0.0f;
          for (int64_t b = b0; b <= b1; ++b) {
            const float* d = slot(b) + 4 * z;
#pragma unroll
            for (int c = 0; c < 4; ++c) r[y][c] += __hip_atomic_load(d + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
        }
      }
    }
    if (write) {
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        const int z = threadIdx.x + y * 64 * kDownWaves, t = z / (kRows / 4);
        const int64_t d = d0 + 4 * (z % (kRows / 4));
        if (z >= quads || d >= p.D) continue;
        const v2bf lo = {(__bf16)r[y][0], (__bf16)r[y][1]}, hi = {(__bf16)r[y][2], (__bf16)r[y][3]};
        *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.D + d) =
            make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
      }
    }
    i += to - from;
    if (i < end) __syncthreads();  // the sums are read before they are cleared
  }
}

template <bool PACKED>
static hipError_t launch_few_t(const MoeFewArgs& a) {
  const int64_t pairs = a.T * a.k, experts = pairs < a.E ? pairs : a.E, most = experts * (a.F / 16);
  const dim3 gu((unsigned)(most < kUpBlocks ? most : kUpBlocks)), gd(kDownBlocks);
  const dim3 bu(64 * kUpWaves), bd(64 * kDownWaves);
  auto go = [&](auto up, auto down) {
    hipLaunchKernelGGL(up, gu, bu, 0, a.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(down, gd, bd, 0, a.stream, a);
    return hipGetLastError();
  };
  // One tile of 16 rows a unit where two would leave half of the CUs without work
  // and a tile is too short to be split (k_moe_down, with one and with two: 5 tokens, 2 of
  // 8 experts, D 1040, F 720: 8.1 and 9.7 us; 32 tokens, 2 of 16 experts, D 4096, F 2048: 40.1
  // and 40.7 us).
  const bool narrow = a.D <= 16 * kDownBlocks && experts * ((a.F + 127) / 128) <= kDownWaves * 32;
  auto by_rows = [&](auto up, auto one, auto two) { return narrow ? go(up, one) : go(up, two); };
  if (a.T <= 16) return by_rows(k_moe_up<1, PACKED>, k_moe_down<1, PACKED, 1>, k_moe_down<1, PACKED, kDownTiles>);
  if (a.T <= 32) return by_rows(k_moe_up<2, PACKED>, k_moe_down<2, PACKED, 1>, k_moe_down<2, PACKED, kDownTiles>);
  return by_rows(k_moe_up<4, PACKED>, k_moe_down<4, PACKED, 1>, k_moe_down<4, PACKED, kDownTiles>);
}

hipError_t launch_moe_few(const MoeFewArgs& a) {
  if (a.T == 0 || a.D == 0 || a.F == 0) return hipSuccess;
  return a.packed ? launch_few_t<true>(a) : launch_few_t<false>(a);
}

}  // namespace fp8dyn
