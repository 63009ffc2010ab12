// adamw.hip -- one AdamW step over many tensors, with 32-bit or 8-bit states, and the
// gradients' norm with the factor that clips them.
//
// Per element, in fp32, each operation rounded by itself (this file is built without
// multiply-add contraction, so that the 8-bit states' codes and scales are those of the
// definition, bit for bit):
//   g = g mul;  m = m b1 + g (1 - b1);  v = v b2 + (g g) (1 - b2);  r = sqrt(v)
//   p = p (1 - lr wd) - (m / (r c2 + eps)) step
//   step = lr / (1 - b1^t), c2 = 1 / sqrt(1 - b2^t), formed in 64 bits.
// The quotient alone is a product with the reciprocal instruction (1 ulp).
//
// 8-bit states: m and r are kept as MXFP8, e4m3 codes with one power of two (E8M0) for
// each 32 elements, the smallest with which the largest is at most 448. r and not v: its
// codes span 2^18 in a group, which is 2^36 in v. A value of r above zero keeps a code
// above zero, since m / (0 c2 + eps) would be a step of any size.
// To nearest, a code of three mantissa bits stands still when a step changes its value by
// less than 1/32 to 1/16 of it: with b2 = 0.999 r would never decay, and stop to grow
// after some ten steps. Stochastic rounding (a seed other than 0) moves it by the right
// amount in the mean: 16 random bits below the code's last place, from Wellons' 32-bit
// integer hash "lowbias32" of (seed, tensor, step, element).
//
// The step is bound by HBM: 28 bytes an element with 32-bit states and an fp32 copy, 10.1 with
// 8-bit states and bf16 parameters; the tensors' table travels in the kernel's arguments, so that
// nothing is copied to the device first. Measured, 176 M elements in five tensors: 32-bit 790 to
// 808 us (6.1 to 6.2 TB/s; a large torch copy reaches 5.3), 8-bit 314 to 323 us (5.5 to 5.7 TB/s; to
// nearest 290). Loads and stores stream (non-temporal): plain loads 879 and 328 us, plain stores of the
// 8-bit form 326. The 8-bit step had been bound by its instructions: 377 us with codes scaled and
// rounded by integer steps and the library's square root, 343 with the scaled converts and a root
// of seven instructions (below), 315 with two pieces a workgroup, the second's loads ahead. Sending what
// that root does not cover to the library's costs 1% (319.5 against 323 us, in turn).
// Held to six waves a SIMD it spills: 392.
#include <cmath>
#include <type_traits>

#include "../../include/fp8dyn.h"
#include "common.hpp"
#include "internal.hpp"

namespace fp8dyn {

namespace {

typedef __bf16 aw_bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kTensorsALaunch = 48;  // their table travels in the kernel's arguments (4 KB)
constexpr int kNormTensorsALaunch = 128;
constexpr int kPiece32 = 256 * 4, kPiece8 = 256 * 8;  // elements a workgroup takes at once, by the states

// Elements of a workgroup of the norm: some 2048 workgroups, so that a small table has them on every CU and a
// large one has few partial sums.
int64_t norm_chunk(int64_t total) {
  const int64_t c = (total / 2048 + 2047) / 2048 * 2048;
  return c < 2048 ? 2048 : c > 32768 ? 32768 : c;
}

// Pieces of a workgroup: two with 8-bit states (one 330 us, four 322), one with 32-bit ones (two 847 us,
// four 880, eight 900: workgroups that run together then reach over more of memory).
int step_iters(bool eight, int64_t pieces) { return eight && pieces >= 8192 ? 2 : 1; }

struct StepTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  float* master;
  int64_t n;
  uint32_t key;
  uint32_t vec;  // every pointer allows the wide loads
};
struct StepArgs {
  StepTensor t[kTensorsALaunch];
  int32_t first[kTensorsALaunch + 1];  // chunks before each tensor
  int32_t count, iters;
  float b1, c1, b2, c2m;  // c1 = 1 - b1, c2m = 1 - b2
  float eps, decay, step, c2;
  uint32_t now;  // the step's number for the random bits
  const float* mul;
  // where given: the step's number and rate on the device, from which the factors are formed there
  const int32_t* step_dev;
  const float* lr_dev;
  double lr, wd, log_b1, log_b2;
};
static_assert(sizeof(StepArgs) <= 4096, "kernel arguments");

struct NormArgs {
  const void* g[kNormTensorsALaunch];
  int64_t n[kNormTensorsALaunch];
  int32_t first[kNormTensorsALaunch + 1];
  uint32_t f32[(kNormTensorsALaunch + 31) / 32];
  int32_t count, chunk;
  double* part;
};
static_assert(sizeof(NormArgs) <= 4000, "kernel arguments, with NormOut");

__host__ __device__ __forceinline__ uint32_t lowbias32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  x ^= x >> 16;
  return x;
}

// the tensor of a chunk: the last one whose first chunk is not behind it
template <class A>
__device__ __forceinline__ int tensor_of(const A& a, int32_t chunk) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// V consecutive values of an fp32 or bf16 array, as they are in memory
template <bool F32, int V>
struct Raw {
  uint32_t w[F32 ? V : V / 2];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (F32) return __uint_as_float(w[j]);
    return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
  // `left` of them exist; the others are zeros
  __device__ __forceinline__ void load(const void* base, int64_t i, bool wide, int left) {
    constexpr int W = F32 ? V : V / 2;
    if (wide) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(base) + i * (F32 ? 4 : 2));
      if constexpr (W == 2) {
        const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
        w[0] = x[0], w[1] = x[1];
      } else {
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          const uint4 x = ld_nt16(p + j);
          w[j] = x.x, w[j + 1] = x.y, w[j + 2] = x.z, w[j + 3] = x.w;
        }
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < left) {
        if constexpr (F32)
          w[j] = reinterpret_cast<const uint32_t*>(base)[i + j];
        else
          w[j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(base)[i + j] << (16 * (j & 1));
      }
  }
};

// eight codes
struct RawCodes {
  uint2 w;
  __device__ __forceinline__ void load(const void* base, int64_t i, bool wide, int left) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + i;
    if (wide) {
      const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
      w = make_uint2(x[0], x[1]);
      return;
    }
    w = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) (j < 4 ? w.x : w.y) |= (uint32_t)p[j] << (8 * (j & 3));
  }
};

__device__ __forceinline__ void store_codes(void* base, int64_t i, bool wide, int left, uint2 c) {
  uint8_t* p = reinterpret_cast<uint8_t*>(base) + i;
  if (wide) {
    st_nt8(p, c);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) p[j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const aw_bf16x2 h = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, h);
}

template <bool F32, int V>
__device__ __forceinline__ void store_v(void* base, int64_t i, bool wide, int left, const float* x) {
  if (wide) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        st_nt16(reinterpret_cast<float*>(base) + i + j,
                make_uint4(__float_as_uint(x[j]), __float_as_uint(x[j + 1]), __float_as_uint(x[j + 2]),
                           __float_as_uint(x[j + 3])));
    } else if constexpr (V == 8) {
      st_nt16(reinterpret_cast<uint16_t*>(base) + i, make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]),
                                                                bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])));
    } else {
      st_nt8(reinterpret_cast<uint16_t*>(base) + i, make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j < left) {
      if constexpr (F32)
        reinterpret_cast<float*>(base)[i + j] = x[j];
      else
        reinterpret_cast<uint16_t*>(base)[i + j] = (uint16_t)bf16_pair(x[j], 0.0f);
    }
}

// eight e4m3 codes times their group's power of two
__device__ __forceinline__ void decode8(uint2 c, uint32_t e8, float* x) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(e8 << 23);
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, s, false);
  const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, s, true);
  const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, s, false);
  const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, s, true);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
  x[4] = d[0], x[5] = d[1], x[6] = e[0], x[7] = e[1];
}

// sqrt(v), correctly rounded for 0 and v in [2^-100, infinity) (compared with the library's root for every mantissa,
// at both parities of the exponent); what lies outside is far(). Seven instructions for the 15 of the root that covers
// everything.
__device__ __forceinline__ float root(float v) {
  const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f)), g = v * y;
  return __builtin_fmaf(__builtin_fmaf(-g, g, v), 0.5f * y, g);
}

// Some v is infinite or in (0, 2^-100), where root()'s remainder would lose bits: as integers, v - 1 of zero is above
// all others.
template <int V>
__device__ __forceinline__ bool far(const float* v) {
  uint32_t lo = ~0u;
  float hi = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t b = __float_as_uint(v[j]) - 1u;
    lo = b < lo ? b : lo;
    hi = fmaxf(hi, v[j]);
  }
  return lo < __builtin_bit_cast(uint32_t, 0x1p-100f) - 1u || hi > 3.402823466e38f;
}

// the largest of a group's 32 magnitudes as bits (those of a NaN are above all others): a lane
// holds 8, four neighbouring lanes the group
__device__ __forceinline__ uint32_t group_top(const float* x) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
    t = b > t ? b : t;
  }
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0xB1, 0xf, 0xf, true);  // lanes 1 0 3 2
  t = o > t ? o : t;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x4E, 0xf, 0xf, true);  // lanes 2 3 0 1
  return o > t ? o : t;
}

// four codes of x / s, s a power of two. SR: rnd[j]'s upper 20 bits are added below the last place (below the
// smallest normal code too, where codes are 2^-9 apart) before the rest is cut off.
template <bool SR>
__device__ __forceinline__ uint32_t codes4(const float* x, const uint32_t* rnd, float s) {
  if constexpr (SR) {
    int w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(0, x[0], rnd[0], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[1], rnd[1], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[2], rnd[2], s, 2);
    return (uint32_t)__builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[3], rnd[3], s, 3);
  } else {
    typedef short v2s __attribute__((ext_vector_type(2)));
    v2s w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], s, true);
    return __builtin_bit_cast(uint32_t, w);
  }
}

// MXFP8 of eight values of a group: codes and the group's E8M0 byte. LIFT: values are not negative, and one
// above zero keeps a code above zero.
template <bool SR, bool LIFT>
__device__ __forceinline__ uint2 encode8(float* x, const uint32_t* rnd, uint32_t& e8) {
  const uint32_t top = group_top(x);
  int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < 12 ? 12 : e;
  const float s = __uint_as_float((uint32_t)e << 23);
  if constexpr (LIFT) {
    // the middle one of x, the smallest code's value and x made large: x, that value, or 0
    const float least = s * 0x1p-9f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_fmed3f(x[j], least, x[j] * 0x1p126f);
  }
  uint2 c = make_uint2(codes4<SR>(x, rnd, s), codes4<SR>(x + 4, rnd + 4, s));
  e8 = (uint32_t)e;
  if (top >= 0x7f800000u) {  // not finite: the whole group stands for NaN
    e8 = 255u;
    c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  return c;
}

// A workgroup takes a.iters pieces of 256 V elements of one tensor, each piece's loads under way while the
// one before it is computed.
template <bool P32, bool G32, bool MASTER, bool EIGHT, bool SR>
__global__ __launch_bounds__(256) void k_adamw(const StepArgs a) {
  constexpr int V = EIGHT ? 8 : 4;
  float mul = 1.0f;
  if (a.mul) {
    mul = *a.mul;
    if (!(fabsf(mul) <= 3.402823466e38f)) return;  // gradients that are not finite: no step
  }
  float step = a.step, c2 = a.c2, decay = a.decay;
  uint32_t now = a.now;
  if (a.step_dev || a.lr_dev) {
    const double t = (double)(a.step_dev ? *a.step_dev : (int32_t)now);
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    now = (uint32_t)(int32_t)t;
    step = (float)(lr / -expm1(t * a.log_b1));
    c2 = (float)(1.0 / sqrt(-expm1(t * a.log_b2)));
    decay = (float)(1.0 - lr * a.wd);
  }
  const int32_t chunks = a.first[a.count];
  for (int32_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int k = tensor_of(a, chunk);
    const StepTensor& T = a.t[k];
    const int64_t n = T.n, begin = (int64_t)(chunk - a.first[k]) * a.iters * (256 * V);
    const uint32_t key = SR ? lowbias32(T.key + now) : 0u;
    struct Piece {
      Raw<G32, V> g;
      Raw<MASTER || P32, V> p;
      std::conditional_t<EIGHT, RawCodes, Raw<true, V>> m, v;
      uint32_t em, ev;
    } next;
    auto load = [&](int it) {
      const int64_t i = begin + (int64_t)(it * 256 + (int)threadIdx.x) * V;
      const int left = n - i < V ? (int)(n - i) : V;
      const bool wide = T.vec && left == V;
      next.g.load(T.g, i, wide, left);
      next.p.load(MASTER ? T.master : T.p, i, wide, left);
      next.m.load(T.m, i, wide, left);
      next.v.load(T.v, i, wide, left);
      next.em = next.ev = 0;
      if constexpr (EIGHT)
        if (left > 0) next.em = T.ms[i >> 5], next.ev = T.vs[i >> 5];
    };
    load(0);
    for (int it = 0; it < a.iters; ++it) {
      const int64_t i = begin + (int64_t)(it * 256 + (int)threadIdx.x) * V;
      if (begin + (int64_t)it * (256 * V) >= n) break;
      const int left = n - i < V ? (int)(n - i) : V;
      const bool wide = T.vec && left == V;
      Piece cur = next;
      if (it + 1 < a.iters) load(it + 1);
      float p[V], m[V], v[V], r[V];
      if constexpr (EIGHT) {
        decode8(cur.m.w, cur.em, m);
        decode8(cur.v.w, cur.ev, v);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (EIGHT) {
          v[j] = v[j] * v[j];
        } else {
          m[j] = cur.m[j];
          v[j] = cur.v[j];
        }
        const float x = a.mul ? cur.g[j] * mul : cur.g[j];
        m[j] = m[j] * a.b1 + x * a.c1;
        v[j] = v[j] * a.b2 + (x * x) * a.c2m;
        r[j] = EIGHT ? root(v[j]) : sqrtf(v[j]);
      }
      if constexpr (EIGHT)
        if (far<V>(v)) {
#pragma unroll
          for (int j = 0; j < V; ++j) r[j] = sqrtf(v[j]);
        }
#pragma unroll
      for (int j = 0; j < V; ++j)
        p[j] = cur.p[j] * decay - (m[j] * __builtin_amdgcn_rcpf(r[j] * c2 + a.eps)) * step;
      uint32_t lo[V], hi[V];
      if constexpr (SR) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          // 16 bits each and a half below them, at the top of a word
          const uint32_t b = lowbias32((uint32_t)i + (uint32_t)j + key);
          lo[j] = b << 16 | 0x8000u, hi[j] = (b & 0xffff0000u) | 0x8000u;
        }
      }
      if constexpr (EIGHT) {
        // lanes past the end hold zeros, and take no part in a group's largest
        if (left < V) {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j >= left) m[j] = r[j] = 0.0f;
        }
        uint32_t em, ev;
        const uint2 cm = encode8<SR, false>(m, lo, em), cv = encode8<SR, true>(r, hi, ev);
        store_codes(T.m, i, wide, left, cm);
        store_codes(T.v, i, wide, left, cv);
        if ((threadIdx.x & 3) == 0 && left > 0) T.ms[i >> 5] = (uint8_t)em, T.vs[i >> 5] = (uint8_t)ev;
      } else {
        store_v<true, V>(T.m, i, wide, left, m);
        store_v<true, V>(T.v, i, wide, left, v);
      }
      if constexpr (MASTER) store_v<true, V>(T.master, i, wide, left, p);
      if constexpr (SR && !P32 && !MASTER) {
#pragma unroll
        for (int j = 0; j < V; ++j) {  // bf16 with 16 random bits below its last place
          const uint32_t b = __float_as_uint(p[j]);
          if ((b & 0x7fffffffu) <= 0x7f800000u) p[j] = __uint_as_float((b + ((lo[j] ^ hi[j]) >> 16)) & 0xffff0000u);
        }
      }
      store_v<P32, V>(T.p, i, wide, left, p);
    }
  }
}

// The part of a piece's sum of squares that thread `tid` of NT takes, in 64 bits, in order.
template <int NT>
__device__ __forceinline__ double square_sum(const NormArgs& a, int32_t chunk, int tid) {
  const int t = tensor_of(a, chunk);
  const int64_t n = a.n[t], begin = (int64_t)(chunk - a.first[t]) * a.chunk;
  const int64_t end = begin + a.chunk < n ? begin + a.chunk : n;
  const bool f32 = (a.f32[t >> 5] >> (t & 31)) & 1u;
  const bool vec = ((uintptr_t)a.g[t] & 15) == 0;
  double s = 0.0;
  const int64_t whole = vec ? begin + ((end - begin) & ~(int64_t)7) : begin;
  if (f32) {
    const float* g = reinterpret_cast<const float*>(a.g[t]);
    for (int64_t i = begin + 4 * tid; i < whole; i += 4 * NT) {
      const uint4 w = ld_nt16(g + i);
      const double x0 = __uint_as_float(w.x), x1 = __uint_as_float(w.y);
      const double x2 = __uint_as_float(w.z), x3 = __uint_as_float(w.w);
      s += x0 * x0 + x1 * x1 + x2 * x2 + x3 * x3;
    }
    for (int64_t i = whole + tid; i < end; i += NT) s += (double)g[i] * (double)g[i];
  } else {
    const uint16_t* g = reinterpret_cast<const uint16_t*>(a.g[t]);
    for (int64_t i = begin + 8 * tid; i < whole; i += 8 * NT) {
      const uint4 w = ld_nt16(g + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double x = bf16_lo(u[j]), y = bf16_hi(u[j]);
        s += x * x + y * y;
      }
    }
    for (int64_t i = whole + tid; i < end; i += NT) {
      const double x = __uint_as_float((uint32_t)g[i] << 16);
      s += x * x;
    }
  }
  return s;
}

__device__ __forceinline__ double wave_sum64(double s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// One partial sum of squares a workgroup: a thread's elements in order, then a tree. HBM-bound: 176 M bf16
// values (352 MB) in 54 us, and 4 us for k_grad_norm, 6.0 TB/s together.
__global__ __launch_bounds__(256) void k_grad_sq(const NormArgs a) {
  __shared__ double red[4];
  const int32_t chunks = a.first[a.count];
  for (int32_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const double s = wave_sum64(square_sum<256>(a, chunk, threadIdx.x));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.part[chunk] = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
  }
}

struct NormOut {
  double grad_scale, max_norm;
  float* norm;
  float* mul;
  int32_t* step;
};

// The sum over 1024 threads, and what follows from it.
__device__ __forceinline__ void finish_norm(double s, const NormOut& o) {
  __shared__ double red[16];
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = red[0];
  for (int w = 1; w < 16; ++w) s += red[w];
  const double x = sqrt(s) * o.grad_scale;
  const float xf = (float)x;
  if (o.norm) *o.norm = xf;
  const double clip = o.max_norm / (x + 1e-6);
  const float mul = (float)(clip < 1.0 ? o.grad_scale * clip : o.grad_scale);
  // the steps that k_adamw takes and no other are counted: not those of a NaN, nor of a factor past fp32
  const bool fine = fabsf(xf) <= 3.402823466e38f && fabsf(mul) <= 3.402823466e38f;
  if (o.mul) *o.mul = fine ? mul : __uint_as_float(0x7fc00000u);
  if (o.step && fine) *o.step += 1;
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* __restrict__ part, int64_t n, const NormOut o) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
  finish_norm(s, o);
}

// Both in one launch, for tables of few pieces: a wavefront takes every sixteenth.
__global__ __launch_bounds__(1024) void k_grad_norm_small(const NormArgs a, const NormOut o) {
  const int32_t chunks = a.first[a.count];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double s = 0.0;
  for (int32_t chunk = wave; chunk < chunks; chunk += 16) s += square_sum<64>(a, chunk, threadIdx.x & 63);
  finish_norm(s, o);
}

template <bool P32, bool G32, bool MASTER>
hipError_t launch_step(const StepArgs& s, bool eight, bool sr, unsigned grid, hipStream_t stream) {
  if (eight) {
    if (sr) hipLaunchKernelGGL((k_adamw<P32, G32, MASTER, true, true>), dim3(grid), dim3(256), 0, stream, s);
    else hipLaunchKernelGGL((k_adamw<P32, G32, MASTER, true, false>), dim3(grid), dim3(256), 0, stream, s);
  } else if constexpr (!P32 && !MASTER) {
    if (sr) hipLaunchKernelGGL((k_adamw<P32, G32, MASTER, false, true>), dim3(grid), dim3(256), 0, stream, s);
    else hipLaunchKernelGGL((k_adamw<P32, G32, MASTER, false, false>), dim3(grid), dim3(256), 0, stream, s);
  } else {
    hipLaunchKernelGGL((k_adamw<P32, G32, MASTER, false, false>), dim3(grid), dim3(256), 0, stream, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a) {
  int64_t total = 0;
  for (int32_t i = 0; i < a.count; ++i) total += a.tensors[i].n;
  const int64_t piece = a.eight ? kPiece8 : kPiece32;
  StepArgs s;
  s.iters = step_iters(a.eight, total / piece);
  const int64_t ch = piece * s.iters;
  s.b1 = (float)a.beta1, s.c1 = (float)(1.0 - a.beta1);
  s.b2 = (float)a.beta2, s.c2m = (float)(1.0 - a.beta2);
  s.eps = (float)a.eps;
  s.decay = (float)(1.0 - a.lr * a.wd);
  s.step = (float)(a.lr / (1.0 - std::pow(a.beta1, (double)a.step)));
  s.c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(a.beta2, (double)a.step)));
  s.now = (uint32_t)a.step;
  s.mul = a.mul, s.step_dev = a.step_dev, s.lr_dev = a.lr_dev;
  s.lr = a.lr, s.wd = a.wd, s.log_b1 = std::log(a.beta1), s.log_b2 = std::log(a.beta2);
  const uint32_t lo = (uint32_t)a.seed, hi = (uint32_t)(a.seed >> 32);
  int64_t chunks = 0;
  s.count = 0;
  auto flush = [&]() -> hipError_t {
    if (s.count == 0) return hipSuccess;
    s.first[s.count] = (int32_t)chunks;
    const unsigned grid = (unsigned)(chunks < kMaxGrid256 ? chunks : kMaxGrid256);
    const bool sr = a.seed != 0;
    hipError_t e;
    if (a.p_f32)
      e = a.g_f32 ? launch_step<true, true, false>(s, a.eight, sr, grid, a.stream)
                  : launch_step<true, false, false>(s, a.eight, sr, grid, a.stream);
    else if (a.master)
      e = a.g_f32 ? launch_step<false, true, true>(s, a.eight, sr, grid, a.stream)
                  : launch_step<false, false, true>(s, a.eight, sr, grid, a.stream);
    else
      e = a.g_f32 ? launch_step<false, true, false>(s, a.eight, sr, grid, a.stream)
                  : launch_step<false, false, false>(s, a.eight, sr, grid, a.stream);
    s.count = 0;
    chunks = 0;
    return e;
  };
  for (int32_t i = 0; i < a.count; ++i) {
    const fp8_adamw_tensor& t = a.tensors[i];
    if (t.n == 0) continue;
    const int64_t c = (t.n + ch - 1) / ch;
    if (s.count == kTensorsALaunch || chunks + c > INT32_MAX) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    const uintptr_t all = (uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.m | (uintptr_t)t.v | (uintptr_t)t.master;
    s.first[s.count] = (int32_t)chunks;
    s.t[s.count++] = {t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n,
                      lowbias32(hi ^ lowbias32(lo ^ lowbias32((uint32_t)i))),
                      (all & 15) == 0 ? 1u : 0u};
    chunks += c;
  }
  return flush();
}

// Pieces of a table of tensors, and the elements of one; with at most kSmallNorm pieces (and one launch's tensors)
// one workgroup takes all: it saves a launch, some 3 us of the host's and as much of the device's time.
constexpr int64_t kSmallNorm = 64;
struct NormPlan {
  int64_t chunk, chunks, tensors;
  bool small() const { return chunks <= kSmallNorm && tensors <= kNormTensorsALaunch; }
};
static NormPlan norm_plan(const fp8_grad_tensor* tensors, int32_t count) {
  int64_t total = 0;
  NormPlan p{0, 0, 0};
  for (int32_t i = 0; i < count; ++i) total += tensors[i].n;
  p.chunk = norm_chunk(total);
  for (int32_t i = 0; i < count; ++i) {
    p.chunks += (tensors[i].n + p.chunk - 1) / p.chunk;
    p.tensors += tensors[i].n > 0;
  }
  return p;
}

int64_t grad_norm_partials(const fp8_grad_tensor* tensors, int32_t count) {
  const NormPlan p = norm_plan(tensors, count);
  return p.small() ? 0 : p.chunks;
}

hipError_t launch_grad_norm(const GradNormArgs& a) {
  const NormPlan plan = norm_plan(a.tensors, a.count);
  const NormOut out{a.grad_scale, a.max_norm, a.norm, a.mul, a.step};
  NormArgs s;
  int64_t chunks = 0, before = 0;
  s.chunk = (int32_t)plan.chunk;
  s.count = 0;
  s.first[0] = 0;
  auto flush = [&]() -> hipError_t {
    if (s.count == 0) return hipSuccess;
    s.part = a.ws + before;
    const unsigned grid = (unsigned)(chunks < kMaxGrid256 ? chunks : kMaxGrid256);
    hipLaunchKernelGGL(k_grad_sq, dim3(grid), dim3(256), 0, a.stream, s);
    before += chunks;
    s.count = 0;
    chunks = 0;
    return hipGetLastError();
  };
  for (int32_t i = 0; i < a.count; ++i) {
    const fp8_grad_tensor& t = a.tensors[i];
    if (t.n == 0) continue;
    const int64_t c = (t.n + plan.chunk - 1) / plan.chunk;
    if (s.count == kNormTensorsALaunch || chunks + c > INT32_MAX) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    if (s.count % 32 == 0) s.f32[s.count / 32] = 0;
    s.f32[s.count / 32] |= (t.type == FP8_OUT_F32 ? 1u : 0u) << (s.count % 32);
    s.g[s.count] = t.g;
    s.n[s.count] = t.n;
    s.first[s.count++] = (int32_t)chunks;
    chunks += c;
    s.first[s.count] = (int32_t)chunks;
  }
  if (plan.small()) {
    hipLaunchKernelGGL(k_grad_norm_small, dim3(1), dim3(1024), 0, a.stream, s, out);
    return hipGetLastError();
  }
  const hipError_t e = flush();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, a.stream, a.ws, before, out);
  return hipGetLastError();
}

}  // namespace fp8dyn
