// internal.hpp -- launcher interfaces between the C-ABI layer (api.hip) and
// the kernels. Host-side only declarations; no validation happens below this
// line, so every launcher assumes arguments the API has already checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

struct fp8_adamw_tensor;  // include/fp8dyn.h
struct fp8_grad_tensor;

namespace fp8dyn {

struct QuantArgs {
  const uint16_t* x;
  int64_t batch, rows, cols;
  bool e5;      // e5m2 (else e4m3)
  double fmax;  // largest finite value of the output format
  double eps;
  uint8_t* q;
  float* scale;
  float* inv;
  hipStream_t stream;
  bool fnuz = false;  // write the fnuz variant by software encoding (rowwise, tensorwise)
};

hipError_t launch_quant_row(const QuantArgs& a);
// codes k-packed in chunks of group_rows (16 or 2) rows x 64 columns; rows % group_rows == 0,
// cols % 64 == 0, cols <= 16384
hipError_t launch_quant_row_kpacked(const QuantArgs& a, int group_rows);
hipError_t launch_quant_col(const QuantArgs& a, void* ws);
// qT k-packed as the [cols][rows] B operand; rows % 64 == 0, cols % 16 == 0, the vector path's conditions
hipError_t launch_quant_col_kpacked(const QuantArgs& a, void* ws);
size_t quant_col_ws_bytes(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_quant_tensor(const QuantArgs& a, void* ws);  // ws >= 256 bytes
// tensorwise scale, transposed output qT[b][c][r]; needs cols % 8 == 0, rows % 16 == 0
hipError_t launch_quant_tensor_transposed(const QuantArgs& a, void* ws);
hipError_t launch_quant_block(const QuantArgs& a, int block_rows, int block_cols);
// Row normalization fused with the rowwise quantization of its bf16 output.
struct NormQuantArgs {
  const uint16_t* x;      // [rows][cols], cols % 8 == 0, cols <= 16384, 16-byte aligned
  const uint16_t* gamma;  // [cols]
  const uint16_t* beta;   // [cols] or nullptr (LayerNorm)
  int64_t rows, cols;
  bool layer;             // LayerNorm (else RMSNorm)
  double norm_eps;
  bool e5;
  double fmax, eps;
  uint16_t* y;            // [rows][cols] bf16 or nullptr
  uint8_t* q;             // [rows][cols] or nullptr (then y only)
  float* scale;
  float* inv;
  hipStream_t stream;
  // launch_add_norm_quant_row only: the row normalized is h = bf16(x + res)
  const uint16_t* res = nullptr;  // or nullptr: h = x
  uint16_t* h = nullptr;          // written when set and res is; may be x or res
  float* mean = nullptr;          // mean32, rstd32 of each row, written when set
  float* rstd = nullptr;
};
hipError_t launch_norm_quant_row(const NormQuantArgs& a);
hipError_t launch_add_norm_quant_row(const NormQuantArgs& a);

// Workgroups of 256 threads a launch has at most: a grid has fewer than 2^32 threads.
constexpr int64_t kMaxGrid256 = (int64_t)1 << 23;

// Backward of the row normalization, with the residual stream's gradient.
struct NormBwdArgs {
  const uint16_t* dy;     // [rows][cols]
  const uint16_t* dh;     // [rows][cols] or nullptr
  const uint16_t* h;      // [rows][cols], the normalized rows
  const uint16_t* gamma;  // [cols]
  const float* mean;      // [rows] (LayerNorm)
  const float* rstd;      // [rows]
  int64_t rows, cols;     // cols % 8 == 0, cols <= 16384
  bool layer;
  uint16_t* dx;           // [rows][cols]; may be dy or dh
  uint16_t* dgamma;       // [cols] or nullptr
  uint16_t* dbeta;        // [cols] or nullptr
  float* ws;              // norm_bwd_ws_floats()
  hipStream_t stream;
};
hipError_t launch_norm_bwd(const NormBwdArgs& a);
int64_t norm_bwd_ws_floats(int64_t rows, int64_t cols, bool layer);

// Limits of the router and of the layer for a few tokens: experts (a token's logits live in
// registers), choices, and the layer's tokens.
constexpr int32_t kMaxMoeE = 1024;
constexpr int32_t kMaxMoeK = 32;
constexpr int kFewT = 64;

// Expert router: the k largest logits of each token, gate weights, and the
// rows sorted by expert.
enum GateKind : int { kGateSoftmax = 0, kGateSoftmaxTopk = 1, kGateSigmoid = 2 };
struct RouteArgs {
  const void* logits;  // [T][E], bf16 or fp32
  bool f32;
  int64_t T;           // T * k < 2^31
  int32_t E, k;        // E <= kMaxMoeE, 1 <= k <= min(E, kMaxMoeK)
  int gate;
  int32_t* ids;        // [T][k]
  float* weights;      // [T][k]
  int32_t* offsets;    // [E + 1], or nullptr (then order and slot too)
  int32_t* order;      // [T * k]
  int32_t* slot;       // [T][k]
  uint32_t* ws;        // route_ws_words()
  hipStream_t stream;
};
hipError_t launch_moe_route(const RouteArgs& a);
int64_t route_ws_words(int64_t T, int32_t E);
struct RouteBwdArgs {
  const void* logits;
  bool f32;
  int64_t T;
  int32_t E, k;
  int gate;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  void* dlogits;       // [T][E], the logits' type; may be logits itself
  hipStream_t stream;
};
hipError_t launch_moe_route_bwd(const RouteBwdArgs& a);

// Mixture-of-experts layer for a few tokens.
struct MoeFewArgs {
  const uint16_t* x;      // [T][D] bf16
  const int32_t* ids;     // [T][k]; outside [0, E): no expert
  const float* weights;   // [T][k]
  const uint8_t* w13;     // [E][2F][D] e4m3, gate rows first
  const float* inv13;     // [E][2F]
  const uint8_t* w2;      // [E][D][F] e4m3
  const float* inv2;      // [E][D]
  int64_t T;              // <= kFewT
  int32_t E, k;           // E <= kMaxMoeE, k <= kMaxMoeK
  int64_t D, F;           // % 16 == 0 (packed: % 64 == 0), < 2^20: 32-bit byte offsets in x and act
  bool packed;
  uint16_t* out;          // [T][D]
  uint16_t* act;          // workspace, moe_few_ws_bytes(): the activations and the experts' tokens
  hipStream_t stream;
};
hipError_t launch_moe_few(const MoeFewArgs& a);  // F > 0
size_t moe_few_ws_bytes(int64_t T, int k, int64_t F);

// One AdamW step over many tensors (adamw.hip).
struct AdamwArgs {
  const fp8_adamw_tensor* tensors;  // host
  int32_t count;
  bool p_f32, g_f32, eight, master;
  double lr, beta1, beta2, eps, wd;
  int64_t step;
  uint64_t seed;
  const float* mul;         // device, or nullptr
  const int32_t* step_dev;  // device, or nullptr: instead of step
  const float* lr_dev;      // device, or nullptr: instead of lr
  hipStream_t stream;
};
hipError_t launch_adamw(const AdamwArgs& a);

// The gradients' norm and the factor that clips them (adamw.hip).
struct GradNormArgs {
  const fp8_grad_tensor* tensors;  // host
  int32_t count;
  double grad_scale, max_norm;
  float* norm;
  float* mul;
  int32_t* step;
  double* ws;  // grad_norm_partials()
  hipStream_t stream;
};
hipError_t launch_grad_norm(const GradNormArgs& a);
int64_t grad_norm_partials(const fp8_grad_tensor* tensors, int32_t count);

// Gradient through a gated product with its rowwise quantization (gated_bwd.hip).
struct GatedBwdArgs {
  const uint16_t* dh;  // [M][F]
  const uint16_t* gu;  // [M][2F]: gate, then up
  int64_t M, F;        // F % 8 == 0, F <= kMaxGatedF
  bool gelu;
  bool e5;
  double fmax, eps;
  uint16_t* dgu;       // [M][2F] or nullptr; may be gu
  uint8_t* q;          // [M][2F] or nullptr (then no scales)
  float* scale;
  float* inv;          // or nullptr
  uint16_t* h;         // [M][F] or nullptr; may be dh
  hipStream_t stream;
};
constexpr int64_t kMaxGatedF = 32768;  // a row's gradient lives in registers
hipError_t launch_gated_bwd(const GatedBwdArgs& a);

// Tensorwise quantization of up to kMaxTJobs tensors in three launches (clear
// the amax words, amax of every tensor, one cast launch): each tensor gets its
// transposed output qT [cols][rows] and, when q is set, its row-major output
// q [rows][cols] from the same read. rows % 16 == 0, cols % 8 == 0,
// rows * cols < 2^30, 16-byte aligned x and qT, 8-byte aligned q.
// amax_words: kMaxTJobs device words.
constexpr int kMaxTJobs = 3;
struct TJobSpec {
  const uint16_t* x;
  int64_t rows, cols;
  bool e5;
  double fmax;
  uint8_t* q;   // or nullptr
  uint8_t* qT;
  float* scale;
  float* inv;   // or nullptr
};
hipError_t launch_quant_tensor_multi_t(const TJobSpec* specs, int n, double eps, uint32_t* amax_words,
                                       hipStream_t stream);
// Tensorwise quantization of two tensors (row-major codes only) in two
// launches: a per-workgroup amax pass into `partials`, then a cast pass that
// reduces them; no word needs clearing first. n % 8 == 0 for both tensors.
struct TPairSpec {
  const uint16_t* x;
  int64_t n;
  uint8_t* q;
  float* scale;
  float* inv;  // or nullptr
};
constexpr int kPairMaxAmaxBlocks = 2048;  // per tensor
hipError_t launch_quant_tensor_pair(const TPairSpec* specs, bool e5, double fmax, double eps, float* partials,
                                    hipStream_t stream);
hipError_t launch_quant_mx(const QuantArgs& a, uint8_t* e8m0, int mode);
hipError_t launch_quant_mx_packed(const QuantArgs& a, uint8_t* e8m0, int mode, int group_rows);

// Probe kernels: results[0..3] = fp8 codes of 1.0 (e4m3, e5m2) and of the
// formats' maxima; results[4..5] = matrix-core dot products of 128 copies of
// the codes 0x38 (e4m3) and 0x3C (e5m2) with themselves.
hipError_t run_probe(float* host_results);

// GEMMs ------------------------------------------------------------------------
enum ScaleKind : int { kScaleTensor = 0, kScaleRow = 1, kScaleBlock = 2, kScaleMX = 3 };

struct GemmArgs {
  const uint8_t* a;   // [Mtot][K]
  const uint8_t* b;   // [E][N][K]
  const void* sa;     // per ScaleKind
  const void* sb;
  const int32_t* offsets;  // device [E+1], or nullptr for a dense problem (E == 1)
  int32_t E;
  int64_t M, N, K;    // M = Mtot
  bool a_e5, b_e5;
  int scale_kind;
  bool out_f32;
  void* out;          // [M][N]
  hipStream_t stream;
  bool b_kpacked = false;  // B in 1 KB chunks of 16 rows x 64 K (fast kernel, ROW/TENSOR/MX scales)
  bool exact = false;      // full-precision accumulation (codes decoded to bf16, BF16 matrix cores)
};
hipError_t launch_gemm_fp8(const GemmArgs& g);
// the direct-to-LDS kernel (K % 128 == 0, aligned operands); launch_gemm_fp8 picks it
bool gemm_fp8_fast_eligible(const GemmArgs& g);
// dense tensorwise / rowwise outputs small enough for the 64 x 64 tile form
// of the generic kernel (at most one tile per CU)
bool gemm_fp8_small_dense(int64_t M, int64_t N);
hipError_t launch_gemm_fp8_fast(const GemmArgs& g);

// Gated product (gemm_gated.hip): b holds [E][2F][K], gate rows before up rows; out [M][F] bf16.
struct GatedMmArgs {
  const uint8_t* a;        // [M][K] e4m3; packed and grouped: pair-interleaved
  const uint8_t* b;        // packed: k-packed
  const float* sa;         // [M], or one
  const float* sb;         // [E][2F], or one
  const int32_t* offsets;  // device [E + 1], or nullptr for a dense problem (E == 1)
  int32_t E;
  int64_t M, F, K;
  bool row_scales;         // else one scale each
  bool packed;
  bool gelu;
  bool exact;              // full-precision accumulation
  uint16_t* gu;            // [M][2F], or nullptr
  uint16_t* out;
  hipStream_t stream;
};
hipError_t launch_gated_mm(const GatedMmArgs& g);
// a shape that the packed form takes (the caller has checked its alignment)
bool gated_mm_packed_ok(const GatedMmArgs& g);

struct WgradArgs {
  const uint16_t* gy;  // [M][N]
  const uint16_t* x;   // [M][K]
  int64_t M, N, K;
  uint16_t* gw;        // [N][K]
  hipStream_t stream;
};
hipError_t launch_wgrad_bf16(const WgradArgs& w);

struct GroupedWgradArgs {
  const uint16_t* gy;       // [Mtot][N]
  const uint16_t* x;        // [Mtot][K]
  const int32_t* offsets;   // device [E+1]
  int32_t E;
  int64_t Mtot, N, K;       // N % 8 == 0, K % 8 == 0, 32 * max(N, K) * 2 < 2^31
  uint16_t* gw;             // [E][N][K]
  hipStream_t stream;
};
hipError_t launch_grouped_wgrad_bf16(const GroupedWgradArgs& w);

// Degenerate sizes (fill.hip): the eps-clamped scale of an empty group into
// scale[0..n) (and inv), and zeros over bytes (2-byte aligned, even count).
hipError_t launch_empty_group_scales(float* scale, float* inv, int64_t n, double fmax, double eps,
                                     hipStream_t stream);
hipError_t launch_zero_fill(void* p, int64_t bytes, hipStream_t stream);

}  // namespace fp8dyn
