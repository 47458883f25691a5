// kernels.h -- launch interfaces between the host API (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "svdq.h"

namespace svdq {

// Raises `kernel`'s dynamic shared-memory limit on the current device to at
// least `bytes`, calling the runtime only the first time a larger limit is
// needed (the call costs microseconds of host time, more than a small
// kernel's launch).
cudaError_t ensure_dynamic_smem(const void* kernel, size_t bytes);

// Launches a kernel that may be scheduled under the previous kernel's tail
// (it waits with grid_dependency_wait before its first global access).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// SVDQ_OK when the current device is supported (compute capability 10.0)
// and holds the handle `w`; the status any entry point would return otherwise.
svdq_status handle_device_status(const svdq_weights* w);

// The current device's SM count and error word, with the status any entry
// point returns when the device is not supported.
struct DeviceInfo {
  int num_sms;
  DeviceErr err;
};
svdq_status current_device_info(DeviceInfo* info);

// 2-D tensor map over row-major [rows][inner], 128-byte swizzled boxes; false
// when the driver refuses it.
bool encode_tensor_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* ptr, uint64_t inner, uint64_t rows,
                          uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows,
                          CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// A CUDA status as an entry point returns it (clears a non-sticky error).
svdq_status cuda_status(cudaError_t e);

// ---------------------------------------------------------------- kernel 1
struct K1Params {
  int M, K, K_pad, r_tot, r_pad;
  int fmt;                 // 0 NVFP4, 1 INT4
  int do_quant, do_lr;     // fused: both; unfused baseline: one of them
  int stages;              // set by the launcher
  int ksplit;              // CTAs per row block (the cluster with the low-rank branch), set by the launcher
  const float* inv_lambda; // [K_pad], permuted per 64-wide stage (see prepare.cu)
  const __nv_bfloat16* L1t; // L1f^T in the staged layout (one contiguous tile per stage)
  float s_t, six_st;       // NVFP4 activation tensor scale and fl32(6 s_t)
  // per-call NVFP4 tensor scale (null: s_t above): the amax partials of X^,
  // reduced after the grid-dependency wait; s_t = fl32(2^j / s_tR) and LR
  // leaves scaled by 2^(k_alpha - j), where 2^k_alpha is the prepared alpha
  const uint32_t* amax_parts;
  int n_parts, k_alpha;
  float s_tR;
  float* dyn_record;       // if set, CTA 0 writes {s_t, j as int32 bits, 2^j}
  uint8_t* qX;             // [M][K_pad/2]
  uint8_t* sX;             // scale layout (see svdq.h)
  __nv_bfloat16* LR;       // [M][r_pad]
  DeviceErr err;
};
// Kernel 1 stages X in [K1_BOX_ROWS x 64] bf16 TMA boxes (128-byte swizzle);
// the host encodes tmX with exactly this box.
constexpr int K1_BOX_ROWS = 64;
cudaError_t launch_quant_down(const CUtensorMap& tmX, K1Params p, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- kernel 2
struct K2Params {
  int M, N, K_pad, r_tot, r_pad, N_pad;
  int num_m_blocks, num_n_blocks;
  int nk;                  // K_pad / 256 4-bit k-tiles
  int nl;                  // r_pad / 64 low-rank k-tiles (0: plain W4A4 GEMM)
  const uint8_t* sX;       // activation scales, replicated layout (sfx_rep_offset)
  const uint8_t* sR;       // weight scales, replicated layout (sfw_rep_offset)
  const float* bias;       // [N_pad]
  float alpha;             // s_tX * s_tR
  const uint32_t* amax_parts;  // per-call tensor scale: alpha = 2^j from these (null: alpha above)
  int n_parts;
  float s_tR;
  int epi;                 // 0 none, 1 GELU (tanh form)
  __nv_bfloat16* Y;        // [M][N]
  DeviceErr err;
  // Emit mode (the next layer's kernel-1 outputs instead of Y): this
  // layer's bf16 output Y is the next layer's activation X2 (its K = N)
  struct Next {
    const float* inv_lambda;   // [N] the next layer's 1/lambda
    const __nv_bfloat16* L1t;  // its first factor (with any LoRA A) in kernel 1's staged layout: per 64 rows
                               // of K one [r_tot x 64] bf16 box, 128-byte swizzled (a K-major MMA B operand)
    float s_t, six_st;         // its static NVFP4 activation tensor scale and fl32(6 s_t)
    int r_tot;                 // <= 64
    uint8_t* qX;               // [M][N_pad / 2]
    uint8_t* sX;               // replicated layout over N_pad (sfx_rep_offset)
    float* part;               // [num_n_blocks][M_128][LR_PART_STRIDE] partial LR, one per column block
  } next;
};
constexpr int LR_PART_STRIDE = 64;   // floats per row of an emit-mode LR partial
// TMA box heights the host encodes for kernel 2's operands (rows of a tile):
// NVFP4 stages 128 rows of qX / LR and 256 rows of qR / L2a per k-tile; INT4
// stages 128 of each.
constexpr int K2_NV_ROWS_A = 128, K2_NV_ROWS_B = 256;
constexpr int K2_I4_ROWS = 128;
cudaError_t launch_gemm_nvfp4(const CUtensorMap& tmA, const CUtensorMap& tmB,
                              const CUtensorMap& tmLR, const CUtensorMap& tmL2, K2Params p,
                              int num_sms, cudaStream_t stream, bool emit_next = false);
// LR of the next layer from the emit mode's partials: bf16 of their sum in
// partial order, zeros for r_tot <= i < r_pad.
cudaError_t launch_next_lr_reduce(const float* part, int parts, int M, int M_128, int r_tot, int r_pad,
                                  __nv_bfloat16* LR, cudaStream_t stream);

struct K2I8Params {
  int M, N, K_pad, r_tot, r_pad, N_pad;
  int num_m_blocks, num_n_blocks;
  int nk;                  // K_pad / 128 k-tiles (two 64-groups each)
  int nl;                  // r_pad / 64 low-rank chunks (0: plain W4A4 GEMM)
  const float* sX;         // binary16 values widened to float32, chunked (int4_scale_offset)
  const float* sR;
  const float* bias;
  int epi;
  __nv_bfloat16* Y;
  DeviceErr err;
};
cudaError_t launch_gemm_int4(const CUtensorMap& tmX8, const CUtensorMap& tmR8, const CUtensorMap& tmLR,
                             const CUtensorMap& tmL2, K2I8Params p, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- per-call activation amax
// One uint32 slot per CTA (the bits of that CTA's amax(|X^|)); at most
// AMAX_MAX_PARTS slots.
constexpr int AMAX_MAX_PARTS = 1024;
static_assert(AMAX_MAX_PARTS <= 1024, "warp_amax_bits reads at most 32 slots a lane");
int act_amax_num_parts(int K, int num_sms);   // slots the pass writes (0: K too large)
cudaError_t launch_act_amax(const __nv_bfloat16* X, int M, int K, const float* inv_lambda, uint32_t* parts,
                            int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- unfused up projection
struct UpParams {
  int M, N, r_tot, r_pad;
  const __nv_bfloat16* LR;   // [M][r_pad]
  const __nv_bfloat16* L2a;  // [N_pad][r_pad]
  float alpha;
  int epi;
  __nv_bfloat16* Y;          // [M][N], read-modify-write
};
cudaError_t launch_lowrank_up(UpParams p, cudaStream_t stream);

// ---------------------------------------------------------------- preparation / calibration
cudaError_t launch_calibrate(int M, int K, int N, const __nv_bfloat16* X, const __nv_bfloat16* Wt,
                             float alpha, float* lambda_out, float* act_scale_out, unsigned* ws,
                             cudaStream_t stream);

struct PrepParams {
  int fmt, K, N, K_pad, N_pad, rank, lora_rank, r_tot, r_pad;
  const __nv_bfloat16* Wt;     // [N][K]
  const float* lambda;         // [K]
  const __nv_bfloat16* L1f;    // [K][rank]
  const __nv_bfloat16* L2;     // [rank][N]
  const __nv_bfloat16* bias;   // [N] or null
  const __nv_bfloat16* loraA;  // [K][lora_rank] or null
  const __nv_bfloat16* loraB;  // [lora_rank][N] or null
  float* R;                    // scratch [N][K]
  unsigned* amax_bits;         // scratch, 1 word
  uint8_t* qR;                 // [N_pad][K_pad/2]
  uint8_t* sR;                 // scales
  uint8_t* sR_rep;             // NVFP4: kernel 2's replicated copy (sfw_rep_offset)
  uint8_t* qR8;                // INT4: kernel 2's copy of the codes as E4M3 bytes [N_pad][K_pad]
  __nv_bfloat16* L1t;          // [K_pad/64][r_tot][64], 128-byte swizzled
  __nv_bfloat16* L2a;          // [N_pad][r_pad]
  float* bias_f;               // [N_pad]
  float* lambda_inv;           // [K]
  float* lambda_inv_k1;        // [K_pad], permuted per 64-wide stage for kernel 1
};
cudaError_t launch_prepare_residual(const PrepParams& p, cudaStream_t stream);
cudaError_t launch_prepare_quantize(const PrepParams& p, float s_tR, float alpha,
                                    cudaStream_t stream);

cudaError_t launch_selftest_timeout(DeviceErr err, cudaStream_t stream);

// Randomized truncated SVD of W^ = diag(lambda) W (see rsvd.cu); synchronous.
// L1f bf16 [K][r], L2 bf16 [r][N] on the device; sigma_out (host, may be
// null) receives the min(r + 8, K, N) estimated singular values.
cudaError_t lowrank_factors(int K, int N, int r, const __nv_bfloat16* Wt, const float* lam, uint64_t seed,
                            __nv_bfloat16* L1f, __nv_bfloat16* L2, double* sigma_out, cudaStream_t s);

// ---------------------------------------------------------------- AWQ W4A16 layer
// Codes: uint8 [K/32][N_pad][16] (chunk c holds k in [32c, 32c+32) of feature
// n, 4 bits each; 32-bit word w of a chunk holds k = 32c + 8w + i at bit
// 4 awq_nibble_pos(i): the even k in the low half-word, the odd in the high,
// so one shift and mask give the bf16 pair (k, k + 1) and the float32
// pairs (k, k + 2)); scale binary16 and zero uint8 [K/64][N_pad]; N_pad = N
// rounded up to 32.
__host__ __device__ constexpr int awq_nibble_pos(int i) { return (i >> 1) + 4 * (i & 1); }
constexpr int AWQ_WARPS = 8;      // warps of a CTA, splitting K
constexpr int AWQ_MB_MAX = 4;     // activation rows per pass over the weights
constexpr int AWQ_STAGES = 4;     // TMA ring depth (stages of 8 groups x 32 features)
static_assert(AWQ_MB_MAX <= AWQ_WARPS, "one warp per row writes the outputs");
struct AwqPrepParams {
  int K, N, N_pad;
  const __nv_bfloat16* Wt;        // [N][K]
  const float* s;                 // [K] AWQ input-channel scales, or null (all 1)
  const __nv_bfloat16* bias;      // [N] or null
  uint8_t* code;
  __half* scale;
  uint8_t* zero;
  float* inv_s;                   // [K] fl32(1/s)
  float* bias_f;                  // [N_pad]
};
struct AwqParams {
  int M, K, N, N_pad, mb;         // mb: activation rows staged per pass
  const __nv_bfloat16* X;         // [M][K]
  const uint8_t* code;
  const __half* scale;
  const uint8_t* zero;
  const float* inv_s;             // [K] fl32(1/s)
  const float* bias;              // [N_pad]
  __nv_bfloat16* Y;               // [M][N]
  DeviceErr err;
};
// The tensor-core form (awq_gemm.cu): 128 x 256 tiles over 64-wide k-tiles.
struct AwqGemmParams {
  int M, K, N, N_pad;
  int num_m_blocks, num_n_blocks;  // ceil(M / 128), ceil(N / 256)
  const float* inv_s;              // [K] fl32(1/s) (read only when the handle has an AWQ scale)
  const float* bias;               // [N_pad]
  __nv_bfloat16* Y;                // [M][N], N % 16 == 0, 32-byte aligned
  DeviceErr err;
};
// tmX: X bf16 [M][K], box {64, 128}, 128-byte swizzle; tmCode: the codes as a
// 3-D uint8 tensor [K/32][N_pad][16], box {16, 256, 2}; tmScale / tmZero:
// [K/64][N_pad] binary16 / uint8, box {256, 1}.
cudaError_t launch_awq_gemm(const CUtensorMap& tmX, const CUtensorMap& tmCode, const CUtensorMap& tmScale,
                            const CUtensorMap& tmZero, AwqGemmParams p, bool has_s, int num_sms,
                            cudaStream_t stream);
cudaError_t launch_awq_quantize(const AwqPrepParams& p, cudaStream_t stream);
// tmCode: codes as a 3-D uint8 tensor [K/32][N_pad][16], box {16, 32, 16};
// tmScale / tmZero: [K/64][N_pad] binary16 / uint8, box {32, 8}.
cudaError_t launch_awq_gemv(const CUtensorMap& tmCode, const CUtensorMap& tmScale, const CUtensorMap& tmZero,
                           AwqParams p, int num_sms, cudaStream_t stream);
int awq_rows_per_block(int K, int M);
size_t awq_smem_bytes(int K, int mb);

// ---------------------------------------------------------------- 16-bit matrix products (gemm16.cu)
// What is multiplied.  NT: both operands with the reduction index innermost
// (X W^T).  GATED: NT with two weights and the gated epilogue.  GRAD: the
// backward products, dZ^T X (both operands with the reduction index outermost)
// and dZ W (B with it outermost), as the jobs of one launch.
enum Gemm16Op { GEMM16_NT, GEMM16_GATED, GEMM16_GRAD };
struct Gemm16Plan {
  Gemm16Op op;
  bool swap;     // the weight is the MMA's 128-row operand, the tokens its N
  int bn;        // MMA N: 128 or 256 (pair form), 16, 32, 64 or 128 (swapped)
  int splits;    // CTAs (pairs) a tile's reduction is split over: a power of two
  bool tall;     // pair form: 512 x 256 tiles (NT and GRAD, not split)
};
struct Gemm16Job {
  int M, N;                    // rows and columns of the output (of each of two stacked ones)
  int tiles_m, tiles_n;        // tiles along the MMA's M and N; 0: no such job
  int tiles_m1;                // row blocks of the first of two stacked A operands (tiles_m: one)
  int nk1, nk;                 // 64-wide k-tiles of the first operand pair, of both
  int group;                   // set by the launcher: row blocks of a group of tiles
  int a_mn;                    // GRAD: A has the reduction index outermost
  uint16_t *Y, *Y2;            // output rows of stride ldy; the second stacked output
  long long ldy;
};
struct Gemm16Params {
  Gemm16Job job[2];            // the second: GRAD only
  int splits, job1_extra;      // set by the launcher
  int fp16;                    // 0 bf16, 1 fp16
  // forward epilogue
  int act;                     // svdq_epilogue
  const uint16_t *bias, *bias2;
  const uint16_t* R;           // residual rows of stride ldr, or null
  long long ldr;
  uint16_t *Z, *Z2;            // pre-activations [M][N], or null
  // GRAD: bias gradients from `parts` column-sum partials [parts][part_n] (0: none)
  int parts, part_n;
  const float *part, *part2;
  uint16_t *dbias, *dbias2;
  DeviceErr err;
};
// A job's tensor maps; a map that nothing uses is a copy of another.
enum Gemm16Map { MAP_A, MAP_A2, MAP_B, MAP_B2, MAP_Y, MAP_Z, MAP_Z2, MAPS, MAP_Y2 = MAP_Z2 };
template <int JOBS>
struct Gemm16Maps {
  CUtensorMap m[JOBS][MAPS];
};
// Tiles of the second job that make up for one of the first.
constexpr int gemm16_extra(int nk0, int nk1) { return nk1 > 0 ? (nk0 + nk1 / 2) / nk1 : 0; }
// Columns of the pair form's store boxes (32 rows high; 128-byte swizzle, 64-byte for 32 columns).
constexpr int gemm16_box_cols(const Gemm16Plan& p) { return p.op == GEMM16_GATED && p.bn == 128 ? 32 : 64; }
cudaError_t launch_gemm16(const Gemm16Plan& plan, const Gemm16Maps<2>& maps, Gemm16Params p, int num_sms,
                          cudaStream_t stream);

// ---------------------------------------------------------------- column sums and activation slopes (act_grad.cu)
// Kinds of the pass over [M][N] gradients: column sums alone; dZ = dY act'(Z);
// dG = dH U act'(G), dU = dH act(G); the last two with optional column sums.
enum ActGradKind { ACT_GRAD_SUM, ACT_GRAD_DENSE, ACT_GRAD_GATED };
struct ActGradParams {
  ActGradKind kind;
  int M, N, fp16, act;
  const uint16_t* dY;          // rows of stride ld
  long long ld;
  const uint16_t *Z, *U;       // [M][N]
  uint16_t *dZ, *dU;           // [M][N]
  float *part, *part2;         // [parts][N] column-sum partials, or null
  int parts;                   // act_grad_parts(M, N)
};
int act_grad_parts(int M, int N);
cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t stream);
// out[n] = round(sum over parts, in order, of part[.][n]), dt svdq_dtype
cudaError_t launch_sum_parts(const float* part, int parts, int N, int dt, void* out, const float* part2, void* out2,
                             cudaStream_t stream);

// ---------------------------------------------------------------- layer norm (layernorm.cu)
struct LayerNormParams {
  int M, C, dt;                // svdq_dtype
  const void *X, *gamma, *beta;
  long long ldx, ldy;
  float eps;
  void* Y;
  float *mean, *rstd;          // [M], or null
};
cudaError_t launch_layernorm(const LayerNormParams& p, cudaStream_t stream);
struct LayerNormGradParams {
  int M, C, dt;
  const void *dY, *X, *gamma;
  long long lddy, ldx, lddx;
  const float *mean, *rstd;
  void* dX;
  float *part_g, *part_b;      // [parts][C] partials of dgamma / dbeta, or null
};
int layernorm_grad_parts(int M, int C);   // partials at most
// *parts: the partials it writes
cudaError_t launch_layernorm_grad(const LayerNormGradParams& p, int* parts, cudaStream_t stream);

}  // namespace svdq
