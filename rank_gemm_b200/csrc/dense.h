// dense.h -- launch interfaces and device helpers of the 16-bit layers (the
// dense linear, the gated feed-forward, the layer norm): between dense.cu and
// its kernels (gemm16.cu, act_grad.cu, layernorm.cu).
#pragma once

#include "kernels.h"

namespace svdq {

// ---------------------------------------------------------------- from the host API (api.cu)
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

// ---------------------------------------------------------------- launching
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
  // GRAD: the reduction in `parts` ranges of k-tiles, a tile each.  More than
  // one: float32 partials P [parts][rows of Y, of Y2][N] instead of Y and Y2,
  // the rows of each rounded up to 32.
  int parts;
  float* P;
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
// A tile's epilogue takes as long as about seven k-tiles (40 x 7840 -> 5232
// backward, whose dW tiles have one: counted as one 147 us, as seven 46).
constexpr int gemm16_weight(int nk) { return nk > 7 ? nk : 7; }
// Tiles of the second job that make up for one of the first.
constexpr int gemm16_extra(int nk0, int nk1) {
  return nk1 > 0 ? (gemm16_weight(nk0) + gemm16_weight(nk1) / 2) / gemm16_weight(nk1) : 0;
}
// Columns of the pair form's store boxes (32 rows high; 128-byte swizzle, 64-byte for 32 columns).
constexpr int gemm16_box_cols(const Gemm16Plan& p) { return p.op == GEMM16_GATED && p.bn == 128 ? 32 : 64; }
// Y (and Y2) = the sum of a job's partials, in order, rounded once; of one or two jobs.
cudaError_t launch_join_parts(const Gemm16Job* jobs, int count, int fp16, cudaStream_t stream);
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

// ---------------------------------------------------------------- device helpers
// Loads of gamma, beta and biases.  Volatile, so that a load guarded by a null
// check is never issued ahead of the check; without a memory clobber, so that
// it may still move ahead of earlier stores.  Not the read-only (.nc) form:
// these kernels start under the previous one's tail, which may be writing
// what they read after grid_dependency_wait.
__device__ __forceinline__ uint4 ld_param(const uint4* p) {
  uint4 u;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}
__device__ __forceinline__ uint32_t ld_param32(const void* p) {
  uint32_t u;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(u) : "l"(p));
  return u;
}
__device__ __forceinline__ uint16_t ld_param(const uint16_t* p) {
  uint16_t u;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(u) : "l"(p));
  return u;
}

// SiLU, y / (1 + e^-y), with the same two approximations (relative error near
// 1e-6 for a 16-bit output).
__device__ __forceinline__ float sigmoid_approx(float y) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-1.4426950408889634f * y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return r;
}
__device__ __forceinline__ float silu(float y) { return y * sigmoid_approx(y); }

// (act(z), act'(z)) of an svdq_epilogue.  Both activations are z s(w) with s
// the logistic function (silu: w = z; tanh-form GELU: w = 2u, u = sqrt(2/pi)
// (z + 0.044715 z^3)), so act' = s + z s (1 - s) w'.  Where s (1 - s) is 0 the
// second term is left out: w' may have overflowed there.
__device__ __forceinline__ void act_and_slope(float z, int act, float& f, float& slope) {
  if (act == 0) {
    f = z;
    slope = 1.f;
    return;
  }
  const bool gelu = act == 1;
  constexpr float k2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
  const float zz = z * z;
  const float w = gelu ? k2 * z * fmaf(0.044715f, zz, 1.0f) : z;
  const float dw = gelu ? k2 * fmaf(0.134145f, zz, 1.0f) : 1.0f;
  const float s = sigmoid_approx(w), q = s * (1.0f - s);
  f = z * s;
  slope = q > 0.f ? fmaf(z * q, dw, s) : s;
}

}  // namespace svdq
