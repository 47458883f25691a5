// dense.cu -- host side of the 16-bit layers declared in include/svdq.h: the
// dense linear, the gated feed-forward and the layer norm, forward and
// backward.  Checks arguments, picks the tiling, encodes the tensor maps and
// launches; nothing is kept between calls.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "svdq.h"
#include "common.cuh"
#include "kernels.h"

using namespace svdq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }

bool type16(svdq_dtype dt) { return dt == SVDQ_BF16 || dt == SVDQ_FP16; }
bool known_act(svdq_epilogue a) { return a == SVDQ_EPI_NONE || a == SVDQ_EPI_GELU_TANH || a == SVDQ_EPI_SILU; }
bool width_ok(int n) { return n > 0 && n % 8 == 0; }
// a row stride in 16-bit elements: covers the row, 16-byte steps, under the TMA limit of 2^40 bytes
bool stride_ok(long long ld, int width) { return ld >= width && ld % 8 == 0 && ld < (1ll << 39); }

const uint16_t* in16(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* out16(void* p) { return static_cast<uint16_t*>(p); }

// ------------------------------------------------------------------ tiling
// A tile's k-tile costs its MMA cycles, or the time its operand bytes take
// into shared memory where that is longer; a tile also costs a fixed part.
Gemm16Plan plan_pair(Gemm16Op op, int rows, int cols, int nk, int num_sms) {
  Gemm16Plan best{op, false, 256, 1};
  double best_t = 0;
  const int pairs = num_sms / 2;
  for (int bn = 256; bn >= 128; bn -= 128) {
    const int out_cols = op == GEMM16_GATED ? bn / 2 : bn;
    const long long tiles = (long long)rows * ceil_div(cols, out_cols);
    for (int s = 1; s <= 4; s *= 2) {
      if (s > 1 && (nk < 4 * s || tiles * s > pairs)) break;
      const double per_k = bn == 256 ? 512 : 320;
      const double waves = (double)((tiles * s + pairs - 1) / pairs);
      const double t = waves * ceil_div(nk, s) * per_k + (s > 1 ? 2500 : 1500);
      if (best_t == 0 || t < best_t) {
        best_t = t;
        best = Gemm16Plan{op, false, bn, s};
      }
    }
  }
  return best;
}

Gemm16Plan plan_swap(Gemm16Op op, int tokens, int features, int nk, int num_sms) {
  int bn = 16;
  while (bn < 128 && bn < tokens) bn *= 2;
  const int tiles = ceil_div(features, 128) * ceil_div(tokens, bn);
  int s = 1;
  while (s < 8 && tiles * s * 2 <= num_sms && nk >= 4 * s) s *= 2;
  return Gemm16Plan{op, true, bn, s};
}
// Up to this many rows of X the swapped form is taken.
constexpr int SWAP_ROWS = 128;

// ------------------------------------------------------------------ operands
struct Operand {
  const void* ptr;
  uint64_t inner, rows, ld;   // innermost extent, rows, row stride in elements
};

// Encodes A (128-row tiles) and B (b_rows of them per CTA) and launches.
svdq_status run_gemm(const DeviceInfo& d, const Gemm16Plan& plan, svdq_dtype dt, const Operand& a0, const Operand* a1,
                     const Operand& b0, const Operand* b1, Gemm16Params p, cudaStream_t stream) {
  const CUtensorMapDataType t =
      dt == SVDQ_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const bool a_mn = plan.op == GEMM16_TN || (plan.swap && plan.op == GEMM16_NN);
  const bool b_mn = plan.op == GEMM16_TN || (!plan.swap && plan.op == GEMM16_NN);
  const uint32_t a_box = a_mn ? 64 : 128, b_box = b_mn ? 64 : plan.swap ? plan.bn : plan.bn / 2;
  CUtensorMap tm[7];
  auto map = [&](CUtensorMap* m, const Operand& o, uint32_t box) {
    return encode_tensor_map_2d(m, t, o.ptr, o.inner, o.rows, o.ld * 2, 64, box);
  };
  if (!map(&tm[0], a0, a_box) || !map(&tm[2], b0, b_box)) return SVDQ_ERR_CUDA;
  if (!a1)
    tm[1] = tm[0];
  else if (!map(&tm[1], *a1, a_box))
    return SVDQ_ERR_CUDA;
  if (!b1)
    tm[3] = tm[2];
  else if (!map(&tm[3], *b1, b_box))
    return SVDQ_ERR_CUDA;
  if (!plan.swap) {   // the outputs' store boxes; maps that nothing uses are copies
    const uint32_t w = gemm16_box_cols(plan);
    auto out = [&](CUtensorMap* m, void* ptr, uint64_t ld) {
      return encode_tensor_map_2d(m, t, ptr, p.N, p.M, ld * 2, w, 32,
                                  w == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    };
    void* z2 = p.Z2 ? p.Z2 : p.Y2;
    if (!out(&tm[4], p.Y, p.ldy)) return SVDQ_ERR_CUDA;
    tm[5] = tm[6] = tm[4];
    if (p.Z && !out(&tm[5], p.Z, p.N)) return SVDQ_ERR_CUDA;
    if (z2 && !out(&tm[6], z2, p.Z2 ? (uint64_t)p.N : (uint64_t)p.ldy)) return SVDQ_ERR_CUDA;
  } else {
    tm[4] = tm[5] = tm[6] = tm[0];
  }
  p.fp16 = dt == SVDQ_FP16;
  p.err = d.err;
  return cuda_status(launch_gemm16(plan, tm, p, d.num_sms, stream));
}

Gemm16Params no_epilogue() {
  Gemm16Params p = {};
  p.act = SVDQ_EPI_NONE;
  return p;
}

// out [M][N] = A B^T of row-major X [M][K] and W [N][K] (two weights: gated)
svdq_status forward_product(const DeviceInfo& d, svdq_dtype dt, int M, int K, int N, const void* X, long long ldx,
                            const void* W, const void* W2, Gemm16Params p, cudaStream_t stream) {
  const Gemm16Op op = W2 ? GEMM16_GATED : GEMM16_NT;
  const int nk = ceil_div(K, 64);
  const Operand x{X, (uint64_t)K, (uint64_t)M, (uint64_t)ldx}, w{W, (uint64_t)K, (uint64_t)N, (uint64_t)K},
      w2{W2, (uint64_t)K, (uint64_t)N, (uint64_t)K};
  p.M = M;
  p.N = N;
  p.nk1 = p.nk = nk;
  if (M <= SWAP_ROWS) {
    const Gemm16Plan plan = plan_swap(op, M, N, nk, d.num_sms);
    p.tiles_m = p.tiles_m1 = ceil_div(N, 128);
    p.tiles_n = ceil_div(M, plan.bn);
    return run_gemm(d, plan, dt, w, W2 ? &w2 : nullptr, x, nullptr, p, stream);
  }
  p.tiles_m = p.tiles_m1 = ceil_div(M, 256);
  const Gemm16Plan plan = plan_pair(op, p.tiles_m, N, nk, d.num_sms);
  p.tiles_n = ceil_div(N, W2 ? plan.bn / 2 : plan.bn);
  return run_gemm(d, plan, dt, x, nullptr, w, W2 ? &w2 : nullptr, p, stream);
}

// dX [M][K] = dZ W (+ dZ2 W2), dZ [M][N] rows of stride ldz, W [N][K]
svdq_status input_gradient(const DeviceInfo& d, svdq_dtype dt, int M, int K, int N, const void* dZ, long long ldz,
                           const void* dZ2, const void* W, const void* W2, void* dX, long long lddx,
                           cudaStream_t stream) {
  const Operand z{dZ, (uint64_t)N, (uint64_t)M, (uint64_t)ldz}, z2{dZ2, (uint64_t)N, (uint64_t)M, (uint64_t)ldz},
      w{W, (uint64_t)K, (uint64_t)N, (uint64_t)K}, w2{W2, (uint64_t)K, (uint64_t)N, (uint64_t)K};
  Gemm16Params p = no_epilogue();
  p.M = M;
  p.N = K;
  p.nk1 = ceil_div(N, 64);
  p.nk = dZ2 ? 2 * p.nk1 : p.nk1;
  p.Y = out16(dX);
  p.ldy = lddx;
  if (M <= SWAP_ROWS) {
    const Gemm16Plan plan = plan_swap(GEMM16_NN, M, K, p.nk, d.num_sms);
    p.tiles_m = p.tiles_m1 = ceil_div(K, 128);
    p.tiles_n = ceil_div(M, plan.bn);
    return run_gemm(d, plan, dt, w, dZ2 ? &w2 : nullptr, z, dZ2 ? &z2 : nullptr, p, stream);
  }
  p.tiles_m = p.tiles_m1 = ceil_div(M, 256);
  const Gemm16Plan plan = plan_pair(GEMM16_NN, p.tiles_m, K, p.nk, d.num_sms);
  p.tiles_n = ceil_div(K, plan.bn);
  return run_gemm(d, plan, dt, z, dZ2 ? &z2 : nullptr, w, dZ2 ? &w2 : nullptr, p, stream);
}

// dW [N][K] = dZ^T X (and dW2 = dZ2^T X, stacked below it as one launch)
svdq_status weight_gradient(const DeviceInfo& d, svdq_dtype dt, int M, int K, int N, const void* dZ, long long ldz,
                            const void* dZ2, const void* X, long long ldx, void* dW, void* dW2, cudaStream_t stream) {
  const Operand z{dZ, (uint64_t)N, (uint64_t)M, (uint64_t)ldz}, z2{dZ2, (uint64_t)N, (uint64_t)M, (uint64_t)ldz},
      x{X, (uint64_t)K, (uint64_t)M, (uint64_t)ldx};
  Gemm16Params p = no_epilogue();
  p.M = N;
  p.N = K;
  p.nk1 = p.nk = ceil_div(M, 64);
  p.tiles_m1 = ceil_div(N, 256);
  p.tiles_m = dZ2 ? 2 * p.tiles_m1 : p.tiles_m1;
  p.Y = out16(dW);
  p.Y2 = out16(dW2);
  p.ldy = K;
  const Gemm16Plan plan = plan_pair(GEMM16_TN, p.tiles_m, K, p.nk, d.num_sms);
  p.tiles_n = ceil_div(K, plan.bn);
  return run_gemm(d, plan, dt, z, dZ2 ? &z2 : nullptr, x, nullptr, p, stream);
}

cudaError_t zero(void* p, size_t bytes, cudaStream_t stream) {
  return p ? cudaMemsetAsync(p, 0, bytes, stream) : cudaSuccess;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ dense linear
svdq_status svdq_dense_linear(svdq_dtype dt, int M, int K, int N, const void* X, long long ldx, const void* W_t,
                              const void* bias, svdq_epilogue act, const void* residual, long long ldr, void* Y,
                              long long ldy, void* Z, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !W_t || (M > 0 && (!X || !Y))) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || !width_ok(K) || !width_ok(N) || !stride_ok(ldx, K) || !stride_ok(ldy, N) ||
      (residual && !stride_ok(ldr, N)))
    return SVDQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(W_t) || !aligned16(bias) || !aligned16(residual) || !aligned16(Y) || !aligned16(Z))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  DeviceInfo d;
  const svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  Gemm16Params p = no_epilogue();
  p.act = act;
  p.bias = in16(bias);
  p.R = in16(residual);
  p.ldr = ldr;
  p.Y = out16(Y);
  p.ldy = ldy;
  p.Z = out16(Z);
  return forward_product(d, dt, M, K, N, X, ldx, W_t, nullptr, p, stream);
}

// [dZ when there is an activation | the bias gradient's partials]
size_t svdq_dense_linear_backward_workspace_bytes(int M, int K, int N, svdq_epilogue act) {
  if (M < 0 || !width_ok(K) || !width_ok(N) || !known_act(act)) return 0;
  return (act == SVDQ_EPI_NONE ? 0 : align256((size_t)M * N * 2)) +
         align256((size_t)act_grad_parts(M, N) * N * 4);
}

svdq_status svdq_dense_linear_backward(svdq_dtype dt, int M, int K, int N, const void* dY, long long lddy,
                                       const void* X, long long ldx, const void* W_t, const void* Z,
                                       svdq_epilogue act, void* dX, long long lddx, void* dW, void* dbias,
                                       void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act)) return SVDQ_ERR_INVALID_ARG;
  if (M > 0 && (!dY || (act != SVDQ_EPI_NONE && !Z) || (dX && !W_t) || (dW && !X))) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || !width_ok(K) || !width_ok(N) || !stride_ok(lddy, N) || (dW && !stride_ok(ldx, K)) ||
      (dX && !stride_ok(lddx, K)))
    return SVDQ_ERR_SHAPE;
  if (!aligned16(dY) || !aligned16(X) || !aligned16(W_t) || !aligned16(Z) || !aligned16(dX) || !aligned16(dW) ||
      !aligned16(dbias) || !aligned16(workspace))
    return SVDQ_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < svdq_dense_linear_backward_workspace_bytes(M, K, N, act)) return SVDQ_ERR_WORKSPACE;
  DeviceInfo d;
  svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  if (M == 0) {
    s = cuda_status(zero(dW, (size_t)N * K * 2, stream));
    return s != SVDQ_OK ? s : cuda_status(zero(dbias, (size_t)N * 2, stream));
  }
  const bool has_act = act != SVDQ_EPI_NONE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part = reinterpret_cast<float*>(ws + (has_act ? align256((size_t)M * N * 2) : 0));
  if (has_act || dbias) {
    ActGradParams p = {};
    p.kind = has_act ? ACT_GRAD_DENSE : ACT_GRAD_SUM;
    p.M = M;
    p.N = N;
    p.fp16 = dt == SVDQ_FP16;
    p.act = act;
    p.dY = in16(dY);
    p.ld = lddy;
    p.Z = in16(Z);
    p.dZ = has_act ? out16(ws) : nullptr;
    p.part = dbias ? part : nullptr;
    p.parts = act_grad_parts(M, N);
    if ((s = cuda_status(launch_act_grad(p, stream))) != SVDQ_OK) return s;
    if (dbias &&
        (s = cuda_status(launch_sum_parts(part, p.parts, N, dt, dbias, nullptr, nullptr, stream))) != SVDQ_OK)
      return s;
  }
  const void* dZ = has_act ? workspace : dY;
  const long long ldz = has_act ? N : lddy;
  if (dX && (s = input_gradient(d, dt, M, K, N, dZ, ldz, nullptr, W_t, nullptr, dX, lddx, stream)) != SVDQ_OK)
    return s;
  return dW ? weight_gradient(d, dt, M, K, N, dZ, ldz, nullptr, X, ldx, dW, nullptr, stream) : SVDQ_OK;
}

// ------------------------------------------------------------------ gated feed-forward
svdq_status svdq_gated_linear(svdq_dtype dt, int M, int K, int F, const void* X, long long ldx, const void* Wg_t,
                              const void* Wu_t, const void* bias_g, const void* bias_u, svdq_epilogue act, void* H,
                              long long ldh, void* G, void* U, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !Wg_t || !Wu_t || (M > 0 && (!X || !H))) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || !width_ok(K) || !width_ok(F) || !stride_ok(ldx, K) || !stride_ok(ldh, F)) return SVDQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(Wg_t) || !aligned16(Wu_t) || !aligned16(bias_g) || !aligned16(bias_u) ||
      !aligned16(H) || !aligned16(G) || !aligned16(U))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  DeviceInfo d;
  const svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  Gemm16Params p = no_epilogue();
  p.act = act;
  p.bias = in16(bias_g);
  p.bias2 = in16(bias_u);
  p.Y = out16(H);
  p.ldy = ldh;
  p.Z = out16(G);
  p.Z2 = out16(U);
  return forward_product(d, dt, M, K, F, X, ldx, Wg_t, Wu_t, p, stream);
}

// [dG | dU | the two bias gradients' partials]
size_t svdq_gated_linear_backward_workspace_bytes(int M, int K, int F) {
  if (M < 0 || !width_ok(K) || !width_ok(F)) return 0;
  return 2 * align256((size_t)M * F * 2) + 2 * align256((size_t)act_grad_parts(M, F) * F * 4);
}

svdq_status svdq_gated_linear_backward(svdq_dtype dt, int M, int K, int F, const void* dH, long long lddh,
                                       const void* X, long long ldx, const void* Wg_t, const void* Wu_t,
                                       const void* G, const void* U, svdq_epilogue act, void* dX, long long lddx,
                                       void* dWg, void* dWu, void* dbias_g, void* dbias_u, void* workspace,
                                       size_t ws_bytes, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !dWg != !dWu || !dbias_g != !dbias_u) return SVDQ_ERR_INVALID_ARG;
  if (M > 0 && (!dH || !G || !U || (dX && (!Wg_t || !Wu_t)) || (dWg && !X))) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || !width_ok(K) || !width_ok(F) || !stride_ok(lddh, F) || (dWg && !stride_ok(ldx, K)) ||
      (dX && !stride_ok(lddx, K)))
    return SVDQ_ERR_SHAPE;
  if (!aligned16(dH) || !aligned16(X) || !aligned16(Wg_t) || !aligned16(Wu_t) || !aligned16(G) || !aligned16(U) ||
      !aligned16(dX) || !aligned16(dWg) || !aligned16(dWu) || !aligned16(dbias_g) || !aligned16(dbias_u) ||
      !aligned16(workspace))
    return SVDQ_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < svdq_gated_linear_backward_workspace_bytes(M, K, F)) return SVDQ_ERR_WORKSPACE;
  DeviceInfo d;
  svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  if (M == 0) {
    void* w[2] = {dWg, dWu};
    void* b[2] = {dbias_g, dbias_u};
    for (int i = 0; i < 2; ++i) {
      if ((s = cuda_status(zero(w[i], (size_t)F * K * 2, stream))) != SVDQ_OK) return s;
      if ((s = cuda_status(zero(b[i], (size_t)F * 2, stream))) != SVDQ_OK) return s;
    }
    return SVDQ_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t dz_bytes = align256((size_t)M * F * 2);
  ActGradParams p = {};
  p.kind = ACT_GRAD_GATED;
  p.M = M;
  p.N = F;
  p.fp16 = dt == SVDQ_FP16;
  p.act = act;
  p.dY = in16(dH);
  p.ld = lddh;
  p.Z = in16(G);
  p.U = in16(U);
  p.dZ = out16(ws);
  p.dU = out16(ws + dz_bytes);
  p.parts = act_grad_parts(M, F);
  float* part = reinterpret_cast<float*>(ws + 2 * dz_bytes);
  float* part2 = reinterpret_cast<float*>(ws + 2 * dz_bytes + align256((size_t)p.parts * F * 4));
  p.part = dbias_g ? part : nullptr;
  p.part2 = part2;
  if ((s = cuda_status(launch_act_grad(p, stream))) != SVDQ_OK) return s;
  if (dbias_g &&
      (s = cuda_status(launch_sum_parts(part, p.parts, F, dt, dbias_g, part2, dbias_u, stream))) != SVDQ_OK)
    return s;
  if (dX && (s = input_gradient(d, dt, M, K, F, p.dZ, F, p.dU, Wg_t, Wu_t, dX, lddx, stream)) != SVDQ_OK) return s;
  return dWg ? weight_gradient(d, dt, M, K, F, p.dZ, F, p.dU, X, ldx, dWg, dWu, stream) : SVDQ_OK;
}

// ------------------------------------------------------------------ layer norm
static size_t elem_bytes(svdq_dtype dt) { return dt == SVDQ_FP32 ? 4 : 2; }
static bool elem_aligned(svdq_dtype dt, const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & (elem_bytes(dt) - 1)) == 0;
}
static bool float_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
static bool known_type(svdq_dtype dt) { return dt == SVDQ_BF16 || dt == SVDQ_FP16 || dt == SVDQ_FP32; }

svdq_status svdq_layernorm(svdq_dtype dt, int M, int C, const void* X, long long ldx, const void* gamma,
                           const void* beta, float eps, void* Y, long long ldy, float* mean, float* rstd,
                           cudaStream_t stream) {
  if (!known_type(dt) || !gamma != !beta || (M > 0 && (!X || !Y)) || !(eps >= 0.f) || !std::isfinite(eps))
    return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || C < 1 || ldx < C || ldy < C) return SVDQ_ERR_SHAPE;
  if (!elem_aligned(dt, X) || !elem_aligned(dt, gamma) || !elem_aligned(dt, beta) || !elem_aligned(dt, Y) ||
      !float_aligned(mean) || !float_aligned(rstd))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  DeviceInfo d;
  const svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  return cuda_status(launch_layernorm({M, C, (int)dt, X, gamma, beta, ldx, ldy, eps, Y, mean, rstd}, stream));
}

// [dgamma partials | dbeta partials]
size_t svdq_layernorm_backward_workspace_bytes(int M, int C) {
  if (M < 0 || C < 1) return 0;
  return 256 + 2 * align256((size_t)layernorm_grad_parts(M, C) * C * 4);
}

svdq_status svdq_layernorm_backward(svdq_dtype dt, int M, int C, const void* dY, long long lddy, const void* X,
                                    long long ldx, const void* gamma, const float* mean, const float* rstd, void* dX,
                                    long long lddx, void* dgamma, void* dbeta, void* workspace, size_t ws_bytes,
                                    cudaStream_t stream) {
  if (!known_type(dt) || !dgamma != !dbeta || (M > 0 && (!dY || !X || !mean || !rstd))) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || C < 1 || lddy < C || ldx < C || (dX && lddx < C)) return SVDQ_ERR_SHAPE;
  if (!elem_aligned(dt, dY) || !elem_aligned(dt, X) || !elem_aligned(dt, gamma) || !elem_aligned(dt, dX) ||
      !elem_aligned(dt, dgamma) || !elem_aligned(dt, dbeta) || !float_aligned(mean) || !float_aligned(rstd) ||
      !aligned16(workspace))
    return SVDQ_ERR_ALIGNMENT;
  if (dgamma && (!workspace || ws_bytes < svdq_layernorm_backward_workspace_bytes(M, C))) return SVDQ_ERR_WORKSPACE;
  DeviceInfo d;
  svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  if (M == 0) {
    s = cuda_status(zero(dgamma, (size_t)C * elem_bytes(dt), stream));
    return s != SVDQ_OK ? s : cuda_status(zero(dbeta, (size_t)C * elem_bytes(dt), stream));
  }
  if (!dX && !dgamma) return SVDQ_OK;
  int parts = layernorm_grad_parts(M, C);
  float* pg = dgamma ? static_cast<float*>(workspace) : nullptr;
  float* pb = dgamma ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t)parts * C * 4))
                     : nullptr;
  s = cuda_status(launch_layernorm_grad(
      {M, C, (int)dt, dY, X, gamma, lddy, ldx, lddx, mean, rstd, dX, pg, pb}, &parts, stream));
  if (s != SVDQ_OK || !dgamma) return s;
  return cuda_status(launch_sum_parts(pg, parts, C, dt, dgamma, pb, dbeta, stream));
}

}  // extern "C"
