// act_grad.cu -- the elementwise half of the 16-bit layers' backward passes,
// with the bias gradients' column sums taken from the same pass.
//
//   sum     db = sum_m dY
//   dense   dZ = dY act'(Z),                       db  = sum_m dZ
//   gated   dG = dH U act'(G), dU = dH act(G),     dbg = sum_m dG, dbu = sum_m dU
//
// The sums take the float32 values before their rounding to 16 bits.  Bound
// by memory: every value is read or written once, 16 bytes a thread.  A block
// owns 256 columns (32 threads of 8) and a contiguous range of rows, 8 rows at
// a time; its 8 row lanes add up in shared memory in a fixed order, the blocks
// of a column write one float32 partial each, and sum_parts_kernel adds those
// in order: no atomics, the same bits on every run.
// Measured, 4608 x 12288 bf16 gated: 99 us for 566 MB (5.7 TB/s, 87% of the
// measured copy rate; instruction issue 63% busy).
#include "common.cuh"
#include "dense.h"

namespace svdq {

namespace {

constexpr int COLS = 256, LANES = 8, THREADS = 256;

__device__ __forceinline__ void unpack8(const uint4& v, bool fp16, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t;
    if (fp16)
      t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    else
      t = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8], bool fp16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (fp16) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int KIND>
__global__ void __launch_bounds__(THREADS) act_grad_kernel(ActGradParams p) {
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int n = blockIdx.x * COLS + cl * 8;
  const int r0 = (int)((long long)p.M * blockIdx.y / gridDim.y);
  const int r1 = (int)((long long)p.M * (blockIdx.y + 1) / gridDim.y);
  const bool fp16 = p.fp16 != 0;
  float s[8] = {}, s2[8] = {};
  grid_launch_dependents();   // the products' kernel may set up as SMs fall idle
  grid_dependency_wait();
  if (n < p.N) {
#pragma unroll 2
    for (int m = r0 + rl; m < r1; m += LANES) {
      const size_t at = (size_t)m * p.N + n;
      float dy[8];
      unpack8(*reinterpret_cast<const uint4*>(p.dY + (size_t)m * p.ld + n), fp16, dy);
      if (KIND == ACT_GRAD_SUM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += dy[i];
      } else if (KIND == ACT_GRAD_DENSE) {
        float z[8];
        unpack8(*reinterpret_cast<const uint4*>(p.Z + at), fp16, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, d;
          act_and_slope(z[i], p.act, f, d);
          z[i] = dy[i] * d;
          s[i] += z[i];
        }
        *reinterpret_cast<uint4*>(p.dZ + at) = pack8(z, fp16);
      } else {
        float g[8], u[8];
        unpack8(*reinterpret_cast<const uint4*>(p.Z + at), fp16, g);
        unpack8(*reinterpret_cast<const uint4*>(p.U + at), fp16, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, d;
          act_and_slope(g[i], p.act, f, d);
          g[i] = dy[i] * u[i] * d;
          u[i] = dy[i] * f;
          s[i] += g[i];
          s2[i] += u[i];
        }
        *reinterpret_cast<uint4*>(p.dZ + at) = pack8(g, fp16);
        *reinterpret_cast<uint4*>(p.dU + at) = pack8(u, fp16);
      }
    }
  }
  if (!p.part) return;
  __shared__ float sh[LANES][COLS];
  auto reduce = [&](const float (&v)[8], float* part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sh[rl][cl * 8 + i] = v[i];
    __syncthreads();
    const int col = blockIdx.x * COLS + threadIdx.x;
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < LANES; ++r) t += sh[r][threadIdx.x];
    if (col < p.N) part[(size_t)blockIdx.y * p.N + col] = t;
    __syncthreads();
  };
  reduce(s, p.part);
  if (KIND == ACT_GRAD_GATED) reduce(s2, p.part2);
}

// 32 columns x 32 part lanes a block: lane l adds parts l, l + 32, ..., then
// the lanes as a tree, the same one every time.
constexpr int SUM_LANES = 32;
__global__ void __launch_bounds__(32 * SUM_LANES) sum_parts_kernel(const float* part, const float* part2, int parts,
                                                                   int N, int dt, void* out, void* out2) {
  grid_dependency_wait();   // launched early: the partials' kernel may still run
  const float* src = blockIdx.y ? part2 : part;
  void* dst = blockIdx.y ? out2 : out;
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5, n = blockIdx.x * 32 + cl;
  float t = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int s = rl; s < parts; s += SUM_LANES) t += src[(size_t)s * N + n];
  }
  __shared__ float sh[SUM_LANES][33];
  sh[rl][cl] = t;
  __syncthreads();
  // warp w takes column w: its 32 lanes' sums, added as a tree
  t = sh[cl][rl];
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int col = blockIdx.x * 32 + rl;
  if (cl == 0 && col < N) {
    if (dt == SVDQ_FP32)
      static_cast<float*>(dst)[col] = t;
    else if (dt == SVDQ_FP16)
      static_cast<__half*>(dst)[col] = __float2half_rn(t);
    else
      static_cast<__nv_bfloat16*>(dst)[col] = __float2bfloat16_rn(t);
  }
}

}  // namespace

// Row ranges: as many blocks as the SMs hold at four each and no more (a
// second, nearly empty round cost 148 us instead of 103 for 4608 x 12288
// gated), and no more than one for every 16 rows (8 to 16 rows each then).
int act_grad_parts(int M, int N) {
  const int cb = (int)(((long long)N + COLS - 1) / COLS);
  int parts = 148 * 4 / cb;
  const int most = (int)(((long long)M + 15) / 16);
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts;
}

cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)(((long long)p.N + COLS - 1) / COLS), p.parts);
  switch (p.kind) {
    case ACT_GRAD_SUM: return launch_early(act_grad_kernel<ACT_GRAD_SUM>, grid, THREADS, 0, stream, p);
    case ACT_GRAD_DENSE: return launch_early(act_grad_kernel<ACT_GRAD_DENSE>, grid, THREADS, 0, stream, p);
    default: return launch_early(act_grad_kernel<ACT_GRAD_GATED>, grid, THREADS, 0, stream, p);
  }
}

cudaError_t launch_sum_parts(const float* part, int parts, int N, int dt, void* out, const float* part2, void* out2,
                             cudaStream_t stream) {
  return launch_early(sum_parts_kernel, dim3((N + 31) / 32, part2 ? 2 : 1), 32 * SUM_LANES, 0, stream, part, part2,
                      parts, N, dt, out, out2);
}

}  // namespace svdq
