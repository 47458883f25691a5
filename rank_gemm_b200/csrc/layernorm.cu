// layernorm.cu -- layer norm and its backward pass.
//
//   forward   mean = sum x / C,  var = sum (x - mean)^2 / C (two passes over
//             the row, which sits in registers), rstd = 1 / sqrt(var + eps),
//             y = (x - mean) rstd gamma + beta
//   backward  xh = (x - mean) rstd,  g = dy gamma,
//             dx = rstd (g - mean(g) - xh mean(g xh)),
//             dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// Bound by memory: each row is read once (forward) or once each of x and dy
// (backward), 16 bytes a thread where the row's length, stride and address
// allow, else one element a thread.  A group of 32 .. 512 threads owns a row
// and a thread the same columns of every row, so in the backward pass
// dgamma / dbeta add up in registers over the rows of a group; the groups'
// float32 partials are added in group order by sum_parts_kernel: no atomics,
// the same bits on every run.  Rows too long for the registers of a group are
// read again from L2 (the streamed forms).
#include "common.cuh"
#include "kernels.h"

namespace svdq {

namespace {

constexpr int MAX_TPR = 512;    // threads of a row
constexpr int MIN_BLOCK = 128;

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive elements (16 bytes, or one element)
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

// Sums of N values over the tpr threads of a row group; every thread of the
// block calls it.  `sh` alternates between two buffers, so one barrier a call
// is enough.
template <int N>
struct Reducer {
  float (*sh)[N];   // [2][32 warps]
  int tpr, warp0, buf;
  __device__ Reducer(float (*s)[N], int tpr_) : sh(s), tpr(tpr_), buf(0) {
    warp0 = (int)(threadIdx.x / tpr) * (tpr >> 5);
  }
  __device__ void sum(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sh[buf * 32 + warp][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = lane < nw ? sh[buf * 32 + warp0 + lane][i] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      v[i] = __shfl_sync(0xffffffffu, t, 0);
    }
    buf ^= 1;
  }
};
static_assert(MAX_TPR <= 16 * 32, "Reducer adds at most 16 warps");

// ------------------------------------------------------------------ forward
// PER packs of VEC elements a thread; PER = 0: streamed (three reads of the row).
template <typename T, int VEC, int PER>
__global__ void __launch_bounds__(MAX_TPR) layernorm_kernel(LayerNormParams p, int tpr) {
  __shared__ float sh[64][1];
  const int rpb = blockDim.x / tpr, t = threadIdx.x % tpr;
  const long long row = (long long)blockIdx.x * rpb + threadIdx.x / tpr;
  const bool live = row < p.M;
  const int nv = p.C / VEC;
  using P = Pack<T, VEC>;
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(p.X) + (live ? row : 0) * p.ldx);
  P* y = reinterpret_cast<P*>(static_cast<T*>(p.Y) + (live ? row : 0) * p.ldy);
  const P* ga = static_cast<const P*>(p.gamma);
  const P* be = static_cast<const P*>(p.beta);
  Reducer<1> red(sh, tpr);
  const float inv_c = 1.0f / (float)p.C;
  P r[PER ? PER : 1];
  float s[1] = {0.f};
  if (PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * tpr;
      if (live && c < nv) r[i] = x[c];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (live && t + i * tpr < nv)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += to_f32(r[i].v[j]);
  } else if (live) {
    for (int c = t; c < nv; c += tpr) {
      const P q = x[c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0] += to_f32(q.v[j]);
    }
  }
  red.sum(s);
  const float mean = s[0] * inv_c;
  s[0] = 0.f;
  if (PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (live && t + i * tpr < nv)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f32(r[i].v[j]) - mean;
          s[0] = fmaf(d, d, s[0]);
        }
  } else if (live) {
    for (int c = t; c < nv; c += tpr) {
      const P q = x[c];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = to_f32(q.v[j]) - mean;
        s[0] = fmaf(d, d, s[0]);
      }
    }
  }
  red.sum(s);
  const float rstd = 1.0f / sqrtf(s[0] * inv_c + p.eps);
  if (!live) return;
  auto put = [&](const P& q, int c) {
    P o, g, b;
    if (ga) {
      g = ga[c];
      b = be[c];
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float v = (to_f32(q.v[j]) - mean) * rstd;
      if (ga) v = fmaf(v, to_f32(g.v[j]), to_f32(b.v[j]));
      o.v[j] = from_f32<T>(v);
    }
    y[c] = o;
  };
  if (PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (t + i * tpr < nv) put(r[i], t + i * tpr);
  } else {
    for (int c = t; c < nv; c += tpr) put(x[c], c);
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// ------------------------------------------------------------------ backward
template <typename T, int VEC, int PER>
__global__ void __launch_bounds__(MAX_TPR) layernorm_grad_kernel(LayerNormGradParams p, int tpr) {
  __shared__ float sh[64][2];
  const int rpb = blockDim.x / tpr, t = threadIdx.x % tpr, group = blockIdx.x * rpb + threadIdx.x / tpr;
  const int groups = gridDim.x * rpb;
  const int nv = p.C / VEC;
  using P = Pack<T, VEC>;
  const P* ga = static_cast<const P*>(p.gamma);
  Reducer<2> red(sh, tpr);
  const float inv_c = 1.0f / (float)p.C;
  float ag[PER][VEC] = {}, ab[PER][VEC] = {};
  // every group of a block runs the same number of rounds (the reduction's barrier)
  for (long long base = (long long)blockIdx.x * rpb; base < p.M; base += groups) {
    const long long row = base + threadIdx.x / tpr;
    const bool live = row < p.M;
    const P* x = reinterpret_cast<const P*>(static_cast<const T*>(p.X) + (live ? row : 0) * p.ldx);
    const P* dy = reinterpret_cast<const P*>(static_cast<const T*>(p.dY) + (live ? row : 0) * p.lddy);
    const float mean = live ? p.mean[row] : 0.f, rstd = live ? p.rstd[row] : 0.f;
    P rx[PER], rd[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * tpr;
      if (live && c < nv) {
        rx[i] = x[c];
        rd[i] = dy[c];
      }
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = t + i * tpr;
      if (live && c < nv) {
        P g;
        if (ga) g = ga[c];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (to_f32(rx[i].v[j]) - mean) * rstd, d = to_f32(rd[i].v[j]);
          const float gv = ga ? d * to_f32(g.v[j]) : d;
          ag[i][j] = fmaf(d, xh, ag[i][j]);
          ab[i][j] += d;
          s[0] += gv;
          s[1] = fmaf(gv, xh, s[1]);
        }
      }
    }
    red.sum(s);
    if (live && p.dX) {
      P* dx = reinterpret_cast<P*>(static_cast<T*>(p.dX) + row * p.lddx);
      const float a = s[0] * inv_c, b = s[1] * inv_c;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = t + i * tpr;
        if (c < nv) {
          P g, o;
          if (ga) g = ga[c];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float xh = (to_f32(rx[i].v[j]) - mean) * rstd, d = to_f32(rd[i].v[j]);
            const float gv = ga ? d * to_f32(g.v[j]) : d;
            o.v[j] = from_f32<T>(rstd * (gv - a - xh * b));
          }
          dx[c] = o;
        }
      }
    }
  }
  if (!p.part_g) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = t + i * tpr;
    if (c < nv) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const size_t at = (size_t)group * p.C + (size_t)c * VEC + j;
        p.part_g[at] = ag[i][j];
        p.part_b[at] = ab[i][j];
      }
    }
  }
}

// Rows too long for registers: dX by reading x and dy twice, one block a row ...
template <typename T>
__global__ void __launch_bounds__(MAX_TPR) layernorm_grad_rows_kernel(LayerNormGradParams p) {
  __shared__ float sh[64][2];
  const T* x = static_cast<const T*>(p.X) + (long long)blockIdx.x * p.ldx;
  const T* dy = static_cast<const T*>(p.dY) + (long long)blockIdx.x * p.lddy;
  T* dx = static_cast<T*>(p.dX) + (long long)blockIdx.x * p.lddx;
  const T* ga = static_cast<const T*>(p.gamma);
  const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x], inv_c = 1.0f / (float)p.C;
  Reducer<2> red(sh, (int)blockDim.x);
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    const float xh = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * (ga ? to_f32(ga[c]) : 1.f);
    s[0] += g;
    s[1] = fmaf(g, xh, s[1]);
  }
  red.sum(s);
  const float a = s[0] * inv_c, b = s[1] * inv_c;
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    const float xh = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * (ga ? to_f32(ga[c]) : 1.f);
    dx[c] = from_f32<T>(rstd * (g - a - xh * b));
  }
}
// ... and the columns' sums over a range of rows, a thread a column.
template <typename T>
__global__ void __launch_bounds__(MAX_TPR) layernorm_grad_cols_kernel(LayerNormGradParams p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.C) return;
  const int r0 = (int)((long long)p.M * blockIdx.y / gridDim.y), r1 = (int)((long long)p.M * (blockIdx.y + 1) / gridDim.y);
  float g = 0.f, b = 0.f;
  for (int m = r0; m < r1; ++m) {
    const float d = to_f32(static_cast<const T*>(p.dY)[(long long)m * p.lddy + c]);
    const float xh = (to_f32(static_cast<const T*>(p.X)[(long long)m * p.ldx + c]) - p.mean[m]) * p.rstd[m];
    g = fmaf(d, xh, g);
    b += d;
  }
  p.part_g[(size_t)blockIdx.y * p.C + c] = g;
  p.part_b[(size_t)blockIdx.y * p.C + c] = b;
}

// ------------------------------------------------------------------ shapes
constexpr int ELEMS_MAX = 32;   // elements a thread holds

struct RowShape {
  int per, tpr, block;   // per = 0: streamed
};
// Packs a thread and threads a row: few threads with several packs each for
// long rows (fewer warps to synchronise), at most max_per packs.
RowShape row_shape(int nv, int max_per) {
  RowShape s;
  s.per = nv >= 256 ? 4 : nv >= 64 ? 2 : 1;
  if (s.per > max_per) s.per = max_per;
  while (s.per < max_per && (long long)s.per * MAX_TPR < nv) s.per *= 2;
  if ((long long)s.per * MAX_TPR < nv) s.per = 0;
  const int need = s.per ? (nv + s.per - 1) / s.per : MAX_TPR;
  s.tpr = (need + 31) / 32 * 32;
  s.block = s.tpr >= MIN_BLOCK ? s.tpr : MIN_BLOCK / s.tpr * s.tpr;
  return s;
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename T>
bool vectors(int C, std::initializer_list<const void*> ptrs, std::initializer_list<long long> lds) {
  if (C * sizeof(T) % 16) return false;
  for (const void* q : ptrs)
    if (!aligned_to(q, 16)) return false;
  for (long long ld : lds)
    if (ld * (long long)sizeof(T) % 16) return false;
  return true;
}

template <typename T, int VEC>
cudaError_t forward(const LayerNormParams& p, cudaStream_t st) {
  constexpr int MP = ELEMS_MAX / VEC < 8 ? ELEMS_MAX / VEC : 8;
  const RowShape s = row_shape(p.C / VEC, MP);
  const int rpb = s.block / s.tpr;
  const unsigned grid = (unsigned)((p.M + rpb - 1) / rpb);
  switch (s.per) {
    case 0: layernorm_kernel<T, VEC, 0><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    case 1: layernorm_kernel<T, VEC, 1><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    case 2: layernorm_kernel<T, VEC, 2><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    case 4: layernorm_kernel<T, VEC, 4><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    default: layernorm_kernel<T, VEC, MP><<<grid, s.block, 0, st>>>(p, s.tpr); break;
  }
  return cudaGetLastError();
}

constexpr int GRAD_GROUPS = 148 * 4;   // row groups of the backward pass at most

template <typename T, int VEC>
cudaError_t backward(const LayerNormGradParams& p, cudaStream_t st) {
  constexpr int MP = 16 / VEC < 4 ? 16 / VEC : 4;
  const RowShape s = row_shape(p.C / VEC, MP);
  if (s.per == 0) {
    if (p.dX) {
      layernorm_grad_rows_kernel<T><<<p.M, MAX_TPR, 0, st>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (p.part_g)
      layernorm_grad_cols_kernel<T><<<dim3((p.C + MAX_TPR - 1) / MAX_TPR, p.parts), MAX_TPR, 0, st>>>(p);
    return cudaGetLastError();
  }
  const int rpb = s.block / s.tpr;
  const unsigned grid = (unsigned)(p.parts / rpb);   // parts is a multiple of every rows-per-block
  switch (s.per) {
    case 1: layernorm_grad_kernel<T, VEC, 1><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    case 2: layernorm_grad_kernel<T, VEC, 2><<<grid, s.block, 0, st>>>(p, s.tpr); break;
    default: layernorm_grad_kernel<T, VEC, MP><<<grid, s.block, 0, st>>>(p, s.tpr); break;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_any(const LayerNormParams& p, cudaStream_t st) {
  return vectors<T>(p.C, {p.X, p.Y, p.gamma, p.beta}, {p.ldx, p.ldy}) ? forward<T, 16 / sizeof(T)>(p, st)
                                                                     : forward<T, 1>(p, st);
}
template <typename T>
cudaError_t backward_any(const LayerNormGradParams& p, cudaStream_t st) {
  return vectors<T>(p.C, {p.X, p.dY, p.dX, p.gamma}, {p.ldx, p.lddy, p.lddx}) ? backward<T, 16 / sizeof(T)>(p, st)
                                                                             : backward<T, 1>(p, st);
}

}  // namespace

// Groups (and partials): a multiple of 4, the most rows a block holds.
int layernorm_grad_parts(int M, int) {
  const int need = (M + 3) / 4 * 4;
  return need < GRAD_GROUPS ? need : GRAD_GROUPS;
}

cudaError_t launch_layernorm(const LayerNormParams& p, cudaStream_t st) {
  switch (p.dt) {
    case SVDQ_BF16: return forward_any<__nv_bfloat16>(p, st);
    case SVDQ_FP16: return forward_any<__half>(p, st);
    default: return forward_any<float>(p, st);
  }
}
cudaError_t launch_layernorm_grad(const LayerNormGradParams& p, cudaStream_t st) {
  switch (p.dt) {
    case SVDQ_BF16: return backward_any<__nv_bfloat16>(p, st);
    case SVDQ_FP16: return backward_any<__half>(p, st);
    default: return backward_any<float>(p, st);
  }
}

}  // namespace svdq
