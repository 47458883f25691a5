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
// allow.  Else one element a thread, and there the instructions bound it: 4608
// x 3001 fp16 26.7 us forward and 39.9 backward, where the bytes take 8.4 and
// 12.7.  A group of 32 .. 512 threads walks over
// rows, a thread the same columns of every row, so in the backward pass gamma
// and the sums of dgamma and dbeta stay in registers over the rows of a group;
// the blocks' float32 partials are added in block order by sum_parts_kernel:
// no atomics, the same bits on every run.  What keeps the memory busy is the
// bytes in flight and the instructions a value costs: the next rows are copied
// ahead (cp.async) into a ring of shared-memory slots that belong to the
// thread that reads them, so no barrier guards the ring, and the arithmetic
// runs two float32 operations an instruction.  Rows too long for the registers
// of a group are streamed: forward they are read three times, 16 bytes a thread
// as above, the second and third time from L2 (4096 x 40960 bf16 131 us, its
// bytes 103).  Backward (above 12288 columns in 16 bits, 6144 in float32) every
// load is one element, dX reads x and dy twice and the columns' sums once more,
// from memory: 4096 x 16384 bf16 354 us (dX alone 217), its bytes 62.
// Measured, 16384 x 3072 bf16: forward 36.5 us (201 MB, 5.5 TB/s, 84% of the
// measured copy rate; instruction issue 68% busy), backward with the weights'
// gradients 61 us (302 MB, 4.9 TB/s, 75%; issue 55% busy at 12 warps a SM,
// which is what the two sums' registers leave room for).
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "dense.h"

namespace svdq {

namespace {

constexpr int MAX_TPR = 512;    // threads of a row
constexpr int SMALL_BLOCK = 128;
constexpr int DEPTH = 2;        // rows in a thread's ring

// ------------------------------------------------------------------ values
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

// VEC consecutive elements as they lie in memory: 16 bytes, or one element.
template <typename T, int VEC>
struct PackOf {
  using type = uint4;
};
template <typename T>
struct PackOf<T, 1> {
  using type = T;
};
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename PackOf<T, VEC>::type& p, float* f) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(p);
  } else {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        f[j] = __uint_as_float(w[j]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
      } else {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}
// A pack of gamma or beta (guarded by a null check: see ld_param).
template <typename T, int VEC>
__device__ __forceinline__ typename PackOf<T, VEC>::type ld_const(const typename PackOf<T, VEC>::type* p) {
  if constexpr (VEC > 1)
    return ld_param(p);
  else
    return *p;
}
template <typename T, int VEC>
__device__ __forceinline__ typename PackOf<T, VEC>::type pack(const float* f) {
  if constexpr (VEC == 1) {
    return from_f32<T>(f[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        w[j] = __float_as_uint(f[j]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------ two float32 operations an instruction
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t bits(F2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ F2 f2(uint64_t r) {
  F2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return f2(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return f2(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return f2(r);
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }

// Loops over the VEC values of a pack, two at a time where there are two.
template <int VEC>
__device__ __forceinline__ void add_to(F2& acc, const float* v) {
  if constexpr (VEC == 1)
    acc.x += v[0];
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) acc = add2(acc, F2{v[j], v[j + 1]});
}
template <int VEC>
__device__ __forceinline__ void fma_to(F2& acc, const float* u, const float* v) {
  if constexpr (VEC == 1)
    acc.x = fmaf(u[0], v[0], acc.x);
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) acc = fma2(F2{u[j], u[j + 1]}, F2{v[j], v[j + 1]}, acc);
}
// o = a + s, o = a s, o = a b + c
template <int VEC>
__device__ __forceinline__ void add_s(float* o, const float* a, float s) {
  if constexpr (VEC == 1)
    o[0] = a[0] + s;
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const F2 r = add2(F2{a[j], a[j + 1]}, both(s));
      o[j] = r.x;
      o[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void add_v(float* o, const float* a, const float* b) {
  if constexpr (VEC == 1)
    o[0] = a[0] + b[0];
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const F2 r = add2(F2{a[j], a[j + 1]}, F2{b[j], b[j + 1]});
      o[j] = r.x;
      o[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void mul_s(float* o, const float* a, float s) {
  if constexpr (VEC == 1)
    o[0] = a[0] * s;
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const F2 r = mul2(F2{a[j], a[j + 1]}, both(s));
      o[j] = r.x;
      o[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void mul_v(float* o, const float* a, const float* b) {
  if constexpr (VEC == 1)
    o[0] = a[0] * b[0];
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const F2 r = mul2(F2{a[j], a[j + 1]}, F2{b[j], b[j + 1]});
      o[j] = r.x;
      o[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void fma_v(float* o, const float* a, const float* b, const float* c) {
  if constexpr (VEC == 1)
    o[0] = fmaf(a[0], b[0], c[0]);
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const F2 r = fma2(F2{a[j], a[j + 1]}, F2{b[j], b[j + 1]}, F2{c[j], c[j + 1]});
      o[j] = r.x;
      o[j + 1] = r.y;
    }
}

// sum / c by one correction of sum * (1 / c), which alone is up to 1.5 steps
// off: a row of one value has to have that value as its mean (1000 in 3584
// columns was off by 6e-5, its output by 0.02).  A sum that is not finite is
// its own mean.
__device__ __forceinline__ float mean_of(float sum, float c, float inv_c) {
  const float m = sum * inv_c, r = fmaf(fmaf(-m, c, sum), inv_c, m);
  return r == r ? r : m;
}

// ------------------------------------------------------------------ sums over a row group
// Sums over the tpr threads of a row group; every thread of the block calls
// it.  `sh` alternates between two buffers, so one barrier a call is enough.
struct Reducer {
  float (*sh)[1];   // [2][16 warps]
  int tpr, warp0, buf;
  __device__ Reducer(float (*s)[1], int tpr_)
      : sh(s), tpr(tpr_), warp0((int)(threadIdx.x / tpr_) * (tpr_ >> 5)), buf(0) {}
  __device__ float sum1(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5;
    if (lane == 0) sh[buf * 16 + warp][0] = v;
    __syncthreads();
    v = lane < nw ? sh[buf * 16 + warp0 + lane][0] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    buf ^= 1;
    return __shfl_sync(0xffffffffu, v, 0);
  }
};
// N = 2 or 4 sums over a group for the price of little more than one: each of
// the first steps halves the number of values a lane carries, so that after
// them the lanes of half (quarter) h carry value h.
template <int N>
__device__ __forceinline__ void fold(float (&s)[N], int lane, float& v) {
  if constexpr (N == 2) {
    const bool h = lane & 16;
    v = (h ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, h ? s[0] : s[1], 16);
  } else {
    const bool h = lane & 16, q = lane & 8;
    const float a = (h ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, h ? s[0] : s[2], 16);
    const float b = (h ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, h ? s[1] : s[3], 16);
    v = (q ? b : a) + __shfl_xor_sync(0xffffffffu, q ? a : b, 8);
  }
#pragma unroll
  for (int o = 16 / N; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
}
template <int N>
__device__ __forceinline__ void group_sums(float (&s)[N], float (*sh)[N], int tpr, int& buf) {
  constexpr int LANES = 32 / N;   // lanes that carry one value
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5, which = lane / LANES;
  float v;
  fold<N>(s, lane, v);
  if (tpr > 32) {
    if (lane % LANES == 0) sh[buf * 16 + warp][which] = v;
    __syncthreads();
    const int warp0 = (int)(threadIdx.x / tpr) * nw;
    v = 0.f;
#pragma unroll
    for (int w = lane % LANES; w < 16; w += LANES)
      if (w < nw) v += sh[buf * 16 + warp0 + w][which];
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    buf ^= 1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = __shfl_sync(0xffffffffu, v, i * LANES);
}
static_assert(MAX_TPR <= 16 * 32, "Reducer adds at most 16 warps");

// ------------------------------------------------------------------ rows ahead
// A thread's ring of row packs in shared memory (16-byte packs); one-element
// packs are loaded one round ahead into registers instead.
template <typename P, int PER, int ROWS>
struct Ring {
  static constexpr bool ON = sizeof(P) == 16;
  static constexpr int BYTES = ON ? DEPTH * ROWS * PER * 16 : 0;   // a thread
  uint32_t base;
  __device__ __forceinline__ uint32_t slot(int stage, int which, int i) const {
    return base + (((stage * ROWS + which) * PER + i) * blockDim.x + threadIdx.x) * 16;
  }
  __device__ __forceinline__ void copy(int stage, int which, int i, const P* src) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot(stage, which, i)), "l"(src) : "memory");
  }
  __device__ __forceinline__ P get(int stage, int which, int i) const {
    if constexpr (ON)
      return lds128(slot(stage, which, i));
    else
      return P();
  }
};
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_oldest() {
  asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
}

// ------------------------------------------------------------------ forward
// TPR threads a row, PER packs a thread, a block of several rows when a row
// is one warp.
template <int TPR>
constexpr int BLOCK_OF = TPR < SMALL_BLOCK ? SMALL_BLOCK : TPR;
template <typename T, int VEC, int TPR, int PER>
__global__ void __launch_bounds__(BLOCK_OF<TPR>, PER <= 4 ? 1024 / BLOCK_OF<TPR> : 1)
    layernorm_kernel(LayerNormParams p) {
  constexpr int RPB = BLOCK_OF<TPR> / TPR;
  __shared__ float sh[32][1];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int t = threadIdx.x % TPR, g0 = threadIdx.x / TPR;
  const int left = p.C / VEC - t;   // pack i is the row's while i TPR < left
  using P = typename PackOf<T, VEC>::type;
  const P* ga = static_cast<const P*>(p.gamma) + t;
  const P* be = static_cast<const P*>(p.beta) + t;
  const bool affine = p.gamma != nullptr;
  Reducer red(sh, TPR);
  using RowRing = Ring<P, PER, 1>;
  const RowRing ring{smem_u32(ring_raw)};
  const float inv_c = 1.0f / (float)p.C;
  const long long stride = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + g0;
  const long long step = stride * p.ldx;
  const T* src = static_cast<const T*>(p.X) + row * p.ldx + t * VEC;   // this row, or (ring) the next to fetch
  auto fetch = [&](long long r, int stage) {
    if (r < p.M)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * TPR < left) ring.copy(stage, 0, i, reinterpret_cast<const P*>(src) + i * TPR);
    cp_commit();
    src += step;
  };
  P ahead[RowRing::ON ? 1 : PER];
  auto load = [&](long long r) {   // one-element packs of the row at src
    if (r < p.M)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * TPR < left) ahead[i] = reinterpret_cast<const P*>(src)[i * TPR];
    src += step;
  };
  grid_launch_dependents();
  grid_dependency_wait();
  if constexpr (RowRing::ON) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(row + d * stride, d);
  } else {
    load(row);
  }
  // One-element packs: gamma and beta stay in registers over the rows (8192 x
  // 1001 fp16 13.3 us, 11.3 so; 4608 x 5001 58.4, 46.0), except where they
  // cost the second block of an SM (4608 x 3001 26.5, 30.2 so).
  constexpr bool KEEP = VEC == 1 && !(TPR == 512 && PER == 8);
  P gam[KEEP ? PER : 1], bet[KEEP ? PER : 1];
  if (KEEP && affine)
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * TPR < left) {
        gam[KEEP ? i : 0] = ld_const<T, VEC>(ga + i * TPR);
        bet[KEEP ? i : 0] = ld_const<T, VEC>(be + i * TPR);
      }
  int stage = 0;
  // every group of a block runs the same number of rounds (the reductions' barriers)
  for (long long base = (long long)blockIdx.x * RPB; base < p.M; base += stride, row += stride) {
    const bool live = row < p.M;
    if (RowRing::ON) cp_wait_oldest();
    float x[PER][VEC];
    F2 acc = both(0.f), acc2 = both(0.f);   // two chains: half the latency
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (live && i * TPR < left) {
        if constexpr (RowRing::ON)
          unpack<T, VEC>(ring.get(stage, 0, i), x[i]);
        else
          unpack<T, VEC>(ahead[i], x[i]);
        add_to<VEC>(i & 1 ? acc2 : acc, x[i]);
      }
    acc = add2(acc, acc2);
    const float mean = mean_of(red.sum1(acc.x + acc.y), (float)p.C, inv_c);
    if constexpr (RowRing::ON) {   // the slots have been read: the sum above needed their values
      fetch(row + DEPTH * stride, stage);
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    } else {
      load(row + stride);
    }
    acc = acc2 = both(0.f);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (live && i * TPR < left) {
        add_s<VEC>(x[i], x[i], -mean);
        fma_to<VEC>(i & 1 ? acc2 : acc, x[i], x[i]);
      }
    acc = add2(acc, acc2);
    const float rstd = 1.0f / sqrtf(red.sum1(acc.x + acc.y) * inv_c + p.eps);
    if (!live) continue;
    P* y = reinterpret_cast<P*>(static_cast<T*>(p.Y) + row * p.ldy) + t;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * TPR < left) {
        mul_s<VEC>(x[i], x[i], rstd);
        if (affine) {
          float g[VEC], b[VEC];
          unpack<T, VEC>(KEEP ? gam[KEEP ? i : 0] : ld_const<T, VEC>(ga + i * TPR), g);
          unpack<T, VEC>(KEEP ? bet[KEEP ? i : 0] : ld_const<T, VEC>(be + i * TPR), b);
          fma_v<VEC>(x[i], x[i], g, b);
        }
        y[i * TPR] = pack<T, VEC>(x[i]);
      }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// Rows too long for registers: one block a row, which is read three times.
template <typename T, int VEC>
__global__ void __launch_bounds__(MAX_TPR) layernorm_streamed_kernel(LayerNormParams p) {
  __shared__ float sh[32][1];
  const int nv = p.C / VEC;
  using P = typename PackOf<T, VEC>::type;
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(p.X) + (long long)blockIdx.x * p.ldx);
  P* y = reinterpret_cast<P*>(static_cast<T*>(p.Y) + (long long)blockIdx.x * p.ldy);
  Reducer red(sh, (int)blockDim.x);
  const float inv_c = 1.0f / (float)p.C;
  float s = 0.f, f[VEC], g[VEC], b[VEC];
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    unpack<T, VEC>(x[c], f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += f[j];
  }
  const float mean = mean_of(red.sum1(s), (float)p.C, inv_c);
  s = 0.f;
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    unpack<T, VEC>(x[c], f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(f[j] - mean, f[j] - mean, s);
  }
  const float rstd = 1.0f / sqrtf(red.sum1(s) * inv_c + p.eps);
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    unpack<T, VEC>(x[c], f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = (f[j] - mean) * rstd;
    if (p.gamma) {
      unpack<T, VEC>(static_cast<const P*>(p.gamma)[c], g);
      unpack<T, VEC>(static_cast<const P*>(p.beta)[c], b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = fmaf(f[j], g[j], b[j]);
    }
    y[c] = pack<T, VEC>(f);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mean;
    if (p.rstd) p.rstd[blockIdx.x] = rstd;
  }
}

// ------------------------------------------------------------------ backward
// dgamma and dbeta add up in registers over a group's rows, then over the
// groups of a block in group order (shared memory), one partial a block.  A
// group takes R rows a round, whose reductions share their steps and barrier.
template <typename T, int VEC, int PER, int R>
__global__ void __launch_bounds__(MAX_TPR) layernorm_grad_kernel(LayerNormGradParams p, int tpr) {
  __shared__ float sh[32][2 * R];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int rpb = blockDim.x / tpr, t = threadIdx.x % tpr, g0 = threadIdx.x / tpr;
  const int left = p.C / VEC - t;   // pack i is the row's while i tpr < left
  using P = typename PackOf<T, VEC>::type;
  using RowRing = Ring<P, PER, 2 * R>;
  const RowRing ring{smem_u32(ring_raw)};
  const float inv_c = 1.0f / (float)p.C;
  // gamma in registers, where they hold it: 16 one-element packs of float32
  // spill with it (4608 x 5002: 325 us, 120 without; in 16 bits 94 with it, 115)
  constexpr bool KEEP = PER * VEC <= (VEC == 1 && sizeof(T) == 4 ? 8 : 16);
  const P* ga = static_cast<const P*>(p.gamma);
  float ag[PER][VEC], ab[PER][VEC], gam[KEEP ? PER : 1][VEC];
  grid_launch_dependents();
  grid_dependency_wait();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[i][j] = ab[i][j] = 0.f;
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) gam[i][j] = 1.f;
      if (ga && i * tpr < left) unpack<T, VEC>(ld_const<T, VEC>(ga + t + i * tpr), gam[i]);
    }
  }
  // round k of this group: rows row + r stride, r < R
  const long long stride = (long long)gridDim.x * rpb, round = R * stride;
  long long row = (long long)blockIdx.x * rpb + g0, ahead = row;
  auto x_of = [&](long long r) { return reinterpret_cast<const P*>(static_cast<const T*>(p.X) + r * p.ldx) + t; };
  auto dy_of = [&](long long r) { return reinterpret_cast<const P*>(static_cast<const T*>(p.dY) + r * p.lddy) + t; };
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long m = ahead + r * stride;
      if (m < p.M) {
        const P *x = x_of(m), *d = dy_of(m);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * tpr < left) {
            ring.copy(stage, 2 * r, i, x + i * tpr);
            ring.copy(stage, 2 * r + 1, i, d + i * tpr);
          }
      }
    }
    cp_commit();
    ahead += round;
  };
  P ax[R][RowRing::ON ? 1 : PER], ad[R][RowRing::ON ? 1 : PER];
  auto load = [&](long long m0) {   // one-element packs of a round
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (m0 + r * stride < p.M) {
        const P *x = x_of(m0 + r * stride), *d = dy_of(m0 + r * stride);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * tpr < left) {
            ax[r][i] = x[i * tpr];
            ad[r][i] = d[i * tpr];
          }
      }
  };
  if constexpr (RowRing::ON) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d);
  } else {
    load(row);
  }
  float next_mean[R], next_rstd[R];
  auto fetch_stats = [&](long long m0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (m0 + r * stride < p.M) {
        next_mean[r] = p.mean[m0 + r * stride];
        next_rstd[r] = p.rstd[m0 + r * stride];
      }
  };
  fetch_stats(row);
  int stage = 0, buf = 0;
  // every group of a block runs the same number of rounds (the reductions' barriers)
  for (long long base = (long long)blockIdx.x * rpb; base < p.M; base += round, row += round) {
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = next_mean[r];
      rstd[r] = next_rstd[r];
    }
    fetch_stats(row + round);
    if (RowRing::ON) cp_wait_oldest();
    float xh[R][PER][VEC], g[R][PER][VEC];   // normalized values; dy, then dy gamma
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 s0 = both(0.f), s1 = both(0.f);
      const bool live = row + r * stride < p.M;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (live && i * tpr < left) {
          if constexpr (RowRing::ON) {
            unpack<T, VEC>(ring.get(stage, 2 * r, i), xh[r][i]);
            unpack<T, VEC>(ring.get(stage, 2 * r + 1, i), g[r][i]);
          } else {
            unpack<T, VEC>(ax[r][i], xh[r][i]);
            unpack<T, VEC>(ad[r][i], g[r][i]);
          }
          add_s<VEC>(xh[r][i], xh[r][i], -mean[r]);
          mul_s<VEC>(xh[r][i], xh[r][i], rstd[r]);
          fma_v<VEC>(ag[i], g[r][i], xh[r][i], ag[i]);
          add_v<VEC>(ab[i], g[r][i], ab[i]);
          if (KEEP) {
            mul_v<VEC>(g[r][i], g[r][i], gam[i]);
          } else if (ga) {
            float w[VEC];
            unpack<T, VEC>(ld_const<T, VEC>(ga + t + i * tpr), w);
            mul_v<VEC>(g[r][i], g[r][i], w);
          }
          add_to<VEC>(s0, g[r][i]);
          fma_to<VEC>(s1, g[r][i], xh[r][i]);
        }
      s[2 * r] = s0.x + s0.y;
      s[2 * r + 1] = s1.x + s1.y;
    }
    group_sums<2 * R>(s, sh, tpr, buf);
    if constexpr (RowRing::ON) {   // the slots have been read: the sums above needed their values
      fetch(stage);
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    } else {
      load(row + round);
    }
    if (p.dX) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row + r * stride >= p.M) continue;
        P* dst = reinterpret_cast<P*>(static_cast<T*>(p.dX) + (row + r * stride) * p.lddx) + t;
        const float a = s[2 * r] * inv_c;
        float b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = -s[2 * r + 1] * inv_c;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * tpr < left) {
            add_s<VEC>(g[r][i], g[r][i], -a);
            fma_v<VEC>(g[r][i], xh[r][i], b, g[r][i]);
            mul_s<VEC>(g[r][i], g[r][i], rstd[r]);
            dst[i * tpr] = pack<T, VEC>(g[r][i]);
          }
      }
    }
  }
  if (!p.part_g) return;
  float* comb = reinterpret_cast<float*>(ring_raw);   // [2][C] when a block holds several rows; the ring is done with
  if (rpb > 1) __syncthreads();
  for (int q = 0; q < rpb; ++q) {   // the block's groups in order; the last one writes
    if (g0 == q) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * tpr < left) {
          const int col = (t + i * tpr) * VEC;
          float* cg = comb + col;
          float* cb = comb + p.C + col;
          if (q > 0)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              ag[i][j] += cg[j];
              ab[i][j] += cb[j];
            }
          if (q + 1 == rpb) {
            cg = p.part_g + (size_t)blockIdx.x * p.C + col;
            cb = p.part_b + (size_t)blockIdx.x * p.C + col;
          }
          if constexpr (VEC > 1) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
              *reinterpret_cast<float4*>(cg + j) = make_float4(ag[i][j], ag[i][j + 1], ag[i][j + 2], ag[i][j + 3]);
              *reinterpret_cast<float4*>(cb + j) = make_float4(ab[i][j], ab[i][j + 1], ab[i][j + 2], ab[i][j + 3]);
            }
          } else {
            cg[0] = ag[i][0];
            cb[0] = ab[i][0];
          }
        }
    }
    if (rpb > 1) __syncthreads();
  }
}

// Rows too long for registers: dX by reading x and dy twice, one block a row ...
template <typename T>
__global__ void __launch_bounds__(MAX_TPR) layernorm_grad_rows_kernel(LayerNormGradParams p) {
  __shared__ float sh[32][2];
  const T* x = static_cast<const T*>(p.X) + (long long)blockIdx.x * p.ldx;
  const T* dy = static_cast<const T*>(p.dY) + (long long)blockIdx.x * p.lddy;
  T* dx = static_cast<T*>(p.dX) + (long long)blockIdx.x * p.lddx;
  const T* ga = static_cast<const T*>(p.gamma);
  const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x], inv_c = 1.0f / (float)p.C;
  int buf = 0;
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    const float xh = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * (ga ? to_f32(ga[c]) : 1.f);
    s[0] += g;
    s[1] = fmaf(g, xh, s[1]);
  }
  group_sums<2>(s, sh, (int)blockDim.x, buf);
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
  const int r0 = (int)((long long)p.M * blockIdx.y / gridDim.y);
  const int r1 = (int)((long long)p.M * (blockIdx.y + 1) / gridDim.y);
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

// Launches a walk over the rows: as many blocks as the SMs hold at once, at
// most `most`.
template <typename Params, typename... Args>
cudaError_t walk(void (*kern)(Params, Args...), const Params& p, int block, int rpb, size_t smem, int most, int* blocks,
                 cudaStream_t st, Args... args) {
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  int grid = (p.M + rpb - 1) / rpb;
  if (grid > 148) {
    int per_sm = 1;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, block, smem);
    if (e != cudaSuccess) return e;
    if (grid > 148 * per_sm) grid = 148 * (per_sm > 0 ? per_sm : 1);
  }
  if (grid > most) grid = most;
  *blocks = grid;
  return launch_early(kern, dim3(grid), block, smem, st, p, args...);
}

// 148 here and in the grids' sizes is the SM count of a B200 (the workspace's
// size is asked for without a device); another count changes times alone.
constexpr int FEW_ROWS = 148 * 4;

template <typename T, int VEC, int TPR, int PER>
cudaError_t forward_as(const LayerNormParams& p, cudaStream_t st) {
  constexpr int BLOCK = BLOCK_OF<TPR>;
  constexpr size_t RING = (size_t)BLOCK * Ring<typename PackOf<T, VEC>::type, PER, 1>::BYTES;
  int blocks;
  return walk<LayerNormParams>(layernorm_kernel<T, VEC, TPR, PER>, p, BLOCK, BLOCK / TPR, RING, 1 << 30, &blocks, st);
}

// Up to four 16-byte packs a thread in 64 registers (1024 threads a SM): more
// values a thread share a reduction's cost, more threads hide its latency.
// Measured, 16384 x 3072 bf16: 3 packs x 128 threads 35.5 us, 6 x 64 39.9,
// 12 x 32 (no barrier at all, 12 warps a SM) 49.9; 4608 x 3072 fp32: 3 packs
// x 256 threads 20.8 us, 2 x 512 25.6 (one-element packs lose by 256: 4608 x
// 3001 fp16 28.8 us for 26.5).  One-element packs: up to 16 a thread.  Few rows
// take fewer packs and more threads, for latency.
template <typename T, int VEC, int TPR>
cudaError_t forward_packs(const LayerNormParams& p, int nv, cudaStream_t st) {
  if (nv <= TPR) return forward_as<T, VEC, TPR, 1>(p, st);
  if (nv <= 2 * TPR) return forward_as<T, VEC, TPR, 2>(p, st);
  if constexpr (VEC == 1) {
    if (nv > 8 * TPR) return forward_as<T, VEC, TPR, 16>(p, st);
    if (nv > 4 * TPR) return forward_as<T, VEC, TPR, 8>(p, st);
  } else {
    if (nv <= 3 * TPR) return forward_as<T, VEC, TPR, 3>(p, st);
  }
  return forward_as<T, VEC, TPR, 4>(p, st);
}
template <typename T, int VEC>
cudaError_t forward(const LayerNormParams& p, cudaStream_t st) {
  constexpr int MOST = VEC == 1 ? 16 : 4;
  const int nv = p.C / VEC, want = p.M <= FEW_ROWS ? (VEC == 1 ? 2 : 1) : MOST;   // packs a thread
  if (nv <= 32 * want) return forward_packs<T, VEC, 32>(p, nv, st);
  if (nv <= 128 * want) return forward_packs<T, VEC, 128>(p, nv, st);
  if constexpr (VEC > 1)
    if (nv <= 256 * want) return forward_packs<T, VEC, 256>(p, nv, st);
  if (nv <= 512 * MOST) return forward_packs<T, VEC, 512>(p, nv, st);
  if (VEC > 1 && nv <= 512 * 8) return forward_as<T, VEC, 512, 8>(p, st);
  layernorm_streamed_kernel<T, VEC><<<p.M, MAX_TPR, 0, st>>>(p);
  return cudaGetLastError();
}

// One 16-byte pack a thread and two rows a round while 512 threads cover the
// row (two sums per column, gamma and two rows' values in registers; measured,
// 16384 x 3072 bf16 with the weights' gradients: 61.0 us, one row a round
// 65.4, two packs and one row 63.4, two packs and two rows, which leave room
// for fewer threads, 98.8), more packs and one row a round for longer rows.
// Eight one-element packs: one row (8192 x 1001 fp16 25.9, two 27.4; 900 x 3001
// 12.4, 14.1; 4608 x 3001 49.8, 46.3).
template <typename T, int VEC, int PER>
cudaError_t backward_as(const LayerNormGradParams& p, int most, int* parts, cudaStream_t st) {
  constexpr int R = PER * VEC <= (VEC == 1 ? 4 : 8) ? 2 : 1;
  const int nv = p.C / VEC, tpr = ((nv + PER - 1) / PER + 31) / 32 * 32;
  const int block = tpr >= SMALL_BLOCK ? tpr : SMALL_BLOCK / tpr * tpr;
  const size_t ring = (size_t)block * Ring<typename PackOf<T, VEC>::type, PER, 2 * R>::BYTES;
  const size_t comb = block > tpr ? (size_t)p.C * 8 : 0;   // tpr <= 64 then: at most 8 KB
  return walk<LayerNormGradParams, int>(layernorm_grad_kernel<T, VEC, PER, R>, p, block, block / tpr,
                                        ring > comb ? ring : comb, most, parts, st, tpr);
}
template <typename T, int VEC>
cudaError_t backward(const LayerNormGradParams& p, int* parts, cudaStream_t st) {
  const int nv = p.C / VEC, most = layernorm_grad_parts(p.M, p.C);
  if constexpr (VEC == 1) {
    if (nv <= (p.M <= FEW_ROWS ? 2 * MAX_TPR : 64)) return backward_as<T, VEC, 2>(p, most, parts, st);
    if (nv <= 8 * MAX_TPR) return backward_as<T, VEC, 8>(p, most, parts, st);
    if (nv <= 16 * MAX_TPR) return backward_as<T, VEC, 16>(p, most, parts, st);
  } else {
    if (nv <= MAX_TPR) return backward_as<T, VEC, 1>(p, most, parts, st);
    if (nv <= 2 * MAX_TPR) return backward_as<T, VEC, 2>(p, most, parts, st);
    if (nv <= 3 * MAX_TPR) return backward_as<T, VEC, 3>(p, most, parts, st);
  }
  if (p.dX) {
    layernorm_grad_rows_kernel<T><<<p.M, MAX_TPR, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  *parts = most < 64 ? most : 64;
  if (p.part_g)
    layernorm_grad_cols_kernel<T><<<dim3((p.C + MAX_TPR - 1) / MAX_TPR, *parts), MAX_TPR, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_any(const LayerNormParams& p, cudaStream_t st) {
  return vectors<T>(p.C, {p.X, p.Y, p.gamma, p.beta}, {p.ldx, p.ldy}) ? forward<T, 16 / sizeof(T)>(p, st)
                                                                     : forward<T, 1>(p, st);
}
template <typename T>
cudaError_t backward_any(const LayerNormGradParams& p, int* parts, cudaStream_t st) {
  return vectors<T>(p.C, {p.X, p.dY, p.dX, p.gamma}, {p.ldx, p.lddy, p.lddx})
             ? backward<T, 16 / sizeof(T)>(p, parts, st)
             : backward<T, 1>(p, parts, st);
}

}  // namespace

// Partials: at most one a block of the walk over the rows.
int layernorm_grad_parts(int M, int C) {
  const int most = 148 * (C <= 1024 ? 8 : 4);
  return M < most ? M : most;
}

cudaError_t launch_layernorm(const LayerNormParams& p, cudaStream_t st) {
  switch (p.dt) {
    case SVDQ_BF16: return forward_any<__nv_bfloat16>(p, st);
    case SVDQ_FP16: return forward_any<__half>(p, st);
    default: return forward_any<float>(p, st);
  }
}
cudaError_t launch_layernorm_grad(const LayerNormGradParams& p, int* parts, cudaStream_t st) {
  switch (p.dt) {
    case SVDQ_BF16: return backward_any<__nv_bfloat16>(p, parts, st);
    case SVDQ_FP16: return backward_any<__half>(p, parts, st);
    default: return backward_any<float>(p, parts, st);
  }
}

}  // namespace svdq
