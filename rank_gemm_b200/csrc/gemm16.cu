// gemm16.cu -- matrix products of 16-bit operands (bf16 or fp16) on the
// 5th-generation tensor core: the dense linear with its bias / activation /
// residual epilogue, the gated feed-forward projection, and the products of
// their backward passes.
//
//   D[m][n] = sum_k A[m][k] B[n][k], float32 accumulation in TMEM,
//   linear:  z = D + b_n;  Y = act(z) + R;  Z = z (kept for the backward pass)
//   gated:   g = D_g + bg_n, u = D_u + bu_n;  H = act(g) u;  G = g, U = u
//   each output rounded once from float32.
//
// One kernel template, warp-specialised: warp 0 feeds a ring of k-tiles
// (64 wide) by TMA, warp 1 issues the MMAs from one thread, the other warps
// drain the accumulators.
//   pair form (CG = 2)    a CTA pair shares one 256 x BN tile
//                         (tcgen05.mma.cta_group::2): each CTA stages its 128
//                         rows of A and its half of B, so an operand byte is
//                         fetched into shared memory once per pair; the two
//                         float32 accumulators of TMEM alternate, so the
//                         epilogue of one tile runs under the next one's MMAs.
//   swapped form (SWAP)   for few rows of X (tokens): the weight is the
//                         128-row operand and the tokens are the MMA's N
//                         (16 .. 128), so a token batch does not fill a
//                         128-row tile with zeros and the weights stream once.
// Operands may be stored with the reduction index innermost (K-major) or
// outermost (MN-major, the tensor core transposes as it reads), so the
// backward products read dZ, X and W as they lie: no transposed copies.
// Gated: the pair form stages 128 features of both weights as one B tile
// (accumulator columns 0-127 are g, 128-255 u), so X is read once; the
// swapped form stages two A tiles.
// Few tiles: the reduction is split over the CTAs of a cluster, whose float32
// partial tiles are summed in rank order through distributed shared memory
// (no workspace, no atomics, the same bits on every run).
// Outputs of whole tiles leave through shared memory, a 32-row box of 128-byte
// rows per warp and TMA store, so they reach L2 as full lines.
// All waits are bounded (mbar_wait); TMEM is freed on every exit path.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace svdq {

namespace {

constexpr int BK = 64;                       // one 128-byte swizzled row of 16-bit values
constexpr int SMEM_LIMIT = 232448;           // 227 KB
constexpr int MAX_STAGES = 8;

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], t_full[2], t_empty[2];
  uint32_t tmem_base;
  int abort;
};

constexpr int pow2_at_least(int x, int lo) { return x <= lo ? lo : pow2_at_least(x, 2 * lo); }

template <int CG, int BN, bool SWAP, bool GATED>
struct Cfg {
  static constexpr int A_TILES = (SWAP && GATED) ? 2 : 1;
  static constexpr int A_TILE_BYTES = 128 * BK * 2;
  static constexpr int A_BYTES = A_TILES * A_TILE_BYTES;
  static constexpr int B_ROWS = BN / CG;                  // per CTA
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int OUT_COLS = (GATED && !SWAP) ? BN / 2 : BN;   // output columns of a tile
  static constexpr int BOX_COLS = OUT_COLS / 2 < 64 ? OUT_COLS / 2 : 64;   // pair form: columns of a store box
  static constexpr int EPI_WARPS = SWAP ? 4 : 8;          // one or two per TMEM sub-partition
  static constexpr int PARK = SWAP ? 0 : EPI_WARPS * 32 * BOX_COLS * 2;   // one store box a warp
  static constexpr int ROOM = (SMEM_LIMIT - 1024 - PARK - (int)sizeof(Ctl)) / STAGE;
  static constexpr int STAGES = ROOM < MAX_STAGES ? ROOM : MAX_STAGES;
  static constexpr int ACC_COLS = A_TILES * BN;
  static constexpr int TMEM_COLS = pow2_at_least(2 * ACC_COLS, 32);
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + PARK + sizeof(Ctl);
  static_assert(STAGE % 1024 == 0, "tiles stay 1024-byte aligned for the 128-byte swizzle");
  static_assert(TMEM_COLS <= 512 && STAGES >= 3, "TMEM or ring too small");
  static_assert(ACC_COLS * 512 <= STAGES * STAGE, "a split's partial tile fits the ring");
};

// ------------------------------------------------------------------ PTX forms this kernel adds
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Load into this CTA's shared memory, completing on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int x, int y, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}
// Store of a box from shared memory; rows and columns past the tensor are left out.
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void tc_alloc(uint32_t dst_smem, uint32_t ncols) {
  if (CG == 1) {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tc_dealloc(uint32_t taddr, uint32_t ncols) {
  if (CG == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on the barrier at the same place in both CTAs of the pair (mask).
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CG == 1)
    mma_bf16(d_tmem, a, b, idesc, accumulate);   // the operand type is the descriptor's
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Tile of one operand, k step j (16 wide).  K-major: 128-byte rows, 8-row
// groups 1024 bytes apart, a step 32 bytes into the row.  MN-major: boxes of
// 64 (MN) x 64 (k), a k row of 64 MN values per 128-byte line, 8-k groups
// 1024 bytes apart, the next 64 MN values one box (8 KB) on, a step 16 lines.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t tile, int j) {
  return MN ? smem_desc(tile + 2048 * j, 8192, 1024, 2) : desc_k_sw128(tile + 32 * j);
}

// ------------------------------------------------------------------ epilogue arithmetic
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float load16(const uint16_t* p, bool fp16) {
  return unpack16((uint32_t)ld_nc(p), fp16).x;
}
__device__ __forceinline__ uint16_t round16(float v, bool fp16) { return (uint16_t)pack16(v, 0.f, fp16); }

// Eight consecutive columns of one row: v += bias.
__device__ __forceinline__ void add_bias8(float (&v)[8], const uint16_t* bias, int n, bool fp16) {
  if (!bias) return;
  const uint4 b = ld_nc(reinterpret_cast<const uint4*>(bias + n));
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16(w[i], fp16);
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}
__device__ __forceinline__ uint4 round8(const float (&v)[8], bool fp16) {
  return make_uint4(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16), pack16(v[4], v[5], fp16),
                    pack16(v[6], v[7], fp16));
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], bool fp16) {
  *reinterpret_cast<uint4*>(p) = round8(v, fp16);
}
__device__ __forceinline__ void add8(float (&v)[8], const uint4& r, bool fp16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16(w[i], fp16);
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}
__device__ __forceinline__ void act8(float (&v)[8], int act) {
  if (act == SVDQ_EPI_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = gelu_tanh(v[i]);
  } else if (act == SVDQ_EPI_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu(v[i]);
  }
}

}  // namespace

template <int CG, int BN, bool SWAP, bool GATED, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(Cfg<CG, BN, SWAP, GATED>::THREADS, 1)
    gemm16_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                  const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                  const __grid_constant__ CUtensorMap tmZ2, Gemm16Params p) {
  using C = Cfg<CG, BN, SWAP, GATED>;
  constexpr int OUT_COLS = C::OUT_COLS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* park = ring + C::STAGES * C::STAGE;
  Ctl* ctl = reinterpret_cast<Ctl*>(park + C::PARK);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cta = CG == 2 ? (int)(rank & 1) : 0;             // CTA of the pair
  const int split = (int)rank / CG, S = p.splits;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ctl->t_full[s]), 1);
      mbar_init(smem_u32(&ctl->t_empty[s]), CG * C::EPI_WARPS);
    }
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc_alloc<CG>(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
  tc_fence_before();
  if (CG * S > 1)
    cluster_sync_all();   // the other CTAs' barriers are set up before anything signals them
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  // The next kernel may be scheduled as SMs fall idle; this one touches
  // global memory only after the previous kernel's writes are visible.
  grid_launch_dependents();
  if (warp != 1) grid_dependency_wait();

  const int num_tiles = p.tiles_m * p.tiles_n;
  const int first = (int)blockIdx.x / (CG * S), step = (int)gridDim.x / (CG * S);
  const int kt0 = (int)((long long)p.nk * split / S), kt1 = (int)((long long)p.nk * (split + 1) / S);
  // tiles run down groups of 8 row blocks, so the tiles in flight share rows
  // of A and columns of B in L2
  auto coords = [&](int tile, int& mb, int& nb) {
    constexpr int GROUP = 8;
    const int per = GROUP * p.tiles_n, g = tile / per, r = tile - g * per;
    const int rows = min(GROUP, p.tiles_m - g * GROUP);
    mb = g * GROUP + r % rows;
    nb = r / rows;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < num_tiles; tile += step) {
        int mb, nb;
        coords(tile, mb, nb);
        const bool second = mb >= p.tiles_m1;                 // the second of two stacked A operands
        const int a_row = (second ? mb - p.tiles_m1 : mb) * 128 * CG + cta * 128;
        const int b_row = (GATED && !SWAP) ? nb * OUT_COLS : nb * BN + cta * C::B_ROWS;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!mbar_wait(smem_u32(&ctl->empty[stage]), phase ^ 1, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const bool seg = kt >= p.nk1;                       // the second part of a two-part reduction
          const int k = (seg ? kt - p.nk1 : kt) * BK;
          const uint32_t a = smem_u32(ring + stage * C::STAGE), b = a + C::A_BYTES;
          const uint32_t bar = smem_u32(&ctl->full[stage]);
          const uint32_t sig = CG == 2 ? dsmem_map(bar, rank & ~1u) : bar;
          if (cta == 0) mbar_arrive_expect_tx(bar, CG * C::STAGE);
          auto load = [&](uint32_t dst, const CUtensorMap* m, int x, int y) {
            if (CG == 2)
              tma_load_2d_pair(dst, m, x, y, sig);
            else
              tma_load_2d(dst, m, x, y, sig);
          };
          auto load_tile = [&](uint32_t dst, const CUtensorMap* m, bool mn, int rows, int row) {
            if (!mn) {
              load(dst, m, k, row);
            } else {
              for (int i = 0; i < rows; i += 64) load(dst + i * 128, m, row + i, k);
            }
          };
          const CUtensorMap* ma = (second || seg) ? &tmA1 : &tmA0;
          load_tile(a, ma, A_MN, 128, a_row);
          if (C::A_TILES == 2) load_tile(a + C::A_TILE_BYTES, &tmA1, A_MN, 128, a_row);
          const bool b1 = (GATED && !SWAP) ? cta == 1 : seg;
          load_tile(b, b1 ? &tmB1 : &tmB0, B_MN, C::B_ROWS, b_row);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the pair's first CTA)
    if (lane == 0 && cta == 0) {
      const uint32_t idesc = (1u << 4) | (p.fp16 ? 0u : (1u << 7) | (1u << 10)) | (A_MN ? 1u << 15 : 0u) |
                             (B_MN ? 1u << 16 : 0u) | ((uint32_t)(BN >> 3) << 17) |
                             ((uint32_t)((128 * CG) >> 4) << 24);
      const uint16_t mask = (uint16_t)(3u << (rank & ~1u));
      auto commit = [&](uint64_t* bar) {
        if (CG == 2)
          tc_commit_pair(smem_u32(bar), mask);
        else
          tc_commit(smem_u32(bar));
      };
      int stage = 0;
      uint32_t phase = 0, tl = 0;
      bool ok = true;
      for (int tile = first; ok && tile < num_tiles; tile += step, ++tl) {
        const uint32_t ab = tl & 1, pt = (tl >> 1) & 1;
        if (!mbar_wait(smem_u32(&ctl->t_empty[ab]), pt ^ 1, abort_flag, p.err)) break;
        tc_fence_after();
        const uint32_t acc = tmem + ab * C::ACC_COLS;
        for (int kt = kt0; kt < kt1; ++kt) {
          if (!mbar_wait(smem_u32(&ctl->full[stage]), phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(ring + stage * C::STAGE), b = a + C::A_BYTES;
#pragma unroll
          for (int j = 0; j < BK / 16; ++j) {
            const uint64_t db = operand_desc<B_MN>(b, j);
#pragma unroll
            for (int t = 0; t < C::A_TILES; ++t)
              mma_f16<CG>(acc + t * BN, operand_desc<A_MN>(a + t * C::A_TILE_BYTES, j), db, idesc,
                          kt != kt0 || j != 0);
          }
          commit(&ctl->empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        commit(&ctl->t_full[ab]);
      }
    }
  }

  // -------------------------------------------------------------- epilogue
  const int e = warp - 2, sub = warp & 3;
  const int row = sub * 32 + lane;                            // TMEM lane: row of this CTA's 128
  const bool fp16 = p.fp16 != 0;

  // Eight columns n .. n + 7 of row m (pair form), r the residual's.
  auto emit8 = [&](uint16_t* out, int m, int n, float (&v)[8], float (&u)[8], const uint4& r) {
    add_bias8(v, p.bias, n, fp16);
    if (GATED) add_bias8(u, p.bias2, n, fp16);
    const size_t at = (size_t)m * p.N + n;
    if (p.Z) store8(p.Z + at, v, fp16);
    if (GATED && p.Z2) store8(p.Z2 + at, u, fp16);
    act8(v, p.act);
    if (GATED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= u[i];
    } else if (p.R) {
      add8(v, r, fp16);
    }
    store8(out + (size_t)m * p.ldy + n, v, fp16);
  };
  // The residual of eight columns; the pointers may be Y's own, so it is
  // loaded before anything of its chunk is stored.
  auto residual8 = [&](int m, int n) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if (!GATED && p.R && m < p.M && n < p.N) r = *reinterpret_cast<const uint4*>(p.R + (size_t)m * p.ldr + n);
    return r;
  };
  // COUNT tokens m0, m0 + step, ... of feature n (swapped form): a warp's
  // lanes are 32 consecutive features.
  float bias_v = 0.f, bias_u = 0.f;
  auto load_bias = [&](int n) {
    if (n < p.N) {
      if (p.bias) bias_v = load16(p.bias + n, fp16);
      if (GATED && p.bias2) bias_u = load16(p.bias2 + n, fp16);
    }
  };
  auto emit_tokens = [&](int m0, int step, int n, const float* v, const float* u, auto count) {
    constexpr int COUNT = decltype(count)::value;
    float r[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int m = m0 + i * step;
      r[i] = (!GATED && p.R && m < p.M && n < p.N) ? unpack16((uint32_t)p.R[(size_t)m * p.ldr + n], fp16).x : 0.f;
    }
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int m = m0 + i * step;
      if (m >= p.M || n >= p.N) continue;
      float f = v[i] + bias_v;
      const float g = GATED ? u[i] + bias_u : 0.f;
      const size_t at = (size_t)m * p.N + n;
      if (p.Z) p.Z[at] = round16(f, fp16);
      if (GATED && p.Z2) p.Z2[at] = round16(g, fp16);
      if (p.act == SVDQ_EPI_GELU_TANH) f = gelu_tanh(f);
      if (p.act == SVDQ_EPI_SILU) f = silu(f);
      f = GATED ? f * g : f + r[i];
      p.Y[(size_t)m * p.ldy + n] = round16(f, fp16);
    }
  };

  if (warp >= 2 && S == 1) {
    uint32_t tl = 0;
    for (int tile = first; tile < num_tiles; tile += step, ++tl) {
      int mb, nb;
      coords(tile, mb, nb);
      const bool second = mb >= p.tiles_m1;
      const int row0 = (second ? mb - p.tiles_m1 : mb) * 128 * CG + cta * 128;
      const uint32_t ab = tl & 1, pt = (tl >> 1) & 1;
      const int m = row0 + row;                               // pair form: row; swapped: feature
      if (SWAP) load_bias(m);
      // pair form: this warp's 32 rows, columns c0 .. c0 + PER - 1 of the tile, in boxes of W
      constexpr int PER = OUT_COLS / 2, W = C::BOX_COLS;
      const int c0 = (e >> 2) * PER, n_tile = nb * OUT_COLS, row_w = row0 + sub * 32;
      uint4 res[2];
      if (!SWAP) {
        res[0] = residual8(m, n_tile + c0);
        res[1] = residual8(m, n_tile + c0 + 8);
      }
      if (!mbar_wait(smem_u32(&ctl->t_full[ab]), pt, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16) + ab * C::ACC_COLS;
      if (!SWAP) {
        const uint32_t box = smem_u32(park) + (uint32_t)e * (32 * W * 2);
        // one output of a W-column box: what(v, u, n, res) turns eight columns' accumulators into its values
        auto emit_box = [&](const CUtensorMap* map, int c, bool last, auto what) {
          if (lane == 0) bulk_wait_read();   // the previous box has left shared memory
          __syncwarp();
#pragma unroll 1
          for (int d = 0; d < W; d += 16) {
            uint32_t r[16], q[16];
            tmem_ld16(taddr + c + d, r);
            if (GATED) tmem_ld16(taddr + BN / 2 + c + d, q);
            const uint4 now[2] = {res[0], res[1]};
            if (last && c + d + 16 < c0 + PER) {
              res[0] = residual8(m, n_tile + c + d + 16);
              res[1] = residual8(m, n_tile + c + d + 24);
            }
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[8], u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v[i] = __uint_as_float(r[8 * h + i]);
                u[i] = GATED ? __uint_as_float(q[8 * h + i]) : 0.f;
              }
              const int n = n_tile + c + d + 8 * h;
              if (n < p.N) {
                add_bias8(v, p.bias, n, fp16);
                if (GATED) add_bias8(u, p.bias2, n, fp16);
              }
              what(v, u, now[h]);
              const int chunk = (d >> 3) + h;   // 16-byte chunk of the row, swizzled as the box's map
              const uint32_t at = W == 64 ? lane * 128 + ((chunk ^ (lane & 7)) << 4)
                                          : lane * 64 + ((chunk ^ ((lane >> 1) & 3)) << 4);
              sts128(box + at, round8(v, fp16));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row_w < p.M && n_tile + c < p.N) tma_store_2d(map, box, n_tile + c, row_w);
        };
#pragma unroll 1
        for (int c = c0; c < c0 + PER; c += W) {
          if (p.Z) emit_box(&tmZ, c, false, [&](float (&)[8], float (&)[8], const uint4&) {});
          if (GATED && p.Z2)
            emit_box(&tmZ2, c, false, [&](float (&v)[8], float (&u)[8], const uint4&) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = u[i];
            });
          emit_box(!GATED && second ? &tmZ2 : &tmY, c, true, [&](float (&v)[8], float (&u)[8], const uint4& r) {
            act8(v, p.act);
            if (GATED) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] *= u[i];
            } else if (p.R) {
              add8(v, r, fp16);
            }
          });
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < BN && nb * BN + c < p.M; c += 16) {
          uint32_t r[16], q[16];
          tmem_ld16(taddr + c, r);
          if (GATED) tmem_ld16(taddr + BN + c, q);
          tmem_wait_ld();
          emit_tokens(nb * BN + c, 1, m, reinterpret_cast<const float*>(r), reinterpret_cast<const float*>(q),
                      std::integral_constant<int, 16>{});
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(dsmem_map(smem_u32(&ctl->t_empty[ab]), rank & ~1u));
        else
          mbar_arrive(smem_u32(&ctl->t_empty[ab]));
      }
    }
    if (!SWAP && lane == 0) bulk_wait_all();
  }
  if (S > 1) {
    // One tile per cluster: every CTA parks its float32 partial in its own
    // ring (free: all of its MMAs are complete) as [column][128 rows], and
    // rank s sums columns s, s + S, ... (blocks of 8 in the pair form) of all
    // ranks in rank order, eight loads in flight a thread.
    const uint32_t part = smem_u32(ring);
    int mb, nb;
    coords(first, mb, nb);
    const bool second = mb >= p.tiles_m1;
    const int m = (second ? mb - p.tiles_m1 : mb) * 128 * CG + cta * 128 + row;
    bool ok = false;
    if (warp >= 2) {
      if (SWAP) load_bias(m);
      ok = mbar_wait(smem_u32(&ctl->t_full[0]), 0, abort_flag, p.err);
      if (ok) {
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16);
        for (int c = (e >> 2) * 16; c < C::ACC_COLS; c += 16 * (C::EPI_WARPS / 4)) {
          if (SWAP && nb * BN + (c & (BN - 1)) >= p.M) continue;   // columns past the last token
          uint32_t r[16];
          tmem_ld16(taddr + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) sts_f32(part + ((c + i) * 128 + row) * 4, __uint_as_float(r[i]));
        }
        tc_fence_before();
      }
    }
    cluster_sync_all();
    if (warp >= 2 && ok) {
      // columns col, col + step, ... (8, none past `last`) summed over the ranks
      auto totals = [&](int col, int step, int last, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        for (int s = 0; s < S; ++s) {
          const uint32_t from = dsmem_map(part + row * 4, s * CG + cta);
          float t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = ld_dsmem_f32(from + min(col + i * step, last) * 512);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += t[i];
        }
      };
      if (!SWAP) {
        uint16_t* out = second ? p.Y2 : p.Y;
        for (int b = (e >> 2) * S + split; b < OUT_COLS / 8; b += 2 * S) {
          const int n = nb * OUT_COLS + 8 * b;
          if (m < p.M && n < p.N) {
            const uint4 res = residual8(m, n);
            float v[8], u[8];
            totals(8 * b, 1, C::ACC_COLS - 1, v);
            if (GATED) totals(BN / 2 + 8 * b, 1, C::ACC_COLS - 1, u);
            emit8(out, m, n, v, u, res);
          }
        }
      } else {
        for (int c = split; c < BN && nb * BN + c < p.M; c += 8 * S) {
          float v[8], u[8];
          totals(c, S, BN - 1, v);
          if (GATED) totals(BN + c, S, 2 * BN - 1, u);
          // fewer than 8 of this rank's columns are left in the tile: one by one
          const int left = (BN - c + S - 1) / S;
          if (left >= 8)
            emit_tokens(nb * BN + c, S, m, v, u, std::integral_constant<int, 8>{});
          else
            for (int i = 0; i < 8; ++i)
              if (i < left) emit_tokens(nb * BN + c + i * S, 1, m, v + i, u + i, std::integral_constant<int, 1>{});
        }
      }
    }
  }

  tc_fence_before();
  if (CG * S > 1)
    cluster_sync_all();   // no CTA leaves while another reads its shared memory or signals its barriers
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc<CG>(tmem, C::TMEM_COLS);
  }
}

namespace {

template <int CG, int BN, bool SWAP, bool GATED, bool A_MN, bool B_MN>
cudaError_t launch(const CUtensorMap (&tm)[7], const Gemm16Params& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<CG, BN, SWAP, GATED>;
  auto kern = gemm16_kernel<CG, BN, SWAP, GATED, A_MN, B_MN>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)p.tiles_m * p.tiles_n;
  const int width = CG * p.splits;
  const long long most = p.splits > 1 ? tiles : num_sms / CG;   // a split cluster owns one tile
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * width));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = width;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], tm[6], p);
}

}  // namespace

cudaError_t launch_gemm16(const Gemm16Plan& plan, const CUtensorMap (&tm)[7], Gemm16Params p, int num_sms,
                          cudaStream_t stream) {
  p.splits = plan.splits;
  if (plan.swap) {
    switch (plan.op) {
#define SVDQ_SWAP(G, MN)                                                                 \
  switch (plan.bn) {                                                                     \
    case 16: return launch<1, 16, true, G, MN, false>(tm, p, num_sms, stream);           \
    case 32: return launch<1, 32, true, G, MN, false>(tm, p, num_sms, stream);           \
    case 64: return launch<1, 64, true, G, MN, false>(tm, p, num_sms, stream);           \
    case 128: return launch<1, 128, true, G, MN, false>(tm, p, num_sms, stream);         \
    default: return cudaErrorInvalidValue;                                               \
  }
      case GEMM16_NT: SVDQ_SWAP(false, false)
      case GEMM16_GATED: SVDQ_SWAP(true, false)
      case GEMM16_NN: SVDQ_SWAP(false, true)
      default: return cudaErrorInvalidValue;
#undef SVDQ_SWAP
    }
  }
#define SVDQ_PAIR(G, AMN, BMN)                                                           \
  return plan.bn == 256 ? launch<2, 256, false, G, AMN, BMN>(tm, p, num_sms, stream)     \
                        : launch<2, 128, false, G, AMN, BMN>(tm, p, num_sms, stream);
  switch (plan.op) {
    case GEMM16_NT: SVDQ_PAIR(false, false, false)
    case GEMM16_GATED: SVDQ_PAIR(true, false, false)
    case GEMM16_NN: SVDQ_PAIR(false, false, true)
    case GEMM16_TN: SVDQ_PAIR(false, true, true)
  }
#undef SVDQ_PAIR
  return cudaErrorInvalidValue;
}

}  // namespace svdq
