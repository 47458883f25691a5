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
// (64 wide) by TMA, warp 1 issues the MMAs, the other warps drain the
// accumulators.  The MMA warp runs its loop whole and elects a lane for each
// issue: state that is uniform over the warp reaches the instructions' uniform
// operands without a move, and that warp's instructions between two MMAs bound
// the shorter tiles (256 rows 3072 -> 9216: 17.5 us with a single-lane loop,
// 15.6 so).
//   pair form (CG = 2)    a CTA pair shares one 256 x BN tile
//                         (tcgen05.mma.cta_group::2): each CTA stages its 128
//                         rows of A and its half of B, so an operand byte is
//                         fetched into shared memory once per pair; the two
//                         float32 accumulators of TMEM alternate, so the
//                         epilogue of one tile runs under the next one's MMAs.
//   tall pair (TALL)      a 512 x 256 tile, two 256-row accumulators over the
//                         same B: a quarter less operand traffic per product.
//                         TMEM holds no second pair of accumulators, so the
//                         first and last k-tiles run for one accumulator and
//                         then for the other, while the epilogue drains or
//                         has drained the other one.
//   swapped form (SWAP)   for few rows of X (tokens): the weight is the
//                         128-row operand and the tokens are the MMA's N
//                         (16 .. 128), so a token batch does not fill a
//                         128-row tile with zeros and the weights stream once.
// Operands may be stored with the reduction index innermost (K-major) or
// outermost (MN-major, the tensor core transposes as it reads), so the
// backward products read dZ, X and W as they lie: no transposed copies.
// Gated: the pair form stages features of both weights as one B tile (the
// accumulator's lower columns are g, the upper u), so X is read once; the
// swapped form stages two A tiles.
// Backward (GRAD): dW and dX are two jobs of one launch, whose tiles share the
// pairs (one tail instead of two), and the bias gradients' partials are added
// by the epilogue warps before their first tile.
// Few tiles: the reduction is split over the CTAs of a cluster, whose float32
// partial tiles are summed in rank order through distributed shared memory
// (no workspace, no atomics, the same bits on every run).  A backward
// product of few tiles and a long reduction (few rows, or many rows of narrow
// layers) is cut into up to 32 parts that are tiles of their own: float32
// partials in the workspace, joined in order by join_parts_kernel.
// Outputs of whole tiles leave through shared memory, a 32-row box of 128-byte
// rows per warp (swapped: one box of 128 features) and TMA store, so they
// reach L2 as full lines.
// What bounds it.  Large products: the power cap (4608 x 3072 -> 9216: 164 us
// in a burst, 1590 TFLOP/s, tensor pipe 86% active at 1.58 GHz; 185 to 195 us
// back to back).  Middle sizes: operand bytes into shared memory, about 13
// TB/s over the chip (777 x 1160 -> 2056: 250 ns a k-tile on 136 SMs), and the
// fixed parts: launch 1 us, first operands 1 to 2 us, an epilogue that nothing
// overlaps 1 to 2.5 us.  Few rows: the weights' bytes (23 x 3072 -> 9216: 57
// MB in 14.3 us, of which 9 us streaming) and the same fixed parts.
// All waits are bounded (mbar_wait).  When one runs out, the whole cluster
// leaves together: after the loads, MMAs and partials that it has in flight (see
// the end of the kernel), with TMEM freed.
#include <type_traits>

#include "common.cuh"
#include "dense.h"

namespace svdq {

namespace {

constexpr int BK = 64;                       // one 128-byte swizzled row of 16-bit values
constexpr int SMEM_LIMIT = 232448;           // 227 KB
constexpr int MAX_STAGES = 8;

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], t_full[2], t_empty[2], inbox, drain;
  uint32_t tmem_base;
  int abort;
};

constexpr int pow2_at_least(int x, int lo) { return x <= lo ? lo : pow2_at_least(x, 2 * lo); }

template <int CG, int BN, bool SWAP, bool GATED, bool TALL>
struct Cfg {
  static constexpr int A_TILES = (SWAP && GATED) || TALL ? 2 : 1;
  static constexpr int TILE_ROWS = 128 * CG * (TALL ? 2 : 1);   // along the MMA's M
  static constexpr int A_TILE_BYTES = 128 * BK * 2;
  static constexpr int A_BYTES = A_TILES * A_TILE_BYTES;
  static constexpr int B_ROWS = BN / CG;                  // per CTA
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int K_TILE = A_BYTES + B_BYTES;          // one 64-wide k-tile
  static constexpr int OUT_COLS = (GATED && !SWAP) ? BN / 2 : BN;   // output columns of a tile
  static constexpr int BOX_COLS = OUT_COLS / 2 < 64 ? OUT_COLS / 2 : 64;   // pair form: columns of a store box
  static constexpr int EPI_WARPS = SWAP ? 4 : 8;          // one or two per TMEM sub-partition
  static constexpr int PARK = SWAP ? BN * 256 : EPI_WARPS * 32 * BOX_COLS * 2;   // the store box, or one a warp
  static constexpr int ACC_COLS = A_TILES * BN;
  // The partials a split tile's ranks send this one: memory of their own where
  // eight k-tiles still fit beside it (the senders need not wait for this
  // rank's MMAs then), else the ring.
  static constexpr int INBOX_WANT = (ACC_COLS + 32 * A_TILES) * 512;
  static constexpr int INBOX =
      SWAP && (SMEM_LIMIT - 1024 - PARK - INBOX_WANT - (int)sizeof(Ctl)) / K_TILE >= 8 ? INBOX_WANT : 0;
  static constexpr int ROOM_BYTES = SMEM_LIMIT - 1024 - PARK - INBOX - (int)sizeof(Ctl);
  // A stage of the ring is one or two k-tiles: two halve the waits and commits
  // between the MMAs, where at least four such stages fit (swapped: three).
  static constexpr int KS = ROOM_BYTES / (2 * K_TILE) >= (SWAP ? 3 : 4) ? 2 : 1;
  static constexpr int STAGE = KS * K_TILE;
  static constexpr int ROOM = ROOM_BYTES / STAGE;
  static constexpr int STAGES = ROOM < MAX_STAGES ? ROOM : MAX_STAGES;
  static constexpr int TMEM_COLS = TALL ? ACC_COLS : pow2_at_least(2 * ACC_COLS, 32);
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + PARK + INBOX + sizeof(Ctl);
  static_assert(STAGE % 1024 == 0, "tiles stay 1024-byte aligned for the 128-byte swizzle");
  static_assert(TMEM_COLS <= 512 && STAGES >= 3, "TMEM or ring too small");
  static_assert(TALL || (ACC_COLS + 4 * A_TILES * 8) * 512 <= STAGES * STAGE, "a split's partial tile fits the ring");
};

// ------------------------------------------------------------------ PTX forms this kernel adds
// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
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
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
// Whether every one of the swapped form's four epilogue warps passes true.
__device__ __forceinline__ bool all_warps_ok(bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Relaxed: what it hands over, TMEM columns, has been read (tcgen05.wait::ld);
// a release would wait for this thread's stores as well.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
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
// The same, counted on a barrier of the receiving CTA (16 bytes each).
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            uint32_t cluster_bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(addr),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(cluster_bar)
      : "memory");
}
// Tells the other CTAs of the cluster that a wait has run out.  Ordered before
// this thread's next arrival on the cluster's barrier.
__device__ __forceinline__ void tell_abort(uint32_t abort_word, int ctas) {
  for (int r = 0; r < ctas; ++r)
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dsmem_map(abort_word, r)), "r"(1) : "memory");
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
// Waits for a phase on the way out: without a look at the abort flag, until `deadline`.
__device__ __forceinline__ void wait_until(uint32_t bar, uint32_t parity, uint64_t deadline) {
  while (!mbar_try_wait(bar, parity) && global_timer_ns() < deadline) {
  }
}
// cluster_sync_all that orders no memory: an arrival with release semantics
// would wait for this thread's stores to global memory.
__device__ __forceinline__ void cluster_sync_last() {
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ void st_dsmem_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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
__device__ __forceinline__ uint64_t operand_desc(bool mn, uint32_t tile, int j) {
  return mn ? smem_desc(tile + 2048 * j, 8192, 1024, 2) : desc_k_sw128(tile + 32 * j);
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
  return unpack16((uint32_t)ld_param(p), fp16).x;
}
__device__ __forceinline__ uint16_t round16(float v, bool fp16) { return (uint16_t)pack16(v, 0.f, fp16); }

// Eight consecutive columns of one row: v += bias.
__device__ __forceinline__ void add_bias8(float (&v)[8], const uint16_t* bias, int n, bool fp16) {
  if (!bias) return;
  const uint4 b = ld_param(reinterpret_cast<const uint4*>(bias + n));
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
template <int COUNT>
__device__ __forceinline__ void activate(float (&v)[COUNT], int act) {
  if (act == SVDQ_EPI_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = gelu_tanh(v[i]);
  } else if (act == SVDQ_EPI_SILU) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = silu(v[i]);
  }
}
enum Out { OUT_Z, OUT_Z2, OUT_Y };   // which output a pass over the accumulators makes

// Token block of a tile of the swapped form.
__device__ __forceinline__ int tile_tokens(const Gemm16Params& p, int tile) {
  const Gemm16Job& j = p.job[0];
  const int per = j.group * j.tiles_n, g = tile / per;
  return (tile - g * per) / min(j.group, j.tiles_m - g * j.group);
}

}  // namespace

template <int CG, int BN, bool SWAP, bool GATED, bool GRAD, bool TALL, bool FP16>
__global__ void __launch_bounds__(Cfg<CG, BN, SWAP, GATED, TALL>::THREADS, 1)
    gemm16_kernel(const __grid_constant__ Gemm16Maps<GRAD ? 2 : 1> maps, const __grid_constant__ Gemm16Params p) {
  using C = Cfg<CG, BN, SWAP, GATED, TALL>;
  constexpr int OUT_COLS = C::OUT_COLS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* park = ring + C::STAGES * C::STAGE;
  Ctl* ctl = reinterpret_cast<Ctl*>(park + C::PARK + C::INBOX);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cta = CG == 2 ? (int)(rank & 1) : 0;             // CTA of the pair
  const int split = (int)rank / CG, S = p.splits;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.m[0][MAP_A]);
    tma_prefetch_desc(&maps.m[0][MAP_B]);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ctl->t_full[s]), 1);
      mbar_init(smem_u32(&ctl->t_empty[s]), CG * C::EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->inbox), 1);
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_barrier_init();
    if (C::INBOX && S > 1) {   // the bytes the ranks will send: whole chunks of 16 columns up to the last token
      const int own = OUT_COLS / S, tokens = p.job[0].M - tile_tokens(p, blockIdx.x / S) * BN;
      const int cols = min(max(min((tokens + 15) / 16 * 16, BN) - split * own, 0), own);
      mbar_arrive_expect_tx(smem_u32(&ctl->inbox), (uint32_t)(cols * 512 * S * C::A_TILES));
    }
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
  // global memory only after the previous kernel's writes are visible.  Every
  // warp waits here: a bounded wait must not count the previous kernel's time.
  grid_launch_dependents();
  grid_dependency_wait();

  // this pair (CTA, cluster), of how many
  const int first = (int)blockIdx.x / (CG * S), slots = (int)gridDim.x / (CG * S);
  auto tiles_of = [&](const Gemm16Job& j) { return j.tiles_m * j.tiles_n * (GRAD ? j.parts : 1); };
  const int tiles0 = tiles_of(p.job[0]), tiles1 = GRAD ? tiles_of(p.job[1]) : 0;
  // The n-th tile of this pair: its job and block coordinates.  Job 0's tiles
  // go round the pairs; the pairs left with one fewer of them take
  // job1_extra tiles of job 1 each, and the rest of job 1 goes round from the
  // last pair.  Within a job tiles run down groups of row blocks, so the tiles
  // in flight share rows of A and columns of B in L2.
  struct Tile {
    bool valid;
    int job, mb, nb;
    bool second;   // of two stacked A operands and outputs; mb counts within it
    int part;      // range of the reduction
  };
  auto tile_at = [&](int n) {
    Tile t;
    int tile = first + n * slots;
    t.job = 0;
    t.valid = tile < tiles0;
    if (GRAD && !t.valid && tiles1 > 0) {
      const int r = tiles0 % slots, few = slots - r, n1 = n - (tiles0 / slots + (first < r));
      const int extra = r ? min(tiles1, p.job1_extra * few) : 0;
      const int mine = first >= r && extra > 0 ? (extra - (first - r) + few - 1) / few : 0;
      tile = n1 < mine ? first - r + n1 * few : extra + (slots - 1 - first) + (n1 - mine) * slots;
      t.job = 1;
      t.valid = tile < tiles1;
    }
    if (t.valid) {
      const Gemm16Job& j = p.job[t.job];
      t.part = GRAD && j.parts > 1 ? tile / (j.tiles_m * j.tiles_n) : 0;
      if (GRAD) tile -= t.part * j.tiles_m * j.tiles_n;
      const int per = j.group * j.tiles_n, g = tile / per, q = tile - g * per;
      const int rows = min(j.group, j.tiles_m - g * j.group);
      t.mb = g * j.group + q % rows;
      t.nb = q / rows;
      t.second = t.mb >= j.tiles_m1;
      if (t.second) t.mb -= j.tiles_m1;
    }
    return t;
  };
  // its k-tiles: one range of a cluster's CTAs, or of the job's parts
  auto k_at = [&](const Gemm16Job& j, int i) { return (int)((long long)j.nk * i / (GRAD ? S * j.parts : S)); };
  auto k_begin = [&](const Gemm16Job& j, const Tile& t) { return k_at(j, t.part * S + split); };
  auto k_end = [&](const Gemm16Job& j, const Tile& t) { return k_at(j, t.part * S + split + 1); };

  int load_stage = 0;          // producer: the first place in the ring that it has not filled,
  uint32_t load_phase = 0;     // and that place's turn
  // The waits that last for a whole reduction have a limit that grows with it:
  // the set one besides for every 65536 k-tiles (30 us a k-tile at 2 s).
  auto reduction_err = [&](const Gemm16Job& j) {
    return DeviceErr{p.err.word, p.err.limit_ns + (p.err.limit_ns >> 16) * (unsigned)j.nk};
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto next = [&] {
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      };
      for (int n = 0; ok; ++n) {
        const Tile t = tile_at(n);
        if (!t.valid) break;
        const Gemm16Job& j = p.job[t.job];
        const CUtensorMap* map = maps.m[t.job];
        const bool a_mn = GRAD && j.a_mn;
        const int a_row = t.mb * C::TILE_ROWS + cta * 128;
        const int b_row = (GATED && !SWAP) ? t.nb * OUT_COLS : t.nb * BN + cta * C::B_ROWS;
        const int kt1 = k_end(j, t);
        for (int k0 = k_begin(j, t); k0 < kt1; k0 += C::KS, next()) {
          if (!(ok = mbar_wait(smem_u32(&ctl->empty[stage]), phase ^ 1, abort_flag, p.err))) break;
          const uint32_t bar = smem_u32(&ctl->full[stage]);
          const uint32_t sig = CG == 2 ? dsmem_map(bar, rank & ~1u) : bar;
          if (cta == 0) mbar_arrive_expect_tx(bar, CG * C::K_TILE * min(C::KS, kt1 - k0));
          for (int s = 0; s < C::KS && k0 + s < kt1; ++s) {
            const bool seg = GRAD && k0 + s >= j.nk1;           // the second part of a two-part reduction
            const int k = (seg ? k0 + s - j.nk1 : k0 + s) * BK;
            const uint32_t a = smem_u32(ring + stage * C::STAGE + s * C::K_TILE), b = a + C::A_BYTES;
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
            const CUtensorMap* map_a = map + (t.second || seg ? MAP_A2 : MAP_A);
            load_tile(a, map_a, a_mn, 128, a_row);
            if (TALL) load_tile(a + C::A_TILE_BYTES, map_a, a_mn, 128, a_row + 256);
            if (SWAP && GATED) load_tile(a + C::A_TILE_BYTES, map + MAP_A2, false, 128, a_row);
            const bool b2 = (GATED && !SWAP) ? cta == 1 : seg;
            load_tile(b, map + (b2 ? MAP_B2 : MAP_B), GRAD, C::B_ROWS, b_row);
          }
        }
      }
      load_stage = stage;
      load_phase = phase;
      // the pair's commits have all arrived before this CTA may leave
      for (int i = 0; CG == 2 && ok && i < C::STAGES; ++i, next())
        ok = mbar_wait(smem_u32(&ctl->empty[stage]), phase ^ 1, abort_flag, p.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the pair's first CTA)
    if (cta == 0) {
      const uint32_t idesc0 = (1u << 4) | (FP16 ? 0u : (1u << 7) | (1u << 10)) | (GRAD ? 1u << 16 : 0u) |
                              ((uint32_t)(BN >> 3) << 17) | ((uint32_t)((128 * CG) >> 4) << 24);
      const uint16_t mask = (uint16_t)(3u << (rank & ~1u));
      auto commit = [&](uint64_t* bar) {   // by the elected lane
        if (CG == 2)
          tc_commit_pair(smem_u32(bar), mask);
        else
          tc_commit(smem_u32(bar));
      };
      // Every lane runs every iteration, also after a wait has run out (`ok`
      // then skips the waits and the issues): elect.sync needs them all.
      bool ok = true;
      struct Slot {   // a place in the ring
        int stage;
        uint32_t phase;
        __device__ __forceinline__ void next() {
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      };
      Slot at{0, 0};
      auto drained = [&](int buf, uint32_t use) {
        if (ok) ok = mbar_wait(smem_u32(&ctl->t_empty[buf]), (use & 1) ^ 1, abort_flag, p.err);
        tc_fence_after();
      };
      for (uint32_t n = 0;; ++n) {
        const Tile tile = tile_at((int)n);
        if (!tile.valid) break;
        const Gemm16Job& job = p.job[tile.job];
        const bool a_mn = GRAD && job.a_mn;
        const uint32_t idesc = idesc0 | (a_mn ? 1u << 15 : 0u);
        const int nk = k_end(job, tile) - k_begin(job, tile);
        // the k-tiles of the stage at x, `left` of the tile's, into accumulators [T0, T1) at column acc
        auto multiply = [&](const Slot& x, uint32_t acc, auto t0, auto t1, int left, bool first_k) {
          constexpr int T0 = decltype(t0)::value, T1 = decltype(t1)::value;
#pragma unroll
          for (int s = 0; s < C::KS; ++s) {
            if (s > 0 && s >= left) break;
            const uint32_t a = smem_u32(ring + x.stage * C::STAGE + s * C::K_TILE), b = a + C::A_BYTES;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              const uint64_t db = operand_desc(GRAD, b, k);
#pragma unroll
              for (int t = T0; t < T1; ++t)
                mma_f16<CG>(acc + t * BN, operand_desc(a_mn, a + t * C::A_TILE_BYTES, k), db, idesc,
                            !first_k || s != 0 || k != 0);
            }
          }
        };
        const std::integral_constant<int, 0> T_0;
        const std::integral_constant<int, 1> T_1;
        const std::integral_constant<int, C::A_TILES> T_ALL;
        // stages from k-tile k0 to k1, one after the other
        auto through = [&](int k0, int k1, uint32_t acc) {
          for (int k = k0; k < k1; k += C::KS) {
            if (ok) ok = mbar_wait(smem_u32(&ctl->full[at.stage]), at.phase, abort_flag, p.err);
            tc_fence_after();
            if (elect_one() && ok) {
              multiply(at, acc, T_0, T_ALL, k1 - k, k == 0);
              commit(&ctl->empty[at.stage]);
            }
            at.next();
          }
        };
        if (!TALL) {
          const uint32_t ab = n & 1;
          drained(ab, n >> 1);
          through(0, nk, tmem + ab * C::ACC_COLS);
          if (elect_one() && ok) commit(&ctl->t_full[ab]);
        } else {
          // the same k-tiles, at most a ring of them, for accumulator 0 and then for 1, with their release
          auto apart = [&](int k0, int k1, bool last) {
            Slot x = at;
            for (int k = k0; k < k1; k += C::KS, x.next()) {
              if (ok) ok = mbar_wait(smem_u32(&ctl->full[x.stage]), x.phase, abort_flag, p.err);
              tc_fence_after();
              if (elect_one() && ok) multiply(x, tmem, T_0, T_1, k1 - k, k == 0);
            }
            if (last && elect_one() && ok) commit(&ctl->t_full[0]);
            if (k0 == 0) drained(1, n);
            for (int k = k0; k < k1; k += C::KS, at.next())
              if (elect_one() && ok) {
                multiply(at, tmem, T_1, T_ALL, k1 - k, k == 0);
                commit(&ctl->empty[at.stage]);
              }
            if (last && elect_one() && ok) commit(&ctl->t_full[1]);
          };
          constexpr int RING = C::STAGES * C::KS;
          const int head = min(nk, RING), rest = nk - head, tail = min(rest, RING);
          const int mid = (rest - tail + C::KS - 1) / C::KS * C::KS;
          drained(0, n);
          apart(0, head, nk == head);
          through(head, head + mid, tmem);
          if (rest > mid) apart(head + mid, nk, true);
        }
      }
    }
  }

  // -------------------------------------------------------------- epilogue
  const int e = warp - 2, sub = warp & 3;
  const int row = sub * 32 + lane;                            // TMEM lane: row of this CTA's 128
  constexpr bool fp16 = FP16;

  if (GRAD && warp >= 2 && p.parts > 0) {
    // The bias gradients, 32 columns a block of CTAs: warp w adds parts w,
    // w + 8, ..., then the warps in order.
    float* sh = reinterpret_cast<float*>(park);
    const int blocks = (p.part_n + 31) / 32, two = p.part2 ? 2 : 1;
    for (int cb = blockIdx.x; cb < two * blocks; cb += gridDim.x) {
      const float* src = cb < blocks ? p.part : p.part2;
      uint16_t* dst = cb < blocks ? p.dbias : p.dbias2;
      const int n = (cb < blocks ? cb : cb - blocks) * 32 + lane;
      float t = 0.f;
      if (n < p.part_n) {
#pragma unroll 4
        for (int s = e; s < p.parts; s += 8) t += src[(size_t)s * p.part_n + n];
      }
      sh[e * 32 + lane] = t;
      named_bar_sync(1, 256);
      if (e == 0 && n < p.part_n) {
        t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sh[w * 32 + lane];
        dst[n] = round16(t, fp16);
      }
      named_bar_sync(1, 256);
    }
  }

  // The residual of eight columns (pair form); the pointers may be Y's own, so
  // it is loaded before anything of its chunk is stored.
  auto residual8 = [&](int m, int n) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if (!GATED && p.R && m < p.job[0].M && n < p.job[0].N)
      r = *reinterpret_cast<const uint4*>(p.R + (size_t)m * p.ldr + n);
    return r;
  };
  // What output `out` holds of accumulators v (and u), biases added: v is
  // overwritten.  r: the residual's values.
  auto finish = [&](Out out, auto& v, auto& u, auto add_residual) {
    constexpr int COUNT = sizeof(v) / sizeof(float);
    if (GATED && out == OUT_Z2) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = u[i];
    } else if (out == OUT_Y) {
      activate(v, p.act);
      if (GATED) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] *= u[i];
      } else if (p.R) {
        add_residual();
      }
    }
  };

  if (!SWAP && warp >= 2 && S == 1) {
    // This warp's 32 rows, PER columns of every tile, in boxes of W columns.
    constexpr int PER = OUT_COLS / 2, W = C::BOX_COLS;
    const int c0 = (e >> 2) * PER;
    const uint32_t box = smem_u32(park) + (uint32_t)e * (32 * W * 2);
    // n counts accumulators: one a tile, or two (TALL)
    constexpr int PARTS = TALL ? 2 : 1;
    Tile t = tile_at(0);
    for (int n = 0; t.valid; ++n) {
      const int part = n % PARTS;
      const Gemm16Job& j = p.job[t.job];
      const CUtensorMap* map = maps.m[t.job];
      const int row_w = t.mb * C::TILE_ROWS + part * 256 + cta * 128 + sub * 32, m = row_w + lane;
      const int n_tile = t.nb * OUT_COLS;
      const uint32_t ab = n & 1, pt = (n >> 1) & 1;
      // the bias of this warp's columns, two a word, words 0-31 and 32-63 over the lanes (gated: g's, u's)
      uint32_t bias_w[2] = {0u, 0u};
      if (!GRAD) {
        const int col = n_tile + c0 + 2 * lane;
        if (p.bias && 2 * lane < PER && col < j.N) bias_w[0] = ld_param32(p.bias + col);
        if (GATED) {
          if (p.bias2 && 2 * lane < PER && col < j.N) bias_w[1] = ld_param32(p.bias2 + col);
        } else if (p.bias && 2 * lane + 64 < PER && col + 64 < j.N) {
          bias_w[1] = ld_param32(p.bias + col + 64);
        }
      }
      // eight columns c .. c + 7 of the warp's: v += bias (words of reg)
      auto add_bias = [&](float (&v)[8], uint32_t words, int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack16(__shfl_sync(0xffffffffu, words, (c / 2 + i) & 31), fp16);
          v[2 * i] += f.x;
          v[2 * i + 1] += f.y;
        }
      };
      uint4 res[2] = {residual8(m, n_tile + c0), residual8(m, n_tile + c0 + 8)};
      if (!mbar_wait(smem_u32(&ctl->t_full[ab]), pt, abort_flag, reduction_err(j))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16) + ab * (TALL ? BN : C::ACC_COLS);
      const bool second = GRAD && t.second;
      auto emit_box = [&](Out out, int at, int c) {
        // the next 16 columns come out of TMEM while these are worked on
        uint32_t r[2][16], q[2][GATED ? 16 : 1];
        auto fetch = [&](int buf, int d) {
          tmem_ld16(taddr + c + d, r[buf]);
          if constexpr (GATED) tmem_ld16(taddr + BN / 2 + c + d, q[buf]);
        };
        fetch(0, 0);
        if (lane == 0) bulk_wait_read();   // the previous box has left shared memory
        __syncwarp();
#pragma unroll
        for (int d = 0; d < W; d += 16) {
          const int buf = (d >> 4) & 1;
          const uint4 now[2] = {res[0], res[1]};
          if (out == OUT_Y && c + d + 16 < c0 + PER) {
            res[0] = residual8(m, n_tile + c + d + 16);
            res[1] = residual8(m, n_tile + c + d + 24);
          }
          tmem_wait_ld();
          if (d + 16 < W) fetch(buf ^ 1, d + 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[8], u[8];
            const int cc = c - c0 + d + 8 * h;   // column of the warp's
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] = __uint_as_float(r[buf][8 * h + i]);
              u[i] = GATED ? __uint_as_float(q[buf][GATED ? 8 * h + i : 0]) : 0.f;
            }
            if (!GRAD && p.bias) add_bias(v, GATED || cc < 64 ? bias_w[0] : bias_w[1], cc);
            if (GATED && p.bias2) add_bias(u, bias_w[1], cc);
            finish(out, v, u, [&] { add8(v, now[h], fp16); });
            const int chunk = (d >> 3) + h;      // 16-byte chunk of the row, swizzled as the box's map
            const uint32_t off = W == 64 ? lane * 128 + ((chunk ^ (lane & 7)) << 4)
                                         : lane * 64 + ((chunk ^ ((lane >> 1) & 3)) << 4);
            sts128(box + off, round8(v, fp16));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row_w < j.M && n_tile + c < j.N) tma_store_2d(map + at, box, n_tile + c, row_w);
      };
      // A part of the reduction: the accumulators as they are, 32 columns a box.
      if (GRAD && j.parts > 1) {
        const int below = (t.part * (j.Y2 ? 2 : 1) + (second ? 1 : 0)) * ((j.M + 31) / 32 * 32);
#pragma unroll 1
        for (int c = c0; c < c0 + PER; c += 32) {
          uint32_t r[2][16];
          tmem_ld16(taddr + c, r[0]);
          tmem_ld16(taddr + c + 16, r[1]);
          if (lane == 0) bulk_wait_read();   // the previous box has left shared memory
          __syncwarp();
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t* v = &r[i >> 2][4 * (i & 3)];
            sts128(box + lane * 128 + ((i ^ (lane & 7)) << 4), make_uint4(v[0], v[1], v[2], v[3]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row_w < j.M && n_tile + c < j.N) tma_store_2d(map + MAP_Y, box, n_tile + c, below + row_w);
        }
      } else {
#pragma unroll 1
        for (int c = c0; c < c0 + PER; c += W) {
          if (!GRAD && p.Z) emit_box(OUT_Z, MAP_Z, c);
          if (GATED && p.Z2) emit_box(OUT_Z2, MAP_Z2, c);
          emit_box(OUT_Y, second ? MAP_Y2 : MAP_Y, c);
        }
      }
      tc_fence_before();
      __syncwarp();
      // not for a buffer no later tile waits for: nothing is left in flight towards the pair's first CTA
      const bool wanted = tile_at((n + 2) / PARTS).valid;
      if (lane == 0 && wanted) mbar_arrive_cluster(dsmem_map(smem_u32(&ctl->t_empty[ab]), rank & ~1u));
      if (part == PARTS - 1) t = tile_at((n + 1) / PARTS);
    }
    if (lane == 0) bulk_wait_all();
  }

  // Swapped form: `own` tokens m0 .. of this CTA's 128 features leave as one
  // box [token][feature].  values(c, v, u): the accumulators of tokens m0 + c ..
  auto emit_tokens = [&](int m0, int f0, int own, auto step_tag, auto values) {
    constexpr int STEP = decltype(step_tag)::value;
    const Gemm16Job& j = p.job[0];
    const int n = f0 + row;
    const bool live = n < j.N;
    float bias_v = 0.f, bias_u = 0.f;
    if (live && p.bias) bias_v = load16(p.bias + n, fp16);
    if (GATED && live && p.bias2) bias_u = load16(p.bias2 + n, fp16);
    const uint32_t box = smem_u32(park) + row * 2;
    auto pass = [&](Out out, int at) {
      if (warp == 2 && lane == 0) bulk_wait_read();   // the previous box has left shared memory
      named_bar_sync(1, 128);
#pragma unroll 1
      for (int c = 0; c < own && m0 + c < j.M; c += STEP) {
        float v[STEP], u[STEP], r[STEP];
#pragma unroll
        for (int i = 0; i < STEP; ++i)
          r[i] = (!GATED && out == OUT_Y && p.R && live && m0 + c + i < j.M)
                     ? unpack16((uint32_t)p.R[(size_t)(m0 + c + i) * p.ldr + n], fp16).x
                     : 0.f;
        values(c, v, u);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          v[i] += bias_v;
          if (GATED) u[i] += bias_u;
        }
        finish(out, v, u, [&] {
#pragma unroll
          for (int i = 0; i < STEP; ++i) v[i] += r[i];
        });
#pragma unroll
        for (int i = 0; i < STEP; ++i) sts16(box + (c + i) * 256, round16(v[i], fp16));
      }
      fence_proxy_async_smem();
      named_bar_sync(1, 128);
      if (warp == 2 && lane == 0 && m0 < j.M) tma_store_2d(&maps.m[0][at], smem_u32(park), f0, m0);
    };
    if (p.Z) pass(OUT_Z, MAP_Z);
    if (GATED && p.Z2) pass(OUT_Z2, MAP_Z2);
    pass(OUT_Y, MAP_Y);
  };

  if (SWAP && warp >= 2 && S == 1) {
    for (int n = 0;; ++n) {
      const Tile t = tile_at(n);
      if (!t.valid) break;
      const uint32_t ab = n & 1, pt = (n >> 1) & 1;
      // the four warps leave together when the wait runs out: emit_tokens joins them
      const bool ok = mbar_wait(smem_u32(&ctl->t_full[ab]), pt, abort_flag, reduction_err(p.job[0]));
      if (!all_warps_ok(ok)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16) + ab * C::ACC_COLS;
      emit_tokens(t.nb * BN, t.mb * 128, BN, std::integral_constant<int, 16>{},
                  [&](int c, float (&v)[16], float (&u)[16]) {
                    tmem_ld16(taddr + c, reinterpret_cast<uint32_t(&)[16]>(v));
                    if (GATED) tmem_ld16(taddr + BN + c, reinterpret_cast<uint32_t(&)[16]>(u));
                    tmem_wait_ld();
                  });
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->t_empty[ab]));
    }
    if (warp == 2 && lane == 0) bulk_wait_all();
  }

  if (S > 1) {
    // One tile per cluster.  Rank q sums output columns q own .. of all ranks:
    // each rank sends its float32 partial of them, four columns a store, into
    // rank q's inbox (or, where shared memory holds none beside the ring, into
    // its ring, free once every rank's MMAs are complete) as [source rank]
    // [128 rows][own + 4 columns] (the pad keeps 16-byte accesses of eight
    // rows on different banks), where q adds the sources in rank order.
    constexpr int HALVES = GATED ? 2 : 1, HALF = C::ACC_COLS / HALVES;   // accumulator halves g and u
    constexpr int LOG_OUT = OUT_COLS == 256 ? 8 : OUT_COLS == 128 ? 7 : OUT_COLS == 64 ? 6 : OUT_COLS == 32 ? 5 : 4;
    const int log_own = LOG_OUT - (31 - __clz(S)), own = 1 << log_own;    // S is a power of two, own >= 4
    const uint32_t line = (own + 4) * 4;
    const uint32_t inbox = smem_u32(C::INBOX ? park + C::PARK : ring) + row * line;
    const Tile t = tile_at(0);
    const Gemm16Job& j = p.job[t.job];
    bool ok = false;
    if (warp >= 2) {
      ok = mbar_wait(smem_u32(&ctl->t_full[0]), 0, abort_flag, reduction_err(j));
      tc_fence_after();
    }
    if (!C::INBOX) cluster_sync_all();
    if (warp >= 2 && ok) {
      const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16);
      for (int c = (e >> 2) * 16; c < C::ACC_COLS; c += 16 * (C::EPI_WARPS / 4)) {
        const int half = c / HALF, oc = c - half * HALF;                // output column
        if (SWAP && t.nb * BN + oc >= j.M) continue;                    // past the last token
        uint32_t r[16];
        tmem_ld16(taddr + c, r);
        tmem_wait_ld();
        const uint32_t slot = inbox + (uint32_t)(split * HALVES + half) * 128 * line;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int q = (oc + i) >> log_own;
          const uint32_t to = dsmem_map(slot + ((oc + i) & (own - 1)) * 4, q * CG + cta);
          if (C::INBOX)
            st_async_v4(to, r[i], r[i + 1], r[i + 2], r[i + 3], dsmem_map(smem_u32(&ctl->inbox), q));
          else
            st_dsmem_v4(to, r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
      }
      tc_fence_before();
    }
    if (!C::INBOX)
      cluster_sync_all();
    else if (warp >= 2)
      ok = mbar_wait(smem_u32(&ctl->inbox), 0, abort_flag, reduction_err(j)) && ok;
    // columns col .. col + 3 of the half
    auto total4 = [&](int half, int col, float* v) {
      const uint32_t from = inbox + half * 128 * line + col * 4;
      v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll 2
      for (int s = 0; s < S; ++s) {
        const uint4 x = lds128(from + (uint32_t)(s * HALVES) * 128 * line);
        v[0] += __uint_as_float(x.x);
        v[1] += __uint_as_float(x.y);
        v[2] += __uint_as_float(x.z);
        v[3] += __uint_as_float(x.w);
      }
    };
    if (!SWAP) {
      const int m = t.mb * 256 + cta * 128 + row;
      if (warp >= 2 && ok && m < j.M) {
        uint16_t* out = GRAD && t.second ? j.Y2 : j.Y;
        for (int c = (e >> 2) * 8; c < own; c += 16) {
          const int n = t.nb * OUT_COLS + split * own + c;
          if (n >= j.N) break;
          const uint4 res = residual8(m, n);
          float v[8], u[8];
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            total4(0, c + i, v + i);
            if (GATED) total4(1, c + i, u + i);
          }
          add_bias8(v, p.bias, n, fp16);
          if (GATED) add_bias8(u, p.bias2, n, fp16);
          const size_t at = (size_t)m * j.N + n;
          if (p.Z) store8(p.Z + at, v, fp16);
          if (GATED && p.Z2) store8(p.Z2 + at, u, fp16);
          finish(OUT_Y, v, u, [&] { add8(v, res, fp16); });
          store8(out + (size_t)m * j.ldy + n, v, fp16);
        }
      }
    } else if (warp >= 2 && all_warps_ok(ok)) {
      emit_tokens(t.nb * BN + split * own, t.mb * 128, own, std::integral_constant<int, 4>{},
                  [&](int c, float (&v)[4], float (&u)[4]) {
                    total4(0, c, v);
                    if (GATED) total4(1, c, u);
                  });
      if (warp == 2 && lane == 0) bulk_wait_all();
    }
  }

  if (*abort_flag && CG * S > 1) tell_abort(smem_u32(&ctl->abort), CG * S);
  tc_fence_before();
  if (CG * S > 1)
    cluster_sync_last();   // no CTA leaves while another reads its shared memory or signals its barriers
  else
    __syncthreads();
  if (*abort_flag) {
    // A wait has run out somewhere in the cluster (every thread of it sees the
    // same here) and no thread issues anything any more.  What has been issued
    // lands before a CTA leaves: loads on their stage's barrier, MMAs on one
    // of their own, the other ranks' partials on the inbox.  A copy within the
    // chip takes microseconds; a barrier that will never complete (some of its
    // operations were not issued) is given up after 10 ms.
    const uint64_t deadline = global_timer_ns() + 10000000ull;
    if (warp == 0 && lane == 0) {
      if (cta == 0) {
        for (int s = 0; s < C::STAGES; ++s)
          wait_until(smem_u32(&ctl->full[s]), s < load_stage ? load_phase : load_phase ^ 1, deadline);
      } else {   // its loads count on the other CTA's barriers, which may not expect them: 1 ms
        while (global_timer_ns() + 9000000ull < deadline) {
        }
      }
    }
    if (warp == 1 && cta == 0) {
      __syncwarp();
      if (elect_one()) {   // the lane that issued the MMAs
        if (CG == 2)
          tc_commit_pair(smem_u32(&ctl->drain), (uint16_t)(1u << rank));
        else
          tc_commit(smem_u32(&ctl->drain));
        wait_until(smem_u32(&ctl->drain), 0, deadline);
      }
      __syncwarp();
    }
    if (C::INBOX && S > 1 && warp == 2 && lane == 0) wait_until(smem_u32(&ctl->inbox), 0, deadline);
    tc_fence_before();
    if (CG * S > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc<CG>(tmem, C::TMEM_COLS);
  }
}

namespace {

// ------------------------------------------------------------------ joining the parts of a reduction
// Eight columns a thread, the parts in order: no atomics, the same bits on
// every run.  Bound by latency: the partials, at most 20 MB, come from L2.
struct JoinParams {
  struct {
    const float* P;
    uint16_t *Y, *Y2;
    long long ldy;
    int M, N, parts;
  } job[2];
};
template <bool FP16>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ JoinParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const auto& j = p.job[blockIdx.y];
  const int per_row = j.N / 8, rows = j.M * (j.Y2 ? 2 : 1), pad = (j.M + 31) / 32 * 32;   // of each stacked output
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
  if (at >= (long long)rows * per_row) return;
  const int row = (int)(at / per_row), col = (int)(at - (long long)row * per_row) * 8;
  const bool second = row >= j.M;
  const float* src = j.P + (size_t)(second ? row - j.M + pad : row) * j.N + col;
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < j.parts; ++s, src += (size_t)pad * (j.Y2 ? 2 : 1) * j.N) {
    const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
    const float part[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += part[i];
  }
  uint16_t* y = second ? j.Y2 + (size_t)(row - j.M) * j.ldy : j.Y + (size_t)row * j.ldy;
  store8(y + col, v, FP16);
}

template <int CG, int BN, bool SWAP, bool GATED, bool GRAD, bool TALL, bool FP16>
cudaError_t launch(const Gemm16Maps<2>& maps, const Gemm16Params& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<CG, BN, SWAP, GATED, TALL>;
  auto kern = gemm16_kernel<CG, BN, SWAP, GATED, GRAD, TALL, FP16>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  long long tiles = 0;
  for (const Gemm16Job& j : p.job) tiles += (long long)j.tiles_m * j.tiles_n * j.parts;
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
  if constexpr (GRAD) {
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
  } else {
    Gemm16Maps<1> one;
    for (int i = 0; i < MAPS; ++i) one.m[0][i] = maps.m[0][i];
    return cudaLaunchKernelEx(&cfg, kern, one, p);
  }
}

// As many row blocks a group as keep the group's rows of A in L2 (40 MB of
// it), at least 9, the row blocks shared out evenly.  Measured, back to back:
// 4608 x 3072 -> 9216 all 18 blocks 189 us, groups of 9 193, 8 195, 4 199;
// 8192 x 8192 -> 8192 groups of 8 828, 18 855, 4 857.
int group_rows(const Gemm16Job& j, bool tall) {
  if (j.tiles_m == 0) return 1;
  const long long block = 2ll * (tall ? 512 : 256) * j.nk * BK;
  const int least = tall ? 5 : 9, most = 40000000 / block > least ? (int)(40000000 / block) : least;
  const int groups = (j.tiles_m + most - 1) / most;
  return (j.tiles_m + groups - 1) / groups;
}

template <bool FP16>
cudaError_t launch_as(const Gemm16Plan& plan, const Gemm16Maps<2>& maps, const Gemm16Params& p, int num_sms,
                      cudaStream_t stream) {
  if (plan.swap) {
#define SVDQ_SWAP(G)                                                                        \
  switch (plan.bn) {                                                                        \
    case 16: return launch<1, 16, true, G, false, false, FP16>(maps, p, num_sms, stream);          \
    case 32: return launch<1, 32, true, G, false, false, FP16>(maps, p, num_sms, stream);          \
    case 64: return launch<1, 64, true, G, false, false, FP16>(maps, p, num_sms, stream);          \
    case 128: return launch<1, 128, true, G, false, false, FP16>(maps, p, num_sms, stream);        \
    default: return cudaErrorInvalidValue;                                                  \
  }
    if (plan.op == GEMM16_NT) SVDQ_SWAP(false)
    if (plan.op == GEMM16_GATED) SVDQ_SWAP(true)
#undef SVDQ_SWAP
    return cudaErrorInvalidValue;
  }
  if (plan.tall) {
    if (plan.op == GEMM16_NT) return launch<2, 256, false, false, false, true, FP16>(maps, p, num_sms, stream);
    if (plan.op == GEMM16_GRAD) return launch<2, 256, false, false, true, true, FP16>(maps, p, num_sms, stream);
    return cudaErrorInvalidValue;
  }
#define SVDQ_PAIR(G, B)                                                                     \
  return plan.bn == 256 ? launch<2, 256, false, G, B, false, FP16>(maps, p, num_sms, stream) \
                        : launch<2, 128, false, G, B, false, FP16>(maps, p, num_sms, stream);
  switch (plan.op) {
    case GEMM16_NT: SVDQ_PAIR(false, false)
    case GEMM16_GATED: SVDQ_PAIR(true, false)
    case GEMM16_GRAD: SVDQ_PAIR(false, true)
  }
#undef SVDQ_PAIR
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm16(const Gemm16Plan& plan, const Gemm16Maps<2>& maps, Gemm16Params p, int num_sms,
                          cudaStream_t stream) {
  p.splits = plan.splits;
  p.job[0].group = group_rows(p.job[0], plan.tall);
  p.job[1].group = group_rows(p.job[1], plan.tall);
  auto tile_nk = [](const Gemm16Job& j) { return j.parts ? (j.nk + j.parts - 1) / j.parts : 0; };
  p.job1_extra = gemm16_extra(tile_nk(p.job[0]), tile_nk(p.job[1]));
  return p.fp16 ? launch_as<true>(plan, maps, p, num_sms, stream) : launch_as<false>(plan, maps, p, num_sms, stream);
}

cudaError_t launch_join_parts(const Gemm16Job* jobs, int count, int fp16, cudaStream_t stream) {
  JoinParams q = {};
  long long most = 0;
  for (int i = 0; i < count; ++i) {
    const Gemm16Job& j = jobs[i];
    const long long chunks = (long long)j.M * (j.Y2 ? 2 : 1) * (j.N / 8);
    q.job[i] = {j.P, j.Y, j.Y2, j.ldy, j.M, j.N, j.parts};
    if (chunks > most) most = chunks;
  }
  const dim3 grid((unsigned)((most + 255) / 256), count);
  return fp16 ? launch_early(join_parts_kernel<true>, grid, 256, 0, stream, q)
              : launch_early(join_parts_kernel<false>, grid, 256, 0, stream, q);
}

}  // namespace svdq
