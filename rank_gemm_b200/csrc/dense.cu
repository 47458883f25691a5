// dense.cu -- host side of the 16-bit layers declared in include/svdq.h: the
// dense linear, the gated feed-forward and the layer norm, forward and
// backward.  Checks arguments, picks the tiling, encodes the tensor maps and
// launches; nothing is kept between calls.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "svdq.h"
#include "common.cuh"
#include "dense.h"

using namespace svdq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }

bool type16(svdq_dtype dt) { return dt == SVDQ_BF16 || dt == SVDQ_FP16; }
bool known_act(svdq_epilogue a) { return a == SVDQ_EPI_NONE || a == SVDQ_EPI_GELU_TANH || a == SVDQ_EPI_SILU; }
// Sizes stay 512 short of 2^31, so that a tile's rows and columns past the
// last still count in 32 bits.
constexpr int MOST = 0x7FFFFE00;
bool width_ok(int n) { return n > 0 && n % 8 == 0 && n <= MOST; }
bool rows_ok(int m) { return m >= 0 && m <= MOST; }
// a row stride in 16-bit elements: covers the row, 16-byte steps, under the TMA limit of 2^40 bytes
bool stride_ok(long long ld, int width) { return ld >= width && ld % 8 == 0 && ld < (1ll << 39); }

const uint16_t* in16(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* out16(void* p) { return static_cast<uint16_t*>(p); }

// ------------------------------------------------------------------ tiling
// Clusters of `width` CTAs an SM-filling grid can hold at once: the SMs of a
// GPC that do not make up a whole cluster stay idle (cudaOccupancy reports
// 148, 74, 33 and 15 for widths 1, 2, 4 and 8 on this part).
int clusters(int width, int num_sms) {
  return width == 1 ? num_sms : width == 2 ? num_sms / 2 : width == 4 ? num_sms * 33 / 148 : num_sms * 15 / 148;
}

// Estimated time of a plan in SM cycles: the longest share of a CTA (pair),
// k-tile by k-tile, or, where that is longer, the time the operand bytes take
// from L2 (8500 a cycle over the chip) or the weights from memory (3400);
// besides, a fixed part (launch, fill, epilogue, drain) and the exchange of a
// split tile's partials.  The constants were fitted to 24 shapes of 1 to 2048
// rows under every tiling.  Of 120 shapes drawn at random, all four operators,
// 112 took at most 1.08 times their best tiling's time; the others, us chosen
// and best: 179 x 8216 -> 6776 46.3, 36.9 (256 columns split in two); gated 1 x
// 12056 -> 104 21.0, 17.1 (pair form split in four); gated backward 6 x 5080 ->
// 11136 156, 135 (not cut); gated 1004 x 1160 -> 1440 15.7, 13.8 and 1580 x 776
// -> 1064 16.3, 15.0 (256 columns); backward 66 x 224 -> 11848 15.0, 13.4 and 77
// x 296 -> 1296 9.3, 8.5 (128 columns, cut); 1319 x 5720 -> 824 31.4, 28.5.  A
// pair's rate for weights from memory is not in the estimate.  Where the
// two forms cross (us, best tilings of each): 64 x 1024 -> 1024 swapped 4.9,
// pair 6.4; 128 x 12288 -> 3072 swapped 24.4, pair 26.7; 128 x 3072 -> 9216
// swapped 15.8, pair 15.6; 256 x 1024 -> 1024 swapped 8.6, pair 6.6.
struct Choice {
  Gemm16Plan plan{};
  int parts[2] = {1, 1};   // of each job's reduction
  double cycles = 0;
  void offer(const Gemm16Plan& p, double t, int parts0 = 1, int parts1 = 1) {
    if (cycles == 0 || t < cycles) {
      plan = p;
      parts[0] = parts0;
      parts[1] = parts1;
      cycles = t;
    }
  }
};
struct JobShape {
  int M, N, nk;        // output rows and columns, k-tiles
  int stacked;         // outputs stacked along the rows
  int most_parts;      // ranges its reduction may be cut into
};
// The longest share of a pair, in cycles (ca, cb a tile), as the kernel deals
// the tiles out: `per` tiles of the second job make up for one of the first.
long long longest_share(long long ta, long long ca, long long tb, long long cb, int per, int slots) {
  if (!tb) return (ta + slots - 1) / slots * ca;
  const long long r = ta % slots, few = slots - r;
  const long long extra = tb && r ? std::min(tb, per * few) : 0, rest = tb - extra;
  long long most = 0;
  const long long at[4] = {0, r > 0 ? r - 1 : 0, r, slots - 1};   // the shares step at these pairs
  for (long long p : at) {
    const long long n0 = ta / slots + (p < r), n1 = p >= r && extra > p - r ? (extra - (p - r) + few - 1) / few : 0;
    const long long q = slots - 1 - p, n2 = rest > q ? (rest - q + slots - 1) / slots : 0;
    most = std::max(most, n0 * ca + (n1 + n2) * cb);
  }
  return most;
}
Choice plan_pair(Gemm16Op op, JobShape a, JobShape b, int num_sms) {
  Choice best;
  struct Form {
    int rows, bn, k_tile, tile, fixed, exchange;
    bool tall;
  };
  // Cycles of a k-tile, of a tile besides, of a launch, of a split's exchange
  // a rank.  512 x 256 tiles take 0.94 of the time of two 256 x 256 at 128
  // k-tiles (8192^3: 826 us, 875), 0.96 at 72 and 1.01 at 48, and leave more
  // pairs idle at the end.
  // The backward products' 64 x 64 boxes cost the narrow forms more (1023
  // rows, 1160 and 2056 wide: 128 columns 26.3 us, 256 24.0).
  const bool grad = op == GEMM16_GRAD;
  const Form forms[3] = {{512, 256, grad ? 1060 : 1020, 6000, 10400, 0, true},
                         {256, 256, grad ? 660 : 537, 0, 10400, 5000, false},
                         {256, 128, grad ? 620 : 365, 0, 6700, 3500, false}};
  // The weights' bytes from memory (backward: less than the work).  Without
  // them one row of a gated 3072 -> 9216 took this form: 31.5 us, swapped 21.2.
  const double stream = grad ? 0 : (op == GEMM16_GATED ? 2.0 : 1.0) * a.N * a.nk * 128 / 3400;
  for (const Form& f : forms) {
    if (f.tall && op == GEMM16_GATED) continue;
    const int out_cols = op == GEMM16_GATED ? f.bn / 2 : f.bn;
    auto tiles_of = [&](const JobShape& j) {
      return j.nk ? (long long)j.stacked * ceil_div(j.M, f.rows) * ceil_div(j.N, out_cols) : 0;
    };
    const long long ta = tiles_of(a), tb = tiles_of(b), tiles = ta + tb;
    const double arrival = ((double)ta * a.nk + (double)tb * b.nk) * (f.rows + f.bn) * 128 / 8500;
    for (int s = 1; s <= (f.tall ? 1 : 4); s *= 2) {
      const int slots = clusters(2 * s, num_sms);
      if (s > 1 && ((ta && a.nk < 4 * s) || (tb && b.nk < 4 * s) || tiles > slots)) break;
      auto cost = [&](int nk) { return (long long)(grad ? gemm16_weight(nk) : nk) * f.k_tile + f.tile; };
      const double share = (double)longest_share(ta, cost(ceil_div(a.nk, s)), tb, cost(ceil_div(b.nk, s)),
                                                 gemm16_extra(a.nk, b.nk), slots);
      best.offer({op, false, f.bn, s, f.tall},
                 f.fixed + std::max(share, std::max(arrival, stream)) + (s > 1 ? f.exchange * s : 0));
      if (!grad || s > 1) continue;
      // Reductions cut so that every pair gets its even share, at least 8
      // k-tiles: float32 partials and a kernel that joins them, 9000 cycles
      // (7 x 96 -> 3168 backward 15.6 us, cut 8.1; 8192 x 512 -> 512 35.0,
      // cut 16.7; counted as 4500: 128 x 1024 -> 1024 8.0, cut 8.8).
      const long long even = std::max((ta * gemm16_weight(a.nk) + tb * gemm16_weight(b.nk) + slots - 1) / slots, 8ll);
      auto cut = [&](const JobShape& j) {
        return j.nk ? std::max(1, std::min(j.most_parts, ceil_div(j.nk, (int)std::min<long long>(even, j.nk)))) : 1;
      };
      const int pa = cut(a), pb = cut(b);
      if (pa == 1 && pb == 1) continue;
      const int ka = ceil_div(a.nk, pa), kb = b.nk ? ceil_div(b.nk, pb) : 0;
      const double cut_share =
          (double)longest_share(ta * pa, cost(ka), tb * pb, cost(kb), gemm16_extra(ka, kb), slots);
      auto floats = [](const JobShape& j, int parts) {
        return parts > 1 ? (double)parts * j.stacked * j.M * j.N : 0.0;
      };
      best.offer({op, false, f.bn, 1, f.tall},
                 f.fixed + std::max(cut_share, arrival) + 9000 + (floats(a, pa) + floats(b, pb)) * 8 / 5000, pa, pb);
    }
  }
  return best;
}
Choice plan_swap(Gemm16Op op, int tokens, int features, int nk, int num_sms) {
  Choice best;
  const int weights = op == GEMM16_GATED ? 2 : 1;
  for (int bn = 16; bn <= 128; bn *= 2) {
    const int tiles = ceil_div(features, 128) * ceil_div(tokens, bn);
    const double per_k = (300 + 1.1 * bn) * (weights == 2 ? 1.5 : 1.0);
    for (int s = 1; s <= 8 && 4 * s <= bn; s *= 2) {   // at least four tokens a rank
      const int slots = clusters(s, num_sms);
      if (s > 1 && (nk < 2 * s || tiles > slots)) break;
      const double share = (double)((tiles + slots - 1) / slots) * ceil_div(nk, s) * per_k;
      // the weights' bytes at memory's rate, or at 41 a cycle and CTA
      const double stream = (double)weights * features * nk * 128 / std::min(3400.0, 41.0 * tiles * s);
      best.offer({op, true, bn, s, false}, 5000 + 50 * bn + std::max(share, stream) + (s > 1 ? 1000 + 70 * bn : 0));
    }
    if (bn >= tokens) break;
  }
  return best;
}
// More rows of X than this never gain from the swapped form.
constexpr int SWAP_ROWS = 256;
// Up to this many rows the pair form is not taken: its 256-row boxes, nearly
// empty, come slower than full ones, which its estimate does not know (gated 2 x
// 1272 -> 4344: 12.7 us, swapped 9.1).  It would gain where a long reduction
// has few features, whose weights the swapped form streams through at most 4
// CTAs a tile for one token (gated 1 x 12056 -> 104: 17.1 us, swapped 21.0).
constexpr int PAIR_ROWS = 32;

// The tiling of a forward product of M rows, N (two weights: of each) features.
Gemm16Plan plan_forward(Gemm16Op op, int M, int N, int nk, int num_sms) {
  const Choice pair = plan_pair(op, {M, N, nk, 1, 1}, {}, num_sms);
  const Choice swapped = M <= SWAP_ROWS ? plan_swap(op, M, N, nk, num_sms) : Choice{};
  return M <= PAIR_ROWS || (swapped.cycles > 0 && swapped.cycles < pair.cycles) ? swapped.plan : pair.plan;
}

// ------------------------------------------------------------------ operands
struct Operand {
  const void* ptr;
  uint64_t inner, rows, ld;   // innermost extent, rows, row stride in elements
};
CUtensorMapDataType map_type(svdq_dtype dt) {
  return dt == SVDQ_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Rows of one part's partials: whole store boxes, so that none reaches into the next part.
long long part_rows(int M, int stacked) { return ((long long)M + 31) / 32 * 32 * stacked; }
// A job's maps: operands in boxes of 64 along their inner extent, outputs in
// the epilogue's store boxes.
bool encode_job(const Gemm16Plan& plan, svdq_dtype dt, const Operand& a, const Operand* a2, const Operand& b,
                const Operand* b2, const Gemm16Job& j, void* Z, void* Z2, CUtensorMap* m) {
  const CUtensorMapDataType t = map_type(dt);
  const bool grad = plan.op == GEMM16_GRAD;
  const uint32_t a_box = grad && j.a_mn ? 64 : 128, b_box = grad ? 64 : plan.swap ? plan.bn : plan.bn / 2;
  auto in = [&](CUtensorMap* to, const Operand& o, uint32_t box) {
    return encode_tensor_map_2d(to, t, o.ptr, o.inner, o.rows, o.ld * 2, 64, box);
  };
  const uint32_t cols = plan.swap ? 128 : gemm16_box_cols(plan), rows = plan.swap ? plan.bn / plan.splits : 32;
  const CUtensorMapSwizzle swz = plan.swap    ? CU_TENSOR_MAP_SWIZZLE_NONE
                                 : cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B
                                              : CU_TENSOR_MAP_SWIZZLE_64B;
  auto out = [&](CUtensorMap* to, void* ptr, uint64_t ld) {
    return encode_tensor_map_2d(to, t, ptr, j.N, j.M, ld * 2, cols, rows, swz);
  };
  auto partials = [&](CUtensorMap* to) {
    return encode_tensor_map_2d(to, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, j.P, j.N,
                                j.parts * part_rows(j.M, j.Y2 ? 2 : 1), (uint64_t)j.N * 4, 32, 32,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!in(&m[MAP_A], a, a_box) || !in(&m[MAP_B], b, b_box)) return false;
  if (!(j.parts > 1 ? partials(&m[MAP_Y]) : out(&m[MAP_Y], j.Y, j.ldy))) return false;
  m[MAP_A2] = m[MAP_A];
  m[MAP_B2] = m[MAP_B];
  m[MAP_Z] = m[MAP_Z2] = m[MAP_Y];
  if (a2 && !in(&m[MAP_A2], *a2, a_box)) return false;
  if (b2 && !in(&m[MAP_B2], *b2, b_box)) return false;
  if (Z && !out(&m[MAP_Z], Z, j.N)) return false;
  if (Z2 && !out(&m[MAP_Z2], Z2, j.N)) return false;
  return !j.Y2 || out(&m[MAP_Y2], j.Y2, j.ldy);
}

// Y [M][N] = epilogue(X W^T) of row-major X [M][K] and W [N][K] (two weights: gated)
svdq_status forward_product(const DeviceInfo& d, svdq_dtype dt, int M, int K, int N, const void* X, long long ldx,
                            const void* W, const void* W2, void* Y, long long ldy, Gemm16Params p,
                            cudaStream_t stream) {
  const Gemm16Op op = W2 ? GEMM16_GATED : GEMM16_NT;
  const int nk = ceil_div(K, 64);
  const Operand x{X, (uint64_t)K, (uint64_t)M, (uint64_t)ldx}, w{W, (uint64_t)K, (uint64_t)N, (uint64_t)K},
      w2{W2, (uint64_t)K, (uint64_t)N, (uint64_t)K};
  Gemm16Job& j = p.job[0];
  j.M = M;
  j.N = N;
  j.nk1 = j.nk = nk;
  j.parts = 1;
  j.Y = out16(Y);
  j.ldy = ldy;
  const Gemm16Plan plan = plan_forward(op, M, N, nk, d.num_sms);
  Gemm16Maps<2> maps;
  bool ok;
  if (plan.swap) {
    j.tiles_m = ceil_div(N, 128);
    j.tiles_n = ceil_div(M, plan.bn);
    ok = encode_job(plan, dt, w, W2 ? &w2 : nullptr, x, nullptr, j, p.Z, p.Z2, maps.m[0]);
  } else {
    j.tiles_m = ceil_div(M, plan.tall ? 512 : 256);
    j.tiles_n = ceil_div(N, W2 ? plan.bn / 2 : plan.bn);
    ok = encode_job(plan, dt, x, nullptr, w, W2 ? &w2 : nullptr, j, p.Z, p.Z2, maps.m[0]);
  }
  j.tiles_m1 = j.tiles_m;
  if (!ok) return SVDQ_ERR_CUDA;
  p.fp16 = dt == SVDQ_FP16;
  p.err = d.err;
  return cuda_status(launch_gemm16(plan, maps, p, d.num_sms, stream));
}

// Ranges the reduction of an output of rows x cols may be cut into: at least 8
// k-tiles each, at most 32 of them and 148 x 256 x 128 float32 partials.
int most_parts(long long rows, int cols, int nk) {
  const long long fit = 148ll * 256 * 128 / (rows * cols);   // rows: of the partials
  return (int)std::max(1ll, std::min(std::min(fit, 32ll), nk / 8ll));
}
// The partials' bytes in a backward pass's workspace: dX's, then dW's.
struct PartBytes {
  size_t dx, dw;
};
PartBytes part_bytes(int M, int K, int N, bool two) {
  auto bytes = [&](long long rows, int nk) {
    const int parts = rows ? most_parts(rows, K, nk) : 1;
    return parts > 1 ? align256((size_t)parts * rows * K * 4) : 0;
  };
  return {bytes(part_rows(M, 1), ceil_div(N, 64) * (two ? 2 : 1)), bytes(part_rows(N, two ? 2 : 1), ceil_div(M, 64))};
}

size_t partials_bytes(int M, int K, int N, bool two) {
  const PartBytes b = part_bytes(M, K, N, two);
  return b.dx + b.dw;
}

// The products of a backward pass: the gradients asked for as jobs, the one of
// the longer tiles first, and their tiling.
struct BackwardPlan {
  int jobs = 0, at_w = -1, at_x = -1;   // of which number
  JobShape shape[2] = {};
  Choice choice;
};
BackwardPlan plan_backward(int M, int K, int N, bool two, bool dW, bool dX, int num_sms) {
  BackwardPlan b;
  const int nk_w = ceil_div(M, 64), nk_x = ceil_div(N, 64) * (two ? 2 : 1);
  const bool x_first = dX && (!dW || nk_x > nk_w);
  if (dW) {
    b.at_w = x_first ? 1 : 0;
    b.shape[b.at_w] = {N, K, nk_w, two ? 2 : 1, most_parts(part_rows(N, two ? 2 : 1), K, nk_w)};
    ++b.jobs;
  }
  if (dX) {
    b.at_x = dW && !x_first ? 1 : 0;
    b.shape[b.at_x] = {M, K, nk_x, 1, most_parts(part_rows(M, 1), K, nk_x)};
    ++b.jobs;
  }
  if (b.jobs) b.choice = plan_pair(GEMM16_GRAD, b.shape[0], b.shape[1], num_sms);
  return b;
}

// The products of a backward pass, dZ (and dZ2) [M][N] of row stride ldz:
//   dW [N][K] = dZ^T X, dW2 = dZ2^T X (stacked below it)   when dW
//   dX [M][K] = dZ W + dZ2 W2                              when dX
// and the bias gradients' sums (p.parts ...), in one launch.
struct Backward {
  int M, K, N;
  const void *dZ, *dZ2, *X, *W, *W2;
  long long ldz, ldx, lddx;
  void *dX, *dW, *dW2;
  uint8_t* partials;   // part_bytes
};
svdq_status backward_products(const DeviceInfo& d, svdq_dtype dt, const Backward& g, Gemm16Params p,
                              cudaStream_t stream) {
  const uint64_t M = g.M, K = g.K, N = g.N, ldz = g.ldz;
  const Operand z{g.dZ, N, M, ldz}, z2{g.dZ2, N, M, ldz}, w{g.W, K, N, K}, w2{g.W2, K, N, K},
      x{g.X, K, M, (uint64_t)g.ldx};
  const bool two = g.dZ2 != nullptr;
  const BackwardPlan b = plan_backward(g.M, g.K, g.N, two, g.dW, g.dX, d.num_sms);
  const int jobs = b.jobs, at_w = b.at_w, at_x = b.at_x;
  if (!jobs) return SVDQ_OK;
  if (at_w >= 0) {
    Gemm16Job& j = p.job[at_w];
    j.M = g.N;
    j.N = g.K;
    j.nk1 = j.nk = b.shape[at_w].nk;
    j.a_mn = 1;
    j.Y = out16(g.dW);
    j.Y2 = out16(g.dW2);
    j.ldy = g.K;
    j.P = reinterpret_cast<float*>(g.partials + part_bytes(g.M, g.K, g.N, two).dx);
  }
  if (at_x >= 0) {
    Gemm16Job& j = p.job[at_x];
    j.M = g.M;
    j.N = g.K;
    j.nk1 = ceil_div(g.N, 64);
    j.nk = b.shape[at_x].nk;
    j.Y = out16(g.dX);
    j.ldy = g.lddx;
    j.P = reinterpret_cast<float*>(g.partials);
  }
  const Gemm16Plan& plan = b.choice.plan;
  for (int i = 0; i < jobs; ++i) {
    p.job[i].tiles_n = ceil_div(g.K, plan.bn);
    p.job[i].tiles_m1 = ceil_div(b.shape[i].M, plan.tall ? 512 : 256);
    p.job[i].tiles_m = b.shape[i].stacked * p.job[i].tiles_m1;
    p.job[i].parts = b.choice.parts[i];
  }
  Gemm16Maps<2> maps;
  if (at_w >= 0 &&
      !encode_job(plan, dt, z, two ? &z2 : nullptr, x, nullptr, p.job[at_w], nullptr, nullptr, maps.m[at_w]))
    return SVDQ_ERR_CUDA;
  if (at_x >= 0 && !encode_job(plan, dt, z, two ? &z2 : nullptr, w, two ? &w2 : nullptr, p.job[at_x], nullptr, nullptr,
                               maps.m[at_x]))
    return SVDQ_ERR_CUDA;
  if (jobs == 1)
    for (int i = 0; i < MAPS; ++i) maps.m[1][i] = maps.m[0][i];
  p.fp16 = dt == SVDQ_FP16;
  p.err = d.err;
  const svdq_status s = cuda_status(launch_gemm16(plan, maps, p, d.num_sms, stream));
  Gemm16Job cut[2];
  int cuts = 0;
  for (int i = 0; i < jobs; ++i)
    if (p.job[i].parts > 1) cut[cuts++] = p.job[i];
  return s != SVDQ_OK || !cuts ? s : cuda_status(launch_join_parts(cut, cuts, p.fp16, stream));
}

cudaError_t zero(void* p, size_t bytes, cudaStream_t stream) {
  return p ? cudaMemsetAsync(p, 0, bytes, stream) : cudaSuccess;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ how products are tiled (test hook)
svdq_status svdq_debug_product_plan(int op, int M, int K, int N, int num_sms, int* plan) {
  if (op < 0 || op > 3 || !plan || num_sms < 8) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || M == 0 || !width_ok(K) || !width_ok(N)) return SVDQ_ERR_SHAPE;
  Gemm16Plan g;
  int parts_x = 1, parts_w = 1;
  if (op < 2) {
    g = plan_forward(op ? GEMM16_GATED : GEMM16_NT, M, N, ceil_div(K, 64), num_sms);
  } else {
    const BackwardPlan b = plan_backward(M, K, N, op == 3, true, true, num_sms);
    g = b.choice.plan;
    parts_x = b.choice.parts[b.at_x];
    parts_w = b.choice.parts[b.at_w];
  }
  const int out[6] = {g.swap, g.bn, g.splits, g.tall, parts_x, parts_w};
  std::copy(out, out + 6, plan);
  return SVDQ_OK;
}

// ------------------------------------------------------------------ dense linear
svdq_status svdq_dense_linear(svdq_dtype dt, int M, int K, int N, const void* X, long long ldx, const void* W_t,
                              const void* bias, svdq_epilogue act, const void* residual, long long ldr, void* Y,
                              long long ldy, void* Z, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !W_t || (M > 0 && (!X || !Y))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !width_ok(K) || !width_ok(N) || !stride_ok(ldx, K) || !stride_ok(ldy, N) ||
      (residual && !stride_ok(ldr, N)))
    return SVDQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(W_t) || !aligned16(bias) || !aligned16(residual) || !aligned16(Y) || !aligned16(Z))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  DeviceInfo d;
  const svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  Gemm16Params p = {};
  p.act = act;
  p.bias = in16(bias);
  p.R = in16(residual);
  p.ldr = ldr;
  p.Z = out16(Z);
  return forward_product(d, dt, M, K, N, X, ldx, W_t, nullptr, Y, ldy, p, stream);
}

// [dZ when there is an activation | the bias gradient's partials | the products' partials]
size_t svdq_dense_linear_backward_workspace_bytes(int M, int K, int N, svdq_epilogue act) {
  if (!rows_ok(M) || !width_ok(K) || !width_ok(N) || !known_act(act)) return 0;
  return (act == SVDQ_EPI_NONE ? 0 : align256((size_t)M * N * 2)) +
         align256((size_t)act_grad_parts(M, N) * N * 4) + partials_bytes(M, K, N, false);
}

svdq_status svdq_dense_linear_backward(svdq_dtype dt, int M, int K, int N, const void* dY, long long lddy,
                                       const void* X, long long ldx, const void* W_t, const void* Z,
                                       svdq_epilogue act, void* dX, long long lddx, void* dW, void* dbias,
                                       void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act)) return SVDQ_ERR_INVALID_ARG;
  if (M > 0 && (!dY || (act != SVDQ_EPI_NONE && !Z) || (dX && !W_t) || (dW && !X))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !width_ok(K) || !width_ok(N) || !stride_ok(lddy, N) || (dW && !stride_ok(ldx, K)) ||
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
  const bool products = dX || dW;
  Gemm16Params q = {};
  if ((has_act && products) || dbias) {
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
    if (dbias) {
      if (!products) return cuda_status(launch_sum_parts(part, p.parts, N, dt, dbias, nullptr, nullptr, stream));
      q.parts = p.parts;
      q.part_n = N;
      q.part = part;
      q.dbias = out16(dbias);
    }
  }
  const void* dZ = has_act ? workspace : dY;
  const long long ldz = has_act ? N : lddy;
  uint8_t* partials = reinterpret_cast<uint8_t*>(part) + align256((size_t)act_grad_parts(M, N) * N * 4);
  return backward_products(d, dt, {M, K, N, dZ, nullptr, X, W_t, nullptr, ldz, ldx, lddx, dX, dW, nullptr, partials}, q,
                           stream);
}

// ------------------------------------------------------------------ gated feed-forward
svdq_status svdq_gated_linear(svdq_dtype dt, int M, int K, int F, const void* X, long long ldx, const void* Wg_t,
                              const void* Wu_t, const void* bias_g, const void* bias_u, svdq_epilogue act, void* H,
                              long long ldh, void* G, void* U, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !Wg_t || !Wu_t || (M > 0 && (!X || !H))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !width_ok(K) || !width_ok(F) || !stride_ok(ldx, K) || !stride_ok(ldh, F)) return SVDQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(Wg_t) || !aligned16(Wu_t) || !aligned16(bias_g) || !aligned16(bias_u) ||
      !aligned16(H) || !aligned16(G) || !aligned16(U))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  DeviceInfo d;
  const svdq_status s = current_device_info(&d);
  if (s != SVDQ_OK) return s;
  Gemm16Params p = {};
  p.act = act;
  p.bias = in16(bias_g);
  p.bias2 = in16(bias_u);
  p.Z = out16(G);
  p.Z2 = out16(U);
  return forward_product(d, dt, M, K, F, X, ldx, Wg_t, Wu_t, H, ldh, p, stream);
}

// [dG | dU | the two bias gradients' partials | the products' partials]
size_t svdq_gated_linear_backward_workspace_bytes(int M, int K, int F) {
  if (!rows_ok(M) || !width_ok(K) || !width_ok(F)) return 0;
  return 2 * align256((size_t)M * F * 2) + 2 * align256((size_t)act_grad_parts(M, F) * F * 4) +
         partials_bytes(M, K, F, true);
}

svdq_status svdq_gated_linear_backward(svdq_dtype dt, int M, int K, int F, const void* dH, long long lddh,
                                       const void* X, long long ldx, const void* Wg_t, const void* Wu_t,
                                       const void* G, const void* U, svdq_epilogue act, void* dX, long long lddx,
                                       void* dWg, void* dWu, void* dbias_g, void* dbias_u, void* workspace,
                                       size_t ws_bytes, cudaStream_t stream) {
  if (!type16(dt) || !known_act(act) || !dWg != !dWu || !dbias_g != !dbias_u) return SVDQ_ERR_INVALID_ARG;
  if (M > 0 && (!dH || !G || !U || (dX && (!Wg_t || !Wu_t)) || (dWg && !X))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !width_ok(K) || !width_ok(F) || !stride_ok(lddh, F) || (dWg && !stride_ok(ldx, K)) ||
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
  if (!dX && !dWg && !dbias_g) return SVDQ_OK;
  if ((s = cuda_status(launch_act_grad(p, stream))) != SVDQ_OK) return s;
  if (!dX && !dWg) return cuda_status(launch_sum_parts(part, p.parts, F, dt, dbias_g, part2, dbias_u, stream));
  Gemm16Params q = {};
  if (dbias_g) {
    q.parts = p.parts;
    q.part_n = F;
    q.part = part;
    q.part2 = part2;
    q.dbias = out16(dbias_g);
    q.dbias2 = out16(dbias_u);
  }
  uint8_t* partials = reinterpret_cast<uint8_t*>(part2) + align256((size_t)p.parts * F * 4);
  return backward_products(
      d, dt, {M, K, F, p.dZ, p.dU, X, Wg_t, Wu_t, F, ldx, lddx, dX, dWg, dWu, partials}, q, stream);
}

// ------------------------------------------------------------------ layer norm
static size_t elem_bytes(svdq_dtype dt) { return dt == SVDQ_FP32 ? 4 : 2; }
static bool elem_aligned(svdq_dtype dt, const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & (elem_bytes(dt) - 1)) == 0;
}
static bool float_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
// covers the row, under the 2^40 bytes that every 16-bit call takes: offsets stay far from 64 bits' end
static bool row_stride_ok(svdq_dtype dt, long long ld, int C) {
  return ld >= C && ld < (1ll << 40) / (long long)elem_bytes(dt);
}
static bool length_ok(int C) { return C >= 1 && C <= MOST; }
static bool known_type(svdq_dtype dt) { return dt == SVDQ_BF16 || dt == SVDQ_FP16 || dt == SVDQ_FP32; }

svdq_status svdq_layernorm(svdq_dtype dt, int M, int C, const void* X, long long ldx, const void* gamma,
                           const void* beta, float eps, void* Y, long long ldy, float* mean, float* rstd,
                           cudaStream_t stream) {
  if (!known_type(dt) || !gamma != !beta || (M > 0 && (!X || !Y)) || !(eps >= 0.f) || !std::isfinite(eps))
    return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !length_ok(C) || !row_stride_ok(dt, ldx, C) || !row_stride_ok(dt, ldy, C)) return SVDQ_ERR_SHAPE;
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
  if (!rows_ok(M) || !length_ok(C)) return 0;
  // the first 256 keep it above zero for M = 0: zero means refused
  return 256 + 2 * align256((size_t)layernorm_grad_parts(M, C) * C * 4);
}

svdq_status svdq_layernorm_backward(svdq_dtype dt, int M, int C, const void* dY, long long lddy, const void* X,
                                    long long ldx, const void* gamma, const float* mean, const float* rstd, void* dX,
                                    long long lddx, void* dgamma, void* dbeta, void* workspace, size_t ws_bytes,
                                    cudaStream_t stream) {
  if (!known_type(dt) || !dgamma != !dbeta || (M > 0 && (!dY || !X || !mean || !rstd))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_ok(M) || !length_ok(C) || !row_stride_ok(dt, lddy, C) || !row_stride_ok(dt, ldx, C) ||
      (dX && !row_stride_ok(dt, lddx, C)))
    return SVDQ_ERR_SHAPE;
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

// ------------------------------------------------------------------ a W4A4 layer behind its norm
static size_t normed_bytes(const svdq_weights_info& i, int M) { return align256((size_t)M * i.K * 2); }

size_t svdq_norm_linear_workspace_bytes(const svdq_weights* w, int M) {
  svdq_weights_info i;
  if (M < 0 || svdq_weights_view(w, &i) != SVDQ_OK) return 0;
  return normed_bytes(i, M) + svdq_linear_workspace_bytes(w, M);
}

svdq_status svdq_norm_linear(const svdq_weights* w, int M, const void* X, const void* gamma, const void* beta,
                             float eps, svdq_epilogue epi, void* Y, void* workspace, size_t ws_bytes,
                             cudaStream_t stream) {
  svdq_weights_info i;
  if (svdq_weights_view(w, &i) != SVDQ_OK || (M > 0 && (!X || !Y))) return SVDQ_ERR_INVALID_ARG;
  if (epi != SVDQ_EPI_NONE && epi != SVDQ_EPI_GELU_TANH) return SVDQ_ERR_INVALID_ARG;
  if (!gamma != !beta || !(eps >= 0.f) || !std::isfinite(eps)) return SVDQ_ERR_INVALID_ARG;
  if (M < 0) return SVDQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(gamma) || !aligned16(beta) || (reinterpret_cast<uintptr_t>(Y) & 31u))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) return SVDQ_OK;
  if (!workspace || ws_bytes < svdq_norm_linear_workspace_bytes(w, M)) return SVDQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SVDQ_ERR_ALIGNMENT;
  svdq_status s = handle_device_status(w);
  if (s != SVDQ_OK) return s;
  uint8_t* rest = static_cast<uint8_t*>(workspace) + normed_bytes(i, M);
  s = svdq_layernorm(SVDQ_BF16, M, i.K, X, i.K, gamma, beta, eps, workspace, i.K, nullptr, nullptr, stream);
  return s != SVDQ_OK ? s : svdq_linear(w, M, workspace, epi, Y, rest, ws_bytes - normed_bytes(i, M), stream);
}

}  // extern "C"
