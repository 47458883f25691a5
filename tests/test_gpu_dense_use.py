"""The 16-bit layers as a program uses them: a pre-norm gated feed-forward
block forward and backward, a quantized layer behind its norm, CUDA graphs,
several streams, empty and padded batches, special values, sizes past 32-bit
offsets.  Parity bars are test_gpu_dense.py's (see there for their
derivation)."""
import math
import random

import pytest
import torch

import test_gpu_dense as D
import workloads
from svdq_harness import GpuLayer, dev_bf16

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from rank_gemm_b200 import binding
    return binding


@pytest.fixture(autouse=True)
def no_device_error(B):
    yield
    assert B.svdq_poll_device_error() == 0


# ---------------------------------------------------------------- one block, forward and backward
class Block:
    """Y = X + act(n Wg^T + bg) * (n Wu^T + bu) Wd^T + bd, n = LayerNorm(X)."""
    NAMES = ("X", "gamma", "beta", "Wg", "Wu", "bg", "bu", "Wd", "bd")

    def __init__(self, t, M, C, F, act, seed):
        g = D.gen(seed)
        self.t, self.M, self.C, self.F, self.act = t, M, C, F, act
        self.X = D.draw(g, t, M, C, scale=2.0)
        self.gamma, self.beta = (1 + D.draw(g, t, C, scale=0.2)).to(t), D.draw(g, t, C, scale=0.2)
        self.Wg, self.Wu = D.draw(g, t, F, C, scale=C ** -0.5), D.draw(g, t, F, C, scale=C ** -0.5)
        self.bg, self.bu = D.draw(g, t, F, scale=0.1), D.draw(g, t, F, scale=0.1)
        self.Wd, self.bd = D.draw(g, t, C, F, scale=F ** -0.5), D.draw(g, t, C, scale=0.1)
        self.dY = D.draw(g, t, M, C)

    def new(self, *shape, dtype=None):
        return D.nan_like(dtype or self.t, *shape)

    def run(self, B):
        """(Y, gradients by name) through the library."""
        t, M, C, F, a = self.t, self.M, self.C, self.F, D.ACTS[self.act]
        n, mean, rstd = self.new(M, C), self.new(M, dtype=torch.float32), self.new(M, dtype=torch.float32)
        G, U, H, Y = self.new(M, F), self.new(M, F), self.new(M, F), self.new(M, C)
        B.svdq_layernorm(M, C, self.X, self.gamma, self.beta, 1e-5, n, mean, rstd)
        B.svdq_gated_linear(M, C, F, n, self.Wg, self.Wu, self.bg, self.bu, a, H, G, U)
        B.svdq_dense_linear(M, F, C, H, self.Wd, self.bd, 0, self.X, Y)
        out = {k: self.new(*getattr(self, k).shape) for k in self.NAMES}
        dH, dn = self.new(M, F), self.new(M, C)
        need = max(B.svdq_dense_linear_backward_workspace_bytes(M, F, C, 0),
                   B.svdq_gated_linear_backward_workspace_bytes(M, C, F),
                   B.svdq_layernorm_backward_workspace_bytes(M, C))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")   # shared by the three: one stream
        B.svdq_dense_linear_backward(M, F, C, self.dY, H, self.Wd, None, 0, dH, out["Wd"], out["bd"], ws)
        B.svdq_gated_linear_backward(M, C, F, dH, n, self.Wg, self.Wu, G, U, a, dn, out["Wg"], out["Wu"], out["bg"],
                                     out["bu"], ws)
        B.svdq_layernorm_backward(M, C, dn, self.X, self.gamma, mean, rstd, out["X"], out["gamma"], out["beta"], ws)
        torch.cuda.synchronize()
        out["X"] = (out["X"].float() + self.dY.float()).to(t)       # the residual's share
        return Y, out

    def forward64(self, v):
        m, r = D.norm64(v["X"], 1e-5)
        n = (v["X"] - m) * r * v["gamma"] + v["beta"]
        h = D.act64(n @ v["Wg"].T + v["bg"], self.act)[0] * (n @ v["Wu"].T + v["bu"])
        return v["X"] + h @ v["Wd"].T + v["bd"]

    def values64(self):
        return {k: getattr(self, k).double() for k in self.NAMES}


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,C,F,act", [(1, 64, 128, "silu"), (70, 136, 328, "gelu"), (300, 264, 520, "silu"),
                                       (1030, 128, 256, "none")])
def test_block_forward_and_gradients(B, t, M, C, F, act):
    """Gradients against central differences of the float64 forward along
    random directions, and against autograd of it.  Every stage rounds to 16
    bits and there are at most six in a row, independent over at least 64
    terms: 12 half steps of the value's norm, in the 2-norm, is a bound with a
    factor of two to spare; a wrong term shows as an error of order one."""
    b = Block(t, M, C, F, act, seed=M)
    Y, grads = b.run(B)
    v = b.values64()
    want = b.forward64(v)
    u = D.half_step(t)
    assert float((Y.double() - want).norm()) <= 12 * u * float(want.norm())
    leaves = {k: x.clone().requires_grad_() for k, x in v.items()}
    auto = dict(zip(leaves, torch.autograd.grad(b.forward64(leaves), list(leaves.values()), b.dY.double())))
    g = D.gen(77)
    for k in b.NAMES:
        got = grads[k].double()
        assert float((got - auto[k]).norm()) <= 12 * u * float(auto[k].norm()), k
        d = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = (b.forward64(dict(v, **{k: v[k] + s * h * d})) for s in (1, -1))
        numeric = float(((up - down) / (2 * h) * b.dY.double()).sum())
        # the difference itself is good to 1e-6 of its terms; the gradient's error enters along d
        bound = 12 * u * float(auto[k].norm()) * float(d.norm()) + 1e-6 * float(((up - down).abs() / (2 * h)
                                                                                 * b.dY.double().abs()).sum())
        assert abs(float((got * d).sum()) - numeric) <= bound, k


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slope_against_differences(B, act):
    """dZ of the dense backward (dX with the identity as weight) against
    central differences of act in float64: truncation h^2 / 6 |act'''| <= 2e-9
    at h = 1e-4, rounding 1e-11; the kernel's slope 2^-18, one half step of dZ
    and one of dX."""
    N = 64
    z = torch.linspace(-12, 12, 64 * N, device="cuda").reshape(64, N).to(torch.float16)
    W = torch.eye(N, device="cuda", dtype=torch.float16)
    dX = D.nan_like(torch.float16, 64, N)
    ws = torch.empty(B.svdq_dense_linear_backward_workspace_bytes(64, N, N, D.ACTS[act]), dtype=torch.uint8, device="cuda")
    B.svdq_dense_linear_backward(64, N, N, torch.ones_like(z), None, W, z, D.ACTS[act], dX, None, None, ws)
    x, h = z.double(), 1e-4
    num = (D.act64(x + h, act)[0] - D.act64(x - h, act)[0]) / (2 * h)
    u = D.half_step(torch.float16)
    assert bool(((dX.double() - num).abs() <= 2 * u * num.abs() + 2.0 ** -18 + 1e-8).all())


# ---------------------------------------------------------------- the quantized layer behind its norm
@pytest.mark.parametrize("M", [1, 130])
@pytest.mark.parametrize("affine", [True, False])
def test_norm_linear_is_the_two_calls(B, M, affine):
    L = workloads.draw_layer("norm_linear", "nvfp4", M, 512, 272, 32, seed=91, n_out=4)
    g = GpuLayer(L.fmt, L.X, L.W, L.bias, L.rank)
    try:
        X = dev_bf16(L.X)
        ga, be = (D.draw(D.gen(1), BF, 512), D.draw(D.gen(2), BF, 512)) if affine else (None, None)
        n, Y, want = D.nan_like(BF, M, 512), D.nan_like(BF, M, L.N), D.nan_like(BF, M, L.N)
        B.svdq_layernorm(M, 512, X, ga, be, 1e-6, n)
        B.svdq_linear(g.h, M, n, 1, want, torch.empty(B.svdq_linear_workspace_bytes(g.h, M), dtype=torch.uint8,
                                                      device="cuda"))
        size = B.svdq_norm_linear_workspace_bytes(g.h, M)
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        B.svdq_norm_linear(g.h, M, X, ga, be, 1e-6, 1, Y, ws)
        assert torch.equal(Y, want)
        for bad in (dict(ws_bytes=size - 1), dict(epi=2), dict(eps=-1.0)):
            kw = dict(dict(eps=1e-6, epi=1, ws_bytes=size), **bad)
            with pytest.raises(B.SvdqError) as e:
                B.svdq_norm_linear(g.h, M, X, ga, be, kw["eps"], kw["epi"], Y, ws, ws_bytes=kw["ws_bytes"])
            assert e.value.status == (5 if "ws_bytes" in bad else 1)
        B.svdq_norm_linear(g.h, 0, X, ga, be, 1e-6, 1, Y, ws)
    finally:
        g.close()


def test_w4a4_layers_refuse_the_silu_epilogue(B):
    L = workloads.draw_layer("silu_refused", "nvfp4", 4, 256, 64, 16, seed=92, n_out=2)
    g = GpuLayer(L.fmt, L.X, L.W, L.bias, L.rank)
    try:
        Y = D.nan_like(BF, 4, 64)
        ws = torch.empty(B.svdq_linear_workspace_bytes(g.h, 4), dtype=torch.uint8, device="cuda")
        with pytest.raises(B.SvdqError) as e:
            B.svdq_linear(g.h, 4, dev_bf16(L.X), B.SVDQ_EPI_SILU, Y, ws)
        assert e.value.status == 1
    finally:
        g.close()


# ---------------------------------------------------------------- graphs, streams, repeats
def all_calls(B, t, M, K, N, seed):
    """Every entry point once on inputs of its own: (run, outputs, inputs)."""
    g = D.gen(seed)
    X, dY, dX = D.draw(g, t, M, K), D.draw(g, t, M, N, scale=0.2), D.nan_like(t, M, K)
    W, W2, b = D.draw(g, t, N, K, scale=0.05), D.draw(g, t, N, K, scale=0.05), D.draw(g, t, N)
    Z, U, R = D.draw(g, t, M, N), D.draw(g, t, M, N), D.draw(g, t, M, N)
    o = {k: D.nan_like(t, M, N) for k in ("Y", "Z", "H", "G", "U")}
    o.update({k: D.nan_like(t, N, K) for k in ("dW", "dWg", "dWu")}, **{k: D.nan_like(t, N) for k in ("db", "dbg", "dbu")},
             dX=dX, dX2=D.nan_like(t, M, K), dX3=D.nan_like(t, M, K), n=D.nan_like(t, M, K), dga=D.nan_like(t, K),
             dbe=D.nan_like(t, K), mean=D.nan_like(torch.float32, M), rstd=D.nan_like(torch.float32, M))
    ga, be = D.draw(g, t, K), D.draw(g, t, K)
    size = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    ws = [size(B.svdq_dense_linear_backward_workspace_bytes(M, K, N, 1)),
          size(B.svdq_gated_linear_backward_workspace_bytes(M, K, N)), size(B.svdq_layernorm_backward_workspace_bytes(M, K))]

    def run(stream=None):
        B.svdq_dense_linear(M, K, N, X, W, b, 1, R, o["Y"], o["Z"], stream=stream)
        B.svdq_dense_linear_backward(M, K, N, dY, X, W, Z, 1, o["dX"], o["dW"], o["db"], ws[0], stream=stream)
        B.svdq_gated_linear(M, K, N, X, W, W2, b, b, 2, o["H"], o["G"], o["U"], stream=stream)
        B.svdq_gated_linear_backward(M, K, N, dY, X, W, W2, Z, U, 2, o["dX2"], o["dWg"], o["dWu"], o["dbg"], o["dbu"],
                                     ws[1], stream=stream)
        B.svdq_layernorm(M, K, X, ga, be, 1e-5, o["n"], o["mean"], o["rstd"], stream=stream)
        B.svdq_layernorm_backward(M, K, o["dX"], X, ga, o["mean"], o["rstd"], o["dX3"], o["dga"], o["dbe"], ws[2],
                                  stream=stream)
    return run, o, (X, dY, Z, U)


def snapshot(o):
    torch.cuda.synchronize()
    return {k: v.clone() for k, v in o.items()}


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


SHAPES = [(1, 256, 384), (40, 1024, 512), (333, 264, 520), (700, 512, 264), (5, 96, 4104), (4100, 136, 96)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_graphs_replay_the_eager_bits(B, M, K, N):
    """Captured, then replayed on inputs written after the capture; a second
    graph of the same calls shares their workspaces."""
    run, o, ins = all_calls(B, BF, M, K, N, seed=3)
    run()
    first = snapshot(o)
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        run()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                run()
            graphs.append(g)
    torch.cuda.synchronize()
    for g in graphs:
        for v in o.values():
            v.fill_(float("nan"))
        g.replay()
        same(snapshot(o), first)
    for x in ins:
        x.copy_(torch.roll(x, 1, 0) * 0.5)
    run()
    second = snapshot(o)
    for v in o.values():
        v.fill_(float("nan"))
    graphs[0].replay()
    graphs[1].replay()
    same(snapshot(o), second)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_two_streams_at_once_and_repeats(B, M, K, N):
    jobs = [all_calls(B, BF, M, K, N, seed=s) for s in (4, 5)]
    want = []
    for run, o, _ in jobs:
        run()
        want.append(snapshot(o))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, o, _), s in zip(jobs, streams):
            run(s)          # handed over, not current
    for (_, o, _), w in zip(jobs, want):
        same(snapshot(o), w)


# ---------------------------------------------------------------- batches
def test_empty_batches(B):
    """M = 0 writes zero weight and bias gradients and nothing else."""
    t, K, N = torch.float16, 64, 136
    _, o, _ = all_calls(B, t, 1, K, N, seed=6)
    e = torch.empty(0, K, dtype=t, device="cuda")
    en = torch.empty(0, N, dtype=t, device="cuda")
    W = torch.zeros(N, K, dtype=t, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    B.svdq_dense_linear(0, K, N, e, W, None, 0, None, en)
    B.svdq_gated_linear(0, K, N, e, W, W, None, None, 2, en)
    B.svdq_layernorm(0, K, e, None, None, 1e-5, e)
    B.svdq_dense_linear_backward(0, K, N, en, e, W, None, 0, e, o["dW"], o["db"], ws)
    B.svdq_gated_linear_backward(0, K, N, en, e, W, W, en, en, 2, e, o["dWg"], o["dWu"], o["dbg"], o["dbu"], ws)
    m = torch.empty(0, dtype=torch.float32, device="cuda")
    B.svdq_layernorm_backward(0, K, e, e, None, m, m, e, o["dga"], o["dbe"], ws)
    torch.cuda.synchronize()
    for k in ("dW", "db", "dWg", "dWu", "dbg", "dbu", "dga", "dbe"):
        assert not bool(o[k].ne(0).any()), k
    assert bool(o["Y"].isnan().all()) and bool(o["dX"].isnan().all())


@pytest.mark.parametrize("M", [3, 33, 130, 257])
def test_rows_behind_the_batch_stay(B, M):
    """Outputs taller and wider than the batch keep what lies behind it, and
    rows of X behind it (NaN here) are not read into it."""
    t, K, N = BF, 136, 200
    g = D.gen(8)
    X = D.nan_like(t, M + 9, K)
    X[:M] = D.draw(g, t, M, K)
    W, b, R = D.draw(g, t, N, K, scale=0.05), D.draw(g, t, N), D.draw(g, t, M + 9, N + 8)
    Y = torch.full((M + 9, N + 8), 7.0, dtype=t, device="cuda")
    H, n, dX = Y.clone(), torch.full((M + 9, K + 8), 7.0, dtype=t, device="cuda"), torch.full((M + 9, K + 8), 7.0, dtype=t,
                                                                                         device="cuda")
    B.svdq_dense_linear(M, K, N, X, W, b, 2, R[:, :N], Y[:, :N])
    B.svdq_gated_linear(M, K, N, X, W, W, b, b, 2, H[:, :N])
    B.svdq_layernorm(M, K, X, None, None, 1e-5, n[:, :K])
    dW = D.nan_like(t, N, K)
    dY = D.nan_like(t, M + 9, N)
    dY[:M] = D.draw(g, t, M, N)
    ws = torch.empty(B.svdq_dense_linear_backward_workspace_bytes(M, K, N, 0), dtype=torch.uint8, device="cuda")
    B.svdq_dense_linear_backward(M, K, N, dY, X, W, None, 0, dX[:, :K], dW, None, ws)
    torch.cuda.synchronize()
    for out, w in ((Y, N), (H, N), (n, K), (dX, K)):
        assert bool(out[:M, :w].isfinite().all())
        assert bool((out[M:] == 7).all()) and bool((out[:, w:] == 7).all())
    assert bool(dW.isfinite().all())


@pytest.mark.parametrize("M", [20, 300])
def test_special_values_stay_in_their_row_and_column(B, M):
    """A NaN row of X, an infinity in a weight: only that row, that column."""
    t, K, N, F = BF, 200, 264, 264
    g = D.gen(9)
    X, W, W2, R = D.draw(g, t, M, K), D.draw(g, t, N, K, scale=0.05), D.draw(g, t, N, K, scale=0.05), D.draw(g, t, M, N)

    def outputs():
        Y, H, n = D.nan_like(t, M, N), D.nan_like(t, M, F), D.nan_like(t, M, K)
        B.svdq_dense_linear(M, K, N, X, W, None, 1, R, Y)
        B.svdq_gated_linear(M, K, F, X, W, W2, None, None, 2, H)
        B.svdq_layernorm(M, K, X, None, None, 1e-5, n)
        return Y, H, n

    clean = outputs()
    X[7, 3] = float("nan")
    R[11] = torch.finfo(t).min
    W[5, 100] = float("inf")
    Y, H, n = outputs()
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[7] = False
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[5] = False
    assert torch.equal(H[rows][:, cols], clean[1][rows][:, cols]) and torch.equal(n[rows], clean[2][rows])
    keep = rows.clone()
    keep[11] = False
    assert torch.equal(Y[keep][:, cols], clean[0][keep][:, cols])
    assert bool(Y[7].isnan().all()) and bool(H[7].isnan().all()) and bool(n[7].isnan().all())
    assert bool((~Y[keep][:, 5].isfinite() | (Y[keep][:, 5] == R[keep][:, 5])).all())   # inf, or act(-inf) + R
    assert bool((Y[11, cols] <= -3e38).all())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_columns_between_rows_are_not_read(B, M):
    """NaN in the columns between a row's end and the next row's start."""
    t, K, N = torch.float16, 72, 136
    g = D.gen(13)
    X, dY, R = D.nan_like(t, M, K + 56), D.nan_like(t, M, N + 56), D.nan_like(t, M, N + 56)
    X[:, :K], dY[:, :N], R[:, :N] = D.draw(g, t, M, K), D.draw(g, t, M, N), D.draw(g, t, M, N)
    W, Z = D.draw(g, t, N, K, scale=0.05), D.draw(g, t, M, N)
    Y, H, dX, dX2, n = (D.nan_like(t, M, w) for w in (N, N, K, K, K))
    dW, dW2, dW3, db = D.nan_like(t, N, K), D.nan_like(t, N, K), D.nan_like(t, N, K), D.nan_like(t, N)
    x, dy = X[:, :K], dY[:, :N]
    ws = torch.empty(B.svdq_gated_linear_backward_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    B.svdq_dense_linear(M, K, N, x, W, None, 0, R[:, :N], Y)
    B.svdq_gated_linear(M, K, N, x, W, W, None, None, 1, H)
    B.svdq_dense_linear_backward(M, K, N, dy, x, W, None, 0, dX, dW, db, ws)
    B.svdq_gated_linear_backward(M, K, N, dy, x, W, W, Z, Z, 1, dX2, dW2, dW3, None, None, ws)
    B.svdq_layernorm(M, K, x, None, None, 1e-5, n)
    for out in (Y, H, dX, dW, db, dX2, dW2, dW3, n):
        assert bool(out.isfinite().all())


@pytest.mark.parametrize("t,M,C,ld", [(BF, 700, 512, 512), (torch.float32, 40, 1001, 1003), (torch.float16, 3, 40000, 40000)])
def test_layernorm_in_place(B, t, M, C, ld):
    X = D.draw(D.gen(14), t, M, ld)[:, :C]
    Y = D.nan_like(t, M, C)
    B.svdq_layernorm(M, C, X, None, None, 1e-5, Y)
    B.svdq_layernorm(M, C, X, None, None, 1e-5, X)
    assert torch.equal(X, Y)


def test_zero_and_constant_rows(B):
    """A constant row: variance 0, rstd = 1 / sqrt(eps), the output is beta; with eps = 0 a NaN, as 0 * inf."""
    t, M, C = torch.float32, 4, 100
    X = torch.zeros(M, C, device="cuda")
    X[1] = 3.0
    X[2] = torch.randn(C, device="cuda")
    be = torch.randn(C, device="cuda")
    Y, mean, rstd = D.nan_like(t, M, C), D.nan_like(t, M), D.nan_like(t, M)
    B.svdq_layernorm(M, C, X, torch.ones(C, device="cuda"), be, 1e-5, Y, mean, rstd)
    assert torch.equal(Y[0], be) and torch.equal(Y[1], be) and torch.equal(Y[3], be)
    assert float(mean[1]) == 3.0 and abs(float(rstd[0]) * math.sqrt(1e-5) - 1) < 1e-6
    B.svdq_layernorm(M, C, X, None, None, 0.0, Y, mean, rstd)
    assert bool(Y[0].isnan().all()) and bool(Y[2].isfinite().all())


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("seed", range(12))
def test_random_sizes(B, seed):
    r = random.Random(seed)
    size = lambda hi: 8 * max(1, int(round(math.exp(r.uniform(0, math.log(hi / 8))))))  # noqa: E731
    M, K, N, t = int(round(math.exp(r.uniform(0, math.log(1500))))), size(2500), size(2500), r.choice(D.TYPES)
    act = r.choice(("none", "gelu", "silu"))
    D.run_linear(B, t, M, K, N, act, bias=r.random() < 0.5, residual=r.random() < 0.5, keep=r.random() < 0.5, seed=seed)
    D.run_linear_backward(B, t, M, K, N, act, seed=seed)
    D.run_gated(B, t, M, K, N, act, bias=r.random() < 0.5, keep=r.random() < 0.5, seed=seed)


def test_offsets_past_32_bits(B):
    """Outputs of more than 2^31 elements and rows of more than 2^31 elements
    apart: the last rows are checked."""
    t, M, K, N = BF, 270000, 64, 8192
    g = D.gen(10)
    X, W = D.draw(g, t, M, K), D.draw(g, t, N, K, scale=0.05)
    Y = torch.empty(M, N, dtype=t, device="cuda")
    B.svdq_dense_linear(M, K, N, X, W, None, 0, None, Y)
    for rows in (slice(0, 64), slice(M - 300, M)):
        D.close(Y[rows], X[rows].double() @ W.double().T, D.dot_bound(X[rows].double(), W.double().T, K), "Y")
    n = torch.empty_like(Y)
    B.svdq_layernorm(M, N, Y, None, None, 1e-5, n)
    x = Y[M - 8:].double()
    m, rs = D.norm64(x, 1e-5)
    assert float((n[M - 8:].double() - (x - m) * rs).norm()) <= 2 * D.half_step(t) * math.sqrt(8 * N)
    del n
    dX, dW = torch.empty_like(X), D.nan_like(t, N, K)
    ws = torch.empty(B.svdq_dense_linear_backward_workspace_bytes(M, K, N, 0), dtype=torch.uint8, device="cuda")
    B.svdq_dense_linear_backward(M, K, N, Y, X, W, None, 0, dX, None, None, ws)
    D.close(dX[M - 300:], Y[M - 300:].double() @ W.double(), D.dot_bound(Y[M - 300:].double(), W.double(), N), "dX")
    # two rows 2^31 + 64 elements apart
    big = torch.empty((1 << 31) + 64 + K, dtype=t, device="cuda")
    pair = torch.as_strided(big, (2, K), ((1 << 31) + 64, 1))
    pair.copy_(X[:2])
    Y2 = D.nan_like(t, 2, N)
    B.svdq_dense_linear(2, K, N, pair, W, None, 0, None, Y2)
    D.close(Y2, X[:2].double() @ W.double().T, D.dot_bound(X[:2].double(), W.double().T, K), "Y2")
