"""GPU parity of the 16-bit layers (svdq_dense_linear, svdq_gated_linear,
svdq_layernorm and their backward passes) against a float64 computation of
the same formulas on the same inputs.

Bars, per element, with u = eps / 2 of the output's type (half a step) and
s = 2^-24 (float32's):
  product      |D' - D| <= 2 K s sum_k |a_k b_k|: the float32 dot-product
               bound (any order of a K-term sum is within K s of the sum of
               magnitudes; the tensor core's truncation instead of rounding
               doubles it)
  activation   slope at most 1.13 (tanh GELU) and 1.1 (SiLU), value error 2^-19
               relative (two approximate instructions of 2^-22 each and their
               arguments' roundings)
  output       u |value|, the rounding to 16 bits, on top
  dZ, dG, dU   are operands of the backward products and rounded to 16 bits,
               so a product of them may be off by u sum |dz w| more
  sums         the float32 column sums are within M s of the magnitudes' sum
The comparison is with the float64 value itself, not its 16-bit rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
S32 = 2.0 ** -24
ACTS = {"none": 0, "gelu": 1, "silu": 2}


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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw(g, t, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)


def nan_like(t, *shape):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


def act64(x, act):
    """(act(x), act'(x)) in float64."""
    if act == "none":
        return x, torch.ones_like(x)
    w, dw = (x, 1.0) if act == "silu" else (
        math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3), math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * x ** 2))
    p = torch.sigmoid(w)
    return x * p, p + x * p * (1 - p) * dw


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps


def close(got, want, bound, what):
    t = got.dtype
    bound = bound + half_step(t) * (want.abs() + bound) + tiny(t)
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst error / bound %g" % (
        what, int(bad.sum()), bad.numel(), float((err / bound).nan_to_num(nan=math.inf).max()))


def dot_bound(a, b, n):
    """2 n s sum |a b| for a [m][k] @ b [k][n]."""
    return 2 * n * S32 * (a.abs() @ b.abs())


# ---------------------------------------------------------------- dense linear
def run_linear(B, t, M, K, N, act, bias=True, residual=True, keep=True, seed=1, pad=0):
    g = gen(seed)
    X, W = draw(g, t, M, K + pad, scale=1.0)[:, :K], draw(g, t, N, K, scale=0.05)
    b = draw(g, t, N) if bias else None
    R = draw(g, t, M, N + 2 * pad)[:, :N] if residual else None
    Y = nan_like(t, M, N + pad)
    Z = nan_like(t, M, N) if keep else None
    B.svdq_dense_linear(M, K, N, X, W, b, ACTS[act], R, Y[:, :N], Z)
    torch.cuda.synchronize()
    z = X.double() @ W.double().T
    zb = dot_bound(X.double(), W.double().T, K)
    if bias:
        z = z + b.double()
        zb = zb + S32 * z.abs()
    f, _ = act64(z, act)
    yb = 1.13 * zb + (2.0 ** -19) * f.abs() if act != "none" else zb
    y = f
    if residual:
        y = y + R.double()
        yb = yb + S32 * y.abs()
    close(Y[:, :N], y, yb, "Y")
    if pad:
        assert bool(Y[:, N:].isnan().all())
    if keep:
        close(Z, z, zb, "Z")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (1, 1024, 1024), (2, 8, 8), (5, 72, 136), (16, 1160, 264),
                                   (17, 192, 2056), (33, 4096, 128), (100, 520, 392), (128, 64, 136)])
def test_linear_few_rows(B, t, M, K, N):
    run_linear(B, t, M, K, N, "gelu")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,N", [(129, 8, 8), (200, 72, 136), (256, 64, 256), (257, 200, 264), (300, 1096, 520),
                                   (513, 2048, 128), (1100, 328, 1160)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_many_rows(B, t, M, K, N, act):
    run_linear(B, t, M, K, N, act)


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("bias,residual,keep", [(False, False, False), (True, False, False), (False, True, True)])
def test_linear_optional_tensors_and_strides(B, M, bias, residual, keep):
    run_linear(B, torch.bfloat16, M, 136, 72, "silu", bias, residual, keep, pad=8)


def test_linear_many_tiles(B):
    """More tiles than CTA pairs: the persistent loop and both accumulators."""
    run_linear(B, torch.bfloat16, 2600, 264, 3080, "none", residual=False, keep=False)


def test_linear_many_feature_tiles_few_rows(B):
    run_linear(B, torch.float16, 7, 264, 24584, "none", residual=False, keep=False)


@pytest.mark.parametrize("M", [4, 300])
def test_linear_into_its_residual(B, M):
    g, t, K, N = gen(3), torch.bfloat16, 256, 200
    X, W, R = draw(g, t, M, K), draw(g, t, N, K, scale=0.05), draw(g, t, M, N)
    Y = nan_like(t, M, N)
    B.svdq_dense_linear(M, K, N, X, W, None, 1, R, Y)
    B.svdq_dense_linear(M, K, N, X, W, None, 1, R, R)
    assert torch.equal(R, Y)


# ---------------------------------------------------------------- dense linear, backward
def run_linear_backward(B, t, M, K, N, act, seed=2, pad=0, want=("dX", "dW", "db")):
    g = gen(seed)
    X, W = draw(g, t, M, K + pad)[:, :K], draw(g, t, N, K, scale=0.05)
    dY, Z = draw(g, t, M, N + pad, scale=0.25)[:, :N], (draw(g, t, M, N, scale=2.0) if act != "none" else None)
    dX = nan_like(t, M, K + pad) if "dX" in want else None
    dW = nan_like(t, N, K) if "dW" in want else None
    db = nan_like(t, N) if "db" in want else None
    ws = torch.full((B.svdq_dense_linear_backward_workspace_bytes(M, K, N, ACTS[act]),), 255, dtype=torch.uint8,
                    device="cuda")
    B.svdq_dense_linear_backward(M, K, N, dY, X, W, Z, ACTS[act], dX[:, :K] if dX is not None else None, dW, db, ws)
    torch.cuda.synchronize()
    dz, off = dY.double(), 0.0
    if act != "none":
        dz = dz * act64(Z.double(), act)[1]
        # the slope is near 1 at most; its error counts on that scale
        off = dY.double().abs() * 2.0 ** -18
        off = off + half_step(t) * (dz.abs() + off) + tiny(t)
    if dX is not None:
        bound = dot_bound(dz.abs() + off, W.double(), N) + (off @ W.double().abs() if act != "none" else 0.0)
        close(dX[:, :K], dz @ W.double(), bound, "dX")
        if pad:
            assert bool(dX[:, K:].isnan().all())
    if dW is not None:
        bound = dot_bound((dz.abs() + off).T, X.double(), M) + (off.T @ X.double().abs() if act != "none" else 0.0)
        close(dW, dz.T @ X.double(), bound, "dW")
    if db is not None:
        close(db, dz.sum(0), M * S32 * dz.abs().sum(0) + (off.sum(0) if act != "none" else 0.0), "db")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (3, 8, 8), (17, 72, 136), (65, 1032, 264), (128, 200, 1160),
                                   (129, 72, 136), (300, 264, 520), (1000, 520, 328), (2100, 136, 72)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_backward(B, t, M, K, N, act):
    run_linear_backward(B, t, M, K, N, act)


@pytest.mark.parametrize("want", [("dX",), ("dW",), ("db",), ("dX", "db")])
def test_linear_backward_parts_and_strides(B, want):
    run_linear_backward(B, torch.bfloat16, 150, 136, 200, "gelu", pad=16, want=want)
    run_linear_backward(B, torch.float16, 20, 136, 200, "none", pad=8, want=want)


def test_linear_backward_many_tiles(B):
    run_linear_backward(B, torch.bfloat16, 2600, 3080, 2568, "none")


# ---------------------------------------------------------------- gated feed-forward
def run_gated(B, t, M, K, F, act, bias=True, keep=True, seed=5, pad=0):
    g = gen(seed)
    X = draw(g, t, M, K + pad)[:, :K]
    Wg, Wu = draw(g, t, F, K, scale=0.05), draw(g, t, F, K, scale=0.05)
    bg, bu = (draw(g, t, F), draw(g, t, F)) if bias else (None, None)
    H = nan_like(t, M, F + pad)
    G, U = (nan_like(t, M, F), nan_like(t, M, F)) if keep else (None, None)
    B.svdq_gated_linear(M, K, F, X, Wg, Wu, bg, bu, ACTS[act], H[:, :F], G, U)
    torch.cuda.synchronize()
    out = []
    for W, b in ((Wg, bg), (Wu, bu)):
        z, zb = X.double() @ W.double().T, dot_bound(X.double(), W.double().T, K)
        if bias:
            z = z + b.double()
            zb = zb + S32 * z.abs()
        out += [z, zb]
    a, ab, u, ub = out
    f = act64(a, act)[0]
    fb = 1.13 * ab + (2.0 ** -19) * f.abs() if act != "none" else ab
    close(H[:, :F], f * u, fb * u.abs() + ub * f.abs() + fb * ub + S32 * (f * u).abs(), "H")
    if pad:
        assert bool(H[:, F:].isnan().all())
    if keep:
        close(G, a, ab, "G")
        close(U, u, ub, "U")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,F", [(1, 1024, 384), (1, 8, 8), (9, 72, 136), (30, 2056, 264), (64, 192, 1160),
                                   (128, 520, 200), (129, 72, 136), (256, 64, 128), (300, 1096, 264), (700, 328, 520)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(B, t, M, K, F, act):
    run_gated(B, t, M, K, F, act)


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("bias,keep", [(False, False), (True, False), (False, True)])
def test_gated_optional_tensors_and_strides(B, M, bias, keep):
    run_gated(B, torch.bfloat16, M, 136, 72, "none", bias, keep, pad=8)


def test_gated_many_tiles(B):
    run_gated(B, torch.bfloat16, 2300, 136, 2056, "silu")
    run_gated(B, torch.float16, 40, 136, 20008, "silu")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,F", [(1, 64, 128), (2, 8, 8), (20, 1032, 136), (128, 72, 328), (130, 136, 72),
                                   (513, 264, 520), (1500, 520, 200)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_gated_backward(B, t, M, K, F, act):
    g = gen(7)
    X, dH = draw(g, t, M, K), draw(g, t, M, F, scale=0.25)
    Wg, Wu, G, U = draw(g, t, F, K, scale=0.05), draw(g, t, F, K, scale=0.05), draw(g, t, M, F, scale=2.0), draw(g, t, M, F)
    dX, dWg, dWu, dbg, dbu = (nan_like(t, *s) for s in ((M, K), (F, K), (F, K), (F,), (F,)))
    ws = torch.full((B.svdq_gated_linear_backward_workspace_bytes(M, K, F),), 255, dtype=torch.uint8, device="cuda")
    B.svdq_gated_linear_backward(M, K, F, dH, X, Wg, Wu, G, U, ACTS[act], dX, dWg, dWu, dbg, dbu, ws)
    torch.cuda.synchronize()
    f, slope = act64(G.double(), act)
    dg, du = dH.double() * U.double() * slope, dH.double() * f
    og, ou = (dH.double() * U.double()).abs() * 2.0 ** -18, du.abs() * 2.0 ** -18
    rg, ru = (o + half_step(t) * (d.abs() + o) + tiny(t) for d, o in ((dg, og), (du, ou)))
    close(dX, dg @ Wg.double() + du @ Wu.double(),
          dot_bound(torch.cat([dg.abs() + rg, du.abs() + ru], 1), torch.cat([Wg, Wu], 0).double(), 2 * F)
          + rg @ Wg.double().abs() + ru @ Wu.double().abs(), "dX")
    for got, d, r, o, gotb, name in ((dWg, dg, rg, og, dbg, "g"), (dWu, du, ru, ou, dbu, "u")):
        close(got, d.T @ X.double(), dot_bound((d.abs() + r).T, X.double(), M) + r.T @ X.double().abs(), "dW" + name)
        close(gotb, d.sum(0), M * S32 * d.abs().sum(0) + o.sum(0), "db" + name)


# ---------------------------------------------------------------- layer norm
def norm64(x, eps):
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    return mean, rstd


@pytest.mark.parametrize("t", TYPES + [torch.float32])
@pytest.mark.parametrize("M,C,pad", [(1, 1, 0), (1, 8, 0), (3, 7, 1), (5, 64, 0), (33, 1001, 0), (130, 512, 8),
                                     (9, 1160, 4), (40, 3080, 0), (6, 12288, 0), (4, 12289, 3), (3, 40000, 0)])
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm(B, t, M, C, pad, affine):
    """Bars: a mean of C values is within C s of the mean magnitude; the
    variance within 2 (C + 3) s relative (and the mean's error squared), rstd
    half of that; the value then takes four more float32 roundings."""
    g, eps = gen(11), 1e-5
    X = (torch.randn(M, C + pad, generator=g, device="cuda") * 3 + 1).to(t)[:, :C]
    ga, be = (draw(g, t, C), draw(g, t, C)) if affine else (None, None)
    Y, mean, rstd = nan_like(t, M, C + pad), nan_like(torch.float32, M), nan_like(torch.float32, M)
    B.svdq_layernorm(M, C, X, ga, be, eps, Y[:, :C], mean, rstd)
    torch.cuda.synchronize()
    x = X.double()
    m, r = norm64(x, eps)
    mb = (C + 2) * S32 * x.abs().mean(1, keepdim=True)
    rb = r * ((C + 6) * S32 + 0.5 * (mb * r) ** 2)
    assert bool(((mean.double()[:, None] - m).abs() <= mb).all())
    assert bool(((rstd.double()[:, None] - r).abs() <= rb).all())
    xh = (x - m) * r
    yb = mb * r + xh.abs() * (rb / r) + 2 * S32 * (xh.abs() + mb * r)
    y = xh
    if affine:
        y = xh * ga.double() + be.double()
        yb = yb * ga.double().abs() + S32 * (y.abs() + yb)
    close(Y[:, :C], y, yb, "Y")
    if pad:
        assert bool(Y[:, C:].isnan().all())


@pytest.mark.parametrize("t", TYPES + [torch.float32])
@pytest.mark.parametrize("M,C,pad", [(1, 1, 0), (2, 8, 0), (3, 7, 1), (700, 64, 0), (33, 1001, 0), (130, 512, 8),
                                     (9, 1160, 4), (1200, 3080, 0), (6, 12288, 0), (5, 12289, 3), (3, 40000, 0)])
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_backward(B, t, M, C, pad, affine):
    g, eps = gen(12), 1e-5
    X = (torch.randn(M, C + pad, generator=g, device="cuda") * 3 + 1).to(t)[:, :C]
    dY = draw(g, t, M, C + pad)[:, :C]
    ga = draw(g, t, C) if affine else None
    m, r = norm64(X.double(), eps)
    m, r = m.float(), r.float()
    dX, dg, db = nan_like(t, M, C + pad), nan_like(t, C), nan_like(t, C)
    ws = torch.full((B.svdq_layernorm_backward_workspace_bytes(M, C),), 255, dtype=torch.uint8, device="cuda")
    B.svdq_layernorm_backward(M, C, dY, X, ga, m.reshape(-1), r.reshape(-1), dX[:, :C], dg, db, ws)
    torch.cuda.synchronize()
    x, dy, m, r = X.double(), dY.double(), m.double(), r.double()
    xh = (x - m) * r
    xb = 2 * S32 * (xh.abs() + m.abs() * r)              # float32 difference and product
    gv = dy * (ga.double() if affine else 1.0)
    a, b = gv.mean(1, keepdim=True), (gv * xh).mean(1, keepdim=True)
    ab = (C + 4) * S32 * gv.abs().mean(1, keepdim=True)
    bb = (C + 4) * S32 * (gv * xh).abs().mean(1, keepdim=True) + (gv.abs() * xb).mean(1, keepdim=True)
    dx = r * (gv - a - xh * b)
    size = gv.abs() + a.abs() + (xh * b).abs()
    dxb = r * (ab + bb * xh.abs() + b.abs() * xb + bb * xb + 5 * S32 * size)
    close(dX[:, :C], dx, dxb, "dX")
    if pad:
        assert bool(dX[:, C:].isnan().all())
    close(db, dy.sum(0), M * S32 * dy.abs().sum(0), "dbeta")
    close(dg, (dy * xh).sum(0), (M + 2) * S32 * (dy * xh).abs().sum(0) + (dy.abs() * xb).sum(0), "dgamma")


# ---------------------------------------------------------------- long reductions over few tiles
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,N", [(5, 96, 9408), (1, 8, 4104), (7002, 80, 64), (2500, 72, 2824), (40, 2056, 5232),
                                   (700, 1024, 4096), (16392, 264, 136)])
def test_linear_backward_reduction_in_parts(B, t, M, K, N):
    run_linear_backward(B, t, M, K, N, "none")


@pytest.mark.parametrize("want", [("dX",), ("dW",), ("dX", "db"), ("dX", "dW")])
def test_linear_backward_reduction_in_parts_one_product(B, want):
    run_linear_backward(B, torch.bfloat16, 4100, 136, 4104, "silu", pad=16, want=want)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,F", [(2, 752, 5856), (6241, 88, 1544), (130, 264, 2056)])
def test_gated_backward_reduction_in_parts(B, t, M, K, F):
    test_gated_backward(B, t, M, K, F, "silu")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,N", [(5, 96, 9408), (4100, 136, 4104), (2, 752, 5856), (300, 264, 520)])
def test_backward_workspace_is_enough(B, gated, M, K, N):
    """Nothing behind the stated bytes is written, and the same bits come out on every run."""
    g, t = gen(9), torch.bfloat16
    X, dY, W, W2, Z, U = (draw(g, t, *s) for s in ((M, K), (M, N), (N, K), (N, K), (M, N), (M, N)))
    size = B.svdq_gated_linear_backward_workspace_bytes(M, K, N) if gated else \
        B.svdq_dense_linear_backward_workspace_bytes(M, K, N, 2)
    runs = []
    for fill in (255, 0):
        ws = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
        dX, dW, dW2, db, db2 = (nan_like(t, *s) for s in ((M, K), (N, K), (N, K), (N,), (N,)))
        if gated:
            B.svdq_gated_linear_backward(M, K, N, dY, X, W, W2, Z, U, 2, dX, dW, dW2, db, db2, ws, size)
            runs.append((dX, dW, dW2, db, db2))
        else:
            B.svdq_dense_linear_backward(M, K, N, dY, X, W, Z, 2, dX, dW, db, ws, size)
            runs.append((dX, dW, db))
        torch.cuda.synchronize()
        assert bool((ws[size:] == fill).all())
    for a, b in zip(*runs):
        assert bool(a.isfinite().all()) and torch.equal(a, b)
