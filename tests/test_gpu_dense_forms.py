"""Every form the 16-bit products can take (tiles, splits over a cluster, cut
reductions) on a size that takes it, against float64, with bias, residual, kept
pre-activations and padded rows; and every measured case of perf/operators.py
against its definition.  test_dense_plan_host.py checks that the sizes take
these forms and that there are no others.  Bars: test_gpu_dense.py's."""
import pytest
import torch

import test_gpu_dense as D
from perf import operators as P

pytestmark = pytest.mark.gpu

B, no_device_error = D.B, D.no_device_error

# {(swapped, MMA columns, ranks, tall, dX cut into parts, dW cut into parts): (M, K, N)}
LINEAR = {
    (0, 128, 1, 0, 0, 0): (258, 144, 160), (0, 128, 2, 0, 0, 0): (270, 2592, 152),
    (0, 128, 4, 0, 0, 0): (260, 5104, 152), (0, 256, 1, 0, 0, 0): (1071, 1224, 1832),
    (0, 256, 1, 1, 0, 0): (3068, 4440, 2936), (0, 256, 2, 0, 0, 0): (792, 9064, 1032),
    (0, 256, 4, 0, 0, 0): (770, 23504, 408),
    (1, 16, 1, 0, 0, 0): (2, 144, 144), (1, 16, 2, 0, 0, 0): (194, 864, 272), (1, 16, 4, 0, 0, 0): (2, 584, 144),
    (1, 32, 1, 0, 0, 0): (241, 144, 1160), (1, 32, 2, 0, 0, 0): (234, 1872, 544),
    (1, 32, 4, 0, 0, 0): (180, 1848, 272), (1, 32, 8, 0, 0, 0): (20, 3408, 144),
    (1, 64, 1, 0, 0, 0): (52, 336, 9768), (1, 64, 2, 0, 0, 0): (94, 3112, 4208),
    (1, 64, 4, 0, 0, 0): (233, 3368, 528), (1, 64, 8, 0, 0, 0): (177, 6872, 264),
    (1, 128, 1, 0, 0, 0): (112, 1048, 9720), (1, 128, 2, 0, 0, 0): (162, 6664, 4240),
    (1, 128, 4, 0, 0, 0): (184, 6952, 2000), (1, 128, 8, 0, 0, 0): (230, 13144, 568),
}
GATED = {
    (0, 128, 1, 0, 0, 0): (270, 144, 152), (0, 128, 2, 0, 0, 0): (271, 2528, 152),
    (0, 128, 4, 0, 0, 0): (257, 5088, 160), (0, 256, 1, 0, 0, 0): (828, 1232, 1160),
    (0, 256, 2, 0, 0, 0): (261, 9240, 1080),
    (0, 256, 4, 0, 0, 0): (269, 22488, 496), (1, 16, 1, 0, 0, 0): (1, 144, 144), (1, 16, 2, 0, 0, 0): (1, 392, 200),
    (1, 16, 4, 0, 0, 0): (2, 464, 144), (1, 32, 1, 0, 0, 0): (49, 144, 4912), (1, 32, 2, 0, 0, 0): (226, 1952, 568),
    (1, 32, 4, 0, 0, 0): (189, 1192, 264), (1, 32, 8, 0, 0, 0): (20, 2408, 144),
    (1, 64, 1, 0, 0, 0): (100, 536, 4920), (1, 64, 2, 0, 0, 0): (164, 5200, 2184),
    (1, 64, 4, 0, 0, 0): (246, 2216, 544), (1, 64, 8, 0, 0, 0): (190, 4424, 280),
    (1, 128, 1, 0, 0, 0): (111, 976, 9688), (1, 128, 2, 0, 0, 0): (102, 5216, 4912),
    (1, 128, 4, 0, 0, 0): (115, 5544, 2440), (1, 128, 8, 0, 0, 0): (211, 9112, 536),
}
LINEAR_BACKWARD = {
    (0, 128, 1, 0, 0, 0): (1, 144, 144), (0, 128, 1, 0, 0, 1): (1617, 152, 144),
    (0, 128, 1, 0, 1, 0): (5, 144, 1512), (0, 128, 1, 0, 1, 1): (966, 144, 2080),
    (0, 128, 2, 0, 0, 0): (514, 152, 1528), (0, 256, 1, 0, 0, 0): (2, 4776, 144),
    (0, 256, 1, 0, 0, 1): (2123, 656, 272), (0, 256, 1, 0, 1, 0): (1, 144, 11920),
    (0, 256, 1, 0, 1, 1): (1008, 152, 2840), (0, 256, 1, 1, 0, 0): (1633, 1512, 1608),
    (0, 256, 1, 1, 0, 1): (4892, 592, 592), (0, 256, 1, 1, 1, 0): (578, 592, 4896),
    (0, 256, 1, 1, 1, 1): (1383, 272, 4152), (0, 256, 2, 0, 0, 0): (979, 432, 3048),
}
GATED_BACKWARD = {
    (0, 128, 1, 0, 0, 0): (1, 144, 144), (0, 128, 1, 0, 0, 1): (1508, 160, 152), (0, 128, 1, 0, 1, 0): (1, 144, 720),
    (0, 128, 1, 0, 1, 1): (2058, 144, 456), (0, 128, 2, 0, 0, 0): (563, 144, 720),
    (0, 256, 1, 0, 0, 0): (1, 3080, 152), (0, 256, 1, 0, 0, 1): (2126, 272, 280),
    (0, 256, 1, 0, 1, 0): (1, 144, 6184), (0, 256, 1, 0, 1, 1): (1050, 184, 1288),
    (0, 256, 1, 1, 0, 0): (1638, 1288, 776), (0, 256, 1, 1, 0, 1): (6957, 272, 264),
    (0, 256, 1, 1, 1, 0): (613, 592, 2384), (0, 256, 1, 1, 1, 1): (1819, 152, 2136),
    (0, 256, 2, 0, 0, 0): (994, 408, 1504),
}
# more tiles than pairs: both accumulators in turn, the tall form's head and tail
LINEAR_MORE = [(2600, 264, 3080), (4192, 12216, 1568), (1299, 6272, 144), (300, 8, 40008)]
GATED_MORE = [(2600, 264, 3080), (984, 8232, 72)]
BACKWARD_MORE = [(7279, 3280, 3544), (5624, 224, 4792)]


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,K,N", list(LINEAR.values()) + LINEAR_MORE)
def test_linear_forms(B, t, M, K, N):
    D.run_linear(B, t, M, K, N, "gelu", pad=8)


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,K,F", list(GATED.values()) + GATED_MORE)
def test_gated_forms(B, t, M, K, F):
    D.run_gated(B, t, M, K, F, "silu", pad=8)


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,K,N", list(LINEAR_BACKWARD.values()) + BACKWARD_MORE)
def test_linear_backward_forms(B, t, M, K, N):
    D.run_linear_backward(B, t, M, K, N, "gelu", pad=8)


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,K,F", list(GATED_BACKWARD.values()) + BACKWARD_MORE[1:])
def test_gated_backward_forms(B, t, M, K, F):
    D.test_gated_backward(B, t, M, K, F, "silu")


# ---------------------------------------------------------------- the measured cases
def product_bounds(c, s, out):
    """Bars of a measured case's outputs (test_gpu_dense.py's), in their order."""
    v = {k: x.double() for k, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    t, M, K = P.TYPES[c["type"]], c["M"], c["K"]

    def pre(w, b):
        z = v["X"] @ v[w].T
        bound = D.dot_bound(v["X"], v[w].T, K)
        return (z + v[b], bound + D.S32 * (z + v[b]).abs()) if c["bias"] else (z, bound)

    if c["op"] == "linear":
        z, zb = pre("W", "b")
        f = D.act64(z, c["epi"])[0]
        yb = 1.13 * zb + 2.0 ** -19 * f.abs() if c["epi"] != "none" else zb
        if c["residual"]:
            yb = yb + D.S32 * (f + v["R"]).abs()
        return [yb, zb][:len(out)]
    if c["op"] == "gated":
        (a, ab), (u, ub) = pre("Wg", "bg"), pre("Wu", "bu")
        f = D.act64(a, c["act"])[0]
        fb = 1.13 * ab + 2.0 ** -19 * f.abs() if c["act"] != "none" else ab
        return [fb * u.abs() + ub * f.abs() + fb * ub + D.S32 * (f * u).abs(), ab, ub][:len(out)]
    if c["op"] == "linear_bwd":
        d, o, act = v["dY"], 0.0, c["epi"] != "none"
        if act:
            d = d * D.act64(v["Z"], c["epi"])[1]
            o = v["dY"].abs() * 2.0 ** -18
        r = o + D.half_step(t) * (d.abs() + o) + D.tiny(t) if act else torch.zeros_like(d)
        terms = [(d, o, r, "W")]
    else:
        f, slope = D.act64(v["G"], c["act"])
        dg, du = v["dH"] * v["U"] * slope, v["dH"] * f
        terms = [(d, o, o + D.half_step(t) * (d.abs() + o) + D.tiny(t), w)
                 for d, o, w in ((dg, (v["dH"] * v["U"]).abs() * 2.0 ** -18, "Wg"), (du, du.abs() * 2.0 ** -18, "Wu"))]
    n = sum(d.shape[1] for d, _, _, _ in terms)
    dx = sum(2 * n * D.S32 * ((d.abs() + r) @ v[w].abs()) + r @ v[w].abs() for d, _, r, w in terms)
    dw = [D.dot_bound((d.abs() + r).T, v["X"], M) + r.T @ v["X"].abs() for d, _, r, _ in terms]
    db = [M * D.S32 * d.abs().sum(0) + (o.sum(0) if torch.is_tensor(o) else 0.0) for d, o, _, _ in terms]
    return ([dx] + dw + db)[:len(out)]


@pytest.mark.parametrize("case", [c for c in P.listed() if not c["op"].startswith("norm")], ids=lambda c: c["name"])
def test_measured_products(B, monkeypatch, case):
    """Against the definition; and the same bits on every run."""
    monkeypatch.setattr(P, "own", True)
    s = P.prepare(case, 3)
    out = P.run(s)
    first = [x.clone() for x in out]
    for name, got, want, bound in zip("abcdefg", first, P.exact(case, 3), product_bounds(case, s, out)):
        D.close(got, want, bound, name)
    for _ in range(3):
        for x in out:
            x.fill_(float("nan"))
        for a, b in zip(P.run(s), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("case", [c for c in P.listed() if c["op"].startswith("norm")], ids=lambda c: c["name"])
def test_measured_norms(B, monkeypatch, case):
    """In the 2-norm: the output's rounding, at most half a step of each value,
    and as much again for the float32 statistics (C 2^-24 of the magnitudes)."""
    monkeypatch.setattr(P, "own", True)
    s = P.prepare(case, 4)
    out = P.run(s)
    first = [x.clone() for x in out]
    for got, want in zip(first, P.exact(case, 4)):
        assert float((got.double() - want).norm()) <= 2 * D.half_step(P.TYPES[case["type"]]) * float(want.norm())
    for a, b in zip(P.run(s), first):
        assert torch.equal(a, b)
