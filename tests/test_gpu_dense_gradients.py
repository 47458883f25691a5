"""The pre-norm block's gradients against differences along directions for
which the comparison can fail: along the gradient itself, where a wrong or
missing gradient shows whole, and along a random direction."""
import pytest
import torch

import test_gpu_dense as D
import test_gpu_dense_use as U

pytestmark = pytest.mark.gpu

B, no_device_error = D.B, D.no_device_error


@pytest.mark.parametrize("t", D.TYPES)
@pytest.mark.parametrize("M,C,F,act", [(1, 64, 128, "silu"), (70, 136, 328, "gelu"), (300, 264, 520, "silu"),
                                       (1030, 128, 256, "none")])
def test_gradients_against_differences(B, t, M, C, F, act):
    """Bars.  The library's gradient e away from the formula's: |e| <= 12 u |g|
    in the 2-norm (at most six 16-bit roundings in a row, a factor of two to
    spare).  Along d = g / |g| the error is at most |e|; along a random unit
    direction its deviation is |e| / sqrt(n), taken five times.  The central
    difference N(h) of the float64 forward is off by its truncation, which
    falls by four when h is halved, so that |N(h) - N(h / 2)| is above
    N(h / 2)'s, and by the forward's rounding, 2^-45 of its terms (2^8 roundings
    a term) over h."""
    b = U.Block(t, M, C, F, act, seed=M)
    _, grads = b.run(B)
    v = b.values64()
    leaves = {k: x.clone().requires_grad_() for k, x in v.items()}
    auto = dict(zip(leaves, torch.autograd.grad(b.forward64(leaves), list(leaves.values()), b.dY.double())))
    dY, u, g = b.dY.double(), D.half_step(t), D.gen(78)
    terms = float((b.forward64(v).abs() * dY.abs()).sum())

    def difference(k, d, h):
        up, down = (b.forward64(dict(v, **{k: v[k] + s * h * d})) for s in (1, -1))
        return float(((up - down) * dY).sum()) / (2 * h)

    for k in b.NAMES:
        got, size, n = grads[k].double(), float(auto[k].norm()), auto[k].numel()
        h = 1e-3 * max(float(v[k].norm()), 1.0)
        random = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
        for d, share in ((auto[k] / size, 1.0), (random / random.norm(), min(1.0, 5 / n ** 0.5))):
            wide, near = difference(k, d, h), difference(k, d, h / 2)
            bound = 12 * u * size * share + abs(wide - near) + 2.0 ** -45 * terms / (h / 2)
            assert abs(float((got * d).sum()) - near) <= bound, k
            if share == 1.0:
                assert bound < 0.25 * abs(near), k     # zeros in the gradient's place would not pass
