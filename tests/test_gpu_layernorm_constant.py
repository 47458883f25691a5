"""Rows of one repeated value: the mean is that value exactly wherever the
row's float32 sum is exact, so the output is beta exactly and rstd is
1 / sqrt(eps), at every width and in every form of the kernel.  The values are
small multiples of a power of two whose sums stay below 2^24 of it: exact in
any order."""
import math

import pytest
import torch

import test_gpu_dense as D

pytestmark = pytest.mark.gpu

B, no_device_error = D.B, D.no_device_error


@pytest.mark.parametrize("t", D.TYPES + [torch.float32])
@pytest.mark.parametrize("C", [1, 3, 7, 13, 56, 112, 896, 1001, 3001, 3584, 7168, 12289, 14336, 57344])
def test_constant_rows_are_beta(B, t, C):
    values = torch.tensor([1000.0, 1.0, -3.0, 0.0, 160.0, -7.0, 0.5, 63.0], device="cuda")
    assert all(abs(float(v)) * C / 0.5 < 2 ** 24 or float(v) % 8 == 0 and abs(float(v)) * C / 8 < 2 ** 24 for v in values)
    for M in (8, 1600):       # few rows; several rows a block
        v = values.repeat(M // 8)
        X = v[:, None].expand(M, C).to(t).contiguous()
        assert torch.equal(X[:, 0].float(), v)
        g = D.gen(15)
        ga, be = D.draw(g, t, C), D.draw(g, t, C)
        Y, mean, rstd = D.nan_like(t, M, C), D.nan_like(torch.float32, M), D.nan_like(torch.float32, M)
        B.svdq_layernorm(M, C, X, ga, be, 1e-5, Y, mean, rstd)
        assert torch.equal(mean, v)
        assert torch.equal(Y, be.expand(M, C))
        # three float32 roundings (eps, the square root, the quotient), the first halved by the root
        assert float((rstd.double() * math.sqrt(1e-5) - 1).abs().max()) <= 3 * D.S32


@pytest.mark.parametrize("C", [56, 1001, 57344])
def test_an_infinite_value_stays_in_its_row(B, C):
    """The mean of a row with an infinity is that infinity, with both a NaN."""
    X = torch.ones(4, C, device="cuda")
    X[1, 5], X[2, 7], X[3, 3], X[3, 9] = math.inf, -math.inf, math.inf, -math.inf
    Y, mean, rstd = torch.empty_like(X), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    B.svdq_layernorm(4, C, X, None, None, 1e-5, Y, mean, rstd)
    assert float(mean[0]) == 1 and float(mean[1]) == math.inf and float(mean[2]) == -math.inf and bool(mean[3].isnan())
    assert not bool(Y[0].any()) and bool(Y[1:].isnan().all())
