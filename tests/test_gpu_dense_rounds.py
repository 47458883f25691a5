"""Layer norms whose blocks take several rounds of rows, in the forms for every
width (16-byte packs, single elements, streamed rows), and random sizes of the
norms and of the gated backward pass.  Bars: test_gpu_dense.py's."""
import math
import random

import pytest
import torch

import test_gpu_dense as D

pytestmark = pytest.mark.gpu

B, no_device_error = D.B, D.no_device_error

# several rounds of rows: rows ahead, gamma and the column sums kept over the rounds, several rows a block
WIDTHS = [(20000, 37, 0), (8192, 1001, 0), (2500, 2002, 2), (4608, 3001, 0), (4608, 5001, 0), (2000, 8190, 0),
          (20000, 64, 0), (3000, 1160, 4), (6000, 5000, 0), (2500, 12288, 0), (700, 12296, 0)]
TYPES = D.TYPES + [torch.float32]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,C,pad", WIDTHS + [(300, 20480, 0), (40, 20481, 1), (600, 32768, 0), (300, 33000, 0)])
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_over_rounds(B, t, M, C, pad, affine):
    D.test_layernorm(B, t, M, C, pad, affine)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,C,pad", WIDTHS + [(200, 20480, 0), (90, 20481, 1)])
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_backward_over_rounds(B, t, M, C, pad, affine):
    D.test_layernorm_backward(B, t, M, C, pad, affine)


@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("M,C", [(3000, 512), (1300, 4096)])
def test_layernorm_at_any_address(B, M, C, offset):
    """Rows of whole packs that start off a 16-byte boundary, forward and
    backward, give the aligned rows' values (the sums' order may differ)."""
    t, g = torch.bfloat16, D.gen(21)

    def shifted(x):
        flat = torch.empty(x.numel() + offset, dtype=t, device="cuda")[offset:]
        return flat.view(x.shape).copy_(x)

    X, dY, ga, be = D.draw(g, t, M, C), D.draw(g, t, M, C), D.draw(g, t, C), D.draw(g, t, C)
    got = []
    for f in (lambda x: x, shifted):
        x, dy, a, b = f(X), f(dY), f(ga), f(be)
        Y, dX = f(D.nan_like(t, M, C)), f(D.nan_like(t, M, C))
        mean, rstd, dg, db = D.nan_like(torch.float32, M), D.nan_like(torch.float32, M), D.nan_like(t, C), D.nan_like(t, C)
        B.svdq_layernorm(M, C, x, a, b, 1e-5, Y, mean, rstd)
        ws = torch.empty(B.svdq_layernorm_backward_workspace_bytes(M, C), dtype=torch.uint8, device="cuda")
        B.svdq_layernorm_backward(M, C, dy, x, a, mean, rstd, dX, dg, db, ws)
        got.append((Y, dX, dg, db))
    for a, b in zip(*got):
        # each within half a step and the float32 sums' error, which is far below it, of the same value
        assert bool(((a.double() - b.double()).abs() <= 2.1 * D.half_step(t) * a.double().abs() + 1e-5).all())


@pytest.mark.parametrize("seed", range(16))
def test_random_sizes(B, seed):
    r = random.Random(100 + seed)
    size = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    t, act = r.choice(D.TYPES), r.choice(("none", "gelu", "silu"))
    D.test_gated_backward(B, t, size(1, 1500), 8 * size(1, 300), 8 * size(1, 300), act)
    for _ in range(3):
        M, C, pad = size(1, 3000), size(1, 9000), r.choice((0, 0, 1, 8))
        D.test_layernorm(B, r.choice(TYPES), M, C, pad, r.random() < 0.5)
        D.test_layernorm_backward(B, r.choice(TYPES), M, C, pad, r.random() < 0.5)
