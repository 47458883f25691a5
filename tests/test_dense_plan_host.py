"""How the 16-bit products are tiled: the sizes that the GPU tests run take
every form there is (no GPU needed)."""
import math
import random

import pytest

import test_gpu_dense_forms as F

LISTS = [F.LINEAR, F.GATED, F.LINEAR_BACKWARD, F.GATED_BACKWARD]


@pytest.fixture(scope="module")
def B():
    from rank_gemm_b200 import build
    build.build()
    from rank_gemm_b200 import binding
    return binding


def form(B, op, M, K, N):
    p = B.svdq_debug_product_plan(op, M, K, N)
    return p[:4] + (int(p[4] > 1), int(p[5] > 1))


@pytest.mark.parametrize("op", range(4))
def test_the_tested_sizes_take_their_forms(B, op):
    for key, size in LISTS[op].items():
        assert form(B, op, *size) == key, size


@pytest.mark.parametrize("op", range(4))
def test_there_are_no_other_forms(B, op):
    r = random.Random(op)
    draw = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    seen = set()
    for _ in range(200000):
        seen.add(form(B, op, draw(1, 40000), 8 * draw(1, 3000), 8 * draw(1, 3000)))
    assert seen <= set(LISTS[op]), seen - set(LISTS[op])


def test_refusals(B):
    plan = (B.ctypes.c_int * 6)()
    f = B.lib.svdq_debug_product_plan
    assert f(4, 8, 8, 8, 148, plan) == f(-1, 8, 8, 8, 148, plan) == f(0, 8, 8, 8, 148, None) == f(0, 8, 8, 8, 4, plan) == 1
    assert f(0, 0, 8, 8, 148, plan) == f(0, 8, 12, 8, 148, plan) == f(0, 8, 8, 0, 148, plan) == 2
