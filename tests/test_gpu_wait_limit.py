"""The products' waits when they run out: with a limit of 1 ms (the library
reads SVDQ_WAIT_LIMIT_MS once a process, so each case is a process of its own,
spawned) a product whose single tile takes several milliseconds gives up. The
call's kernel then ends by itself, svdq_poll_device_error reports a timeout,
and the next call in the same process is right: the cluster left only after
what it had in flight had landed, and gave its tensor memory back.

The limit of a wait for a whole reduction grows with the reduction, so that a
long one is not taken for a stuck one: sizes up to 2^31 - 512 are allowed."""
import multiprocessing as mp
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _long_call(B, form):
    """A call of few tiles and a long reduction: at least 10 ms (40 bytes of
    operands a cycle and CTA in the swapped form, 500 cycles a k-tile in the
    pair form)."""
    new = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    if form == "swapped, split":            # 4 ranks, partials by st.async: 2^18 / 4 k-tiles
        K = 1 << 24
        return lambda a=(new(1, K), new(8, K), new(1, 8)): B.svdq_dense_linear(1, K, 8, a[0], a[1], None, 0, None, a[2])
    if form == "gated, swapped":
        K = 1 << 23
        return lambda a=(new(1, K), new(8, K), new(8, K), new(1, 8)): B.svdq_gated_linear(
            1, K, 8, a[0], a[1], a[2], None, None, 2, a[3])
    if form == "pair, split":               # 4 pairs, partials into the ring: 2^17 / 4 k-tiles
        M, K = 300, 1 << 23
        return lambda a=(new(M, K), new(8, K), new(M, 8)): B.svdq_dense_linear(M, K, 8, a[0], a[1], None, 0, None, a[2])
    M, K = 1 << 20, 2048                    # dW alone: 2^14 k-tiles a tile, too large to be cut
    ws = torch.empty(B.svdq_dense_linear_backward_workspace_bytes(M, K, K, 0), dtype=torch.uint8, device="cuda")
    return lambda a=(new(M, K), new(M, K), new(K, K)): B.svdq_dense_linear_backward(
        M, K, K, a[0], a[1], None, None, 0, None, a[2], None, ws)


def _child(form, queue):
    try:
        from rank_gemm_b200 import binding as B
        assert B.svdq_poll_device_error() == 0
        seen = []
        call = _long_call(B, form)
        for _ in range(2):
            call()
            seen.append(B.svdq_poll_device_error())
        del call
        g = torch.Generator(device="cuda").manual_seed(1)
        right = []
        for M in (5, 300):
            X, W = (torch.randn(s, 256, generator=g, device="cuda").to(BF) for s in (M, 264))
            Y = torch.full((M, 264), float("nan"), dtype=BF, device="cuda")
            B.svdq_dense_linear(M, 256, 264, X, W, None, 0, None, Y)
            want = X.double() @ W.double().T
            # half a step of bf16, and the float32 sum's 2 K 2^-24 of the magnitudes
            bound = 2.0 ** -8 * want.abs() + 2 * 256 * 2.0 ** -24 * 1.01 * (X.double().abs() @ W.double().abs().T)
            right.append(bool(((Y.double() - want).abs() <= bound).all()))
        seen.append(B.svdq_poll_device_error())
        queue.put((seen, right))
    except BaseException as e:  # noqa: BLE001  (reported by the parent)
        queue.put("%s: %s" % (type(e).__name__, str(e)[:300]))


def run_child(target, args, limit_ms):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=target, args=args + (q,))
    old = os.environ.get("SVDQ_WAIT_LIMIT_MS")
    os.environ["SVDQ_WAIT_LIMIT_MS"] = str(limit_ms)
    try:
        p.start()
    finally:
        if old is None:
            del os.environ["SVDQ_WAIT_LIMIT_MS"]
        else:
            os.environ["SVDQ_WAIT_LIMIT_MS"] = old
    try:
        return q.get(timeout=150)
    finally:
        p.join(30)
        if p.is_alive():
            p.terminate()


@pytest.mark.parametrize("form", ["swapped, split", "gated, swapped", "pair, split", "backward"])
def test_a_product_that_runs_out_of_time(form):
    assert run_child(_child, (form,), 1) == ([7, 7, 0], [True, True])


def _long_reduction(gated, queue):
    """2^21 k-tiles over 4 ranks (at least 150 cycles each: 40 ms and more,
    twice the limit of 20 ms), zero but for a few products that are exact."""
    try:
        from rank_gemm_b200 import binding as B
        K = 1 << 27
        X, W = torch.zeros(1, K, dtype=BF, device="cuda"), torch.zeros(8, K, dtype=BF, device="cuda")
        at = torch.tensor([0, 63, K // 4, K // 2 + 77, K - 1], device="cuda")
        X[0, at] = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0], device="cuda").to(BF)
        W[:, at] = torch.arange(40, device="cuda").reshape(8, 5).to(BF)
        want = X[:, at].float() @ W[:, at].float().T
        Y = torch.full((1, 8), float("nan"), dtype=BF, device="cuda")
        if gated:      # act none: the product of the two sums
            B.svdq_gated_linear(1, K, 8, X, W, W, None, None, 0, Y)
            want = want * want
        else:
            B.svdq_dense_linear(1, K, 8, X, W, None, 0, None, Y)
        status = B.svdq_poll_device_error()
        queue.put((status, bool(torch.equal(Y, want.to(BF)))))
    except BaseException as e:  # noqa: BLE001  (reported by the parent)
        queue.put("%s: %s" % (type(e).__name__, str(e)[:300]))


@pytest.mark.parametrize("gated", [False, True])
def test_a_long_reduction_is_not_taken_for_a_stuck_one(gated):
    assert run_child(_long_reduction, (gated,), 20) == (0, True)
