"""Refusals of the 16-bit layers' calls, before anything is launched (no GPU
needed): each bad argument on its own, in an otherwise good call."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5
P = 1 << 20          # an address that is never read: every call below is refused or is a no-op
BIG = 1 << 40


@pytest.fixture(scope="module")
def B():
    from rank_gemm_b200 import build
    build.build()
    from rank_gemm_b200 import binding
    return binding


CALLS = {
    "svdq_dense_linear": dict(dt=0, M=4, K=64, N=128, X=P, ldx=64, W_t=P, bias=P, act=1, residual=P, ldr=128, Y=P,
                              ldy=128, Z=P, stream=None),
    "svdq_dense_linear_backward": dict(dt=0, M=4, K=64, N=128, dY=P, lddy=128, X=P, ldx=64, W_t=P, Z=P, act=1, dX=P,
                                       lddx=64, dW=P, dbias=P, workspace=P, ws_bytes=BIG, stream=None),
    "svdq_gated_linear": dict(dt=1, M=4, K=64, F=128, X=P, ldx=64, Wg_t=P, Wu_t=P, bias_g=P, bias_u=None, act=2, H=P,
                              ldh=128, G=P, U=None, stream=None),
    "svdq_gated_linear_backward": dict(dt=1, M=4, K=64, F=128, dH=P, lddh=128, X=P, ldx=64, Wg_t=P, Wu_t=P, G=P, U=P,
                                       act=2, dX=P, lddx=64, dWg=P, dWu=P, dbias_g=P, dbias_u=P, workspace=P,
                                       ws_bytes=BIG, stream=None),
    "svdq_layernorm": dict(dt=2, M=4, C=33, X=P, ldx=40, gamma=P, beta=P, eps=1e-5, Y=P, ldy=40, mean=P, rstd=P,
                           stream=None),
    "svdq_layernorm_backward": dict(dt=2, M=4, C=33, dY=P, lddy=40, X=P, ldx=40, gamma=P, mean=P, rstd=P, dX=P,
                                    lddx=40, dgamma=P, dbeta=P, workspace=P, ws_bytes=BIG, stream=None),
}


def call(B, name, **change):
    args = dict(CALLS[name], **change)
    return getattr(B.lib, name)(*args.values())


COMMON = [(dict(dt=7), INVALID), (dict(M=-1), SHAPE)]
PRODUCT = COMMON + [(dict(M=(1 << 31) - 511), SHAPE), (dict(K=(1 << 31) - 8, ldx=(1 << 31) - 8), SHAPE),
                    (dict(dt=2), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(K=0), SHAPE),
                    (dict(K=-8), SHAPE), (dict(K=60), SHAPE), (dict(ldx=56), SHAPE), (dict(ldx=68), SHAPE),
                    (dict(ldx=1 << 39), SHAPE), (dict(X=P + 8), ALIGN)]
REFUSALS = {
    "svdq_dense_linear": PRODUCT + [
        (dict(X=None), INVALID), (dict(W_t=None), INVALID), (dict(Y=None), INVALID), (dict(N=0), SHAPE),
        (dict(N=100), SHAPE), (dict(ldy=120), SHAPE), (dict(ldr=120), SHAPE), (dict(ldr=132), SHAPE),
        (dict(W_t=P + 8), ALIGN), (dict(bias=P + 2), ALIGN), (dict(residual=P + 4), ALIGN), (dict(Y=P + 8), ALIGN),
        (dict(Z=P + 8), ALIGN)],
    "svdq_dense_linear_backward": PRODUCT + [
        (dict(dY=None), INVALID), (dict(Z=None), INVALID), (dict(W_t=None), INVALID), (dict(X=None), INVALID),
        (dict(N=100), SHAPE), (dict(lddy=120), SHAPE), (dict(lddx=56), SHAPE), (dict(dW=P + 8), ALIGN),
        (dict(dbias=P + 2), ALIGN), (dict(workspace=P + 8), ALIGN), (dict(workspace=None), WORKSPACE),
        (dict(ws_bytes=16), WORKSPACE)],
    "svdq_gated_linear": PRODUCT + [
        (dict(X=None), INVALID), (dict(Wg_t=None), INVALID), (dict(Wu_t=None), INVALID), (dict(H=None), INVALID),
        (dict(F=0), SHAPE), (dict(F=12), SHAPE), (dict(ldh=120), SHAPE), (dict(Wu_t=P + 8), ALIGN),
        (dict(G=P + 8), ALIGN), (dict(bias_u=P + 2), ALIGN)],
    "svdq_gated_linear_backward": PRODUCT + [
        (dict(dH=None), INVALID), (dict(G=None), INVALID), (dict(U=None), INVALID), (dict(Wg_t=None), INVALID),
        (dict(X=None), INVALID), (dict(dWu=None), INVALID), (dict(dbias_g=None), INVALID), (dict(F=12), SHAPE),
        (dict(lddh=120), SHAPE), (dict(lddx=60), SHAPE), (dict(dWu=P + 8), ALIGN), (dict(workspace=None), WORKSPACE),
        (dict(ws_bytes=16), WORKSPACE)],
    "svdq_layernorm": COMMON + [
        (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(beta=None), INVALID), (dict(gamma=None), INVALID),
        (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
        (dict(C=0), SHAPE), (dict(M=(1 << 31) - 511), SHAPE), (dict(C=(1 << 31) - 511, ldx=1 << 31, ldy=1 << 31), SHAPE),
        (dict(ldx=32), SHAPE), (dict(ldy=32), SHAPE), (dict(X=P + 2), ALIGN),
        (dict(mean=P + 2), ALIGN), (dict(dt=0, Y=P + 1), ALIGN)],
    "svdq_layernorm_backward": COMMON + [
        (dict(dY=None), INVALID), (dict(X=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
        (dict(dbeta=None), INVALID), (dict(C=0), SHAPE), (dict(M=(1 << 31) - 511), SHAPE),
        (dict(lddy=32), SHAPE), (dict(ldx=32), SHAPE),
        (dict(lddx=32), SHAPE), (dict(dX=P + 2), ALIGN), (dict(workspace=None), WORKSPACE),
        (dict(ws_bytes=16), WORKSPACE)],
}


@pytest.mark.parametrize("name,change,status", [(n, c, s) for n, l in REFUSALS.items() for c, s in l])
def test_refusals(B, name, change, status):
    assert call(B, name, **change) == status, (name, change)


def test_empty_forward_calls_are_no_ops(B):
    assert call(B, "svdq_dense_linear", M=0, X=None, Y=None) == OK
    assert call(B, "svdq_gated_linear", M=0, X=None, H=None) == OK
    assert call(B, "svdq_layernorm", M=0, X=None, Y=None) == OK


def test_good_calls_reach_the_device_check(B):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name in CALLS:
        assert call(B, name) == UNSUPPORTED, name
    # what a call does not need may be absent
    assert call(B, "svdq_dense_linear", bias=None, residual=None, ldr=0, Z=None) == UNSUPPORTED
    assert call(B, "svdq_dense_linear_backward", dX=None, lddx=0, W_t=None, act=0, Z=None) == UNSUPPORTED
    assert call(B, "svdq_dense_linear_backward", dW=None, X=None, ldx=0, dbias=None) == UNSUPPORTED
    assert call(B, "svdq_gated_linear_backward", dWg=None, dWu=None, X=None, ldx=0) == UNSUPPORTED
    assert call(B, "svdq_layernorm_backward", dgamma=None, dbeta=None, workspace=None, ws_bytes=0) == UNSUPPORTED


def test_norm_linear_refuses_a_null_handle(B):
    assert B.lib.svdq_norm_linear(None, 4, P, P, P, 1e-5, 0, P, P, BIG, None) == INVALID
    assert B.lib.svdq_norm_linear_workspace_bytes(None, 4) == 0


def test_workspace_sizes(B):
    L = B.lib
    assert L.svdq_dense_linear_backward_workspace_bytes(-1, 64, 64, 0) == 0
    assert L.svdq_dense_linear_backward_workspace_bytes(4, 60, 64, 0) == 0
    assert L.svdq_dense_linear_backward_workspace_bytes(4, 64, 64, 9) == 0
    assert L.svdq_gated_linear_backward_workspace_bytes(4, 64, 4) == 0
    assert L.svdq_layernorm_backward_workspace_bytes(4, 0) == 0
    # past 32 bits
    assert L.svdq_gated_linear_backward_workspace_bytes(1 << 20, 4096, 16384) > 2 * (1 << 20) * 16384 * 2
    assert L.svdq_dense_linear_backward_workspace_bytes(1 << 20, 4096, 16384, 2) > (1 << 20) * 16384 * 2


def test_binding_refuses_what_it_cannot_read(B):
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the current device"):
        B.svdq_dense_linear(4, 64, 64, t, torch.zeros(64, 64, dtype=torch.bfloat16), None, 0, None, t)
    with pytest.raises(ValueError, match="tensor"):
        B.svdq_layernorm(4, 64, t.int(), None, None, 1e-5, t)
    with pytest.raises(ValueError, match="tensor"):
        B.svdq_gated_linear_backward(4, 64, 64, None, t, t, t, t, t, 0, t, t, t, None, None, None)
