"""The library's first call of a process may stand inside a graph capture: the
16-bit layers need no prepared handle, so a program can capture its step
without having called the library before, on a stream of either kind (an
ordinary one, which synchronizes with the legacy default stream, and the
non-blocking one of PyTorch's pool).  Each case runs in a process of its own
(`spawn`: the parent may hold a CUDA context)."""
import ctypes
import multiprocessing as mp

import pytest
import torch

pytestmark = pytest.mark.gpu

M, K, N = 40, 136, 264
CALLS = ("linear", "linear_backward", "gated", "gated_backward", "layernorm", "layernorm_backward")


def _step(B, which):
    """(the call on inputs of its own, its outputs)"""
    g, t = torch.Generator(device="cuda").manual_seed(1), torch.bfloat16
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)   # noqa: E731
    out = lambda *s: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    X, W, W2, dY, Z, U = draw(M, K), draw(N, K), draw(N, K), draw(M, N), draw(M, N), draw(M, N)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    stats = torch.ones(M, device="cuda")
    if which == "linear":
        o = [out(M, N)]
        return lambda: B.svdq_dense_linear(M, K, N, X, W, None, 1, None, o[0]), o
    if which == "linear_backward":
        o = [out(M, K), out(N, K), out(N)]
        return lambda: B.svdq_dense_linear_backward(M, K, N, dY, X, W, Z, 2, *o, ws), o
    if which == "gated":
        o = [out(M, N)]
        return lambda: B.svdq_gated_linear(M, K, N, X, W, W2, None, None, 2, o[0]), o
    if which == "gated_backward":
        o = [out(M, K), out(N, K), out(N, K), out(N), out(N)]
        return lambda: B.svdq_gated_linear_backward(M, K, N, dY, X, W, W2, Z, U, 2, *o, ws), o
    if which == "layernorm":
        o = [out(M, K)]
        return lambda: B.svdq_layernorm(M, K, X, None, None, 1e-5, o[0]), o
    o = [out(M, K), out(K), out(K)]
    return lambda: B.svdq_layernorm_backward(M, K, X, dY[:, :K].contiguous(), None, stats, stats, *o, ws), o


def _blocking_stream():
    """cudaStreamCreate's kind, from the runtime that PyTorch has loaded."""
    torch.cuda.init()
    rt = next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line)
    s = ctypes.c_void_p()
    assert ctypes.CDLL(rt).cudaStreamCreate(ctypes.byref(s)) == 0
    return torch.cuda.ExternalStream(s.value)


def _child(which, blocking, queue):
    try:
        from rank_gemm_b200 import binding as B
        call, o = _step(B, which)
        g = torch.cuda.CUDAGraph()
        s = _blocking_stream() if blocking else torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            call()
        g.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in o]
        for x in o:
            x.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        same = all(bool(a.isfinite().all()) and torch.equal(a, b) for a, b in zip(o, replayed))
        queue.put("same" if same else "replay and eager call differ")
    except BaseException as e:  # noqa: BLE001  (reported by the parent)
        queue.put("%s: %s" % (type(e).__name__, str(e)[:300]))


@pytest.mark.parametrize("which,blocking", [(w, True) for w in CALLS] + [("linear", False)])
def test_first_call_inside_a_capture(which, blocking):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=_child, args=(which, blocking, q))
    p.start()
    try:
        got = q.get(timeout=120)
    finally:
        p.join(30)
        if p.is_alive():
            p.terminate()
    assert got == "same", got
