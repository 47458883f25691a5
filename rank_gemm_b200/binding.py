"""ctypes binding of libsvdq.so (include/svdq.h): argument marshalling only.

Each function has the C entry point's name and argument order.  Device
buffers are passed as torch CUDA tensors (their data pointers are handed to
the library), the stream defaults to torch's current stream, and a non-OK
status raises SvdqError.  No arithmetic of the layer happens here: every step
runs in the library's CUDA kernels.  If the library is missing this module
raises at import time; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvdq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libsvdq.so is not built (expected at %s); run `python -m rank_gemm_b200.build` "
        "(needs nvcc); there is no CPU fallback" % LIB_PATH)

lib = ctypes.CDLL(LIB_PATH)

SVDQ_NVFP4, SVDQ_INT4 = 0, 1
SVDQ_EPI_NONE, SVDQ_EPI_GELU_TANH, SVDQ_EPI_SILU = 0, 1, 2
SVDQ_BF16, SVDQ_FP16, SVDQ_FP32 = 0, 1, 2
DTYPES = {torch.bfloat16: SVDQ_BF16, torch.float16: SVDQ_FP16, torch.float32: SVDQ_FP32}
STATUS = {0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_SHAPE", 3: "SVDQ_ERR_ALIGNMENT",
          4: "SVDQ_ERR_UNSUPPORTED_DEVICE", 5: "SVDQ_ERR_WORKSPACE", 6: "SVDQ_ERR_CUDA",
          7: "SVDQ_ERR_TIMEOUT", 8: "SVDQ_ERR_DEVICE_FAULT", 9: "SVDQ_ERR_NO_MEMORY"}
FORMATS = {"nvfp4": SVDQ_NVFP4, "int4": SVDQ_INT4}


class SvdqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.svdq_status_string(status).decode()
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), msg))


class WeightsInfo(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int), ("rank", ctypes.c_int),
                ("lora_rank", ctypes.c_int), ("r_tot", ctypes.c_int), ("K_pad", ctypes.c_int),
                ("N_pad", ctypes.c_int), ("r_pad", ctypes.c_int), ("qR", ctypes.c_void_p),
                ("sR", ctypes.c_void_p), ("L1t", ctypes.c_void_p), ("L2a", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("lambda_inv", ctypes.c_void_p), ("s_tR", ctypes.c_float),
                ("s_tX", ctypes.c_float), ("alpha", ctypes.c_float)]


class AwqInfo(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int), ("N", ctypes.c_int), ("N_pad", ctypes.c_int), ("code", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p), ("inv_s", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
_SIGS = {
    "svdq_status_string": (ctypes.c_char_p, [_i]),
    "svdq_calibrate_workspace_bytes": (_sz, [_i]),
    "svdq_calibrate": (_i, [_i, _i, _i, _vp, _vp, _f, _vp, _vp, _vp, _sz, _vp]),
    "svdq_prepare_weights": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _f, _vp,
                                  ctypes.POINTER(_vp)]),
    "svdq_free_weights": (_i, [_vp]),
    "svdq_lowrank_factors": (_i, [_i, _i, _i, _vp, _vp, ctypes.c_ulonglong, _vp, _vp, _vp, _vp]),
    "svdq_weights_view": (_i, [_vp, ctypes.POINTER(WeightsInfo)]),
    "svdq_act_buffer_sizes": (_i, [_vp, _i, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
    "svdq_quantize_act_lowrank_down": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp]),
    "svdq_w4a4_gemm_lowrank_up": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "svdq_linear_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_linear": (_i, [_vp, _i, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_linear_dynamic_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_linear_dynamic": (_i, [_vp, _i, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_linear_emit_next_workspace_bytes": (_sz, [_vp, _vp, _i]),
    "svdq_linear_emit_next": (_i, [_vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_mlp_workspace_bytes": (_sz, [_vp, _vp, _i]),
    "svdq_mlp": (_i, [_vp, _vp, _i, _vp, _i, _i, _vp, _vp, _sz, _vp]),
    "svdq_quantize_act": (_i, [_vp, _i, _vp, _vp, _vp, _vp]),
    "svdq_lowrank_down": (_i, [_vp, _i, _vp, _vp, _vp]),
    "svdq_w4a4_gemm": (_i, [_vp, _i, _vp, _vp, _vp, _vp]),
    "svdq_lowrank_up": (_i, [_vp, _i, _vp, _i, _vp, _vp]),
    "svdq_linear_unfused": (_i, [_vp, _i, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_linear_noalloc": (_i, [_vp, _i, _vp, _i, _vp, _vp]),
    "svdq_awq_prepare": (_i, [_i, _i, _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)]),
    "svdq_awq_free": (_i, [_vp]),
    "svdq_awq_view": (_i, [_vp, ctypes.POINTER(AwqInfo)]),
    "svdq_awq_linear": (_i, [_vp, _i, _vp, _vp, _vp]),
    "svdq_awq_gemm": (_i, [_vp, _i, _vp, _vp, _vp]),
    "svdq_linear_host_workspace_bytes": (ctypes.c_size_t, [_vp, _i]),
    "svdq_linear_host": (_i, [_vp, _i, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]),
    "svdq_dense_linear": (_i, [_i, _i, _i, _i, _vp, _ll, _vp, _vp, _i, _vp, _ll, _vp, _ll, _vp, _vp]),
    "svdq_dense_linear_backward_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "svdq_dense_linear_backward": (_i, [_i, _i, _i, _i, _vp, _ll, _vp, _ll, _vp, _vp, _i, _vp, _ll, _vp, _vp, _vp,
                                        _sz, _vp]),
    "svdq_gated_linear": (_i, [_i, _i, _i, _i, _vp, _ll, _vp, _vp, _vp, _vp, _i, _vp, _ll, _vp, _vp, _vp]),
    "svdq_gated_linear_backward_workspace_bytes": (_sz, [_i, _i, _i]),
    "svdq_gated_linear_backward": (_i, [_i, _i, _i, _i, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _i, _vp, _ll, _vp, _vp,
                                        _vp, _vp, _vp, _sz, _vp]),
    "svdq_layernorm": (_i, [_i, _i, _i, _vp, _ll, _vp, _vp, _f, _vp, _ll, _vp, _vp, _vp]),
    "svdq_layernorm_backward_workspace_bytes": (_sz, [_i, _i]),
    "svdq_layernorm_backward": (_i, [_i, _i, _i, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _sz, _vp]),
    "svdq_norm_linear_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_norm_linear": (_i, [_vp, _i, _vp, _vp, _vp, _f, _i, _vp, _vp, _sz, _vp]),
    "svdq_poll_device_error": (_i, [_vp]),
    "svdq_selftest_wait_timeout": (_i, [ctypes.c_uint, _vp]),
    "svdq_debug_override_cc": (None, [_i, _i]),
    "svdq_debug_product_plan": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(_i)]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


def _ptr(t) -> Optional[int]:
    """Device address of a tensor argument (every tensor the ABI takes is
    device memory read as a packed array): a host tensor or a strided view
    is refused here, before the call, instead of being read as raw memory."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, torch.Tensor):
        if not t.is_cuda:
            raise ValueError("svdq: a tensor argument is in host memory; the library takes device memory")
        if not t.is_contiguous():
            raise ValueError("svdq: a tensor argument is not contiguous; the library reads packed arrays")
    return t.data_ptr()


def _stream(s, dev=None) -> Optional[int]:
    if s is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice() if dev is None else dev)
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def _check(status: int, where: str):
    if status != 0:
        raise SvdqError(status, where)


# ------------------------------------------------------------------ entry points
def svdq_status_string(status: int) -> str:
    return lib.svdq_status_string(status).decode()


def svdq_calibrate_workspace_bytes(K: int) -> int:
    return lib.svdq_calibrate_workspace_bytes(K)


def svdq_calibrate(M, K, N, X, W_t, alpha, lambda_out, act_scale_out, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_calibrate(M, K, N, _ptr(X), _ptr(W_t), alpha, _ptr(lambda_out), _ptr(act_scale_out),
                              _ptr(workspace), ws_bytes, _stream(stream)), "svdq_calibrate")


def svdq_prepare_weights(fmt, K, N, rank, W_t, lam, L1f, L2, bias=None, lora_A=None, lora_B=None,
                         lora_rank=0, act_scale=1.0, stream=None) -> int:
    """Returns the opaque handle (an int); release it with svdq_free_weights."""
    h = _vp()
    fmt = FORMATS.get(fmt, fmt)
    _check(lib.svdq_prepare_weights(fmt, K, N, rank, _ptr(W_t), _ptr(lam), _ptr(L1f), _ptr(L2), _ptr(bias),
                                    _ptr(lora_A), _ptr(lora_B), lora_rank, float(act_scale), _stream(stream),
                                    ctypes.byref(h)), "svdq_prepare_weights")
    return h.value


SVDQ_SPLIT_SEED = 0x5EED


def svdq_lowrank_factors(K, N, rank, W_t, lam, L1f, L2, seed=SVDQ_SPLIT_SEED, stream=None):
    """The device's randomized split of diag(lam) W; fills L1f / L2 and returns
    the estimated singular values (a list of min(rank + 8, K, N) floats)."""
    n_sig = min(rank + 8, K, N)
    sig = (ctypes.c_double * n_sig)()
    _check(lib.svdq_lowrank_factors(K, N, rank, _ptr(W_t), _ptr(lam), seed, _ptr(L1f), _ptr(L2), sig,
                                    _stream(stream)), "svdq_lowrank_factors")
    return list(sig)


def svdq_free_weights(w):
    _check(lib.svdq_free_weights(w), "svdq_free_weights")


def svdq_weights_view(w) -> WeightsInfo:
    info = WeightsInfo()
    _check(lib.svdq_weights_view(w, ctypes.byref(info)), "svdq_weights_view")
    return info


def svdq_act_buffer_sizes(w, M):
    q, s, l = _sz(), _sz(), _sz()
    _check(lib.svdq_act_buffer_sizes(w, M, ctypes.byref(q), ctypes.byref(s), ctypes.byref(l)),
           "svdq_act_buffer_sizes")
    return q.value, s.value, l.value


def svdq_quantize_act_lowrank_down(w, M, X, qX, sX, LR, stream=None):
    _check(lib.svdq_quantize_act_lowrank_down(w, M, _ptr(X), _ptr(qX), _ptr(sX), _ptr(LR), _stream(stream)),
           "svdq_quantize_act_lowrank_down")


def svdq_w4a4_gemm_lowrank_up(w, M, qX, sX, LR, epi, Y, stream=None):
    _check(lib.svdq_w4a4_gemm_lowrank_up(w, M, _ptr(qX), _ptr(sX), _ptr(LR), epi, _ptr(Y), _stream(stream)),
           "svdq_w4a4_gemm_lowrank_up")


def svdq_linear_workspace_bytes(w, M) -> int:
    return lib.svdq_linear_workspace_bytes(w, M)


def svdq_linear(w, M, X, epi, Y, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_linear(w, M, _ptr(X), epi, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)),
           "svdq_linear")


def _host_ptr(t) -> Optional[int]:
    """Address of a host tensor argument (svdq_linear_host's X and Y)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if t.is_cuda:
            raise ValueError("svdq: this argument is host memory; a device tensor was given")
        if not t.is_contiguous():
            raise ValueError("svdq: a tensor argument is not contiguous; the library reads packed arrays")
    return t.data_ptr()


def svdq_linear_host_workspace_bytes(w, M) -> int:
    return lib.svdq_linear_host_workspace_bytes(w, M)


def svdq_linear_host(w, M, X_host, epi, Y_host, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_linear_host(w, M, _host_ptr(X_host), epi, _host_ptr(Y_host), _ptr(workspace), ws_bytes,
                                _stream(stream)), "svdq_linear_host")


def svdq_linear_dynamic_workspace_bytes(w, M) -> int:
    return lib.svdq_linear_dynamic_workspace_bytes(w, M)


def svdq_linear_dynamic(w, M, X, epi, Y, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_linear_dynamic(w, M, _ptr(X), epi, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)),
           "svdq_linear_dynamic")


def svdq_linear_emit_next_workspace_bytes(w1, w2, M) -> int:
    return lib.svdq_linear_emit_next_workspace_bytes(w1, w2, M)


def svdq_linear_emit_next(w1, w2, M, X, epi, qX2, sX2, LR2, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_linear_emit_next(w1, w2, M, _ptr(X), epi, _ptr(qX2), _ptr(sX2), _ptr(LR2), _ptr(workspace),
                                     ws_bytes, _stream(stream)), "svdq_linear_emit_next")


def svdq_mlp_workspace_bytes(w1, w2, M) -> int:
    return lib.svdq_mlp_workspace_bytes(w1, w2, M)


def svdq_mlp(w1, w2, M, X, epi1, epi2, Y, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_mlp(w1, w2, M, _ptr(X), epi1, epi2, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)),
           "svdq_mlp")


def svdq_quantize_act(w, M, X, qX, sX, stream=None):
    _check(lib.svdq_quantize_act(w, M, _ptr(X), _ptr(qX), _ptr(sX), _stream(stream)), "svdq_quantize_act")


def svdq_lowrank_down(w, M, X, LR, stream=None):
    _check(lib.svdq_lowrank_down(w, M, _ptr(X), _ptr(LR), _stream(stream)), "svdq_lowrank_down")


def svdq_w4a4_gemm(w, M, qX, sX, Y, stream=None):
    _check(lib.svdq_w4a4_gemm(w, M, _ptr(qX), _ptr(sX), _ptr(Y), _stream(stream)), "svdq_w4a4_gemm")


def svdq_lowrank_up(w, M, LR, epi, Y, stream=None):
    _check(lib.svdq_lowrank_up(w, M, _ptr(LR), epi, _ptr(Y), _stream(stream)), "svdq_lowrank_up")


def svdq_linear_unfused(w, M, X, epi, Y, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_linear_unfused(w, M, _ptr(X), epi, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)),
           "svdq_linear_unfused")


def svdq_linear_noalloc(w, M, X, epi, Y, stream=None):
    """svdq_linear with the intermediates in the library's own scratch array
    (no workspace, no allocation); see include/svdq.h for its size limit and
    the rule that calls overlapping on the GPU race."""
    _check(lib.svdq_linear_noalloc(w, M, _ptr(X), epi, _ptr(Y), _stream(stream)), "svdq_linear_noalloc")


SVDQ_NOALLOC_SCRATCH_BYTES = 32 << 20


def svdq_awq_prepare(K, N, W_t, s=None, bias=None, stream=None) -> int:
    """Returns the opaque AWQ W4A16 handle (an int); release it with svdq_awq_free."""
    h = _vp()
    _check(lib.svdq_awq_prepare(K, N, _ptr(W_t), _ptr(s), _ptr(bias), _stream(stream), ctypes.byref(h)),
           "svdq_awq_prepare")
    return h.value


def svdq_awq_free(w):
    _check(lib.svdq_awq_free(w), "svdq_awq_free")


def svdq_awq_view(w) -> AwqInfo:
    info = AwqInfo()
    _check(lib.svdq_awq_view(w, ctypes.byref(info)), "svdq_awq_view")
    return info


def svdq_awq_linear(w, M, X, Y, stream=None):
    _check(lib.svdq_awq_linear(w, M, _ptr(X), _ptr(Y), _stream(stream)), "svdq_awq_linear")


def svdq_awq_gemm(w, M, X, Y, stream=None):
    _check(lib.svdq_awq_gemm(w, M, _ptr(X), _ptr(Y), _stream(stream)), "svdq_awq_gemm")


# ------------------------------------------------------------------ 16-bit layers
# The element type and the row strides the C calls take come from the tensors;
# every tensor has to have the stated shape, X's (or dY's) type, and to lie on
# the current device.
def _rows(t, rows, cols, dt, dev, what):
    """(address, row stride) of an activation: a [>= rows][cols] tensor whose
    rows are contiguous."""
    if t is None:
        return None, 0
    if t.dtype is dt and t.get_device() == dev and t.shape == (rows, cols) and t.is_contiguous():
        return t.data_ptr(), cols
    st, sh = t.stride(), t.shape
    if t.dtype is not dt or t.get_device() != dev or len(sh) != 2 or sh[1] != cols or sh[0] < rows or \
            (cols > 1 and st[1] != 1):
        raise ValueError("svdq: %s has to be a %s tensor [%d][%d] with contiguous rows on the current device, not %s %s "
                         "on %s" % (what, dt, rows, cols, t.dtype, tuple(sh), t.device))
    return t.data_ptr(), (st[0] if rows > 1 else cols)   # the stride of a single row is never used


def _flat(t, n, dt, dev, what):
    """Address of a packed tensor of n elements."""
    if t is None:
        return None
    if t.dtype is not dt or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise ValueError("svdq: %s has to be a packed %s tensor of %d elements on the current device, not %s %s on %s"
                         % (what, dt, n, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _workspace(t, ws_bytes, dev):
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("svdq: the workspace has to be packed memory of the current device")
    return t.data_ptr(), t.numel() * t.element_size() if ws_bytes is None else ws_bytes


def _type_of(t, what):
    """(dtype, its code, the current device) for a call whose types follow t."""
    dt = None if t is None else t.dtype
    code = DTYPES.get(dt)
    if code is None:
        raise ValueError("svdq: %s has to be a bfloat16, float16 or float32 tensor" % what)
    return dt, code, torch._C._cuda_getDevice() if t.is_cuda else -2


def svdq_dense_linear(M, K, N, X, W_t, bias, act, residual, Y, Z=None, stream=None):
    dt, code, dev = _type_of(X, "X")
    x, ldx = _rows(X, M, K, dt, dev, "X")
    r, ldr = _rows(residual, M, N, dt, dev, "residual")
    y, ldy = _rows(Y, M, N, dt, dev, "Y")
    _check(lib.svdq_dense_linear(code, M, K, N, x, ldx, _flat(W_t, N * K, dt, dev, "W_t"),
                                 _flat(bias, N, dt, dev, "bias"), act, r, ldr, y, ldy,
                                 _flat(Z, M * N, dt, dev, "Z"), _stream(stream, dev)), "svdq_dense_linear")


def svdq_dense_linear_backward_workspace_bytes(M, K, N, act) -> int:
    return lib.svdq_dense_linear_backward_workspace_bytes(M, K, N, act)


def svdq_dense_linear_backward(M, K, N, dY, X, W_t, Z, act, dX, dW, dbias, workspace, ws_bytes=None, stream=None):
    dt, code, dev = _type_of(dY, "dY")
    dy, lddy = _rows(dY, M, N, dt, dev, "dY")
    x, ldx = _rows(X, M, K, dt, dev, "X")
    dx, lddx = _rows(dX, M, K, dt, dev, "dX")
    ws, ws_bytes = _workspace(workspace, ws_bytes, dev)
    _check(lib.svdq_dense_linear_backward(code, M, K, N, dy, lddy, x, ldx, _flat(W_t, N * K, dt, dev, "W_t"),
                                          _flat(Z, M * N, dt, dev, "Z"), act, dx, lddx,
                                          _flat(dW, N * K, dt, dev, "dW"), _flat(dbias, N, dt, dev, "dbias"), ws,
                                          ws_bytes, _stream(stream, dev)), "svdq_dense_linear_backward")


def svdq_gated_linear(M, K, F, X, Wg_t, Wu_t, bias_g, bias_u, act, H, G=None, U=None, stream=None):
    dt, code, dev = _type_of(X, "X")
    x, ldx = _rows(X, M, K, dt, dev, "X")
    h, ldh = _rows(H, M, F, dt, dev, "H")
    _check(lib.svdq_gated_linear(code, M, K, F, x, ldx, _flat(Wg_t, F * K, dt, dev, "Wg_t"),
                                 _flat(Wu_t, F * K, dt, dev, "Wu_t"), _flat(bias_g, F, dt, dev, "bias_g"),
                                 _flat(bias_u, F, dt, dev, "bias_u"), act, h, ldh, _flat(G, M * F, dt, dev, "G"),
                                 _flat(U, M * F, dt, dev, "U"), _stream(stream, dev)), "svdq_gated_linear")


def svdq_gated_linear_backward_workspace_bytes(M, K, F) -> int:
    return lib.svdq_gated_linear_backward_workspace_bytes(M, K, F)


def svdq_gated_linear_backward(M, K, F, dH, X, Wg_t, Wu_t, G, U, act, dX, dWg, dWu, dbias_g, dbias_u, workspace,
                               ws_bytes=None, stream=None):
    dt, code, dev = _type_of(dH, "dH")
    dh, lddh = _rows(dH, M, F, dt, dev, "dH")
    x, ldx = _rows(X, M, K, dt, dev, "X")
    dx, lddx = _rows(dX, M, K, dt, dev, "dX")
    ws, ws_bytes = _workspace(workspace, ws_bytes, dev)
    _check(lib.svdq_gated_linear_backward(code, M, K, F, dh, lddh, x, ldx, _flat(Wg_t, F * K, dt, dev, "Wg_t"),
                                          _flat(Wu_t, F * K, dt, dev, "Wu_t"), _flat(G, M * F, dt, dev, "G"),
                                          _flat(U, M * F, dt, dev, "U"), act, dx, lddx,
                                          _flat(dWg, F * K, dt, dev, "dWg"), _flat(dWu, F * K, dt, dev, "dWu"),
                                          _flat(dbias_g, F, dt, dev, "dbias_g"),
                                          _flat(dbias_u, F, dt, dev, "dbias_u"), ws, ws_bytes, _stream(stream, dev)),
           "svdq_gated_linear_backward")


def svdq_layernorm(M, C, X, gamma, beta, eps, Y, mean=None, rstd=None, stream=None):
    dt, code, dev = _type_of(X, "X")
    x, ldx = _rows(X, M, C, dt, dev, "X")
    y, ldy = _rows(Y, M, C, dt, dev, "Y")
    _check(lib.svdq_layernorm(code, M, C, x, ldx, _flat(gamma, C, dt, dev, "gamma"), _flat(beta, C, dt, dev, "beta"),
                              eps, y, ldy, _flat(mean, M, torch.float32, dev, "mean"),
                              _flat(rstd, M, torch.float32, dev, "rstd"), _stream(stream, dev)), "svdq_layernorm")


def svdq_layernorm_backward_workspace_bytes(M, C) -> int:
    return lib.svdq_layernorm_backward_workspace_bytes(M, C)


def svdq_layernorm_backward(M, C, dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace, ws_bytes=None, stream=None):
    dt, code, dev = _type_of(dY, "dY")
    dy, lddy = _rows(dY, M, C, dt, dev, "dY")
    x, ldx = _rows(X, M, C, dt, dev, "X")
    dx, lddx = _rows(dX, M, C, dt, dev, "dX")
    ws, ws_bytes = _workspace(workspace, ws_bytes, dev)
    _check(lib.svdq_layernorm_backward(code, M, C, dy, lddy, x, ldx, _flat(gamma, C, dt, dev, "gamma"),
                                       _flat(mean, M, torch.float32, dev, "mean"),
                                       _flat(rstd, M, torch.float32, dev, "rstd"), dx, lddx,
                                       _flat(dgamma, C, dt, dev, "dgamma"), _flat(dbeta, C, dt, dev, "dbeta"), ws,
                                       ws_bytes, _stream(stream, dev)), "svdq_layernorm_backward")


def svdq_norm_linear_workspace_bytes(w, M) -> int:
    return lib.svdq_norm_linear_workspace_bytes(w, M)


def svdq_norm_linear(w, M, X, gamma, beta, eps, epi, Y, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(lib.svdq_norm_linear(w, M, _ptr(X), _ptr(gamma), _ptr(beta), eps, epi, _ptr(Y), _ptr(workspace), ws_bytes,
                                _stream(stream)), "svdq_norm_linear")


def svdq_poll_device_error(stream=None) -> int:
    """Returns the status code (does not raise): 0, SVDQ_ERR_TIMEOUT, ..."""
    return lib.svdq_poll_device_error(_stream(stream))


def svdq_selftest_wait_timeout(limit_us, stream=None):
    _check(lib.svdq_selftest_wait_timeout(limit_us, _stream(stream)), "svdq_selftest_wait_timeout")


def svdq_debug_override_cc(major, minor):
    lib.svdq_debug_override_cc(major, minor)


def svdq_debug_product_plan(op, M, K, N, num_sms=148):
    """(swapped form, MMA columns, ranks, tall tiles, parts of dX, parts of the weight gradient)"""
    plan = (_i * 6)()
    _check(lib.svdq_debug_product_plan(op, M, K, N, num_sms, plan), "svdq_debug_product_plan")
    return tuple(plan)
