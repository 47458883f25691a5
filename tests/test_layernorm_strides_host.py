"""The layer norm's row strides: refused from 2^40 bytes on, as include/svdq.h
states for every 16-bit call (no GPU needed)."""
import pytest

import test_dense_host as H

B = H.B   # the fixture that builds and loads the library

CALLS = [("svdq_layernorm", k) for k in ("ldx", "ldy")] + \
    [("svdq_layernorm_backward", k) for k in ("lddy", "ldx", "lddx")]


@pytest.mark.parametrize("dt,elem", [(0, 2), (1, 2), (2, 4)])
@pytest.mark.parametrize("name,stride", CALLS)
def test_strides_of_2_to_40_bytes_are_refused(B, name, stride, dt, elem):
    limit = (1 << 40) // elem
    for bad in (limit, limit + 8, 1 << 62):
        assert H.call(B, name, dt=dt, **{stride: bad}) == H.SHAPE, (stride, bad)
    # one element below the limit passes the shape check: an empty batch is a no-op
    if name == "svdq_layernorm":
        assert H.call(B, name, dt=dt, M=0, **{stride: limit - 1}) == H.OK


def test_a_gradient_that_is_not_asked_for_has_no_stride(B):
    status = H.call(B, "svdq_layernorm_backward", M=0, dX=None, lddx=1 << 62, dgamma=None, dbeta=None)
    assert status in (H.OK, H.UNSUPPORTED)   # nothing to write: OK where there is a device
