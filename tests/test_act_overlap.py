"""Outputs at an input's address, on the CPU: the activation operators' entry
points refuse what their kernels would read after it is written, before any HIP
call (the pointers here are never dereferenced).  A matrix may be written over
another that lies alike; one of another stride or type, or codes, may not."""
import os

import pytest

from fp4_quantization_block_amd import mx

A, B, C, D, E, F = (0x100000 * k for k in range(1, 7))
BF16, F32, LAYER, RMS = mx.MX_SRC_BF16, mx.MX_SRC_F32, mx.MX_NORM_LAYER, mx.MX_NORM_RMS


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("libmx.so not built")
    return mx.load()


def _refused(lib, status):
    assert status == mx.MX_ERR_INVALID_ARG
    assert "over" in lib.mx_last_error_message().decode()


def _norm(lib, x=A, ld_x=64, res=None, ld_res=64, sum=None, ld_sum=64, y=D, ld_y=64, out=BF16, qy=None, sy=None,
          qx=None, sx=None, rows=4):
    return lib.mx_norm_forward(x, ld_x, res, ld_res, BF16, rows, 64, RMS, None, None, 0, 1e-5, sum, ld_sum, y, ld_y,
                               out, 0, qy, sy, 0, qx, sx, None, E, None)


@pytest.mark.parametrize("kw", [
    dict(y=A, ld_y=80), dict(y=A, ld_x=80), dict(y=A, out=F32), dict(y=A, out=F32, rows=1),
    dict(res=B, sum=A, ld_sum=72), dict(res=B, sum=B, ld_res=72), dict(res=B, sum=C, y=B, ld_y=72),
    dict(res=B, sum=C, y=C, ld_y=72), dict(res=B, sum=C, y=B, out=F32), dict(res=B, sum=C, y=C, out=F32),
    dict(qy=A, sy=F), dict(qy=F, sy=A), dict(qx=A, sx=F), dict(qx=F, sx=A), dict(res=B, sum=C, qx=B, sx=F),
])
def test_norm_forward(lib, kw):
    _refused(lib, _norm(lib, **kw))


def _norm_grad(lib, dy=A, ld_dy=64, x=B, ld_x=64, qx=None, sx=None, dsum=C, ld_dsum=64, dx=D, ld_dx=64):
    return lib.mx_norm_backward(dy, ld_dy, BF16, 4, 64, x, ld_x, 0, qx, sx, None, E, RMS, None, 0, dsum, ld_dsum, dx,
                                ld_dx, None, None, None, 0, None)


@pytest.mark.parametrize("kw", [
    dict(dx=A, ld_dx=72), dict(dx=A, ld_dy=72), dict(dx=B, ld_dx=72), dict(dx=B, ld_x=72), dict(dx=C, ld_dx=72),
    dict(dx=C, ld_dsum=72), dict(x=None, qx=D, sx=F), dict(x=None, qx=F, sx=D),
])
def test_norm_backward(lib, kw):
    _refused(lib, _norm_grad(lib, **kw))


def _glu(lib, ld_g=64, ld_u=64, h=C, ld_h=64, out=BF16, qh=None, sh=None, q=(None,) * 4, rows=4):
    return lib.mx_glu_forward(A, ld_g, B, ld_u, BF16, rows, 64, 0, h, ld_h, out, 0, qh, sh, 0, *q, None)


@pytest.mark.parametrize("kw", [
    dict(h=A, ld_h=72), dict(h=A, ld_g=72), dict(h=B, ld_u=72), dict(h=A, out=F32), dict(h=B, out=F32, rows=1),
    dict(qh=A, sh=D), dict(qh=D, sh=B), dict(q=(A, D, E, F)), dict(q=(D, A, E, F)), dict(q=(D, E, B, F)),
    dict(q=(D, E, F, B)), dict(q=(B, D, E, F)),
])
def test_glu_forward(lib, kw):
    _refused(lib, _glu(lib, **kw))


TENSORS, COPIES = (B, 64, C, 64, 0, None, None, None, None), (None, 0, None, 0, 0, B, C, D, E)


@pytest.mark.parametrize("inputs", [TENSORS, COPIES])
@pytest.mark.parametrize("k", range(3))
def test_glu_backward(lib, inputs, k):
    for p in {v for v in (A, *inputs) if v and v >= A}:
        outs = [0x10 * A, 0x20 * A, 0x30 * A]
        outs[k] = p
        lds = [64, 64, 64]
        lds[k] = 72
        args = [v for pair in zip(outs, lds) for v in pair]
        _refused(lib, lib.mx_glu_backward(A, 64, BF16, 64, 64, *inputs, 0, *args, None))


@pytest.mark.parametrize("inputs", [TENSORS, COPIES])
@pytest.mark.parametrize("k", range(6))
def test_glu_backward_dual_layout(lib, inputs, k):
    for p in {v for v in (A, *inputs) if v and v >= A}:
        o = [0x10 * A, 0x20 * A, 0x30 * A, 0x40 * A, 0x50 * A, 0x60 * A]
        o[k] = p
        _refused(lib, lib.mx_glu_backward_dual_layout(A, 64, BF16, 64, 64, *inputs, 0, 1, *o[:4], 0, *o[4:], None))
