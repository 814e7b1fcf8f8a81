"""Argument checks of the activation operators, on the CPU: the C entry points
refuse before any HIP call (the pointers here are never dereferenced), and the
binding refuses tensors of the wrong type, shape or layout before it calls."""
import os

import pytest
import torch

from fp4_quantization_block_amd import mx

INV, UNS, ALI = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGNMENT
P = 0x10000
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("libmx.so not built")
    return mx.load()


def _norm_fwd(lib, x=P, ld_x=64, res=None, ld_res=64, src=1, rows=4, cols=64, kind=1, w=P, b=None, pd=0, eps=1e-5,
              sum=None, ld_sum=64, y=P, ld_y=64, out=1, yf=0, qy=None, sy=None, cf=0, qx=None, sx=None, mean=None,
              rstd=P):
    return lib.mx_norm_forward(x, ld_x, res, ld_res, src, rows, cols, kind, w, b, pd, eps, sum, ld_sum, y, ld_y, out,
                               yf, qy, sy, cf, qx, sx, mean, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(src=2), INV), (dict(rows=0), INV), (dict(cols=0), INV), (dict(rows=-1), INV),
    (dict(rows=BIG), INV), (dict(cols=BIG, ld_x=BIG, ld_y=BIG), INV), (dict(ld_x=63), INV), (dict(x=P + 1), ALI),
    (dict(x=P + 2, src=0, out=0), ALI), (dict(res=P), INV), (dict(sum=P), INV), (dict(res=P, sum=P, ld_res=1), INV),
    (dict(res=P, sum=P, ld_sum=1), INV), (dict(res=P + 1, sum=P), ALI), (dict(res=P, sum=P + 1), ALI),
    (dict(kind=2), INV), (dict(pd=3), INV), (dict(w=P + 2), ALI), (dict(b=P + 1, pd=1), ALI), (dict(eps=-1e-5), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(y=None), INV), (dict(out=2), INV),
    (dict(ld_y=63), INV), (dict(y=P + 1), ALI), (dict(qy=P), INV), (dict(sy=P), INV), (dict(qy=P, sy=P, yf=2), UNS),
    (dict(qy=P, sy=P, yf=3), INV), (dict(qy=P + 8, sy=P), ALI), (dict(qx=P), INV), (dict(qx=P, sx=P, cf=2), UNS),
    (dict(qx=P, sx=P, cols=40), INV), (dict(qy=P, sy=P, y=None, cols=33), INV), (dict(rstd=P + 2), ALI),
    (dict(mean=P + 1), ALI),
])
def test_norm_forward_refuses(lib, kw, status):
    assert _norm_fwd(lib, **kw) == status
    assert lib.mx_last_error_message().decode() != ""


def _norm_bwd(lib, dy=P, ld_dy=64, src=1, rows=4, cols=64, x=P, ld_x=64, cf=0, qx=None, sx=None, mean=None, rstd=P,
              kind=1, w=P, pd=0, dsum=None, ld_dsum=64, dx=P, ld_dx=64, dw=P, db=None, work=P, nbytes=1 << 30):
    return lib.mx_norm_backward(dy, ld_dy, src, rows, cols, x, ld_x, cf, qx, sx, mean, rstd, kind, w, pd, dsum,
                                ld_dsum, dx, ld_dx, dw, db, work, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(dx=None), INV), (dict(src=5), INV), (dict(rows=0), INV), (dict(cols=0), INV),
    (dict(rows=BIG), INV), (dict(ld_dy=1), INV), (dict(ld_dx=1), INV), (dict(ld_x=1), INV), (dict(dy=P + 1), ALI),
    (dict(dx=P + 1), ALI), (dict(x=P + 1), ALI), (dict(x=None), INV), (dict(qx=P, sx=P), INV),
    (dict(x=None, qx=P), INV), (dict(x=None, qx=P, sx=P, cf=2), UNS), (dict(x=None, qx=P, sx=P, cols=40), INV),
    (dict(x=None, qx=P + 4, sx=P), ALI), (dict(kind=7), INV), (dict(kind=0), INV), (dict(rstd=None), INV),
    (dict(rstd=P + 1), ALI), (dict(kind=0, mean=P + 2), ALI), (dict(pd=9), INV), (dict(w=P + 1, pd=1), ALI),
    (dict(dsum=P, ld_dsum=2), INV), (dict(dsum=P + 1), ALI), (dict(dw=P + 2), ALI), (dict(db=P + 2), ALI),
    (dict(work=None), INV), (dict(work=P + 2), ALI), (dict(nbytes=100), INV), (dict(dw=None, db=P, work=None), INV),
    (dict(cols=16385, ld_dy=16385, ld_x=16385, ld_dx=16385, x=2 * P), UNS),
    (dict(cols=16385, ld_dy=16385, ld_x=16385, ld_dx=16385, dy=2 * P), UNS),
])
def test_norm_backward_refuses(lib, kw, status):
    assert _norm_bwd(lib, **kw) == status
    assert lib.mx_last_error_message().decode() != ""


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 64), (509, 2051), (8192, 4096), (5, 20000), (100000, 512)])
def test_norm_workspace(lib, rows, cols):
    n = lib.mx_norm_backward_workspace_bytes(rows, cols)
    assert n > 0 and n % (8 * cols) == 0 and n <= 8 * cols * max(2048, rows)
    assert _norm_bwd(lib, rows=rows, cols=cols, ld_dy=cols, ld_x=cols, ld_dx=cols, nbytes=n - 1) == INV
    assert lib.mx_norm_backward_workspace_bytes(0, cols) == 0
    assert lib.mx_norm_backward_workspace_bytes(rows, -1) == 0


def _glu_fwd(lib, g=P, ld_g=64, u=P, ld_u=64, src=1, rows=4, cols=64, act=0, h=P, ld_h=64, out=1, hf=0, qh=None,
             sh=None, cf=0, qg=None, sg=None, qu=None, su=None):
    return lib.mx_glu_forward(g, ld_g, u, ld_u, src, rows, cols, act, h, ld_h, out, hf, qh, sh, cf, qg, sg, qu, su, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), INV), (dict(u=None), INV), (dict(src=4), INV), (dict(rows=0), INV), (dict(cols=-2), INV),
    (dict(cols=BIG), INV), (dict(ld_g=63), INV), (dict(ld_u=63), INV), (dict(ld_h=63), INV), (dict(g=P + 1), ALI),
    (dict(u=P + 1), ALI), (dict(h=P + 1), ALI), (dict(h=P + 2, out=0), ALI), (dict(act=3), INV), (dict(act=-1), INV),
    (dict(h=None), INV), (dict(out=7), INV), (dict(qh=P), INV), (dict(sh=P), INV), (dict(qh=P, sh=P, hf=2), UNS),
    (dict(qh=P + 1, sh=P), ALI), (dict(qh=P, sh=P, cols=33), INV), (dict(qg=P, sg=P), INV), (dict(qu=P, su=P), INV),
    (dict(qg=P, sg=P, qu=P), INV), (dict(qg=P, sg=P, qu=P, su=P, cf=2), UNS), (dict(qg=P, sg=P, qu=P + 8, su=P), ALI),
    (dict(qg=P, sg=P, qu=P, su=P, cf=5), INV),
])
def test_glu_forward_refuses(lib, kw, status):
    assert _glu_fwd(lib, **kw) == status
    assert lib.mx_last_error_message().decode() != ""


def _head(dh=P, ld_dh=64, src=1, rows=64, cols=64, g=P, ld_g=64, u=P, ld_u=64, cf=0, qg=None, sg=None, qu=None,
          su=None, act=0):
    return (dh, ld_dh, src, rows, cols, g, ld_g, u, ld_u, cf, qg, sg, qu, su, act)


CK = dict(g=None, u=None, qg=P, sg=P, qu=P, su=P)
INPUTS = [
    (dict(dh=None), INV), (dict(src=3), INV), (dict(rows=0), INV), (dict(cols=0), INV), (dict(rows=BIG), INV),
    (dict(ld_dh=1), INV), (dict(ld_g=1), INV), (dict(ld_u=1), INV), (dict(dh=P + 1), ALI), (dict(g=P + 1), ALI),
    (dict(u=P + 1), ALI), (dict(g=None), INV), (dict(u=None), INV), (dict(g=None, u=None), INV),
    (dict(qg=P, sg=P, qu=P, su=P), INV), (dict(CK, su=None), INV), (dict(CK, qu=None, su=None), INV),
    (dict(CK, cf=2), UNS), (dict(CK, cf=8), INV), (dict(CK, qg=P + 8), ALI), (dict(CK, cols=48), INV), (dict(act=5), INV),
]


@pytest.mark.parametrize("kw,status", INPUTS)
def test_glu_backward_refuses_inputs(lib, kw, status):
    assert lib.mx_glu_backward(*_head(**kw), P, 64, P, 64, None, 0, None) == status
    assert lib.mx_last_error_message().decode() != ""
    assert lib.mx_glu_backward_dual_layout(*_head(**kw), 1, P, P, P, P, 0, None, None, None) == status


@pytest.mark.parametrize("args,status", [
    ((None, 64, P, 64, None, 0), INV), ((P, 64, None, 64, None, 0), INV), ((P, 63, P, 64, None, 0), INV),
    ((P, 64, P, 63, None, 0), INV), ((P, 64, P, 64, P, 63), INV), ((P + 1, 64, P, 64, None, 0), ALI),
    ((P, 64, P + 1, 64, None, 0), ALI), ((P, 64, P, 64, P + 1, 64), ALI),
])
def test_glu_backward_refuses_outputs(lib, args, status):
    assert lib.mx_glu_backward(*_head(), *args, None) == status


@pytest.mark.parametrize("kw,args,status", [
    (dict(rows=40), (1, P, P, P, P, 0, None, None), INV), (dict(cols=40), (1, P, P, P, P, 0, None, None), INV),
    ({}, (1, None, P, P, P, 0, None, None), INV), ({}, (1, P, None, P, P, 0, None, None), INV),
    ({}, (1, P, P, None, P, 0, None, None), INV), ({}, (1, P, P, P, None, 0, None, None), INV),
    ({}, (2, P, P, P, P, 0, None, None), UNS), ({}, (4, P, P, P, P, 0, None, None), INV),
    ({}, (1, P + 8, P, P, P, 0, None, None), ALI), ({}, (1, P, P, P + 8, P, 0, None, None), ALI),
    ({}, (1, P, P, P, P, 0, P, None), INV), ({}, (1, P, P, P, P, 2, P, P), UNS), ({}, (1, P, P, P, P, 0, P + 8, P), ALI),
    (dict(rows=(1 << 30), cols=1 << 30, ld_dh=1 << 30, ld_g=1 << 30, ld_u=1 << 30), (1, P, P, P, P, 0, None, None), INV),
    (dict(rows=(1 << 23) + 32), (1, P, P, P, P, 0, None, None), INV),           # 32-bit offsets in a tile
    (dict(cols=(1 << 23) + 32, ld_dh=1 << 24, ld_g=1 << 24, ld_u=1 << 24), (1, P, P, P, P, 0, None, None), INV),
    (dict(ld_dh=(1 << 23) + 1), (1, P, P, P, P, 0, None, None), INV),
    (dict(ld_g=(1 << 23) + 1), (1, P, P, P, P, 0, None, None), INV),
    (dict(ld_u=(1 << 23) + 1), (1, P, P, P, P, 0, None, None), INV),
    (dict(rows=1 << 23, cols=1 << 23, ld_dh=1 << 23, ld_g=1 << 23, ld_u=1 << 23), (1, P, P, P, P, 0, None, None), INV),
])
def test_glu_backward_dual_refuses(lib, kw, args, status):
    assert lib.mx_glu_backward_dual_layout(*_head(**kw), *args, None) == status
    assert lib.mx_last_error_message().decode() != ""


# ---- the binding: refused before the library is asked
X, B16 = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
V, CODES, SC = torch.zeros(64), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
R4 = torch.zeros(4)


@pytest.mark.parametrize("call,error", [
    (lambda: mx.mx_norm_forward(X.half()), TypeError),
    (lambda: mx.mx_norm_forward(X[0]), ValueError),
    (lambda: mx.mx_norm_forward(X.t()), ValueError),
    (lambda: mx.mx_norm_forward(X, kind="group"), KeyError),
    (lambda: mx.mx_norm_forward(X, weight=V.half()), TypeError),
    (lambda: mx.mx_norm_forward(X, weight=V[:63]), ValueError),
    (lambda: mx.mx_norm_forward(X, weight=V, bias=V.bfloat16()), TypeError),
    (lambda: mx.mx_norm_forward(X, weight=torch.zeros(128)[::2]), ValueError),
    (lambda: mx.mx_norm_forward(X, residual=B16), TypeError),
    (lambda: mx.mx_norm_forward(X, residual=X[:3]), ValueError),
    (lambda: mx.mx_norm_forward(X, sum_out=X), ValueError),
    (lambda: mx.mx_norm_forward(X, out_dtype=torch.float16), TypeError),
    (lambda: mx.mx_norm_forward(X, y=B16), TypeError),
    (lambda: mx.mx_norm_forward(X, qy=CODES), ValueError),
    (lambda: mx.mx_norm_forward(X, y_fmt="e4m3", qy=CODES[:, :32]), ValueError),
    (lambda: mx.mx_norm_forward(X, ckpt_fmt="e4m3", sx=SC[:, :1]), ValueError),
    (lambda: mx.mx_norm_forward(X, rstd=V), ValueError),
    (lambda: mx.mx_norm_backward(X, V, x=X), ValueError),
    (lambda: mx.mx_norm_backward(X, R4, x=B16), TypeError),
    (lambda: mx.mx_norm_backward(X, R4, ckpt=mx.checkpoint("e4m3", CODES, SC[:2])), ValueError),
    (lambda: mx.mx_norm_backward(X, R4, x=X, dsum=X[:, :32]), ValueError),
    (lambda: mx.mx_norm_backward(X, R4, x=X, dweight=V.double()), TypeError),
    (lambda: mx.mx_glu_forward(X, B16), TypeError),
    (lambda: mx.mx_glu_forward(X, X[:, :32]), ValueError),
    (lambda: mx.mx_glu_forward(X, X, h=X[:2]), ValueError),
    (lambda: mx.mx_glu_forward(X, X, qg=CODES), ValueError),
    (lambda: mx.mx_glu_backward(X, gate=X, up=B16), TypeError),
    (lambda: mx.mx_glu_backward(X, gate=X, up=X, act="relu"), KeyError),
    (lambda: mx.mx_glu_backward(X, gate_ckpt=mx.checkpoint("e4m3", CODES, SC),
                                up_ckpt=mx.checkpoint("e5m2", CODES, SC)), ValueError),
    (lambda: mx.mx_glu_backward(X, gate=X, up=X, dgate=X.t()), ValueError),
    (lambda: mx.mx_glu_backward_dual_layout(X, X, X, q_row=CODES), ValueError),
    (lambda: mx.mx_glu_backward_dual_layout(X, X, X, qh_col=CODES), ValueError),
    (lambda: mx.mx_norm_forward(X), ValueError),                      # host tensors
    (lambda: mx.mx_norm_backward(X, R4, x=X), ValueError),
    (lambda: mx.mx_glu_forward(X, X), ValueError),
    (lambda: mx.mx_glu_backward(X, gate=X, up=X), ValueError),
    (lambda: mx.mx_norm_forward(X, weight=torch.empty(64, device="meta")), ValueError),
])
def test_binding_refuses(call, error):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("work", [torch.empty(1 << 16, device="meta", dtype=torch.uint8)[::2],
                                  torch.empty((64, 64), dtype=torch.float32).t()])
def test_binding_refuses_a_strided_workspace(work):
    with pytest.raises(ValueError, match="work must be contiguous"):
        mx.mx_norm_backward(X, R4, x=X, work=work)
