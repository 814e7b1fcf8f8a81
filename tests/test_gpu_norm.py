"""mx_norm_forward and mx_norm_backward against their definitions in 64 bits,
with bounds that count fp32 roundings (act_ref.py); quantized outputs and
checkpoints against the oracle's quantizer, bit for bit."""
import numpy as np
import pytest
import torch

import act_ref as R
from act_util import DT, Guarded, assert_row_copy, dev, make_checkpoint, rand, restored
from fp4_quantization_block_amd import mx
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5

# row lengths at which the kernels, or the last chunk, change
COLS = [1, 2, 7, 8, 16, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 384, 509, 512, 513, 520, 1000, 1024,
        1025, 1536, 1537, 2048, 2049, 2056, 3080, 4096, 4097, 5000, 5121, 6144, 6145, 8192, 8193, 12288, 12289, 16384, 16385, 20000,
        24577]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rows(cols):
    return 5 if cols > 4096 else 67


def _stream(seed, rows, cols, mean=0.5):
    """Rows of different size, an offset, one channel far above the others."""
    x = rand(seed, rows, cols) * torch.exp(rand(seed + 1, rows, 1)) + mean
    x[:, cols // 2] *= 30
    return x


def _check_forward(r, s, w, b, layer, dtype, what):
    one = torch.ones(1, dtype=torch.float64)
    y, err, mu, mu_err, rs, r_err = R.norm(s, one if w is None else w.cpu().double(),
                                           0 * one if b is None else b.cpu().double(), EPS, layer)
    if r.y is not None:
        R.within(r.y, y, err, f"{what} y")
    R.within(r.rstd, rs, r_err, f"{what} rstd")
    if layer:
        R.within(r.mean, mu, mu_err, f"{what} mean")
    else:
        assert r.mean is None


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_forward(cols, dtype, kind):
    dt, rows = DT[dtype], _rows(cols)
    x = dev(_stream(1, rows, cols), dt)
    w, b = dev(rand(3, cols), dt), dev(rand(4, cols), dt)
    bias = b if kind == "layer" else None
    r = mx.mx_norm_forward(x, w, bias, eps=EPS, kind=kind)
    _check_forward(r, x.cpu().double(), w, bias, kind == "layer", dt, f"{rows}x{cols} {dtype} {kind}")


@pytest.mark.parametrize("params", ["f32", "bf16", "none", "bias only"])
@pytest.mark.parametrize("src,out", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_forward_types(src, out, params):
    rows, cols = 33, 1031
    x = dev(_stream(1, rows, cols), DT[src])
    p = DT["bf16" if params == "bf16" else "f32"]
    w = None if params in ("none", "bias only") else dev(rand(3, cols), p)
    b = None if params == "none" else dev(rand(4, cols), p)
    r = mx.mx_norm_forward(x, w, b, eps=EPS, kind="layer", out_dtype=DT[out])
    assert r.y.dtype == DT[out]
    _check_forward(r, x.cpu().double(), w, b, True, DT[out], f"{src} {out} {params}")


@pytest.mark.parametrize("cols", [33, 96, 4096, 5000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("alias", [None, "x", "residual"])
def test_forward_residual(alias, dtype, cols):
    """The sum is the fp32 sum rounded to the type, and what is normalised is
    that; it may be written over one of its terms."""
    dt, rows = DT[dtype], 9
    x, res = dev(_stream(1, rows, cols), dt), dev(rand(7, rows, cols), dt)
    want = (x.float() + res.float()).to(dt)
    into = {"x": x, "residual": res, None: None}[alias]
    r = mx.mx_norm_forward(x, None, None, eps=EPS, kind="layer", residual=res, sum_out=into)
    assert torch.equal(r.sum, want)
    assert alias is None or r.sum.data_ptr() == into.data_ptr()
    _check_forward(r, want.cpu().double(), None, None, True, dt, f"residual {cols}")


@pytest.mark.parametrize("cols", [32, 96, 512, 544, 4096, 8224, 20000])
@pytest.mark.parametrize("fmt,other", [("e4m3", "e5m2"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_copies(dtype, fmt, other, cols):
    """The row copy of y encodes the fp32 y that the fp32 output shows; the
    checkpoint is the row copy of the sum; neither changes y, and both come
    out the same without it."""
    dt, rows = DT[dtype], 7
    x, res, w = dev(_stream(1, rows, cols), dt), dev(rand(7, rows, cols), dt), dev(rand(3, cols), dt)
    kw = dict(eps=EPS, kind="rms", residual=res)
    r = mx.mx_norm_forward(x, w, out_dtype=torch.float32, y_fmt=fmt, ckpt_fmt=other, **kw)
    assert_row_copy(r.qy, r.sy, r.y, fmt, "y copy")
    assert_row_copy(r.qx, r.sx, r.sum, other, "checkpoint")
    alone = mx.mx_norm_forward(x, w, write_y=False, y_fmt=fmt, stats=False, **kw)
    assert alone.y is None and alone.rstd is None
    assert torch.equal(alone.qy, r.qy) and torch.equal(alone.sy, r.sy)
    assert torch.equal(mx.mx_norm_forward(x, w, out_dtype=torch.float32, **kw).y, r.y)


@pytest.mark.parametrize("cols", [40, 41, 520, 4100, 20001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (3, 0), (5, 1)])
def test_forward_strides_and_alignment(offset, pad, dtype, cols):
    """Matrices inside larger buffers, at odd elements: nothing outside is
    written, and the results are those of dense matrices."""
    dt, rows = DT[dtype], 11
    a, b = rand(1, rows, cols).to(dt), rand(2, rows, cols).to(dt)
    x, res = Guarded(rows, cols, dt, offset, pad, a), Guarded(rows, cols, dt, offset + 2, pad + 1, b)
    y, total = Guarded(rows, cols, dt, offset + 1, pad + 3), Guarded(rows, cols, dt, offset + 3, pad)
    w = Guarded(1, cols, dt, offset, 0, rand(3, 1, cols).to(dt))
    r = mx.mx_norm_forward(x.view, w.view[0], eps=EPS, kind="layer", residual=res.view, sum_out=total.view, y=y.view)
    want = mx.mx_norm_forward(dev(a, dt), w.view[0].clone(), eps=EPS, kind="layer", residual=dev(b, dt))
    assert torch.equal(r.y, want.y) and torch.equal(r.sum, want.sum) and torch.equal(r.rstd, want.rstd)
    for g, what in ((x, "x"), (res, "residual"), (y, "y"), (total, "sum"), (w, "weight")):
        g.check(what)


@pytest.mark.parametrize("cols", [3, 32, 513, 4096, 20000])
def test_forward_special_rows(cols):
    """Rows that are constant, zero, huge, tiny, or hold an Inf or a NaN: each
    as its formula says, and no other row is touched."""
    x = rand(1, 8, cols).float()
    x[0] = 3.25
    x[1] = 0.0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, cols // 2] = float("inf")
    x[5, cols - 1] = float("nan")
    x[6] += 1e4                                  # a mean far above the deviation
    x = x.to(DEV)
    for kind in ("layer", "rms"):
        r = mx.mx_norm_forward(x, eps=EPS, kind=kind)
        keep = [0, 1, 2, 3, 6, 7]
        got = r._replace(y=r.y[keep], rstd=r.rstd[keep], mean=r.mean[keep] if kind == "layer" else None)
        _check_forward(got, x[keep].cpu().double(), None, None, kind == "layer", torch.float32, f"special {kind}")
        assert bool(torch.isnan(r.y[5]).all())
        if kind == "layer":
            assert bool(torch.isnan(r.y[4]).all()) and bool((r.y[0] == 0).all())
        else:
            # 1 / sqrt(inf) = 0: finite elements give 0 and inf * 0 is NaN
            assert bool(torch.isnan(r.y[4, cols // 2])) and int(torch.isnan(r.y[4]).sum()) == 1
    c = mx.mx_norm_forward(x[:, :cols // 32 * 32], eps=EPS, kind="rms", y_fmt="e4m3", ckpt_fmt="e4m3",
                           out_dtype=torch.float32) if cols >= 32 else None
    if c is not None:
        assert_row_copy(c.qx, c.sx, x[:, :cols // 32 * 32].contiguous(), "e4m3", "special checkpoint")
        assert_row_copy(c.qy, c.sy, c.y, "e4m3", "special y copy")


def test_forward_zero_eps():
    """eps = 0 with a constant row divides by zero, as the formula does."""
    x = torch.full((1, 48), 2.0, device=DEV)
    assert bool(torch.isnan(mx.mx_norm_forward(x, eps=0.0, kind="layer").y).all())
    assert bool((mx.mx_norm_forward(x, eps=0.0, kind="rms").y == 1.0).all())


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def _backward_case(rows, cols, dt, kind, seed=1):
    x = dev(_stream(seed, rows, cols), dt)
    dy = dev(rand(seed + 5, rows, cols) * torch.exp(rand(seed + 6, rows, 1)) * 1e-2, dt)
    w = dev(1 + 0.3 * rand(seed + 7, cols), dt)
    mu, r = R.stats(x.cpu().double(), EPS, kind == "layer")
    return x, dy, w, mu.float().to(DEV), r.float().to(DEV)


def _check_backward(out, dy, s, mean, rstd, w, dsum, kind, what):
    rows, cols = dy.shape
    z = torch.zeros(1, dtype=torch.float64)
    dx, dx_err, dw, dw_err, db, db_err = R.norm_grad(
        dy.cpu().double(), s, mean.cpu().double() if kind == "layer" else torch.zeros(rows, dtype=torch.float64),
        rstd.cpu().double(), torch.ones(1, dtype=torch.float64) if w is None else w.cpu().double(),
        z if dsum is None else dsum.cpu().double(), kind == "layer", rows + 16)
    R.within(out.dx, dx, dx_err, f"{what} dx")
    if out.dweight is not None:
        R.within(out.dweight, dw, dw_err, f"{what} dweight")
    if out.dbias is not None:
        R.within(out.dbias, db, db_err, f"{what} dbias")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_backward(cols, dtype, kind):
    rows = _rows(cols)
    x, dy, w, mean, rstd = _backward_case(rows, cols, DT[dtype], kind)
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean if kind == "layer" else None, weight=w, kind=kind,
                              want_dbias=True)
    _check_backward(out, dy, x.cpu().double(), mean, rstd, w, None, kind, f"{rows}x{cols} {dtype} {kind}")


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 255, 511, 513, 1300, 2600])
@pytest.mark.parametrize("cols", [24, 100, 136, 200, 640, 641])
def test_backward_rows(rows, cols):
    """Row counts around the number of workgroups and of rows they share."""
    x, dy, w, mean, rstd = _backward_case(rows, cols, torch.float32, "layer")
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
    _check_backward(out, dy, x.cpu().double(), mean, rstd, w, None, "layer", f"{rows}x{cols}")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 7, 255, 511, 513, 1023, 1025, 1300, 2600])
@pytest.mark.parametrize("cols", [1056, 1100, 2304, 2305])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_rows_in_groups(rows, cols, dtype):
    """Row counts around the number of rows that a workgroup takes at a time."""
    x, dy, w, mean, rstd = _backward_case(rows, cols, dtype, "layer")
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
    _check_backward(out, dy, x.cpu().double(), mean, rstd, w, None, "layer", f"{rows}x{cols} {dtype}")


@pytest.mark.parametrize("rows", [1, 2, 257, 600])
@pytest.mark.parametrize("cols", [8200, 10243, 12288])
def test_backward_rows_of_three_chunks(rows, cols):
    x, dy, w, mean, rstd = _backward_case(rows, cols, torch.bfloat16, "layer")
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
    _check_backward(out, dy, x.cpu().double(), mean, rstd, w, None, "layer", f"{rows}x{cols}")


@pytest.mark.parametrize("rows", [1, 70, 130])
def test_backward_wide_rows(rows):
    x, dy, w, mean, rstd = _backward_case(rows, 16416, torch.bfloat16, "layer")
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
    _check_backward(out, dy, x.cpu().double(), mean, rstd, w, None, "layer", f"{rows} wide rows")


@pytest.mark.parametrize("cols", [32, 160, 512, 1056, 4096, 8192, 12000 // 32 * 32, 16416])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind,dtype", [("rms", "bf16"), ("layer", "f32")])
def test_backward_from_checkpoint(kind, dtype, fmt, cols):
    """From the checkpoint, the gradients are those at the values its codes
    stand for, with the residual path's gradient added."""
    rows, dt = 19, DT[dtype]
    x, dy, w, mean, rstd = _backward_case(rows, cols, dt, kind)
    dsum = dev(rand(20, rows, cols, scale=1e-2), dt)
    c = make_checkpoint(x, fmt)
    out = mx.mx_norm_backward(dy, rstd, ckpt=c, mean=mean if kind == "layer" else None, weight=w, kind=kind,
                              dsum=dsum, want_dbias=kind == "layer")
    _check_backward(out, dy, restored(c.q, c.s, fmt), mean, rstd, w, dsum, kind, f"{fmt} {cols}")


def test_backward_every_code_and_scale():
    """Every code under every scale byte 1 .. 254, and byte 0 (2^-127), in
    checkpoints no quantizer writes: codes as the oracle decodes them."""
    rows, cols = 255, 256
    q = torch.arange(256, dtype=torch.uint8).repeat(rows, 1).to(DEV)
    s = torch.arange(rows, dtype=torch.uint8)[:, None].repeat(1, cols // 32).to(DEV)
    for fmt in ("e4m3", "e5m2"):
        h = restored(q, s, fmt)
        # rstd takes the scale back out, up to the ends of fp32
        rstd = torch.exp2((127.0 - torch.arange(rows)).clamp(-126, 126)).float().to(DEV)
        dy = torch.ones(rows, cols, device=DEV)
        out = mx.mx_norm_backward(dy, rstd, ckpt=mx.checkpoint(fmt, q, s), kind="rms", want_dweight=True)
        unit = h * rstd.cpu().double()[:, None]
        want = unit.sum(0)
        finite = torch.isfinite(want)
        assert torch.equal(torch.isfinite(out.dweight.cpu()), finite)
        err = ((out.dweight.cpu().double() - want).abs() <= (rows + 20) * R.U * unit.abs().sum(0))
        assert bool(err[finite].all())


@pytest.mark.parametrize("what", ["no weight", "bf16 weight f32 x", "no dweight", "dbias only", "dsum in place",
                                  "dy in place", "x in place"])
@pytest.mark.parametrize("cols", [5, 99, 777, 6145, 12001, 12000])
def test_backward_options(what, cols):
    rows = 21
    x, dy, w, mean, rstd = _backward_case(rows, cols, torch.float32, "layer")
    dsum, kw = None, dict(want_dbias=True)
    dy0 = dy.clone()
    if what == "no weight":
        w = None
    elif what == "bf16 weight f32 x":
        w = w.bfloat16()
    elif what == "no dweight":
        kw = dict(want_dweight=False)
    elif what == "dbias only":
        kw = dict(want_dweight=False, want_dbias=True)
    elif what == "dsum in place":
        dsum = dev(rand(9, rows, cols), torch.float32)
        kw = dict(dsum=dsum, dx=dsum)
        dsum = dsum.clone()
    elif what == "dy in place":
        kw = dict(dx=dy)
    else:
        kw = dict(dx=x)
    x0 = x.cpu().double()
    out = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", **kw)
    _check_backward(out, dy0, x0, mean, rstd, w, dsum, "layer", f"{what} {cols}")


@pytest.mark.parametrize("offset,pad", [(1, 3), (3, 0), (0, 8)])
@pytest.mark.parametrize("cols", [41, 520, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_strides_and_alignment(dtype, cols, offset, pad):
    rows, dt = 13, DT[dtype]
    x, dy, w, mean, rstd = _backward_case(rows, cols, dt, "layer")
    dsum = dev(rand(9, rows, cols), dt)
    gx, gdy = Guarded(rows, cols, dt, offset, pad, x), Guarded(rows, cols, dt, offset + 1, pad + 2, dy)
    gs, gdx = Guarded(rows, cols, dt, offset + 2, pad + 1, dsum), Guarded(rows, cols, dt, offset + 3, pad + 5)
    want = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", dsum=dsum, want_dbias=True)
    nbytes = int(mx.load().mx_norm_backward_workspace_bytes(rows, cols))
    work = torch.full((nbytes + 256,), 7, dtype=torch.uint8, device=DEV)
    got = mx.mx_norm_backward(gdy.view, rstd, x=gx.view, mean=mean, weight=w, kind="layer", dsum=gs.view, dx=gdx.view,
                              want_dbias=True, work=work[:nbytes])
    assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
    assert torch.equal(got.dbias, want.dbias)
    for g, name in ((gx, "x"), (gdy, "dy"), (gs, "dsum"), (gdx, "dx")):
        g.check(name)
    assert bool((work[nbytes:] == 7).all()), "written past the workspace"


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_are_difference_quotients(kind):
    """The directional derivative of sum(dy * norm(x, w, b)) by the forward
    definition in 64 bits, against the kernel's gradients in fp32: the
    quotient's own error is O(h^2), below the gradients' bound."""
    rows, cols = 6, 135
    x, dy, w, _, _ = _backward_case(rows, cols, torch.float32, kind)
    b = dev(rand(30, cols), torch.float32)
    r = mx.mx_norm_forward(x, w, b, eps=EPS, kind=kind)
    out = mx.mx_norm_backward(dy, r.rstd, x=x, mean=r.mean, weight=w, kind=kind, want_dbias=True)
    X, W, B, G = (t.cpu().double() for t in (x, w, b, dy))
    for k in range(5):
        dX, dW, dB = rand(40 + k, rows, cols), rand(50 + k, cols), rand(60 + k, cols)
        h = 1e-6
        f = [float((G * R.norm(X + s * h * dX, W + s * h * dW, B + s * h * dB, EPS, kind == "layer")[0]).sum())
             for s in (1, -1)]
        want = (f[0] - f[1]) / (2 * h)
        terms = [(out.dx.cpu().double() * dX), (out.dweight.cpu().double() * dW), (out.dbias.cpu().double() * dB)]
        size = sum(float(t.abs().sum()) for t in terms)
        # every gradient within 300 U of the size of its terms, and the quotient within 1e-7
        assert abs(sum(float(t.sum()) for t in terms) - want) <= (300 * R.U + 1e-7) * size * 4


def test_runs_repeat_bit_for_bit():
    rows, cols = 3000, 2048
    x, dy, w, mean, rstd = _backward_case(rows, cols, torch.bfloat16, "layer")
    first = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
    for _ in range(5):
        again = mx.mx_norm_backward(dy, rstd, x=x, mean=mean, weight=w, kind="layer", want_dbias=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_side_stream_and_graph():
    """On a stream of its own and captured into a graph: each replay, with the
    program's own work between, gives the eager result on the inputs of then."""
    rows, cols = 130, 4096
    x, dy, w, _, _ = _backward_case(rows, cols, torch.bfloat16, "rms")
    res = dev(rand(9, rows, cols), torch.bfloat16)

    def step():
        f = mx.mx_norm_forward(x, w, eps=EPS, kind="rms", residual=res, ckpt_fmt="e4m3")
        return f, mx.mx_norm_backward(dy, f.rstd, ckpt=mx.checkpoint("e4m3", f.qx, f.sx), weight=w, kind="rms", dsum=dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f0, b0 = step()
    side.synchronize()
    f1, b1 = step()
    torch.cuda.synchronize()
    assert torch.equal(f0.y, f1.y) and torch.equal(b0.dx, b1.dx) and torch.equal(b0.dweight, b1.dweight)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fg, bg = step()
    for k in range(4):
        x.copy_(dev(_stream(100 + k, rows, cols), torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        fe, be = step()
        torch.cuda.synchronize()
        for a, b in ((fg.y, fe.y), (fg.sum, fe.sum), (fg.qx, fe.qx), (fg.sx, fe.sx), (bg.dx, be.dx),
                     (bg.dweight, be.dweight)):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """A matrix of more than 2^32 bytes of bf16: its last rows come out as
    they do alone."""
    rows, cols = 540_001, 4096                   # 2.2e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    w = dev(rand(3, cols), torch.bfloat16)
    f = mx.mx_norm_forward(x, w, eps=EPS, kind="rms", ckpt_fmt="e4m3")
    tail = mx.mx_norm_forward(x[-3:], w, eps=EPS, kind="rms", ckpt_fmt="e4m3")
    for a, b in ((f.y[-3:], tail.y), (f.qx[-3:], tail.qx), (f.sx[-3:], tail.sx), (f.rstd[-3:], tail.rstd)):
        assert torch.equal(a, b)
    ck = mx.checkpoint("e4m3", f.qx, f.sx)
    b = mx.mx_norm_backward(x, f.rstd, ckpt=ck, weight=w, kind="rms", want_dweight=False)
    ct = mx.checkpoint("e4m3", tail.qx, tail.sx)
    bt = mx.mx_norm_backward(x[-3:], tail.rstd, ckpt=ct, weight=w, kind="rms", want_dweight=False)
    assert torch.equal(b.dx[-3:], bt.dx)


def test_more_rows_than_one_launch_counts():
    """2^26 rows and some: 64 threads a row are more than 2^32, which no one
    launch counts.  Every row against the same rows in another place."""
    rows, cols = (1 << 26) + 37, 8
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    w = dev(rand(3, cols), torch.bfloat16)
    f = mx.mx_norm_forward(x, w, eps=EPS, kind="layer")
    for first in (0, (1 << 25) - 50, (1 << 26) - 60, rows - 100):
        part = slice(first, first + 100)
        alone = mx.mx_norm_forward(x[part], w, eps=EPS, kind="layer")
        assert torch.equal(f.y[part], alone.y) and torch.equal(f.rstd[part], alone.rstd)
        assert torch.equal(f.mean[part], alone.mean)
    b = mx.mx_norm_backward(x, f.rstd, x=x, mean=f.mean, weight=w, kind="layer", want_dweight=False)
    part = slice(rows - 100, rows)
    alone = mx.mx_norm_backward(x[part], f.rstd[part], x=x[part], mean=f.mean[part], weight=w, kind="layer",
                                want_dweight=False)
    assert torch.equal(b.dx[part], alone.dx)


def test_wide_rows_in_slices_of_a_launch():
    """More than 2^21 rows beyond 16384 columns need two launches of the wide
    kernels (bf16, 69 GB in, as much out)."""
    rows, cols = (1 << 21) + 3, 16392
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-5:] = dev(rand(1, 5, cols), torch.bfloat16)
    x[:5] = dev(rand(2, 5, cols), torch.bfloat16)
    f = mx.mx_norm_forward(x, eps=EPS, kind="rms")
    for part in (slice(0, 5), slice(rows - 5, rows)):
        alone = mx.mx_norm_forward(x[part], eps=EPS, kind="rms")
        assert torch.equal(f.y[part], alone.y) and torch.equal(f.rstd[part], alone.rstd)
    del f
