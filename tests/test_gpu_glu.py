"""mx_glu_forward, mx_glu_backward and mx_glu_backward_dual_layout against
their definitions in 64 bits, with bounds that count fp32 roundings
(act_ref.py); quantized outputs and checkpoints against the oracle's
quantizer, bit for bit."""
import pytest
import torch

import act_ref as R
from act_util import DT, Guarded, assert_col_copy, assert_row_copy, dev, make_checkpoint, rand, restored
from fp4_quantization_block_amd import mx
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu", "gelu_tanh"]
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 33), (5, 256), (1, 2047), (37, 2048), (64, 2731), (7, 14336), (300, 41)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _inputs(rows, cols, dt, seed=1):
    g = dev(2.5 * rand(seed, rows, cols), dt)
    return g, dev(rand(seed + 1, rows, cols), dt), dev(rand(seed + 2, rows, cols, scale=1e-2), dt)


def _check(out_h, out_dg, out_du, dh, g, u, act, what):
    """g, u: the values the gradients are taken at (float64, host)."""
    a, d, a_err, d_err = R.gate(g, act)
    if out_h is not None:
        R.within(out_h, a * u, a_err * u.abs() + 2 * R.U * (a * u).abs(), f"{what} h")
    if out_dg is not None:
        dh = dh.cpu().double()
        R.within(out_dg, dh * u * d, d_err * (dh * u).abs() + 3 * R.U * (dh * u * d).abs(), f"{what} dgate")
        R.within(out_du, dh * a, a_err * dh.abs() + 2 * R.U * (dh * a).abs(), f"{what} dup")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, dtype, act):
    dt = DT[dtype]
    g, u, dh = _inputs(rows, cols, dt)
    f = mx.mx_glu_forward(g, u, act)
    b = mx.mx_glu_backward(dh, g, u, act, recompute_h=True)
    _check(f.h, b.dgate, b.dup, dh, g.cpu().double(), u.cpu().double(), act, f"{rows}x{cols} {dtype} {act}")
    assert torch.equal(b.h, f.h)
    other = mx.mx_glu_forward(g, u, act, out_dtype=torch.float32 if dtype == "bf16" else torch.bfloat16)
    _check(other.h, None, None, None, g.cpu().double(), u.cpu().double(), act, "other output type")


@pytest.mark.parametrize("act", ACTS)
def test_every_bf16_gate(act):
    """Every bf16 value as the gate, with up = dh = 1: the gate function and
    its slope over their whole range; Inf and NaN as the formulas give them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(256, 256)
    g, one = bits.to(DEV), torch.ones(256, 256, device=DEV)
    gate32 = g.float()
    f = mx.mx_glu_forward(gate32, one, act)
    b = mx.mx_glu_backward(one, gate32, one, act)
    x = bits.double()
    fine = torch.isfinite(x) & (x.abs() < 1e12)          # x^3 of the reference stays finite
    a, d, a_err, d_err = R.gate(x[fine], act)
    R.within(f.h.cpu()[fine], a, a_err + 2 * R.U * a.abs(), "all bf16 h")
    R.within(b.dgate.cpu()[fine], d, d_err + 3 * R.U * d.abs(), "all bf16 dgate")
    big = torch.isfinite(x) & (x.abs() >= 1e12)
    assert torch.equal(f.h.cpu()[big], torch.where(x > 0, x, -0.0).float()[big])
    assert torch.equal(b.dgate.cpu()[big].abs(), torch.where(x > 0, 1.0, 0.0).float()[big])
    nan = torch.isnan(x)
    assert bool(torch.isnan(f.h.cpu()[nan]).all()) and bool(torch.isnan(b.dgate.cpu()[nan]).all())
    assert bool((f.h.cpu()[x == float("inf")] == float("inf")).all())
    assert not bool(torch.isinf(f.h.cpu()[x == float("-inf")]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,other", [("e4m3", "e5m2"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (65, 2048), (2, 14336), (33, 1056)])
def test_forward_copies(rows, cols, fmt, other, dtype):
    dt = DT[dtype]
    g, u, _ = _inputs(rows, cols, dt)
    f = mx.mx_glu_forward(g, u, "silu", out_dtype=torch.float32, h_fmt=fmt, ckpt_fmt=other)
    assert_row_copy(f.qh, f.sh, f.h, fmt, "h copy")
    assert_row_copy(f.qg, f.sg, g, other, "gate checkpoint")
    assert_row_copy(f.qu, f.su, u, other, "up checkpoint")
    alone = mx.mx_glu_forward(g, u, "silu", write_h=False, h_fmt=fmt)
    assert alone.h is None and torch.equal(alone.qh, f.qh) and torch.equal(alone.sh, f.sh)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_from_checkpoints(dtype, fmt, act):
    rows, cols, dt = 37, 1056, DT[dtype]
    g, u, dh = _inputs(rows, cols, dt)
    cg, cu = make_checkpoint(g, fmt), make_checkpoint(u, fmt)
    b = mx.mx_glu_backward(dh, act=act, gate_ckpt=cg, up_ckpt=cu, recompute_h=True)
    _check(b.h, b.dgate, b.dup, dh, restored(cg.q, cg.s, fmt), restored(cu.q, cu.s, fmt), act, f"{fmt} {act}")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_code_and_scale(fmt):
    """Every code of the up checkpoint under every scale byte, Inf and NaN
    among them, as the oracle decodes them (gate = 20, so that act is linear)."""
    rows, cols = 256, 256
    q = torch.arange(256, dtype=torch.uint8).repeat(rows, 1).to(DEV)
    s = torch.arange(rows, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, cols // 32).to(DEV)
    gate = make_checkpoint(torch.full((rows, cols), 16.0, device=DEV), fmt)
    one = torch.ones(rows, cols, device=DEV)
    h = mx.mx_glu_backward(one, act="silu", gate_ckpt=gate, up_ckpt=mx.checkpoint(fmt, q, s), recompute_h=True).h
    up = restored(q, s, fmt)
    a, _, _, _ = R.gate(torch.full((1,), 16.0, dtype=torch.float64), "silu")
    want = up * a
    got = h.cpu().double()
    # beyond fp32 the product is an infinity
    over = want.abs() > torch.finfo(torch.float32).max * (1 - 1e-6)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    rest = ~over & ~torch.isnan(want)
    # an fp32 subnormal result is off by at most one of its steps
    assert bool(((got - want).abs() <= 50 * R.U * want.abs() + 2.0 ** -148)[rest].all())
    assert bool((got.abs() > 3e38)[over].all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 41, 2048, 2049])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (3, 0)])
def test_strides_and_alignment(offset, pad, cols, dtype):
    """Halves of fused buffers and matrices at odd elements; the gradients may
    be written over the inputs."""
    rows, dt = 11, DT[dtype]
    g, u, dh = _inputs(rows, cols, dt)
    both = Guarded(rows, 2 * cols, dt, offset, pad, torch.cat([g, u], 1))
    gdh = Guarded(rows, cols, dt, offset + 1, pad + 1, dh)
    gh = Guarded(rows, cols, dt, offset + 2, pad)
    gate, up = both.view[:, :cols], both.view[:, cols:]
    f = mx.mx_glu_forward(gate, up, "gelu_tanh", h=gh.view)
    want = mx.mx_glu_forward(g, u, "gelu_tanh")
    assert torch.equal(f.h, want.h)
    for x, what in ((both, "gate, up"), (gh, "h")):
        x.check(what)
    wb = mx.mx_glu_backward(dh, g, u, "gelu_tanh", recompute_h=True)
    b = mx.mx_glu_backward(gdh.view, gate, up, "gelu_tanh", recompute_h=True, dgate=gate, dup=up, h=gh.view)
    assert torch.equal(gate, wb.dgate) and torch.equal(up, wb.dup) and torch.equal(b.h, wb.h)
    for x, what in ((both, "gate, up"), (gdh, "dh"), (gh, "h")):
        x.check(what)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_are_difference_quotients(act):
    """sum(dh * h) along random directions in 64 bits against the fp32 gradients."""
    rows, cols = 5, 101
    g, u, dh = _inputs(rows, cols, torch.float32)
    b = mx.mx_glu_backward(dh, g, u, act)
    G, Up, D = (t.cpu().double() for t in (g, u, dh))
    for k in range(5):
        dG, dU, h = rand(40 + k, rows, cols), rand(50 + k, rows, cols), 1e-6
        f = [float((D * R.gate(G + s * h * dG, act)[0] * (Up + s * h * dU)).sum()) for s in (1, -1)]
        terms = [b.dgate.cpu().double() * dG, b.dup.cpu().double() * dU]
        size = sum(float(t.abs().sum()) for t in terms)
        assert abs(sum(float(t.sum()) for t in terms) - (f[0] - f[1]) / (2 * h)) <= (300 * R.U + 1e-7) * size


# ---------------------------------------------------------------------------
# dual layout
# ---------------------------------------------------------------------------
def _check_dual(d, b, fmt, h_fmt, what):
    """d's copies are the oracle's copies of the fp32 gradients b."""
    both = torch.cat([b.dgate, b.dup], 1)
    assert_row_copy(d.q_row, d.s_row, both, fmt, f"{what} row copy")
    assert_col_copy(d.q_col, d.s_col, both, fmt, f"{what} column copy")
    if h_fmt is None:
        assert d.qh_col is None and d.sh_col is None
    else:
        assert_col_copy(d.qh_col, d.sh_col, b.h, h_fmt, f"{what} column copy of h")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt,h_fmt", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", None)])
@pytest.mark.parametrize("rows,cols", [(32, 32), (64, 96), (128, 64), (160, 160), (288, 1056), (96, 4096), (1056, 128), (2080, 2144), (4128, 1056)])
def test_dual_layout(rows, cols, fmt, h_fmt, act):
    """The codes encode the fp32 gradients that mx_glu_backward gives for
    fp32 inputs, in both layouts."""
    g, u, dh = _inputs(rows, cols, torch.float32)
    dh *= torch.exp(dev(rand(9, rows, 1), torch.float32))
    b = mx.mx_glu_backward(dh, g, u, act, recompute_h=True)
    d = mx.mx_glu_backward_dual_layout(dh, g, u, act, fmt=fmt, h_fmt=h_fmt)
    _check_dual(d, b, fmt, h_fmt, f"{rows}x{cols} {act}")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(32, 32), (160, 2080), (256, 512), (2144, 2080), (96, 40960), (128, 40960), (160, 40992)])
def test_dual_layout_from_checkpoints(rows, cols, fmt):
    """From checkpoints, with bf16 dh: the fp32 gradients come from the same
    values through fp32 inputs."""
    g, u, dh = _inputs(rows, cols, torch.bfloat16)
    cg, cu = make_checkpoint(g, fmt), make_checkpoint(u, fmt)
    b = mx.mx_glu_backward(dh.float(), act="silu", gate_ckpt=cg, up_ckpt=cu, recompute_h=True)
    d = mx.mx_glu_backward_dual_layout(dh, act="silu", gate_ckpt=cg, up_ckpt=cu, fmt="e5m2", h_fmt="e4m3")
    _check_dual(d, b, "e5m2", "e4m3", f"{rows}x{cols} {fmt}")
    d16 = mx.mx_glu_backward_dual_layout(dh, g, u, "silu", fmt="e5m2", h_fmt="e4m3")
    b16 = mx.mx_glu_backward(dh.float(), g.float(), u.float(), "silu", recompute_h=True)
    _check_dual(d16, b16, "e5m2", "e4m3", f"{rows}x{cols} bf16")


@pytest.mark.parametrize("rows,cols", [(96, 96), (4096, 1024), (4096, 1088)])
def test_dual_layout_special_blocks(rows, cols):
    """Zero, subnormal, huge, Inf and NaN places: blocks in both directions as
    the quantizer encodes them, in both kernels' tiles."""
    g, u, dh = _inputs(rows, cols, torch.float32)
    dh[:32] = 0.0
    dh[40, 5] = float("inf")
    dh[70, 33] = float("nan")
    u[64:, 64:] = 0.0
    dh[33] *= 1e-38
    dh[34] *= 1e36
    b = mx.mx_glu_backward(dh, g, u, "silu", recompute_h=True)
    d = mx.mx_glu_backward_dual_layout(dh, g, u, "silu", fmt="e5m2", h_fmt="e4m3")
    _check_dual(d, b, "e5m2", "e4m3", "special")


def test_dual_layout_strides_and_guards():
    rows, cols = 64, 96
    g, u, dh = _inputs(rows, cols, torch.bfloat16)
    both = Guarded(rows, 2 * cols, torch.bfloat16, 1, 3, torch.cat([g, u], 1))
    gdh = Guarded(rows, cols, torch.bfloat16, 3, 5, dh)
    want = mx.mx_glu_backward_dual_layout(dh, g, u, "silu", fmt="e5m2", h_fmt="e4m3")
    sizes = [t.numel() for t in want]
    bufs = [torch.full((n + 64,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
    outs = [b[:n].view(t.shape) for b, n, t in zip(bufs, sizes, want)]
    got = mx.mx_glu_backward_dual_layout(gdh.view, both.view[:, :cols], both.view[:, cols:], "silu", fmt="e5m2",
                                         h_fmt="e4m3", q_row=outs[0], s_row=outs[1], q_col=outs[2], s_col=outs[3],
                                         qh_col=outs[4], sh_col=outs[5])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((b[n:] == 7).all()) for b, n in zip(bufs, sizes))


def test_side_stream_and_graph():
    rows, cols = 160, 1056
    g, u, dh = _inputs(rows, cols, torch.bfloat16)

    def step():
        f = mx.mx_glu_forward(g, u, "silu", h_fmt="e4m3", ckpt_fmt="e4m3")
        c = dict(gate_ckpt=mx.checkpoint("e4m3", f.qg, f.sg), up_ckpt=mx.checkpoint("e4m3", f.qu, f.su))
        return (*f, *mx.mx_glu_backward(dh, act="silu", recompute_h=True, **c),
                *mx.mx_glu_backward_dual_layout(dh, act="silu", h_fmt="e4m3", **c))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        g.copy_(dev(rand(70 + k, rows, cols), torch.bfloat16))
        dh.copy_(dev(rand(80 + k, rows, cols), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("rows,cols", [(153_000, 14336), (150_001, 14337)])
def test_offsets_beyond_32_bits(rows, cols):
    """More than 2^31 elements and 2^32 bytes: the last rows come out as they
    do alone, in kernels that count places in 32 bits."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    g = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    u = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    fmt = "e4m3" if cols % 32 == 0 else None
    f = mx.mx_glu_forward(g, u, "silu", ckpt_fmt=fmt, h_fmt=fmt)
    ft = mx.mx_glu_forward(g[-3:], u[-3:], "silu", ckpt_fmt=fmt, h_fmt=fmt)
    for a, b in zip(f, ft):
        assert a is None and b is None or torch.equal(a[-3:], b)
    kw = dict(gate=g, up=u)
    kt = dict(gate=g[-3:], up=u[-3:])
    if fmt:
        kw = dict(gate_ckpt=mx.checkpoint(fmt, f.qg, f.sg), up_ckpt=mx.checkpoint(fmt, f.qu, f.su))
        kt = dict(gate_ckpt=mx.checkpoint(fmt, ft.qg, ft.sg), up_ckpt=mx.checkpoint(fmt, ft.qu, ft.su))
    b = mx.mx_glu_backward(f.h, act="silu", recompute_h=True, **kw)
    bt = mx.mx_glu_backward(f.h[-3:], act="silu", recompute_h=True, **kt)
    for x, y in zip(b, bt):
        assert torch.equal(x[-3:], y)


def test_dual_layout_offsets_beyond_32_bits():
    """Copies of more than 2^32 bytes: the last 32 rows and the last columns
    come out as they do alone."""
    rows, cols = 160_000, 14336
    gen = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.full((rows, cols // 32), 120, dtype=torch.uint8, device=DEV)
    dh = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    d = mx.mx_glu_backward_dual_layout(dh, act="silu", gate_ckpt=mx.checkpoint("e4m3", q, s),
                                       up_ckpt=mx.checkpoint("e4m3", q, s), h_fmt="e4m3")
    ct = mx.checkpoint("e4m3", q[-32:].contiguous(), s[-32:].contiguous())
    t = mx.mx_glu_backward_dual_layout(dh[-32:], act="silu", gate_ckpt=ct, up_ckpt=ct, h_fmt="e4m3")
    assert torch.equal(d.q_row[-32:], t.q_row) and torch.equal(d.s_row[-32:], t.s_row)
    assert torch.equal(d.q_col[:, -32:], t.q_col) and torch.equal(d.s_col[:, -1:], t.s_col)
    assert torch.equal(d.qh_col[:, -32:], t.qh_col) and torch.equal(d.sh_col[:, -1:], t.sh_col)
