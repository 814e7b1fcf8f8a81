"""Calls that write an output over one of their inputs: rows whose
length is no multiple of eight end in a chunk that overlaps the one before, so
that another wave's thread may read what a thread has written already, unless
each element is taken by one thread."""
import pytest
import torch

import act_ref as R
from act_util import DT, Guarded, dev, rand
from fp4_quantization_block_amd import mx
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# rows that end in many places of a wave (64 chunks) and of a workgroup (256)
@pytest.mark.parametrize("rows,cols", [(1, 5), (3, 9), (700, 11), (513, 509), (300, 2051), (64, 4104), (40, 14337)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("over", ["gate", "up"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_glu_forward(act, over, dtype, rows, cols):
    dt = DT[dtype]
    g, u = dev(2 * rand(1, rows, cols), dt), dev(rand(2, rows, cols), dt)
    want = mx.mx_glu_forward(g, u, act).h
    into = g if over == "gate" else u
    got = mx.mx_glu_forward(g, u, act, h=into).h
    assert got is into and torch.equal(got, want)


@pytest.mark.parametrize("over", [0, 1])
def test_glu_forward_over_a_half(over):
    """Over one half of a fused projection: the other half stays."""
    rows, cols = 200, 2051
    g, u = dev(rand(1, rows, cols), torch.bfloat16), dev(rand(2, rows, cols), torch.bfloat16)
    both = Guarded(rows, 2 * cols, torch.bfloat16, 3, 1, torch.cat([g, u], 1))
    half = both.view[:, :cols], both.view[:, cols:]
    mx.mx_glu_forward(*half, "silu", h=half[over])
    assert torch.equal(half[over], mx.mx_glu_forward(g, u, "silu").h) and torch.equal(half[1 - over], (u, g)[over])
    both.check("gate, up")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("over", ["x", "x beside a sum", "residual", "sum"])
@pytest.mark.parametrize("cols", [5, 40, 99, 515, 4097, 16383, 16385, 16392, 20001, 40967])
def test_norm_forward(cols, over, dtype, kind):
    """Up to 16384 columns a row is in registers before y is written, and y is
    the same bit for bit; wider rows are read again, and each y is within the
    bounds of its definition (the order of the sums may be another)."""
    rows, dt = 9 if cols > 4096 else 300, DT[dtype]
    x, w, b = dev(rand(1, rows, cols) + 0.5, dt), dev(rand(3, cols), dt), dev(rand(4, cols), dt)
    res = None if over == "x" else dev(rand(2, rows, cols), dt)
    s = x.clone() if res is None else (x.float() + res.float()).to(dt)
    total = None if res is None else torch.empty_like(x)
    want = mx.mx_norm_forward(x, w, b, kind=kind, residual=res).y
    into = {"x": x, "x beside a sum": x, "residual": res, "sum": total}[over]
    r = mx.mx_norm_forward(x, w, b, kind=kind, residual=res, sum_out=total, y=into)
    assert r.y is into
    if cols <= 16384:
        assert torch.equal(r.y, want)
    y, err, *_ = R.norm(s.cpu().double(), w.cpu().double(), b.cpu().double(), 1e-5, kind == "layer")
    R.within(r.y, y, err, f"y over {over}")
    assert over in ("x", "sum") or torch.equal(total, s)
