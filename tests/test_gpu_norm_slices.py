"""Norms of more rows than one launch counts.  A launch takes at most 2^31
threads' worth of rows, and a row has a fixed number of threads for its length:
8 up to 64 columns, 1024 beyond 16384.  Every pointer of a call moves on with
its rows from one launch to the next, so rows of the first launch, at its end,
and of the second one are compared with the same rows in a call of their own."""
import gc

import pytest
import torch

from act_util import dev, rand
from fp4_quantization_block_amd import mx
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _parts(rows, threads):
    most = (1 << 31) // threads
    assert most + 20 < rows < 2 * most
    return slice(0, 40), slice(most - 40, most), slice(most, rows), slice(most - 20, most + 20)


def _matrix(seed, rows, cols, parts):
    """bf16, random in the parts that are looked at."""
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    for k, p in enumerate(parts):
        x[p] = dev(rand(seed + k, p.stop - p.start, cols), torch.bfloat16)
    return x


def _same(whole, alone, part, what):
    for name, a, b in zip(whole._fields, whole, alone):
        if a is None:
            assert b is None
        elif a.dim() and a.shape[0] != b.shape[0]:
            assert torch.equal(a[part], b), f"{what}: {name} of rows {part.start}.."


def test_short_rows():
    """8 columns: a layer norm of a residual sum, with its statistics, and its gradient."""
    rows, cols = (1 << 28) + 37, 8
    parts = _parts(rows, 8)
    x, res = _matrix(1, rows, cols, parts), _matrix(11, rows, cols, parts)
    w, b = dev(rand(3, cols), torch.bfloat16), dev(rand(4, cols), torch.bfloat16)
    f = mx.mx_norm_forward(x, w, b, kind="layer", residual=res)
    for p in parts:
        _same(f, mx.mx_norm_forward(x[p], w, b, kind="layer", residual=res[p]), p, "forward")
    g = mx.mx_norm_backward(x, f.rstd, x=f.sum, mean=f.mean, weight=w, kind="layer", dsum=res, want_dweight=False)
    for p in parts:
        _same(g, mx.mx_norm_backward(x[p], f.rstd[p], x=f.sum[p], mean=f.mean[p], weight=w, kind="layer", dsum=res[p],
                                     want_dweight=False), p, "gradient")


def test_short_rows_odd():
    """9 columns, whose last chunk overlaps the first."""
    rows, cols = (1 << 28) + 37, 9
    parts = _parts(rows, 8)
    x = _matrix(1, rows, cols, parts)
    f = mx.mx_norm_forward(x, kind="rms", out_dtype=torch.float32)
    for p in parts:
        _same(f, mx.mx_norm_forward(x[p], kind="rms", out_dtype=torch.float32), p, "forward")


def test_short_rows_with_copies():
    """32 columns: the row copy of y and the checkpoint."""
    rows, cols = (1 << 28) + 37, 32
    parts = _parts(rows, 8)
    x = _matrix(1, rows, cols, parts)
    f = mx.mx_norm_forward(x, kind="rms", write_y=False, y_fmt="e4m3", ckpt_fmt="e5m2")
    for p in parts:
        _same(f, mx.mx_norm_forward(x[p], kind="rms", write_y=False, y_fmt="e4m3", ckpt_fmt="e5m2"), p, "forward")


def test_wide_rows():
    """16416 columns (69 GB a matrix): the sum written over x, statistics and
    both copies; then the gradient of the sum, with itself as dy."""
    rows, cols = (1 << 21) + 27, 16416
    parts = _parts(rows, 1024)
    x = _matrix(1, rows, cols, parts)
    before = [x[p].clone() for p in parts]
    kw = dict(kind="layer", write_y=False, y_fmt="e4m3", ckpt_fmt="e5m2")
    f = mx.mx_norm_forward(x, residual=x, sum_out=x, **kw)
    for p, b in zip(parts, before):
        _same(f, mx.mx_norm_forward(b, residual=b, **kw), p, "forward")
    f = f._replace(qy=None, sy=None, qx=None, sx=None)
    torch.cuda.empty_cache()
    w = dev(rand(3, cols), torch.bfloat16)
    g = mx.mx_norm_backward(x, f.rstd, x=x, mean=f.mean, weight=w, kind="layer", want_dweight=False)
    for p in parts:
        _same(g, mx.mx_norm_backward(x[p], f.rstd[p], x=x[p], mean=f.mean[p], weight=w, kind="layer",
                                     want_dweight=False), p, "gradient")


def test_column_sums_of_very_wide_rows():
    """2^27 and some columns, at 32 threads each: 2^32 threads and more, which
    the column sums take in three launches.  With rstd = 1 the products of bf16 values are exact in fp32, and a
    sum of two of them is rounded once."""
    rows, cols = 2, (1 << 27) + 40
    x, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(
        generator=torch.Generator(device=DEV).manual_seed(k)) for k in (1, 2))
    one = torch.ones(rows, device=DEV)
    g = mx.mx_norm_backward(dy, one, x=x, kind="rms", want_dbias=True)
    p = dy.float() * x.float()
    assert torch.equal(g.dweight, p[0] + p[1]) and torch.equal(g.dbias, dy[0].float() + dy[1].float())
    alone = mx.mx_norm_backward(dy, one, x=x, kind="rms", want_dweight=False, want_dbias=True)
    assert torch.equal(alone.dbias, g.dbias) and torch.equal(alone.dx, g.dx)
