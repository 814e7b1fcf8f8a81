"""Marshalling shared by the GPU tests of the activation operators."""
import numpy as np
import torch

import oracle as O
from fp4_quantization_block_amd import mx
from gpu_util import DEV, assert_codes_equal, u8

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale


def dev(x, dtype):
    return x.to(dtype).to(DEV)


class Guarded:
    """A matrix inside a larger buffer of a known pattern: `view` starts
    `offset` elements in and has a row stride of cols + pad; check() says
    whether anything outside it was written."""

    def __init__(self, rows, cols, dtype, offset=0, pad=0, fill=None):
        self.ld, self.rows, self.cols, self.offset = cols + pad, rows, cols, offset
        self.buf = torch.full((offset + rows * self.ld + 64,), 7.0, dtype=dtype, device=DEV)
        self.view = self.buf[offset:offset + rows * self.ld].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.view.copy_(fill)

    def check(self, what):
        outside = torch.ones_like(self.buf, dtype=torch.bool)
        outside[self.offset:self.offset + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = False
        assert bool((self.buf[outside] == 7.0).all()), f"{what}: written outside the matrix"


def np_source(t):
    """Device tensor as the oracle's source array (fp32, or bf16 bits)."""
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def assert_row_copy(q, s, source, fmt, what):
    """q, s are the row copy mx_quantize defines for `source`."""
    qo, so, _ = O.quantize(np_source(source), O.AXIS_ROW, fmt)
    assert_codes_equal(u8(s), so, f"{what} scales")
    assert_codes_equal(u8(q), qo, f"{what} codes")


def assert_col_copy(q, s, source, fmt, what):
    qo, so, _ = O.quantize(np_source(source), O.AXIS_COL, fmt)
    assert_codes_equal(u8(s), so, f"{what} scales")
    assert_codes_equal(u8(q), qo, f"{what} codes")


def restored(q, s, fmt):
    """What a checkpoint's codes and scales stand for (float64, on the host)."""
    rows, cols = q.shape
    return torch.from_numpy(np.asarray(O.dequantize(u8(q), u8(s), None, fmt, rows, cols, O.AXIS_ROW), np.float64))


def make_checkpoint(x, fmt):
    q, s, _ = mx.mx_quantize(x, mx.MX_AXIS_ROW, mx.qconfig(fmt))
    return mx.checkpoint(fmt, q, s)
