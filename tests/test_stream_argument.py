"""Calls with stream=: what the binding allocates for them.

torch's allocator orders the reuse of memory by the stream that was current at
the allocation.  Memory that a call's kernels use on another stream must belong
to that one: the memory may be handed out again as soon as the call has dropped
it (a workspace), and may still be in use by earlier work of the stream it came
from.  Shown on the CPU: torch's streams and the library are stand-ins, which
record who allocated what and what the library was passed."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from fp4_quantization_block_amd import mx

ROWS, COLS = 64, 64
X = torch.zeros(ROWS, COLS)
V, R = torch.zeros(COLS), torch.zeros(ROWS)
CODES, SCALES = torch.zeros(ROWS, COLS, dtype=torch.uint8), torch.zeros(ROWS, COLS // 32, dtype=torch.uint8)


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _World(TorchDispatchMode):
    """The streams, who owns which memory, and what the library was passed."""

    def __init__(self):
        super().__init__()
        self.main, self.side = _Stream(11), _Stream(22)
        self.current = self.main
        self.owner, self.kept, self.passed, self.on, self.recorded = {}, [], set(), [], []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in func.name():
            self.kept.append(out)                  # so that no address comes twice
            self.owner[out.data_ptr()] = self.current.cuda_stream
        return out

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, next(k for k in (self.main, self.side) if k.cuda_stream == s.cuda_stream)
        try:
            yield
        finally:
            self.current = before

    def __getattr__(self, name):                   # the library
        if not name.startswith("mx_"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("_bytes"):
                return 4096
            values = [getattr(a, "value", a) for a in args]
            self.passed.update(v for v in values if isinstance(v, int))
            self.on.append(values[-1])
            return mx.MX_OK

        return call


@pytest.fixture
def world(monkeypatch):
    w = _World()
    monkeypatch.setattr(mx, "load", lambda: w)
    monkeypatch.setattr(torch.cuda, "stream", w.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: w.current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(mx, "_device", lambda: 0)
    monkeypatch.setattr(mx, "_raw_stream", lambda at: w.current.cuda_stream)
    monkeypatch.setattr(mx, "_stream_on", lambda s, at: w.current.cuda_stream if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.recorded.append((t.data_ptr(), s.cuda_stream)))
    return w


def _check(world, call, new):
    """`new`: how many of the call's results are new tensors."""
    with world:
        out = call(world.side)
    used = {p: s for p, s in world.owner.items() if p in world.passed}
    assert world.on == [22] and used, "the call ran elsewhere, or used no memory of its own"
    assert set(used.values()) == {22}, "memory of another stream than the one its kernels run on"
    # results may be used on the caller's stream too, and dropped there
    out = [out] if isinstance(out, torch.Tensor) else out
    results = {t.data_ptr() for t in out if t is not None and t.data_ptr() in world.owner}
    assert len(results) == new and set(world.recorded) == {(p, 11) for p in results}


def test_norm_backward(world):
    _check(world, lambda s: mx.mx_norm_backward(X, R, x=X, want_dbias=True, stream=s), 3)


def test_norm_backward_given_outputs(world):
    """The workspace alone is the call's own; the caller's tensors are not touched."""
    _check(world, lambda s: mx.mx_norm_backward(X, R, x=X, dx=X.clone(), dweight=V.clone(), stream=s), 0)


def test_the_current_stream_given(world):
    """Nothing is handed over where the given stream is the current one."""
    with world:
        mx.mx_norm_backward(X, R, x=X, stream=world.main)
    assert world.on == [11] and set(world.owner.values()) == {11} and not world.recorded


def test_predict_tensor_scale(world):
    _check(world, lambda s: mx.mx_predict_tensor_scale(X, X, 1e-3, "e4m3", stream=s), 1)
    world.on.clear()
    world.recorded.clear()
    _check(world, lambda s: mx.mx_predict_tensor_scale(X, X, 1e-3, "e4m3", None, V[:1], s), 0)


E4M3 = mx.qconfig("e4m3")
A = (CODES, SCALES, None, "e4m3")
CK = dict(gate_ckpt=mx.checkpoint("e4m3", CODES, SCALES), up_ckpt=mx.checkpoint("e4m3", CODES, SCALES))
CALLS = {
    "quantize": (lambda s: mx.mx_quantize(X, mx.MX_AXIS_ROW, E4M3, stream=s), 2),
    "quantize, two levels": (lambda s: mx.mx_quantize(X, mx.MX_AXIS_ROW, mx.qconfig("e4m3", two_level=True), stream=s), 3),
    "quantize, positional": (lambda s: mx.mx_quantize(X, 0, E4M3, CODES, None, None, s), 1),
    "dual layout": (lambda s: mx.mx_quantize_dual_layout(X, E4M3, stream=s), 4),
    "gemm": (lambda s: mx.mx_gemm(*A, *A, ROWS, ROWS, COLS, stream=s), 1),
    "gemm, quantized": (lambda s: mx.mx_gemm_quantized(*A, *A, ROWS, ROWS, COLS, stream=s), 2),
    "predict, no workspace": (lambda s: mx.mx_predict_tensor_scale_noalloc(X, X, 1e-3, "e4m3", stream=s), 1),
    "dequantize": (lambda s: mx.mx_dequantize(CODES, SCALES, None, "e4m3", ROWS, COLS, 0, stream=s), 1),
    "quantize optstate": (lambda s: mx.mx_quantize_optstate(X.view(-1), stream=s), 3),
    "dequantize optstate": (lambda s: mx.mx_dequantize_optstate(CODES.view(-1), V, V, stream=s), 1),
    "quantize nvfp": (lambda s: mx.mx_quantize_nvfp(X, stream=s), 3),
    "dequantize nvfp": (lambda s: mx.mx_dequantize_nvfp(CODES, SCALES, V, ROWS, COLS, stream=s), 1),
    "gemm nvfp": (lambda s: mx.mx_gemm_nvfp(CODES, SCALES, V, False, CODES, SCALES, V, False, ROWS, ROWS, COLS, stream=s), 1),
    "norm": (lambda s: mx.mx_norm_forward(X, kind="layer", residual=X, y_fmt="e4m3", ckpt_fmt="e4m3", stream=s), 8),
    "glu": (lambda s: mx.mx_glu_forward(X, X, h_fmt="e4m3", ckpt_fmt="e4m3", stream=s), 7),
    "glu gradient": (lambda s: mx.mx_glu_backward(X, X, X, recompute_h=True, stream=s), 3),
    "glu gradient, dual layout": (lambda s: mx.mx_glu_backward_dual_layout(X, h_fmt="e4m3", stream=s, **CK), 6),
}


@pytest.mark.parametrize("name", CALLS)
def test_results(name, world):
    _check(world, *CALLS[name])
