"""Calls with stream=, on a stream that is busy, while the caller's own stream
goes on allocating and writing: results as without it, and nobody's memory
written by the other."""
import pytest
import torch

from act_util import dev, rand
from fp4_quantization_block_amd import mx
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _beside(call, sizes):
    """call(stream) behind other work on a side stream; meanwhile memory of
    these sizes (bytes) is taken and filled on the current one."""
    side = torch.cuda.Stream()
    work = torch.ones(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):                        # some milliseconds
            work = work * 0.999 + 0.001
    out = call(side)
    own = [torch.full((n,), 90 + k, dtype=torch.uint8, device=DEV) for k, n in enumerate(sizes * 3)]
    torch.cuda.synchronize()
    for k, t in enumerate(own):
        assert bool((t == 90 + k).all()), "memory of the current stream was written by the call"
    return out


@pytest.mark.parametrize("rows,cols", [(3000, 4096), (130, 640), (40, 20000)])
def test_norm_backward(rows, cols):
    x, dy = dev(rand(1, rows, cols), torch.bfloat16), dev(rand(2, rows, cols), torch.bfloat16)
    w, r = dev(rand(3, cols), torch.bfloat16), dev(rand(4, rows).abs(), torch.float32)
    want = mx.mx_norm_backward(dy, r, x=x, weight=w, want_dbias=True)
    sizes = [int(mx.load().mx_norm_backward_workspace_bytes(rows, cols)), rows * cols * 2, cols * 4]
    for _ in range(3):
        got = _beside(lambda s: mx.mx_norm_backward(dy, r, x=x, weight=w, want_dbias=True, stream=s), sizes)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (96, 160)])
def test_predict_tensor_scale(rows, cols):
    w, g = dev(rand(1, rows, cols), torch.bfloat16), dev(rand(2, rows, cols), torch.bfloat16)
    want = mx.mx_predict_tensor_scale(w, g, 1e-3, "e4m3")
    for _ in range(3):
        got = _beside(lambda s: mx.mx_predict_tensor_scale(w, g, 1e-3, "e4m3", stream=s), [4096, 512])
        assert torch.equal(got, want)


def test_other_calls():
    """The calls that write new tensors: quantizers, the GEMM, and the activation operators."""
    rows, cols = 256, 1024
    x, u, r = (dev(rand(k, rows, cols), torch.bfloat16) for k in (1, 2, 3))
    xf, cfg = x.float().view(-1), mx.qconfig("e4m3", two_level=True)
    q, s, t = mx.mx_quantize(x, mx.MX_AXIS_ROW, cfg)
    c = dict(gate_ckpt=mx.checkpoint("e4m3", q, s), up_ckpt=mx.checkpoint("e4m3", q, s))
    torch.cuda.synchronize()
    calls = [
        lambda k: mx.mx_quantize(x, mx.MX_AXIS_COL, cfg, stream=k),
        lambda k: mx.mx_quantize_dual_layout(x, cfg, stream=k),
        lambda k: (mx.mx_gemm(q, s, t, "e4m3", q, s, t, "e4m3", rows, rows, cols, stream=k),),
        lambda k: mx.mx_gemm_quantized(q, s, t, "e4m3", q, s, t, "e4m3", rows, rows, cols, stream=k),
        lambda k: (mx.mx_dequantize(q, s, t, "e4m3", rows, cols, mx.MX_AXIS_ROW, stream=k),),
        lambda k: mx.mx_quantize_nvfp(x, stream=k),
        lambda k: mx.mx_quantize_optstate(xf, stream=k),
        lambda k: mx.mx_norm_forward(x, kind="layer", residual=r, y_fmt="e4m3", ckpt_fmt="e5m2", stream=k),
        lambda k: mx.mx_glu_forward(x, u, h_fmt="e4m3", ckpt_fmt="e4m3", stream=k),
        lambda k: mx.mx_glu_backward(r, x, u, recompute_h=True, stream=k),
        lambda k: mx.mx_glu_backward_dual_layout(r, h_fmt="e4m3", stream=k, **c),
    ]
    for n, call in enumerate(calls):
        want = call(None)
        got = _beside(call, [rows * cols * b for b in (1, 2, 4)])
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want)), f"call {n}"


def test_captured_on_a_joined_stream():
    """A graph whose gradient runs on a side stream that the capture has been
    joined to: every replay, with eager work between, gives the eager result."""
    rows, cols = 200, 2048
    x, dy = dev(rand(1, rows, cols), torch.bfloat16), dev(rand(2, rows, cols), torch.bfloat16)
    w, r = dev(rand(3, cols), torch.bfloat16), dev(rand(4, rows).abs(), torch.float32)
    side = torch.cuda.Stream()

    def step(stream):
        return mx.mx_norm_backward(dy, r, x=x, weight=w, want_dbias=True, stream=stream)

    step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        held = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        x.copy_(dev(rand(10 + k, rows, cols), torch.bfloat16))
        dy.copy_(dev(rand(20 + k, rows, cols), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = step(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
