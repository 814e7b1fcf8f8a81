"""One training step of a pre-norm gated MLP block on the library's operators,
with its activations kept in 8 bits.

    python examples/mlp_block.py [--tokens 8192 --hidden 4096 --ffn 14336]

    s   = x + residual                  mx_norm_forward: s, its RMS norm, and
    xn  = rmsnorm(s) * w                    the E4M3 checkpoint of s
    gu  = xn . W_gu                     mx_quantize_dual_layout, mx_gemm
    h   = silu(gate) * up               mx_glu_forward: h as the next GEMM's
                                            operand, checkpoints of gate and up
    out = s + h . W_d                   mx_gemm

The backward needs s, gate and up again (from their checkpoints), xn (its
column copy, which is the wgrad GEMM's operand) and h, which it recomputes:
2 bytes an element in bf16 become 1.03, and h is not kept at all.  mx_glu_backward_dual_layout
writes the gradients of gate and up, and h, as the operands of the backward
GEMMs; mx_norm_backward adds the gradient that goes round the block.

Data and weights are random.  The step's gradients are compared with torch's
autograd in fp32 for up to 1024 tokens, and the step is timed.
"""
import argparse
import os
import sys
import time
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp4_quantization_block_amd import mx  # noqa: E402

EPS = 1e-5
ACT_FMT, GRAD_FMT = "e4m3", "e5m2"
ACT, GRAD = mx.qconfig(ACT_FMT), mx.qconfig(GRAD_FMT)


class Weights(NamedTuple):
    """Weights and their quantized copies (row copy for dgrad, column copy for fprop)."""
    norm: torch.Tensor                # [hidden]
    w_gu: torch.Tensor                # [hidden][2 ffn], gate then up
    w_d: torch.Tensor                 # [ffn][hidden]
    gu_row: tuple
    gu_col: tuple
    d_row: tuple
    d_col: tuple


class Saved(NamedTuple):
    """What the backward needs."""
    s: mx.Checkpoint
    rstd: torch.Tensor
    xn_col: tuple
    gate: mx.Checkpoint
    up: mx.Checkpoint

    def nbytes(self) -> int:
        tensors = [self.s.q, self.s.s, self.rstd, *self.xn_col, self.gate.q, self.gate.s, self.up.q, self.up.s]
        return sum(t.numel() * t.element_size() for t in tensors)


def make_weights(hidden: int, ffn: int, device, seed: int = 0) -> Weights:
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    norm = (1 + 0.1 * normal(hidden)).bfloat16()
    w_gu = (normal(hidden, 2 * ffn) * hidden ** -0.5).bfloat16()
    w_d = (normal(ffn, hidden) * ffn ** -0.5).bfloat16()
    gq, gs, gqc, gsc, _ = mx.mx_quantize_dual_layout(w_gu, ACT)
    dq, ds, dqc, dsc, _ = mx.mx_quantize_dual_layout(w_d, ACT)
    return Weights(norm, w_gu, w_d, (gq, gs), (gqc, gsc), (dq, ds), (dqc, dsc))


def _gemm(a, fa, b, fb, out=mx.MX_OUT_BF16):
    (qa, sa), (qb, sb) = a, b
    return mx.mx_gemm(qa, sa, None, fa, qb, sb, None, fb, qa.shape[0], qb.shape[0], qa.shape[1], out_dtype=out)


def forward(x: torch.Tensor, residual: torch.Tensor, w: Weights):
    """(out, Saved) for x, residual [tokens][hidden] in bf16."""
    ffn = w.w_d.shape[0]
    n = mx.mx_norm_forward(x, w.norm, eps=EPS, kind="rms", residual=residual, ckpt_fmt=ACT_FMT)
    xq, xs, xqc, xsc, _ = mx.mx_quantize_dual_layout(n.y, ACT)
    gu = _gemm((xq, xs), ACT_FMT, w.gu_col, ACT_FMT)
    g = mx.mx_glu_forward(gu[:, :ffn], gu[:, ffn:], "silu", write_h=False, h_fmt=ACT_FMT, ckpt_fmt=ACT_FMT)
    out = n.sum + _gemm((g.qh, g.sh), ACT_FMT, w.d_col, ACT_FMT)
    return out, Saved(mx.checkpoint(ACT_FMT, n.qx, n.sx), n.rstd, (xqc, xsc),
                      mx.checkpoint(ACT_FMT, g.qg, g.sg), mx.checkpoint(ACT_FMT, g.qu, g.su))


def backward(dout: torch.Tensor, saved: Saved, w: Weights):
    """Gradients of x (and residual), the norm's weight (fp32), W_gu and W_d (bf16)."""
    yq, ys, yqc, ysc, _ = mx.mx_quantize_dual_layout(dout, GRAD)
    dh = _gemm((yq, ys), GRAD_FMT, w.d_row, ACT_FMT)
    d = mx.mx_glu_backward_dual_layout(dh, act="silu", gate_ckpt=saved.gate, up_ckpt=saved.up, fmt=GRAD_FMT,
                                       h_fmt=ACT_FMT)
    dw_d = _gemm((d.qh_col, d.sh_col), ACT_FMT, (yqc, ysc), GRAD_FMT)
    dxn = _gemm((d.q_row, d.s_row), GRAD_FMT, w.gu_row, ACT_FMT)
    dw_gu = _gemm(saved.xn_col, ACT_FMT, (d.q_col, d.s_col), GRAD_FMT)
    n = mx.mx_norm_backward(dxn, saved.rstd, ckpt=saved.s, weight=w.norm, kind="rms", dsum=dout)
    return n.dx, n.dweight, dw_gu, dw_d


def reference(x, residual, dout, w: Weights):
    """out and the same gradients by torch's autograd in fp32."""
    s = (x + residual).float().requires_grad_()
    norm, w_gu, w_d = (t.float().detach().requires_grad_() for t in (w.norm, w.w_gu, w.w_d))
    xn = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * norm
    gate, up = (xn @ w_gu).chunk(2, 1)
    out = s + (torch.nn.functional.silu(gate) * up) @ w_d
    out.backward(dout.float())
    return out.detach(), s.grad, norm.grad, w_gu.grad, w_d.grad


def inputs(tokens: int, hidden: int, device, seed: int = 1):
    g = torch.Generator(device=device).manual_seed(seed)
    x, r, d = (torch.randn(tokens, hidden, generator=g, device=device) for _ in range(3))
    return x.bfloat16(), r.bfloat16(), (d * 1e-3).bfloat16()


def errors(tokens: int, hidden: int, ffn: int, device="cuda"):
    """{name: relative error} of out and the gradients against fp32."""
    w = make_weights(hidden, ffn, device)
    x, r, dout = inputs(tokens, hidden, device)
    out, saved = forward(x, r, w)
    got = (out, *backward(dout, saved, w))
    names = ("out", "dx", "dnorm", "dW_gu", "dW_d")
    return {n: float((a.float() - b).norm() / b.norm()) for n, a, b in zip(names, got, reference(x, r, dout, w))}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=14336)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    for name, e in errors(min(a.tokens, 1024), a.hidden, a.ffn).items():
        print(f"{name}: relative error against fp32 {e:.3f}", flush=True)
    w = make_weights(a.hidden, a.ffn, "cuda")
    x, r, dout = inputs(a.tokens, a.hidden, "cuda")
    kept = forward(x, r, w)[1].nbytes()
    bf16 = 2 * a.tokens * (2 * a.hidden + 3 * a.ffn)
    print(f"kept for the backward: {kept / 2**20:.0f} MiB (in bf16: s, xn, gate, up, h {bf16 / 2**20:.0f} MiB)", flush=True)
    for _ in range(3):
        backward(dout, forward(x, r, w)[1], w)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        backward(dout, forward(x, r, w)[1], w)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / a.steps * 1e3
    flops = 18 * a.tokens * a.hidden * a.ffn
    print(f"forward and backward: {ms:.3f} ms, {flops / ms / 1e9:.0f} TFLOP/s over everything", flush=True)


if __name__ == "__main__":
    main()
