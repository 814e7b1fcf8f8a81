"""The activation operators with the quantizers and GEMMs around them: a
training step of a gated MLP block (examples/mlp_block.py) against autograd in
fp32.

Every operand that is quantized is off by at most half a step of its format
relative to the value: E4M3 2^-4, E5M2 2^-3 (subnormal codes of small elements
less in the norm).  An output's relative error is taken to be at most the sum
of the half steps on its way; a wrong layout, scale or operand gives about 1."""
import os
import sys

import pytest
import torch

from gpu_util import require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
E4, E5 = 2.0 ** -4, 2.0 ** -3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("tokens,hidden,ffn", [(128, 256, 384), (160, 512, 1056), (256, 1024, 2048)])
def test_step_against_fp32(tokens, hidden, ffn):
    import mlp_block as B

    err = B.errors(tokens, hidden, ffn)
    way = {
        "out": 4 * E4,                           # xn, W_gu; h, W_d
        "dW_d": E5 + E4 + 2 * E4 + 2 * E4,       # dout; h: its code, gate and up's codes, and xn, W_gu before them
        "dx": E5 + E4 + E5 + E4 + 5 * E4,        # dout, W_d; D, W_gu; gate, up; xn, W_gu before; s in the norm
        "dW_gu": E5 + E4 + E5 + E4 + 4 * E4,     # dout, W_d; D, xn; gate, up; xn, W_gu before
        "dnorm": E5 + E4 + E5 + E4 + 5 * E4,
    }
    for name, most in way.items():
        assert err[name] <= most, f"{name}: relative error {err[name]:.3f}, at most {most:.3f}"


def test_step_repeats_bit_for_bit():
    import mlp_block as B

    w = B.make_weights(256, 384, "cuda")
    x, r, dout = B.inputs(160, 256, "cuda")
    runs = []
    for _ in range(2):
        out, saved = B.forward(x, r, w)
        runs.append((out, *B.backward(dout, saved, w)))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_checkpoints_take_about_half():
    """1 + 1/32 bytes for s, xn, gate and up, and none for h."""
    import mlp_block as B

    w = B.make_weights(256, 384, "cuda")
    x, r, _ = B.inputs(128, 256, "cuda")
    _, saved = B.forward(x, r, w)
    assert saved.nbytes() == 128 * (2 * 256 + 2 * 384) * 33 // 32 + 128 * 4
