"""The activation operators' reference against what it does not use: finite
differences of the forward definitions, torch's own layer norm, RMS norm and
activations in 64 bits, and an fp32 evaluation staying inside the bounds."""
import pytest
import torch
import torch.nn.functional as F

import act_ref as R


def _rand(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale


@pytest.mark.parametrize("layer", [True, False])
def test_norm_matches_torch(layer):
    s, w, b = _rand(5, 37, seed=1) + 3, _rand(37, seed=2), _rand(37, seed=3)
    y = R.norm(s, w, b, 1e-5, layer)[0]
    want = F.layer_norm(s, (37,), w, b, 1e-5) if layer else F.rms_norm(s, (37,), w, 1e-5) + b
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("layer", [True, False])
def test_norm_grad_is_the_difference_quotient(layer):
    """Central differences of sum(dy * norm(s)): error O(h^2) = 1e-10 times
    third derivatives of order one, plus 1e-16 / h = 1e-11 of rounding."""
    s, w, b, dy = _rand(3, 11, seed=1) + 1, _rand(11, seed=2), _rand(11, seed=3), _rand(3, 11, seed=4)
    mu, r = R.stats(s, 1e-3, layer)
    dx, _, dw, _, db, _ = R.norm_grad(dy, s, mu, r, w, torch.zeros_like(s), layer, 1)
    h = 1e-5

    def f(s, w, b):
        return float((dy * R.norm(s, w, b, 1e-3, layer)[0]).sum())

    for got, args, k in ((dx, [s, w, b], 0), (dw, [s, w, b], 1), (db, [s, w, b], 2)):
        for i in range(got.numel()):
            up, dn = args[k].clone(), args[k].clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            a, c = list(args), list(args)
            a[k], c[k] = up, dn
            assert abs((f(*a) - f(*c)) / (2 * h) - float(got.view(-1)[i])) < 1e-7


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gate_matches_torch_and_differences(act):
    x = torch.linspace(-12, 12, 997, dtype=torch.float64)
    a, d, _, _ = R.gate(x, act)
    want = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[act](x)
    assert torch.allclose(a, want, rtol=1e-12, atol=1e-13)
    h = 1e-5
    assert torch.allclose(d, (R.gate(x + h, act)[0] - R.gate(x - h, act)[0]) / (2 * h), rtol=0, atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gate_bounds_hold_for_fp32(act):
    """torch's fp32 gates (another evaluation of the same formulas) are inside
    the bounds, and a value off by 1e-4 is not."""
    x = torch.linspace(-80, 80, 4001, dtype=torch.float32)
    a, _, err, _ = R.gate(x.double(), act)
    fp32 = {"silu": F.silu, "gelu": lambda t: t * (0.5 * torch.erfc(t * -0.70710678)),
            "gelu_tanh": lambda t: t * torch.sigmoid(1.5957691216 * (t + 0.044715 * t ** 3))}[act](x)
    keep = a.abs() > 1e-30                       # torch's tails below are not of interest
    R.within(torch.where(keep, fp32.double(), a).float(), a, err, act)
    with pytest.raises(AssertionError):
        R.within((a * (1 + 1e-4)).float(), a, err, act)


def test_norm_bounds_hold_for_fp32_and_catch_errors():
    s = (_rand(4, 515, seed=1) + 30).float()
    w, b = _rand(515, seed=2).float(), _rand(515, seed=3).float()
    y, err, mu, mu_err, r, r_err = R.norm(s.double(), w.double(), b.double(), 1e-5, True)
    R.within(F.layer_norm(s, (515,), w, b, 1e-5), y, err, "layer norm")
    R.within(s.mean(1), mu, mu_err, "mean")
    with pytest.raises(AssertionError):          # a mean over one column too many
        R.within((s.double().sum(1) / 516).float(), mu, mu_err, "mean")
    with pytest.raises(AssertionError):          # the unbiased variance
        R.within((1 / torch.sqrt(s.double().var(1) + 1e-5)).float(), r, r_err, "rstd")
