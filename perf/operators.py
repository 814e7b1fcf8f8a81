"""Cases for measuring the activation operators around the MX GEMMs of a
pre-norm gated MLP block: the normalisation forward and backward (with the
reduction of its parameters' gradients), and the gated activation forward and
backward, each with activation checkpoints in 8 bits (FP8 codes in 1x32 blocks
with a power-of-two scale) and with outputs in the form the GEMMs take.

`own = False` computes them with elementary torch operations in 32 bits,
`own = True` with the library's kernels.  `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

# smallest exponent of a normal, exponent of the largest value, stored mantissa bits, largest value
_FORMATS = {"e4m3": (-6, 8, 3, 448.0), "e5m2": (-14, 15, 2, 57344.0)}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_EPS = 1e-5


def listed():
    return [
        # serving one token: residual add, norm, and the row copy the gate/up GEMM reads
        dict(name="norm one token", op="norm", rows=1, cols=4096, dtype="bf16", kind="rms", residual=True, y=False,
             y_fmt="e4m3", ckpt=""),
        # the training forward of a block: the sum, the norm for the dual-layout quantizer, the 8-bit checkpoint
        dict(name="norm train", op="norm", rows=8192, cols=4096, dtype="bf16", kind="rms", residual=True, y=True,
             y_fmt="", ckpt="e4m3"),
        # a layer norm with weight and bias over rows of no round length, in 32 bits
        dict(name="norm layer f32 odd", op="norm", rows=2047, cols=4097, dtype="f32", kind="layer", residual=False,
             y=True, y_fmt="", ckpt=""),
        # the training backward from the 8-bit checkpoint, with the gradient that skips the block
        dict(name="norm grad train", op="norm_grad", rows=8192, cols=4096, dtype="bf16", kind="rms", residual=True,
             ckpt="e4m3"),
        # a layer norm's backward from the stored input, few rows, weight and bias gradients
        dict(name="norm grad layer odd", op="norm_grad", rows=509, cols=2051, dtype="bf16", kind="layer",
             residual=False, ckpt=""),
        # serving one token: the gated activation as the row copy the down GEMM reads
        dict(name="glu one token", op="glu", rows=1, cols=14336, dtype="bf16", act="silu", h=False, h_fmt="e4m3",
             ckpt=""),
        # the training forward: the down GEMM's operand and the 8-bit checkpoints of gate and up
        dict(name="glu train", op="glu", rows=8192, cols=14336, dtype="bf16", act="silu", h=False, h_fmt="e4m3",
             ckpt="e4m3"),
        # the exact GELU gate in 32 bits, odd lengths
        dict(name="glu gelu f32 odd", op="glu", rows=771, cols=4099, dtype="f32", act="gelu", h=True, h_fmt="",
             ckpt=""),
        # the training backward from the checkpoints, gradients in bf16 beside each other
        dict(name="glu grad train", op="glu_grad", rows=8192, cols=14336, dtype="bf16", act="silu", h=False,
             ckpt="e4m3"),
        # the tanh GELU's backward from the stored inputs, odd lengths, with the product recomputed
        dict(name="glu grad tanh odd", op="glu_grad", rows=1001, cols=2731, dtype="bf16", act="gelu_tanh", h=True,
             ckpt=""),
        # the training backward straight into the dgrad and wgrad GEMMs' operands
        dict(name="glu grad dual train", op="glu_dual", rows=8192, cols=14336, dtype="bf16", act="silu",
             fmt="e5m2", h_fmt="e4m3", ckpt="e4m3"),
        # the same for a small batch from the stored inputs
        dict(name="glu grad dual small", op="glu_dual", rows=288, cols=4096, dtype="bf16", act="gelu_tanh",
             fmt="e4m3", h_fmt="", ckpt=""),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(v) // step * step)

    op = rng.choice(["norm", "norm_grad", "glu", "glu_grad", "glu_dual"])
    c = dict(op=op, rows=size(1, 8192), cols=size(64, 8192 if op.startswith("norm") else 14336))
    c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    c["ckpt"] = rng.choice(["e4m3", "e5m2", ""])
    if op.startswith("norm"):
        c["kind"] = rng.choice(["rms", "layer"])
        c["residual"] = rng.random() < 0.5
    else:
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
    if op == "norm":
        c["y_fmt"] = rng.choice(["e4m3", "e5m2", "", ""])
        c["y"] = c["y_fmt"] == "" or rng.random() < 0.3
    elif op == "glu":
        c["h_fmt"] = rng.choice(["e4m3", "e5m2", "", ""])
        c["h"] = c["h_fmt"] == "" or rng.random() < 0.3
    elif op == "glu_grad":
        c["h"] = rng.random() < 0.5
    elif op == "glu_dual":
        c["fmt"] = rng.choice(["e4m3", "e5m2"])
        c["h_fmt"] = rng.choice(["e4m3", ""])
        c["rows"] = -(-c["rows"] // 32) * 32
    if op == "glu_dual" or c["ckpt"] or c.get("y_fmt") or c.get("h_fmt"):
        c["cols"] = -(-c["cols"] // 32) * 32
    most = max(work(k)["bytes"] for k in listed())
    while work(c)["bytes"] > most:
        c["rows"] = max(32, c["rows"] // 64 * 32)
    return c


def work(case):
    c, n, b = case, case["rows"] * case["cols"], _BYTES[case["dtype"]]
    copy = 1 + 1 / 32                                   # a code and its share of the block's scale
    if c["op"] == "norm":
        per = b + (2 * b if c["residual"] else 0) + (b if c["y"] else 0) + (copy if c["y_fmt"] else 0)
        per += copy if c["ckpt"] else 0
        return {"bytes": n * per + 4 * c["cols"] + 8 * c["rows"], "flops": 8 * n}
    if c["op"] == "norm_grad":
        per = 2 * b + (copy if c["ckpt"] else b) + (b if c["residual"] else 0)
        return {"bytes": n * per + 12 * c["cols"] + 8 * c["rows"], "flops": 14 * n}
    inputs = 2 * (copy if c["ckpt"] and c["op"] != "glu" else b)
    if c["op"] == "glu":
        per = inputs + (b if c["h"] else 0) + (copy if c["h_fmt"] else 0) + (2 * copy if c["ckpt"] else 0)
        return {"bytes": n * per, "flops": 8 * n}
    if c["op"] == "glu_grad":
        return {"bytes": n * (b + inputs + 2 * b + (b if c["h"] else 0)), "flops": 14 * n}
    return {"bytes": n * (b + inputs + 4 * copy + (copy if c["h_fmt"] else 0)), "flops": 24 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, rows, cols):
    """A residual stream: tokens of different size, an offset, a few channels that are 20 times the rest."""
    x = _normal(g, rows, cols) * torch.exp(0.5 * _normal(g, rows, 1)) + 0.1
    at = torch.randint(0, cols, (max(1, cols // 1024),), generator=g, device="cuda")
    x[:, at] *= 20.0
    return x


def _gradient(g, rows, cols):
    """Gradients: small, and of a size of its own for each token."""
    return _normal(g, rows, cols) * (1e-3 * torch.exp(_normal(g, rows, 1)))


def _codes(x, fmt):
    """The 8-bit checkpoint of x as bytes: codes [rows][cols] and block scales [rows][cols / 32]."""
    q, s = _encode(x.float(), fmt)
    return q.view(torch.uint8), s.view(torch.uint8)


def prepare(case, seed):
    c, rows, cols, dt = case, case["rows"], case["cols"], _DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if c["op"] in ("norm", "norm_grad"):
        s["weight"] = (1.0 + 0.2 * _normal(g, cols)).to(dt)
        s["bias"] = (0.1 * _normal(g, cols)).to(dt) if c["kind"] == "layer" else None
        x = _stream(g, rows, cols).to(dt)
        if c["op"] == "norm":
            s["x"] = x
            s["residual"] = _normal(g, rows, cols).to(dt) if c["residual"] else None
            if rows == 1:                               # a decoding loop writes into the same buffers each step
                s["buffers"] = {k: torch.empty(*n, dtype=t, device="cuda") for k, n, t in (
                    ("sum_out", (rows, cols), dt), ("y", (rows, cols), dt), ("qy", (rows, cols), torch.uint8),
                    ("sy", (rows, cols // 32), torch.uint8), ("mean", (rows,), torch.float32),
                    ("rstd", (rows,), torch.float32))}
            return s
        s["dy"] = _gradient(g, rows, cols).to(dt)
        s["dsum"] = _gradient(g, rows, cols).to(dt) if c["residual"] else None
        f = x.float()
        s["mean"] = f.mean(1) if c["kind"] == "layer" else None
        centred = f - s["mean"][:, None] if c["kind"] == "layer" else f
        s["rstd"] = torch.rsqrt(centred.square().mean(1) + _EPS)
        s["x"], s["codes"] = (None, _codes(x, c["ckpt"])) if c["ckpt"] else (x, None)
        return s
    # gate and up: the halves of one fused projection's output
    both = (1.5 * _normal(g, rows, 2 * cols) * torch.exp(0.3 * _normal(g, rows, 1))).to(dt)
    s["gate"], s["up"] = both[:, :cols], both[:, cols:]
    if c["op"] == "glu":
        if rows == 1:
            s["buffers"] = {"h": torch.empty(rows, cols, dtype=dt, device="cuda"),
                            "qh": torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                            "sh": torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")}
        return s
    s["dh"] = _gradient(g, rows, cols).to(dt)
    if c["ckpt"]:
        s["codes"] = _codes(s["gate"], c["ckpt"]) + _codes(s["up"], c["ckpt"])
        s["gate"] = s["up"] = None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _encode(v, fmt):
    """FP8 codes of 1x32 blocks along the last axis (saturating, to nearest even) and their power-of-two scales."""
    _, emax, _, top = _FORMATS[fmt]
    b = v.reshape(v.shape[0], -1, 32)
    field = b.abs().amax(2).view(torch.int32) >> 23     # the largest value's exponent
    e = torch.where(field == 0, -127, (field - 127 - emax).clamp(min=-127))
    y = b * ((127 - e) << 23).view(torch.float32)[:, :, None]
    return y.clamp(-top, top).to(_FP8[fmt]).reshape(v.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _decode(codes, scales, fmt):
    q = codes.view(_FP8[fmt]).float().reshape(codes.shape[0], -1, 32)
    return (q * (scales.int() << 23).view(torch.float32)[:, :, None]).reshape(codes.shape)


def _gate(x, act):
    """act(x) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * x * x)


def _plain(s):
    c, out, dt = s["case"], {}, _DTYPES[s["case"]["dtype"]]
    if c["op"] == "norm":
        x = s["x"].float()
        if c["residual"]:
            out["sum"] = (x + s["residual"].float()).to(dt)
            x = out["sum"].float()
        if c["ckpt"]:
            out["qx"], out["sx"] = _encode(x, c["ckpt"])
        if c["kind"] == "layer":
            out["mean"] = x.mean(1)
            x = x - out["mean"][:, None]
        out["rstd"] = 1.0 / torch.sqrt((x * x).mean(1) + _EPS)
        y = x * out["rstd"][:, None] * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if c["y"]:
            out["y"] = y.to(dt)
        if c["y_fmt"]:
            out["qy"], out["sy"] = _encode(y, c["y_fmt"])
        return out
    if c["op"] == "norm_grad":
        dy = s["dy"].float()
        x = _decode(*s["codes"], c["ckpt"]) if c["ckpt"] else s["x"].float()
        if c["kind"] == "layer":
            x = x - s["mean"][:, None]
        x = x * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = g - x * (g * x).mean(1, keepdim=True)
        if c["kind"] == "layer":
            dx = dx - g.mean(1, keepdim=True)
            out["dbias"] = dy.sum(0, dtype=torch.float64).float()
        dx = dx * s["rstd"][:, None]
        if c["residual"]:
            dx = dx + s["dsum"].float()
        out["dx"] = dx.to(dt)
        out["dweight"] = (dy * x).sum(0, dtype=torch.float64).float()
        return out
    if c["ckpt"] and c["op"] != "glu":
        gate, up = _decode(*s["codes"][:2], c["ckpt"]), _decode(*s["codes"][2:], c["ckpt"])
    else:
        gate, up = s["gate"].float(), s["up"].float()
    a, slope = _gate(gate, c["act"])
    if c["op"] == "glu":
        if c["h"]:
            out["h"] = (a * up).to(dt)
        if c["h_fmt"]:
            out["qh"], out["sh"] = _encode(a * up, c["h_fmt"])
        if c["ckpt"]:
            out["qg"], out["sg"] = _encode(gate, c["ckpt"])
            out["qu"], out["su"] = _encode(up, c["ckpt"])
        return out
    dh = s["dh"].float()
    both = torch.cat([dh * up * slope, dh * a], 1)
    if c["op"] == "glu_grad":
        out["dboth"] = both.to(dt)
        if c["h"]:
            out["h"] = (a * up).to(dt)
        return out
    out["q_row"], out["s_row"] = _encode(both, c["fmt"])
    out["q_col"], out["s_col"] = _encode(both.t().contiguous(), c["fmt"])
    if c["h_fmt"]:
        out["qh_col"], out["sh_col"] = _encode((a * up).t().contiguous(), c["h_fmt"])
    return out


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _values(q, s, fmt):
    """Codes and scale bytes seen as the values they stand for."""
    return q.view(_FP8[fmt]), s.view(torch.float8_e8m0fnu)


def _library(s):
    from fp4_quantization_block_amd import mx

    c, out = s["case"], {}
    fmt = c["ckpt"] or None
    if c["op"] == "norm":
        kept = {k: v for k, v in s.get("buffers", {}).items()
                if (k != "y" or c["y"]) and (k != "sum_out" or c["residual"]) and (k != "mean" or c["kind"] == "layer")
                and (k not in ("qy", "sy") or c["y_fmt"])}
        r = mx.mx_norm_forward(s["x"], s["weight"], s["bias"], eps=_EPS, kind=c["kind"], residual=s["residual"],
                               write_y=c["y"], y_fmt=c["y_fmt"] or None, ckpt_fmt=fmt, **kept)
        if c["residual"]:
            out["sum"] = r.sum
        if fmt:
            out["qx"], out["sx"] = _values(r.qx, r.sx, fmt)
        if c["kind"] == "layer":
            out["mean"] = r.mean
        out["rstd"] = r.rstd
        if c["y"]:
            out["y"] = r.y
        if c["y_fmt"]:
            out["qy"], out["sy"] = _values(r.qy, r.sy, c["y_fmt"])
        return out
    if c["op"] == "norm_grad":
        ckpt = mx.checkpoint(fmt, *s["codes"]) if fmt else None
        r = mx.mx_norm_backward(s["dy"], s["rstd"], x=s["x"], ckpt=ckpt, mean=s["mean"], weight=s["weight"],
                                kind=c["kind"], dsum=s["dsum"], want_dbias=c["kind"] == "layer")
        out["dx"], out["dweight"] = r.dx, r.dweight
        if c["kind"] == "layer":
            out["dbias"] = r.dbias
        return out
    if c["op"] == "glu":
        kept = {k: v for k, v in s.get("buffers", {}).items()
                if (k != "h" or c["h"]) and (k not in ("qh", "sh") or c["h_fmt"])}
        r = mx.mx_glu_forward(s["gate"], s["up"], c["act"], write_h=c["h"], h_fmt=c["h_fmt"] or None, ckpt_fmt=fmt,
                              **kept)
        if c["h"]:
            out["h"] = r.h
        if c["h_fmt"]:
            out["qh"], out["sh"] = _values(r.qh, r.sh, c["h_fmt"])
        if fmt:
            out["qg"], out["sg"] = _values(r.qg, r.sg, fmt)
            out["qu"], out["su"] = _values(r.qu, r.su, fmt)
        return out
    if fmt:
        source = dict(gate_ckpt=mx.checkpoint(fmt, *s["codes"][:2]), up_ckpt=mx.checkpoint(fmt, *s["codes"][2:]))
    else:
        source = dict(gate=s["gate"], up=s["up"])
    if c["op"] == "glu_grad":
        both = torch.empty(c["rows"], 2 * c["cols"], dtype=s["dh"].dtype, device=s["dh"].device)
        r = mx.mx_glu_backward(s["dh"], act=c["act"], dgate=both[:, :c["cols"]], dup=both[:, c["cols"]:],
                               recompute_h=c["h"], **source)
        out["dboth"] = both
        if c["h"]:
            out["h"] = r.h
        return out
    r = mx.mx_glu_backward_dual_layout(s["dh"], act=c["act"], fmt=c["fmt"], h_fmt=c["h_fmt"] or None, **source)
    out["q_row"], out["s_row"] = _values(r.q_row, r.s_row, c["fmt"])
    out["q_col"], out["s_col"] = _values(r.q_col, r.s_col, c["fmt"])
    if c["h_fmt"]:
        out["qh_col"], out["sh_col"] = _values(r.qh_col, r.sh_col, c["h_fmt"])
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in 64 bits for whole e, from the bits of the number."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    return torch.frexp(v)[1].long() - 1


def _block_values(v, fmt):
    """What the codes stand for, and the block scales: the nearest multiple of the step that the value's binade has."""
    emin, emax, mbits, top = _FORMATS[fmt]
    b = v.unflatten(1, (v.shape[1] // 32, 32))
    big = b.abs().amax(2)
    e = torch.where(big == 0, -127, (_floor_log2(big) - emax).clamp(min=-127))
    y = b / _power(e).unsqueeze(2)
    step = _power(_floor_log2(y.abs()).clamp(min=emin) - mbits)
    return (torch.round(y / step) * step).clamp(-top, top).flatten(1), _power(e)


def _restored(codes, scales, fmt):
    return (codes.view(_FP8[fmt]).double().unflatten(1, (-1, 32)) * _power(scales.long() - 127).unsqueeze(2)).flatten(1)


def _slope(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * torch.special.expit(-g)
    if act == "gelu":
        return (g * torch.special.ndtr(g),
                torch.special.ndtr(g) + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi))
    inner = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    p = torch.special.expit(inner)                      # (1 + tanh(z)) / 2 is the logistic function of 2 z
    return g * p, p + g * p * torch.special.expit(-inner) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    c, r = case, {}
    if c["op"] == "norm":
        x = s["x"].double()
        if c["residual"]:
            # the sum is rounded to the stream's type, and what is normalised is that
            r["sum"] = x + s["residual"].double()
            x = r["sum"].float().to(s["x"].dtype).double()
        if c["ckpt"]:
            r["qx"], r["sx"] = _block_values(x, c["ckpt"])
        mean = x.sum(1, keepdim=True) / c["cols"] if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
        if c["kind"] == "layer":
            r["mean"] = mean[:, 0]
        rstd = ((x - mean).square().sum(1, keepdim=True) / c["cols"] + _EPS).pow(-0.5)
        r["rstd"] = rstd[:, 0]
        y = (x - mean) * rstd * s["weight"].double() + (0.0 if s["bias"] is None else s["bias"].double())
        if c["y"]:
            r["y"] = y
        if c["y_fmt"]:
            r["qy"], r["sy"] = _block_values(y, c["y_fmt"])
        return r
    if c["op"] == "norm_grad":
        x = _restored(*s["codes"], c["ckpt"]) if c["ckpt"] else s["x"].double()
        rstd, dy = s["rstd"].double().unsqueeze(1), s["dy"].double()
        unit = (x - s["mean"].double().unsqueeze(1)) * rstd if c["kind"] == "layer" else x * rstd
        wdy = dy * s["weight"].double()
        along = (wdy * unit).sum(1, keepdim=True) / c["cols"]
        across = wdy.sum(1, keepdim=True) / c["cols"] if c["kind"] == "layer" else 0.0
        r["dx"] = rstd * (wdy - unit * along - across) + (s["dsum"].double() if c["residual"] else 0.0)
        r["dweight"] = (dy * unit).sum(0)
        if c["kind"] == "layer":
            r["dbias"] = dy.sum(0)
        return r
    if c["ckpt"] and c["op"] != "glu":
        gate, up = _restored(*s["codes"][:2], c["ckpt"]), _restored(*s["codes"][2:], c["ckpt"])
    else:
        gate, up = s["gate"].double(), s["up"].double()
    a, da = _slope(gate, c["act"])
    if c["op"] == "glu":
        if c["h"]:
            r["h"] = a * up
        if c["h_fmt"]:
            r["qh"], r["sh"] = _block_values(a * up, c["h_fmt"])
        if c["ckpt"]:
            r["qg"], r["sg"] = _block_values(gate, c["ckpt"])
            r["qu"], r["su"] = _block_values(up, c["ckpt"])
        return r
    dh = s["dh"].double()
    both = torch.cat([dh * up * da, dh * a], 1)
    if c["op"] == "glu_grad":
        r["dboth"] = both
        if c["h"]:
            r["h"] = a * up
        return r
    r["q_row"], r["s_row"] = _block_values(both, c["fmt"])
    r["q_col"], r["s_col"] = _block_values(both.t(), c["fmt"])
    if c["h_fmt"]:
        r["qh_col"], r["sh_col"] = _block_values((a * up).t(), c["h_fmt"])
    return r
