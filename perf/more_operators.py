"""Cases for measuring the gate and up projections of a gated MLP block with
their activation and product in one kernel (MX operands, 8-bit outputs and
checkpoints), and the optimizer's side of the block's training step: the
global gradient norm over many tensors, and the AdamW step over many tensors
with states in 32 bits or in FP8 with a dynamic range expansion per group.

`own = False` computes them with elementary torch operations in 32 bits (64
for the norm's sum, and for the powers, whose results lie next to the borders
of an 8-bit format), `own = True` with the library's kernels.  `exact` gives
the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# exponent of the largest value, largest value, smallest subnormal
_FORMATS = {"e4m3": (8, 448.0, 2.0 ** -9), "e5m2": (15, 57344.0, 2.0 ** -16), "e2m1": (2, 6.0, 0.5)}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_LR, _BETAS, _EPS, _DECAY, _MAX_NORM = 3e-4, (0.9, 0.95), 1e-8, 0.1, 1.0


def listed():
    return [
        # serving one token: the projections' product as the row copy that the down projection reads
        dict(name="glu one token", op="glu", rows=1, inner=4096, cols=14336, fa="e4m3", fb="e4m3", act="silu",
             h="", h_fmt="e4m3", keep=False, ckpt=""),
        # serving a batch of sequences from FP4 weights, one token each
        dict(name="glu batch fp4", op="glu", rows=24, inner=4096, cols=14336, fa="e2m1", fb="e2m1", act="gelu_tanh",
             h="bf16", h_fmt="", keep=False, ckpt=""),
        # odd lengths, an inner dimension that no tile divides, gate and up kept in 16 bits for the backward pass
        dict(name="glu odd", op="glu", rows=771, inner=1056, cols=1003, fa="e5m2", fb="e4m3", act="gelu",
             h="bf16", h_fmt="", keep=True, ckpt=""),
        # a long prompt through FP4 weights
        dict(name="glu prompt fp4", op="glu", rows=2047, inner=4096, cols=14336, fa="e2m1", fb="e2m1", act="silu",
             h="bf16", h_fmt="", keep=False, ckpt=""),
        # the training forward: the down projection's operand, gate and up as 8-bit checkpoints
        dict(name="glu train", op="glu", rows=8192, inner=4096, cols=14336, fa="e4m3", fb="e4m3", act="silu",
             h="", h_fmt="e4m3", keep=False, ckpt="e4m3"),
        # the gains of a few layers
        dict(name="norm small", op="norm", count=8, size=4096, packed=False, grad="f32"),
        # the weight gradients of an MLP block, as the GEMMs write them
        dict(name="norm train", op="norm", count=3, size=4096 * 14336, packed=False, grad="bf16"),
        # a step over a few vectors
        dict(name="adamw small", op="adamw", count=8, size=4096, packed=False, param="f32", grad="f32", states="f32",
             group=0, copy=False, clip=False),
        # many small tensors packed without gaps into one buffer, 16-bit parameters
        dict(name="adamw odd", op="adamw", count=150, size=20011, packed=True, param="bf16", grad="bf16",
             states="f32", group=0, copy=False, clip=True),
        # tensors whose last group is not full
        dict(name="adamw odd 8 bit", op="adamw", count=41, size=77777, packed=False, param="f32", grad="f32",
             states="e4m3", group=64, copy=False, clip=False),
        # an MLP block's weights: 32-bit weights and states, and the 16-bit weights that the next step reads
        dict(name="adamw train", op="adamw", count=3, size=4096 * 14336, packed=False, param="f32", grad="bf16",
             states="f32", group=0, copy=True, clip=True),
        # the same with the states in FP8
        dict(name="adamw train 8 bit", op="adamw", count=3, size=4096 * 14336, packed=False, param="f32",
             grad="bf16", states="e4m3", group=128, copy=True, clip=True),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(v) // step * step)

    op = rng.choice(["glu", "glu", "norm", "adamw", "adamw"])
    if op == "glu":
        c = dict(op=op, rows=size(1, 8192), inner=size(64, 8192, 32), cols=size(48, 14336))
        c["fa"], c["fb"] = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e2m1", "e2m1")])
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
        c["h"], c["h_fmt"] = rng.choice([("bf16", ""), ("", "e4m3"), ("bf16", "e4m3")])
        c["keep"], c["ckpt"] = rng.choice([(False, ""), (False, "e4m3"), (True, "")])
        if c["h_fmt"] or c["ckpt"]:
            c["cols"] = -(-c["cols"] // 32) * 32
        most = max(work(k)["flops"] for k in listed())
        while work(c)["flops"] > most:
            c["rows"] //= 2
        return c
    c = dict(op=op, count=size(1, 200), size=size(1, 4096 * 4096), packed=rng.random() < 0.4)
    while c["count"] * c["size"] > 2 ** 27:
        c["count"] = (c["count"] + 1) // 2
    c["grad"] = rng.choice(["bf16", "f32"])
    if op == "norm":
        return c
    c["param"] = rng.choice(["f32", "f32", "bf16"])
    c["states"] = rng.choice(["f32", "e4m3"])
    c["group"] = rng.choice([32, 64, 128, 256]) if c["states"] != "f32" else 0
    c["packed"] = c["packed"] and c["states"] == "f32"
    c["copy"] = c["param"] == "f32" and rng.random() < 0.5
    c["clip"] = rng.random() < 0.5
    return c


def _sizes(c):
    """Lengths of a case's tensors: the largest first, then odd ones down to a third of it."""
    n = c["size"]
    return [n - i * 37 % (2 * n // 3 + 1) if n % 4096 else n for i in range(c["count"])]


def _places(c):
    """(where each tensor begins in one buffer, the buffer's length): without gaps, or each at a whole group."""
    at, places, whole = 0, [], 1 if c["packed"] else c.get("group") or 256
    for n in _sizes(c):
        places.append(at)
        at += -(-n // whole) * whole
    return places, at


def work(case):
    c = case
    if c["op"] == "glu":
        per, mf = (1 / 2 if c["fa"] == "e2m1" else 1) + 1 / 32, c["rows"] * c["cols"]
        out = (2 if c["h"] else 0) + (33 / 32 if c["h_fmt"] else 0)
        out += (4 if c["keep"] else 0) + (33 / 16 if c["ckpt"] else 0)
        return {"bytes": (c["rows"] + 2 * c["cols"]) * c["inner"] * per + mf * out, "flops": 4 * mf * c["inner"]}
    n = sum(_sizes(c))
    if c["op"] == "norm":
        return {"bytes": n * _BYTES[c["grad"]] + 8, "flops": 2 * n}
    states = 16 if c["states"] == "f32" else 4 + 32 / c["group"]
    per = 2 * _BYTES[c["param"]] + _BYTES[c["grad"]] + states + (2 if c["copy"] else 0)
    # a power of each state in and out is counted as two functions of eight operations
    return {"bytes": n * per, "flops": n * (14 if c["states"] == "f32" else 78)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _operand(x, fmt):
    """Codes (two FP4 codes a byte, the first in the low half) of 1x32 blocks of a matrix, and their scale bytes."""
    if fmt != "e2m1":
        q, s = _encode(x, fmt)
        return q.view(torch.uint8), s.view(torch.uint8)
    e, s = _exponents(x, fmt)
    y = (x.unflatten(1, (-1, 32)) * _pow2(-e)).flatten(1)
    steps = torch.tensor(_E2M1, device=x.device)
    codes = torch.bucketize(y.abs(), (steps[1:] + steps[:-1]) / 2).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    return codes[:, 0::2] + 16 * codes[:, 1::2], s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "glu":
        rows, inner, cols = c["rows"], c["inner"], c["cols"]
        # a normalised stream: tokens of different size, a few channels that are 20 times the rest
        x = _normal(g, rows, inner) * torch.exp(0.3 * _normal(g, rows, 1))
        x[:, torch.randint(0, inner, (max(1, inner // 1024),), generator=g, device="cuda")] *= 20.0
        s["a"] = _operand(x, c["fa"])
        # one fused projection's weights, gate then up
        q, b = _operand(_normal(g, 2 * cols, inner) * inner ** -0.5, c["fb"])
        s["gate"], s["up"] = (q[:cols], b[:cols]), (q[cols:], b[cols:])
        if rows == 1 and c["h_fmt"] and not (c["h"] or c["keep"] or c["ckpt"]):
            # a decoding loop writes into the same buffers each step
            s["buffers"] = {"qh": torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                            "sh": torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")}
        return s
    places, total = _places(c)
    spans = list(zip(places, _sizes(c)))
    held = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, n in spans:
        held[at:at + n] = True

    def flat(values, dtype):
        return (values * held).to(dtype)

    size = torch.exp(_normal(g, total // 256 + 1)).repeat_interleave(256)[:total]   # rows of different size
    # the second moment's root, and an average that is less than it
    root = 1e-4 * size * torch.exp(0.7 * _normal(g, total))
    mean = 0.4 * root * _normal(g, total)
    # the gradient has the average's sign: where the two cancel, the smallest magnitude of a group, which sets its
    # exponent, is known only as far as the average's own last bits, and so is the exponent
    s["g"] = flat(root * _normal(g, total).abs() * mean.sign(), _DTYPES[c["grad"]])
    if c["op"] == "norm":
        s["spans"] = spans
        if own:
            from fp4_quantization_block_amd import mx

            s["list"] = mx.tensor_list([s["g"][at:at + n] for at, n in spans])
        return s
    s["p"] = flat(0.02 * _normal(g, total), _DTYPES[c["param"]])
    s["scale"] = 0.5 + torch.rand(1, generator=g, device="cuda") / 2 if c["clip"] else None
    s["step"] = 100
    states = [flat(mean, torch.float32), flat(root.square(), torch.float32)]
    names = ["m", "v"]
    if c["states"] == "f32":
        s["m"], s["v"] = states
    else:
        names = [a + b for a in names for b in ("", "_amax", "_k")]
        for k, x in zip(("m", "v"), states):
            q, s[k + "_amax"], s[k + "_k"] = _expand(x, c["states"], c["group"])
            s[k] = q.view(torch.uint8)
    # the step is written beside the last one's result, so that a run can go back to it
    for k in ["p"] + names:
        s[k + "_out"] = torch.zeros_like(s[k])
    if c["copy"]:
        s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    if own:
        s["plan"] = _plan(s, spans)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)[:, :, None]


def _exponents(v, fmt):
    """Shared exponents of the 1x32 blocks of a matrix, and their scale bytes."""
    emax = _FORMATS[fmt][0]
    field = v.unflatten(1, (-1, 32)).abs().amax(2).view(torch.int32) >> 23      # the largest value's exponent
    e = torch.where(field == 0, -126, (field - 127 - emax).clamp(min=-126))
    return e, (torch.where(field == 0, -127, e) + 127).to(torch.uint8)


def _encode(v, fmt):
    """FP8 codes of 1x32 blocks along the last axis (saturating, to nearest even) and their power-of-two scales."""
    top = _FORMATS[fmt][1]
    e, s = _exponents(v, fmt)
    y = v.unflatten(1, (-1, 32)) * _pow2(-e)
    return y.clamp(-top, top).to(_FP8[fmt]).flatten(1), s.view(torch.float8_e8m0fnu)


def _values(codes, scales, fmt):
    """What an operand's codes and scale bytes stand for."""
    if fmt == "e2m1":
        both = torch.stack([codes & 15, codes >> 4], 2).flatten(1).int()
        steps = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=codes.device)
        q = steps[both]
    else:
        q = codes.view(_FP8[fmt]).float()
    return (q.unflatten(1, (-1, 32)) * (scales.int() << 23).view(torch.float32)[:, :, None]).flatten(1)


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _expand(x, fmt, group):
    """FP8 codes of a state after |x| -> |x|^k with one k a group, the groups' largest magnitudes and their k.
    Powers in 64 bits, of the 32-bit k."""
    _, top, low = _FORMATS[fmt]
    b = x.unflatten(0, (-1, group)).double()
    a = b.abs()
    amax = a.amax(1)
    amin = torch.where(a > 0, a, math.inf).amin(1)
    spread = torch.log2(amax / amin)
    k = torch.where((amax > 0) & (spread > 0), math.log2(top / low) / spread, 1.0).float()
    amax = torch.where(amax > 0, amax, 1.0)
    y = torch.sign(b) * (a / amax[:, None]).pow(k.double()[:, None]) * top
    return y.float().clamp(-top, top).to(_FP8[fmt]).flatten(), amax.float(), k


def _restore(q, amax, k, fmt, group):
    """The state that codes stand for."""
    c = q.view(_FP8[fmt]).float().double().unflatten(0, (-1, group))
    power = (c.abs() / _FORMATS[fmt][1]).pow(1.0 / k.double()[:, None])
    return (torch.sign(c) * amax.double()[:, None] * power).float().flatten()


def _plain(s):
    c, out = s["case"], {}
    if c["op"] == "glu":
        a = _values(*s["a"], c["fa"])
        gate = a @ _values(*s["gate"], c["fb"]).t()
        up = a @ _values(*s["up"], c["fb"]).t()
        h = _act(gate, c["act"]) * up
        if c["h"]:
            out["h"] = h.bfloat16()
        if c["h_fmt"]:
            out["qh"], out["sh"] = _encode(h, c["h_fmt"])
        if c["keep"]:
            out["gate"], out["up"] = gate.bfloat16(), up.bfloat16()
        if c["ckpt"]:
            out["qg"], out["sg"] = _encode(gate, c["ckpt"])
            out["qu"], out["su"] = _encode(up, c["ckpt"])
        return out
    if c["op"] == "norm":
        norm = s["g"].double().square().sum().sqrt()
        return torch.stack([norm, (_MAX_NORM / norm).clamp(max=1.0)]).float()
    g, p = s["g"].float(), s["p"].float()
    if c["clip"]:
        g = g * s["scale"]
    if c["states"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = _restore(s["m"], s["m_amax"], s["m_k"], c["states"], c["group"])
        v = _restore(s["v"], s["v_amax"], s["v_k"], c["states"], c["group"])
    (b1, b2), t = _BETAS, s["step"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    update = m / (torch.sqrt(v) * (1.0 - b2 ** t) ** -0.5 + _EPS)
    p = p - (_LR * _DECAY) * p - (_LR / (1.0 - b1 ** t)) * update
    out["p"] = p.to(s["p"].dtype)
    if c["copy"]:
        out["copy"] = p.bfloat16()
    if c["states"] == "f32":
        out["m"], out["v"] = m, v
        return out
    out["m"], out["m_amax"], out["m_k"] = _expand(m, c["states"], c["group"])
    out["v"], out["v_amax"], out["v_k"] = _expand(v, c["states"], c["group"])
    return out


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _plan(s, spans):
    from fp4_quantization_block_amd import mx

    c = s["case"]

    def views(x):
        return [x[at:at + n] for at, n in spans]

    def state(k, to=""):
        if c["states"] == "f32":
            return views(s[k + to])
        at = [(a // c["group"], -(-n // c["group"])) for a, n in spans]
        amax, power = s[k + "_amax" + to], s[k + "_k" + to]
        return [(q, amax[a:a + n], power[a:a + n]) for q, (a, n) in zip(views(s[k + to]), at)]

    return mx.adamw_plan(views(s["p"]), views(s["g"]), state("m"), state("v"),
                         fmt=None if c["states"] == "f32" else c["states"], group=c["group"] or 128,
                         copies=views(s["copy"]) if c["copy"] else None,
                         out=(views(s["p_out"]), state("m", "_out"), state("v", "_out")))


def _library(s):
    from fp4_quantization_block_amd import mx

    c, out = s["case"], {}
    if c["op"] == "glu":
        r = mx.mx_gemm_glu(*s["a"], None, c["fa"], *s["gate"], None, *s["up"], None, c["fb"], c["rows"], c["cols"],
                           c["inner"], act=c["act"], write_h=bool(c["h"]), h_fmt=c["h_fmt"] or None,
                           keep=c["keep"], ckpt_fmt=c["ckpt"] or None, **s.get("buffers", {}))
        if c["h"]:
            out["h"] = r.h
        if c["h_fmt"]:
            out["qh"], out["sh"] = r.qh.view(_FP8[c["h_fmt"]]), r.sh.view(torch.float8_e8m0fnu)
        if c["keep"]:
            out["gate"], out["up"] = r.gate, r.up
        if c["ckpt"]:
            out["qg"], out["sg"] = r.qg.view(_FP8[c["ckpt"]]), r.sg.view(torch.float8_e8m0fnu)
            out["qu"], out["su"] = r.qu.view(_FP8[c["ckpt"]]), r.su.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "norm":
        return mx.mx_grad_norm(s["list"], max_norm=_MAX_NORM)
    mx.mx_adamw_step(s["plan"], lr=_LR, step=s["step"], betas=_BETAS, eps=_EPS, weight_decay=_DECAY,
                     scale=s["scale"])
    out["p"] = s["p_out"]
    if c["copy"]:
        out["copy"] = s["copy"]
    if c["states"] == "f32":
        out["m"], out["v"] = s["m_out"], s["v_out"]
        return out
    out["m"], out["m_amax"], out["m_k"] = s["m_out"].view(_FP8[c["states"]]), s["m_amax_out"], s["m_k_out"]
    out["v"], out["v_amax"], out["v_k"] = s["v_out"].view(_FP8[c["states"]]), s["v_amax_out"], s["v_k_out"]
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _matrix64(codes, scales, fmt):
    if fmt == "e2m1":
        one = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
        for half in (0, 1):
            c = (codes >> (4 * half)) % 16
            e, frac = (c % 8) // 2, c % 2
            size = torch.where(e == 0, 0.5 * frac, torch.exp2(e.double() - 1) * (1 + 0.5 * frac))
            one[:, half::2] = torch.where(c >= 8, -size, size)
    else:
        one = codes.view(_FP8[fmt]).double()
    return (one.unflatten(1, (-1, 32)) * torch.exp2(scales.double() - 127).unsqueeze(2)).flatten(1)


def _scaled(v, fmt):
    """What the codes of 1x32 blocks round: the values over their block's power of two."""
    b = v.unflatten(1, (-1, 32))
    e = torch.frexp(b.abs().amax(2, keepdim=True))[1].long() - 1 - _FORMATS[fmt][0]
    return torch.ldexp(b, -e).clamp(-_FORMATS[fmt][1], _FORMATS[fmt][1]).flatten(1)


def _kept(x, fmt, group):
    """What an expanded state's codes round, its largest magnitudes and exponents."""
    a = x.unflatten(0, (-1, group))
    size = a.abs()
    most = size.max(1, keepdim=True).values
    least = size.masked_fill(size == 0, math.inf).min(1, keepdim=True).values
    ratio = math.log(_FORMATS[fmt][1] / _FORMATS[fmt][2])
    k = ratio / (torch.log(most) - torch.log(least))
    k[~torch.isfinite(k) | (most == 0) | (most == least)] = 1.0
    most = torch.where(most == 0, torch.ones_like(most), most)
    y = torch.exp(k * torch.log(size / most)) * _FORMATS[fmt][1]
    return torch.copysign(y, a).flatten(), most[:, 0], k[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    c, r = case, {}
    if c["op"] == "glu":
        a = _matrix64(*s["a"], c["fa"])
        g, u = (torch.mm(a, _matrix64(*s[k], c["fb"]).t()) for k in ("gate", "up"))
        if c["act"] == "silu":
            h = u * g * torch.sigmoid(g)
        elif c["act"] == "gelu":
            h = u * g * torch.special.ndtr(g)
        else:
            h = u * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) / 2
        if c["h"]:
            r["h"] = h
        # codes: the value that is rounded; a scale is a whole power of two, which nothing lies between
        for name, v, fmt in (("h", h, c["h_fmt"]), ("g", g, c["ckpt"]), ("u", u, c["ckpt"])):
            if fmt:
                r["q" + name], r["s" + name] = _scaled(v, fmt), None
        if c["keep"]:
            r["gate"], r["up"] = g, u
        return r
    if c["op"] == "norm":
        norm = torch.linalg.vector_norm(s["g"].double())
        return torch.stack([norm, torch.minimum(norm.new_tensor(1.0), _MAX_NORM / norm)])
    g = s["g"].double() * (s["scale"].double() if c["clip"] else 1.0)

    def state(k):
        if c["states"] == "f32":
            return s[k].double()
        q = s[k].view(_FP8[c["states"]]).double().unflatten(0, (-1, c["group"]))
        log = torch.log(q.abs() / _FORMATS[c["states"]][1]) / s[k + "_k"].double().unsqueeze(1)
        return (torch.copysign(torch.exp(log), q) * s[k + "_amax"].double().unsqueeze(1)).flatten()

    m = state("m").mul_(_BETAS[0]).add_(g, alpha=1 - _BETAS[0])
    v = state("v").mul_(_BETAS[1]).addcmul_(g, g, value=1 - _BETAS[1])
    correct = [1 - b ** s["step"] for b in _BETAS]
    p = s["p"].double()
    r["p"] = p * (1 - _LR * _DECAY) - _LR * (m / correct[0]) / ((v / correct[1]).sqrt() + _EPS)
    if c["copy"]:
        r["copy"] = r["p"]
    if c["states"] == "f32":
        r["m"], r["v"] = m, v
        return r
    r["m"], r["m_amax"], r["m_k"] = _kept(m, c["states"], c["group"])
    r["v"], r["v_amax"], r["v_k"] = _kept(v, c["states"], c["group"])
    return r
