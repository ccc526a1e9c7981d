"""The feed-forward sublayer's operators, measured: the RMS norm that adds the
residual and also writes its output in 8 bits, its backward pass, the gated
feed-forward block, its backward pass from 8-bit activation checkpoints, and
the gate's part of that backward pass on its own.

A case is one call (or a store and the load that reads it back) on inputs like
those of a training or serving step.  `run` computes it in plain torch
operations, in 32 bits, where `own` is false, and through the library
(fsdp_emulated_ranks_gb300.cr) where it is true.

An 8-bit matrix is e4m3 codes and one fp32 scale per row and 128 columns: with
m the group's largest finite magnitude, scale = max(m / 448, 2^-126) and code =
e4m3(value / scale).  Where a case returns such a matrix, it returns the values
it stands for, code * scale, as bf16.
"""
import math

import torch

own = False

GROUP = 128
TINY = 2.0 ** -126
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One generated token through the norm: the latency of a small call.
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 2048, "dtype": "bf16", "residual": True},
        # A micro-batch of 8192 tokens at the width of the benchmark's transformer.
        {"name": "norm_step", "op": "norm", "rows": 8192, "cols": 2048, "dtype": "bf16", "residual": True},
        # fp32 activations of a width that is not a multiple of anything.
        {"name": "norm_odd_f32", "op": "norm", "rows": 1777, "cols": 4099, "dtype": "f32", "residual": False},
        # The norm's backward pass in the same training step.
        {"name": "norm_back_step", "op": "norm_back", "rows": 8192, "cols": 2048, "dtype": "bf16", "held": "full"},
        # The same from an 8-bit checkpoint of the norm's input, ragged.
        {"name": "norm_back_odd_q8", "op": "norm_back", "rows": 3001, "cols": 1111, "dtype": "bf16", "held": "q8"},
        # The gate's backward pass from 8-bit checkpoints at the benchmark's feed-forward width.
        {"name": "act_back_step", "op": "act_back", "rows": 8192, "cols": 8192, "act": "silu"},
        # A last, ragged micro-batch and a width two thirds of 4 * 1024 rounded up to an odd number.
        {"name": "act_back_odd", "op": "act_back", "rows": 1025, "cols": 2731, "act": "gelu"},
        # One generated token: the block streams its weights.
        {"name": "glu_token", "op": "glu", "tokens": 1, "dim": 2048, "ffn": 8192, "act": "silu", "keep": False},
        # The forward pass of a training step: gate and up are kept in 8 bits.
        {"name": "glu_step", "op": "glu", "tokens": 8192, "dim": 2048, "ffn": 8192, "act": "silu", "keep": True},
        # A long prompt at odd sizes: nothing is kept.
        {"name": "glu_odd", "op": "glu", "tokens": 1531, "dim": 1001, "ffn": 2731, "act": "gelu", "keep": False},
        # The backward pass of the training step, from 8-bit gate and up.
        {"name": "glu_back_step", "op": "glu_back", "tokens": 8192, "dim": 2048, "ffn": 8192, "act": "silu", "held": "full"},
        # A small ragged micro-batch whose input is an 8-bit checkpoint too.
        {"name": "glu_back_small_q8", "op": "glu_back", "tokens": 257, "dim": 512, "ffn": 2048, "act": "silu", "held": "q8"},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd numbers and multiples of 128 among them."""
    k = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    if kind == 0 and k >= 128:
        k -= k % 128
    elif kind == 1 and k < hi:
        k |= 1
    return max(lo, min(hi, k))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "act_back", "glu", "glu_back"])
    if op in ("norm", "norm_back"):
        rows, cols = _size(rng, 1, 8192), _size(rng, 64, 8192)
        while rows * cols > 8192 * 2048:
            rows = max(1, rows // 2)
        c = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "norm":
            c["residual"] = rng.random() < 0.7
        else:
            c["held"] = rng.choice(["full", "q8"])
        return c
    act = rng.choice(["silu", "gelu"])
    if op == "act_back":
        return {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 64, 8192), "act": act}
    c = {"op": op, "tokens": _size(rng, 1, 8192), "dim": _size(rng, 64, 2048), "ffn": _size(rng, 64, 8192), "act": act}
    if op == "glu":
        c["keep"] = rng.random() < 0.5
    else:
        c["held"] = rng.choice(["full", "q8"])
    return c


def _groups(cols):
    return -(-cols // GROUP)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        r, c, e = case["rows"], case["cols"], 4 if case["dtype"] == "f32" else 2
        q8 = r * c + 4 * r * _groups(c)
        if op == "norm":
            # x (and the residual, and their sum), w, y, rstd, and the 8-bit output, given as bf16 values
            moved = r * c * e * (4 if case["residual"] else 2) + c * e + 4 * r + r * c * 2
            return {"bytes": moved, "flops": 6 * r * c}
        held = q8 if case["held"] == "q8" else r * c * e
        return {"bytes": held + 3 * r * c * e + c * e + 4 * r + 4 * c, "flops": 10 * r * c}
    if op == "act_back":
        r, c = case["rows"], case["cols"]
        return {"bytes": 8 * r * c + 2 * (r * c + 4 * r * _groups(c)), "flops": 20 * r * c}
    t, d, f = case["tokens"], case["dim"], case["ffn"]
    weights = 2 * 2 * d * f
    if op == "glu":
        return {"bytes": 2 * t * d + weights + 2 * t * f * (3 if case["keep"] else 1), "flops": 4 * t * d * f + 10 * t * f}
    held = t * d + 4 * t * _groups(d) if case["held"] == "q8" else 2 * t * d
    kept = 2 * (t * f + 4 * t * _groups(f))
    return {"bytes": 2 * t * f + kept + held + 2 * weights + 2 * t * d + 2 * t * f, "flops": 8 * t * d * f + 20 * t * f}


def _quantise(v):
    """e4m3 codes (as float8) and fp32 scales of a matrix, in 32 bits."""
    rows, cols = v.shape
    g = _groups(cols)
    p = torch.zeros(rows, g * GROUP, dtype=torch.float32, device=v.device)
    p[:, :cols] = v
    p = p.view(rows, g, GROUP)
    m = torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax(-1)
    s = (m * (1.0 / 448.0)).clamp_min(TINY)
    codes = (p * (1.0 / s).unsqueeze(-1)).clamp(-448.0, 448.0)
    codes = torch.where(torch.isfinite(p), codes, torch.full_like(p, math.nan)).to(torch.float8_e4m3fn)
    return codes.view(rows, g * GROUP)[:, :cols].contiguous(), s


def _restore(codes, scales):
    cols = codes.shape[1]
    return codes.to(torch.float32) * scales.repeat_interleave(GROUP, 1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def bf(t):
        return t.to(torch.bfloat16)

    s = dict(case)
    dev = torch.device("cuda")
    if case["op"] in ("norm", "norm_back"):
        r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        # a residual stream: rows of different size, a few channels far larger than the rest
        scale = torch.exp(normal(r, 1, std=0.5)) * torch.where(torch.rand(1, c, generator=g, device=dev) < 0.01, 20.0, 1.0)
        x = normal(r, c) * scale
        s["w"] = (1.0 + normal(c, std=0.1)).to(dt)
        if case["op"] == "norm":
            s["x"] = x.to(dt)
            s["res"] = (normal(r, c) * scale).to(dt) if case["residual"] else None
            s["sum"] = torch.empty(r, c, dtype=dt, device=dev) if case["residual"] else None
            s["y"] = torch.empty(r, c, dtype=dt, device=dev)
            s["codes"] = torch.empty(r, c, dtype=torch.uint8, device=dev)
            s["scales"] = torch.empty(r, _groups(c), dtype=torch.float32, device=dev)
            s["back"] = torch.empty(r, c, dtype=torch.bfloat16, device=dev)
            s["rstd"] = torch.empty(r, dtype=torch.float32, device=dev)
            return s
        x = x.to(dt).float()
        s["rstd"] = torch.rsqrt(x.square().mean(1) + EPS)
        if case["held"] == "q8":
            codes, s["scales"] = _quantise(x)
            s["codes"] = codes.view(torch.uint8)
        else:
            s["x"] = x.to(dt)
        s["dy"] = normal(r, c, std=1e-3).to(dt)
        s["dres"] = normal(r, c, std=1e-3).to(dt)
        s["dx"] = torch.empty(r, c, dtype=dt, device=dev)
        s["dw"] = torch.empty(c, dtype=torch.float32, device=dev)
        s["work"] = torch.empty(32 << 20, dtype=torch.uint8, device=dev)
        return s
    if case["op"] == "act_back":
        r, c = case["rows"], case["cols"]
        s["da"] = bf(normal(r, c, std=1e-3))
        for name in ("g", "u"):
            codes, s[name + "s"] = _quantise(normal(r, c))
            s[name + "c"] = codes.view(torch.uint8)
        for name in ("dg", "du", "a"):
            s[name] = torch.empty(r, c, dtype=torch.bfloat16, device=dev)
        return s
    t, d, f = case["tokens"], case["dim"], case["ffn"]
    x = bf(normal(t, d))
    s["wg"], s["wu"] = bf(normal(f, d, std=d ** -0.5)), bf(normal(f, d, std=d ** -0.5))
    s["work"] = torch.empty(2 * t * f * 2 + 2 * t * d + 6 * d * f + 2 * (t + f) * 256 + (64 << 20), dtype=torch.uint8, device=dev)
    if case["op"] == "glu":
        s["x"] = x
        s["a"] = torch.empty(t, f, dtype=torch.bfloat16, device=dev)
        if case["keep"]:
            for name in ("g", "u"):
                s[name + "c"] = torch.empty(t, f, dtype=torch.uint8, device=dev)
                s[name + "s"] = torch.empty(t, _groups(f), dtype=torch.float32, device=dev)
                s[name] = torch.empty(t, f, dtype=torch.bfloat16, device=dev)
        return s
    for name, w in (("g", s["wg"]), ("u", s["wu"])):
        # what the forward pass kept, with the spread of a gate's and an up projection's values
        codes, s[name + "s"] = _quantise(normal(t, f))
        s[name + "c"] = codes.view(torch.uint8)
    if case["held"] == "q8":
        codes, s["xs"] = _quantise(x.float())
        s["xc"] = codes.view(torch.uint8)
    else:
        s["x"] = x
    s["da"] = bf(normal(t, f, std=1e-3))
    s["dx"] = torch.empty(t, d, dtype=torch.bfloat16, device=dev)
    s["dwg"], s["dwu"] = (torch.empty(f, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    s["a"] = torch.empty(t, f, dtype=torch.bfloat16, device=dev)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---- plain form: 32 bits, rounded once at the end ----------------------------------

def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    k, c = math.sqrt(2.0 / math.pi), 0.044715
    th = torch.tanh(k * (g + c * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3.0 * c * g * g)


def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _act_back(s):
    g, u, da = _restore(_f8(s["gc"]), s["gs"]), _restore(_f8(s["uc"]), s["us"]), s["da"].float()
    a, slope = _act(g, s["act"])
    return da * u * slope, da * a, a * u


def _run_plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "norm":
        dt = s["x"].dtype
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * rstd.unsqueeze(1) * s["w"].float()
        out = {"y": y.to(dt), "y8": _restore(*_quantise(y)).to(bf), "rstd": rstd}
        if s["res"] is not None:
            out["sum"] = h.to(dt)
        return out
    if op == "norm_back":
        dt = s["dy"].dtype
        h = s["x"].float() if "x" in s else _restore(_f8(s["codes"]), s["scales"])
        rstd = s["rstd"].unsqueeze(1)
        xh, dy = h * rstd, s["dy"].float()
        t = dy * s["w"].float()
        dx = rstd * (t - xh * (t * xh).mean(1, keepdim=True)) + s["dres"].float()
        return {"dx": dx.to(dt), "dw": (dy * xh).sum(0)}
    if op == "act_back":
        dg, du, a = _act_back(s)
        return {"dg": dg.to(bf), "du": du.to(bf), "a": a.to(bf)}
    wg, wu = s["wg"].float(), s["wu"].float()
    if op == "glu":
        x = s["x"].float()
        g, u = x @ wg.T, x @ wu.T
        out = {"a": (_act(g, s["act"])[0] * u).to(bf)}
        if s["keep"]:
            out["g8"], out["u8"] = _restore(*_quantise(g)).to(bf), _restore(*_quantise(u)).to(bf)
        return out
    x = s["x"].float() if "x" in s else _restore(_f8(s["xc"]), s["xs"])
    dg, du, a = _act_back(s)
    return {"dx": (dg @ wg + du @ wu).to(bf), "dwg": (dg.T @ x).to(bf), "dwu": (du.T @ x).to(bf), "a": a.to(bf)}


# ---- the library's calls -----------------------------------------------------------

def _run_own(s):
    from fsdp_emulated_ranks_gb300 import cr
    op = s["op"]
    if op == "norm":
        r, c, dt = s["rows"], s["cols"], s["dtype"]
        q8 = cr.Q8(s["codes"], s["scales"])
        cr.cr_rms_norm(s["x"], s["res"], s["w"], r, c, dt, EPS, s["sum"], s["y"], q8, s["rstd"])
        cr.cr_q8_load(q8, r, c, s["back"], "bf16")
        out = {"y": s["y"], "y8": s["back"], "rstd": s["rstd"]}
        if s["res"] is not None:
            out["sum"] = s["sum"]
        return out
    if op == "norm_back":
        r, c, dt = s["rows"], s["cols"], s["dtype"]
        x8 = cr.Q8(s["codes"], s["scales"]) if s["held"] == "q8" else None
        cr.cr_rms_norm_backward(s["dy"], s.get("x"), x8, s["w"], s["rstd"], s["dres"], r, c, dt,
                                s["dx"], s["dw"], "f32", s["work"], s["work"].numel())
        return {"dx": s["dx"], "dw": s["dw"]}
    g8 = u8 = None
    if "gc" in s:
        g8, u8 = cr.Q8(s["gc"], s["gs"]), cr.Q8(s["uc"], s["us"])
    if op == "act_back":
        cr.cr_glu_act_backward(s["da"], g8, u8, s["rows"], s["cols"], "bf16", s["act"],
                               s["dg"], s["du"], s["a"])
        return {"dg": s["dg"], "du": s["du"], "a": s["a"]}
    t, d, f = s["tokens"], s["dim"], s["ffn"]
    if op == "glu":
        cr.cr_glu(s["x"], s["wg"], s["wu"], t, d, f, "bf16", s["act"], s["a"], g8, u8,
                  s["work"], s["work"].numel())
        out = {"a": s["a"]}
        if s["keep"]:
            cr.cr_q8_load(g8, t, f, s["g"], "bf16")
            cr.cr_q8_load(u8, t, f, s["u"], "bf16")
            out["g8"], out["u8"] = s["g"], s["u"]
        return out
    x8 = cr.Q8(s["xc"], s["xs"]) if s["held"] == "q8" else None
    cr.cr_glu_backward(s["da"], g8, u8, s.get("x"), x8, s["wg"], s["wu"], t, d, f, "bf16", s["act"],
                       s["dx"], s["dwg"], s["dwu"], "bf16", s["a"], s["work"], s["work"].numel())
    return {"dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"], "a": s["a"]}


# ---- the definition in 64 bits -----------------------------------------------------

def _e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even: 3 fraction bits, lowest exponent -6, largest 448."""
    mag = v.abs()
    e = torch.floor(torch.log2(torch.where(mag > 0, mag, torch.ones_like(mag)))).clamp(min=-6.0)
    e = torch.where(torch.ldexp(torch.ones_like(mag), e) > mag, (e - 1).clamp(min=-6.0), e)
    step = torch.ldexp(torch.ones_like(mag), e - 3)
    return torch.sign(v) * (torch.round(mag / step) * step).clamp(max=448.0)


def _held(v):
    """The values that the 8-bit form of the 64-bit matrix v stands for."""
    out = torch.empty_like(v)
    for lo in range(0, v.shape[1], GROUP):
        part = v[:, lo:lo + GROUP]
        s = (part.abs().amax(1, keepdim=True) / 448.0).clamp(min=TINY)
        out[:, lo:lo + GROUP] = _e4m3(part / s) * s
    return out


def _decoded(codes, scales):
    """code * scale from the codes' bits: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = codes.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1.0 + m / 8.0, (e - 7).double()), torch.ldexp(m / 8.0, torch.full_like(m, -6.0)))
    v = torch.where(b >= 128, -mag, mag)
    rows, cols = v.shape
    idx = torch.arange(cols, device=v.device) // GROUP
    return v * scales.double()[:, idx]


def _gate64(g, kind):
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1.0 - p)
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    dz = math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g ** 2)
    # 0.5 (1 + tanh z) = sigmoid(2 z)
    p = torch.sigmoid(2.0 * z)
    return g * p, p + g * 2.0 * p * (1.0 - p) * dz


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = h + s["res"].double()
        rstd = 1.0 / torch.sqrt((h ** 2).sum(1) / case["cols"] + EPS)
        y = h * rstd[:, None] * s["w"].double()
        out = {"y": y, "y8": _held(y), "rstd": rstd}
        if case["residual"]:
            out["sum"] = h
        return out
    if op == "norm_back":
        h = s["x"].double() if case["held"] == "full" else _decoded(s["codes"], s["scales"])
        r, dy, w = s["rstd"].double()[:, None], s["dy"].double(), s["w"].double()
        # with rstd given: d/dx of sum(dy * w * x * rstd(x)), rstd' = -rstd^3 x / cols
        lead = dy * w * r
        dx = lead - h * r ** 3 * (dy * w * h).sum(1, keepdim=True) / case["cols"] + s["dres"].double()
        return {"dx": dx, "dw": torch.einsum("rc,rc,r->c", dy, h, s["rstd"].double())}
    if op == "glu":
        x = s["x"].double()
        g, u = torch.einsum("td,fd->tf", x, s["wg"].double()), torch.einsum("td,fd->tf", x, s["wu"].double())
        out = {"a": _gate64(g, case["act"])[0] * u}
        if case["keep"]:
            out["g8"], out["u8"] = _held(g), _held(u)
        return out
    g, u, da = _decoded(s["gc"], s["gs"]), _decoded(s["uc"], s["us"]), s["da"].double()
    val, slope = _gate64(g, case["act"])
    dg, du, a = da * u * slope, da * val, val * u
    if op == "act_back":
        return {"dg": dg, "du": du, "a": a}
    x = s["x"].double() if case["held"] == "full" else _decoded(s["xc"], s["xs"])
    dx = torch.einsum("tf,fd->td", dg, s["wg"].double()) + torch.einsum("tf,fd->td", du, s["wu"].double())
    return {"dx": dx, "dwg": torch.einsum("tf,td->fd", dg, x), "dwu": torch.einsum("tf,td->fd", du, x), "a": a}
