"""The whole feed-forward sublayer's gradients: a 64-bit reference, an emulation of
what the calls compute, with mistakes to plant in it, and the two tests that a set
of gradients has to pass.

    h = x + r,  y = rms_norm(h) w,  a = act(y Wg^T) (y Wu^T),  L = sum(a k)

The calls keep y, gate and up as 8-bit checkpoints (y8, g8, u8) and h in bf16."""
from __future__ import annotations

import math

import torch

import ffn_ref as R

EPS = 1e-6
NAMES = ("dx", "dw", "dwg", "dwu")


def quantised(v):
    """The values that v's 8-bit form stands for (64 bits)."""
    s = R.scales_of(v).float()
    idx = torch.arange(v.shape[1], device=v.device) // R.GROUP
    codes = (v.float() * (1 / s)[:, idx]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.double() * s.double()[:, idx]


def inputs(gen, rows=48, dim=136, ffn=200):
    dev = gen.device

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std
    b = torch.bfloat16
    return {"x": normal(rows, dim).to(b), "r": normal(rows, dim).to(b), "w": (1 + normal(dim, std=0.1)).to(b),
            "wg": normal(ffn, dim, std=dim ** -0.5).to(b), "wu": normal(ffn, dim, std=dim ** -0.5).to(b),
            "k": normal(rows, ffn).to(b)}


def reference(s, held, kind="gelu"):
    """torch's 64-bit autograd of L, each kept value in the place of the computed one: held =
    the values of h (as bf16), y8, g8 and u8."""
    x, w, wg, wu = (s[n].double().requires_grad_() for n in ("x", "w", "wg", "wu"))

    def put(v, kept):
        return v + (kept - v).detach()
    h = put(x + s["r"].double(), held["h"])
    y = put(h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w, held["y"])
    g, u = put(y @ wg.T, held["g"]), put(y @ wu.T, held["u"])
    act = (torch.nn.functional.gelu(g, approximate="tanh") if kind == "gelu" else torch.nn.functional.silu(g))
    (act * u * s["k"].double()).sum().backward()
    return {n: t.grad for n, t in zip(NAMES, (x, w, wg, wu))}


MUTATIONS = ("dx without the mean", "dx 1.2 times", "dwg 1.2 times", "dw without 4 rows", "dwu without 4 tokens",
             "slope without its second term", "dx a row off", "dw without rstd")


def emulate(s, kind="gelu", mutation=None):
    """What the calls compute, and what they hold: bf16 where they round to it, 64 bits elsewhere."""
    h, rstd, y = R.norm(s["x"], s["r"], s["w"], EPS)
    held = {"h": R.bf16(h), "y": quantised(y)}
    g, u, _ = R.glu(R.bf16(y), s["wg"], s["wu"], kind)
    held["g"], held["u"] = quantised(g), quantised(u)
    dg, du, _ = R.glu_act_backward(s["k"], held["g"], held["u"], kind)
    if mutation == "slope without its second term":
        some = held["g"].where(held["g"] != 0, torch.ones_like(dg))
        dg = s["k"].double() * held["u"] * R.act(some, kind)[0] / some
    dy = R.bf16(R.bf16(dg) @ s["wg"].double() + R.bf16(du) @ s["wu"].double())
    keep = slice(0, -4 if mutation == "dwu without 4 tokens" else None)
    dwg, dwu = dg.T @ held["y"], du[keep].T @ held["y"][keep]
    dx, dw, _, _ = R.norm_backward(dy, held["h"], s["w"], rstd, None)
    n = held["h"] * rstd[:, None]
    if mutation == "dx without the mean":
        dx = rstd[:, None] * dy * s["w"].double()
    elif mutation == "dx 1.2 times":
        dx = 1.2 * dx
    elif mutation == "dwg 1.2 times":
        dwg = 1.2 * dwg
    elif mutation == "dw without 4 rows":
        dw = (dy * n)[:-4].sum(0)
    elif mutation == "dx a row off":
        dx = dx.roll(1, 0)
    elif mutation == "dw without rstd":
        dw = (dy * held["h"]).sum(0)
    return {m: R.bf16(v) for m, v in zip(NAMES, (dx, dw, dwg, dwu))}, held


def off_formula(got, want):
    """Gradients whose norm of error, against the reference, passes its bound.  Rounding to bf16
    is off by U16 of a value at most and by U16 / sqrt 3 in the root mean square, where a
    binade begins; each rounding adds at most that part of a gradient's norm, independently.
    dwg and dwu pass two (dg or du, the result), dx and dw four (dg or du, dy, h against its
    statistics, the result): at most 2 / sqrt 3 = 1.15 U16, and 2 U16 is allowed."""
    return [n for n in NAMES if not R.rel_norm(got[n], want[n]) <= 2 * R.U16]


def directions(s, got, held, kind):
    """Directions in which the gradients are looked at: each along itself, and x along h, to which
    the norm's dx is orthogonal, as far as every row's dx would point there without the
    mean that the norm takes off."""
    for n, t in zip(NAMES, ("x", "w", "wg", "wu")):
        yield n, t, got[n].double()
    rstd = torch.rsqrt(held["h"].square().mean(1, keepdim=True) + EPS)
    normed = (held["h"] * rstd).requires_grad_()
    a = R.glu(normed * s["w"].double(), s["wg"], s["wu"], kind)[2]
    (a * s["k"].double()).sum().backward()
    normed, at = normed.detach(), normed.grad
    yield "dx", "x", rstd * normed * (at * normed).mean(1, keepdim=True)


def off_differences(s, got, held, kind="gelu"):
    """Gradients whose derivative along a direction d is not the central difference of the
    64-bit forward pass.  The checkpoints are rounded to e4m3, 2^-4 of a value at most and
    2^-4 / sqrt 3 in the root mean square; a term of a gradient has two such factors, so its
    error has a norm of less than 2^-4 |grad| and signs of its own.  Along d that adds up to
    about 2^-4 |grad| |d| / sqrt(values of d): six times that is allowed, and 2^-6 of the
    derivative for what is left in the errors' squares (2^-8) with a factor of four."""

    def loss(v):
        y = R.norm(v["x"], s["r"], v["w"], EPS)[2]
        return float((R.glu(y, v["wg"], v["wu"], kind)[2] * s["k"].double()).sum())
    base = {n: s[n].double() for n in ("x", "w", "wg", "wu")}
    bad = []
    for n, t, d in directions(s, got, held, kind):
        step = 1e-4 / float(d.abs().max())
        want = (loss({**base, t: base[t] + step * d}) - loss({**base, t: base[t] - step * d})) / (2 * step)
        along = float((got[n].double() * d).sum())
        noise = 6 * 2.0 ** -4 * float(got[n].double().norm() * d.norm()) / math.sqrt(d.numel())
        if not abs(along - want) <= noise + 2.0 ** -6 * abs(want):
            bad.append(n)
    return bad
