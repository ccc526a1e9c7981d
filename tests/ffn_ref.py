"""The feed-forward operators' formulas in 64 bits (include/cr_ffn.h), and the
error bounds their tests use.

Bounds.  U16 = 2^-8 is bf16's unit roundoff, U32 = 2^-24 fp32's.  A result
rounded once to bf16 is within U16 of the exact value, relatively, plus what
the fp32 arithmetic before the rounding loses.  A sum of d fp32 terms added in
any order is within d * U32 * sum|terms|; the tensor cores may truncate where
they align addends, so their sums are given 2 * U32 per addition."""
from __future__ import annotations

import math

import torch

GROUP = 128
U16, U32 = 2.0 ** -8, 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
U_OUT = {"bf16": U16, "f32": U32}


def groups(cols):
    return -(-cols // GROUP)


def decode(codes, scales):
    """code * scale in 64 bits, from the codes' bits."""
    b = codes.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
    mag = torch.where((b & 127) == 127, torch.full_like(mag, math.nan), mag)
    idx = torch.arange(codes.shape[1], device=codes.device) // GROUP
    return torch.where(b >= 128, -mag, mag) * scales.double()[:, idx]


def scales_of(v):
    """The exact scales of the 64-bit matrix v."""
    rows, cols = v.shape
    p = torch.zeros(rows, groups(cols) * GROUP, dtype=torch.float64, device=v.device)
    p[:, :cols] = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    return (p.view(rows, -1, GROUP).amax(-1) / 448).clamp(min=2.0 ** -126)


def assert_q8(codes, scales, v, slack=0.0, what=""):
    """codes and scales are the 8-bit form of v, whose fp32 values may be off by
    `slack` (a matrix, or 0).  A code is the nearest e4m3 value: within half a
    step, 2^-4 of its magnitude or 2^-10 below 2^-6, of value / scale; the
    scale and the division carry 4 U32."""
    want = scales_of(v)
    rows, cols = v.shape
    idx = torch.arange(cols, device=v.device) // GROUP
    if torch.is_tensor(slack):
        p = torch.zeros(rows, groups(cols) * GROUP, dtype=torch.float64, device=v.device)
        p[:, :cols] = torch.where(torch.isfinite(slack), slack, torch.zeros_like(slack))
        ds = p.view(rows, -1, GROUP).amax(-1) / 448
    else:
        ds = slack / 448
    assert torch.all((scales.double() - want).abs() <= 4 * U32 * want + ds), f"{what}: scales"
    got, s = decode(codes, scales), scales.double()[:, idx]
    fine = torch.isfinite(v)
    assert torch.all(torch.isnan(got) == ~fine), f"{what}: codes of values that are not finite"
    # a value just above 448 scales (rounding of the scale) saturates
    half = torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10)
    err = (got - v).abs()
    bad = fine & (err > half * (1 + 2.0 ** -18) + slack + 8 * U32 * v.abs())
    assert not bad.any(), f"{what}: {int(bad.sum())} codes are not the nearest"


def act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def norm(x, residual, w, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def norm_depth(cols):
    """Additions one term of a row's sum of squares may pass through."""
    return 8 * max(4, -(-cols // 8192)) + 5 + 32


def norm_backward(dy, h, w, rstd, dres):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    n = h * r
    t = dy * w
    c = (t * n).mean(1, keepdim=True)
    dx = r * (t - n * c)
    if dres is not None:
        dx = dx + dres.double()
    # what each output may lose in fp32: terms, and the row's or column's sum
    dw = (dy * n).sum(0)
    mag = r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
    return dx, dw, mag, (dy * n).abs().sum(0)


def glu(x, wg, wu, kind):
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.T, x @ wu.T
    return g, u, act(g, kind)[0] * u


def glu_act_backward(da, g, u, kind):
    a, slope = act(g, kind)
    return da.double() * u * slope, da.double() * a, a * u


def bf16(v):
    """v rounded to bf16, as 64 bits."""
    return v.float().to(torch.bfloat16).double()


def rel_norm(got, want):
    d = (got.double() - want).norm()
    n = want.norm()
    return float(d / n) if n > 0 else float(d)
