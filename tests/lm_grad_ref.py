"""The gradient of log probabilities, entropies and log-sum-exps in 64 bits, from the logits alone
(lm_ref.log_probs_backward takes the lse that the call was given, rounded to fp32), and its error bound."""
from __future__ import annotations

import math

import torch

import lm_ref as R

SHARE = 256.0  # |lse| from which the call goes by the row's maximum and sum in place of its lse


def gradient(logits, targets, scale, dlogp, dentropy, dlse):
    """The gradient and its error bound before the last rounding.

    Every row goes by p = exp(z - max) / sum.  Below SHARE the call has exp(z - lse): its lse is off by
    half a step, U32 of itself, beside the sum's own error, and log p is off by both.  From SHARE on, log p is
    a difference of (x - max) scale, off by 2 U32 of itself, and the sum's logarithm.  The power of two adds what
    lm_ref.log_probs_backward counts (4 U32 of log p, 24 U32), the given entropy its own error."""
    v = logits.shape[1]
    s = R.f32(scale)
    z = logits.double() * s
    most = z.amax(1, keepdim=True)
    dead = torch.isneginf(most)
    near = z - torch.where(dead, torch.zeros_like(most), most)
    total = torch.where(dead, torch.zeros_like(most), torch.log(torch.exp(near).sum(1, keepdim=True)))
    none = most + total <= -2.0 ** 100  # such a row gets zeros
    logs = torch.where(none, torch.full_like(z, -math.inf), near - total)
    p = torch.exp(logs)
    left = p > 0
    logs = torch.where(left, logs, torch.zeros_like(logs))
    near = torch.where(left, near, torch.zeros_like(near))
    h = -(p * logs).sum(1, keepdim=True)
    zero = torch.zeros(logits.shape[0], dtype=torch.float64, device=logits.device)
    d, e, q = (zero if t is None else t.double() for t in (dlogp, dentropy, dlse))
    if targets is not None:
        d = torch.where(R.valid(targets, v), d, zero)
    d, e, q = (t[:, None] for t in (d, e, q))
    want = s * p * (q - d - e * (logs + h))
    _, _, lse, _, sum_bound, ent_bound = R.log_probs(logits, None, scale)
    lse = torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)).clamp_max(SHARE)
    off = R.U32 * (4 * logs.abs() + 2 * near.abs() + lse[:, None] + 24) + sum_bound[:, None]
    factor = abs(s) * (q.abs() + d.abs() + e.abs() * (logs.abs() + h))
    bound = p * (off * factor + abs(s) * e.abs() * (off + ent_bound[:, None] + R.U32 * (logs.abs() + h)))
    bound = bound + 2.0 ** -126 * (1 + factor)
    if targets is not None and dlogp is not None:
        hit = torch.zeros_like(z).scatter_(1, targets.long().clamp(0, v - 1)[:, None], 1.0) * s * d * ~none
        want = want + hit
        bound = bound + 4 * R.U32 * hit.abs()
    return want, bound
