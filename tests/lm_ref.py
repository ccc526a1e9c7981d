"""The language model operators' formulas in 64 bits (include/cr_lm.h), and the error
bounds their tests use.

U16 = 2^-8 is bf16's unit roundoff, U32 = 2^-24 fp32's.  A value rounded once to its
type is within U_OUT of it, relatively; every fp32 operation before that adds U32 of
its result."""
from __future__ import annotations

import math

import torch

from ffn_ref import TORCH, U16, U32, U_OUT  # noqa: F401


def f32(x: float) -> float:
    """x rounded to fp32, as the calls round their scales."""
    return float(torch.tensor(x, dtype=torch.float32))


def valid(ids, vocab):
    return (ids >= 0) & (ids < vocab)


def embedding(table, ids, scale):
    v = table.shape[0]
    rows = table.double()[ids.long().clamp(0, v - 1)] * f32(scale)
    return torch.where(valid(ids, v)[:, None], rows, torch.zeros_like(rows))


def embedding_backward(dout, ids, vocab, scale, base):
    """The gradient and its error bound before the last rounding: a sum of n fp32
    terms in any order is within n U32 of the sum of magnitudes; the product with the
    scale and base's addition round once each."""
    ok = valid(ids, vocab)
    d, k = dout.double()[ok], ids.long()[ok]
    total, size = (torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device) for _ in range(2))
    total.index_add_(0, k, d)
    size.index_add_(0, k, d.abs())
    n = torch.zeros(vocab, dtype=torch.float64, device=dout.device).index_add_(0, k, torch.ones_like(k, dtype=torch.float64))
    s = f32(scale)
    want = total * s
    bound = (n[:, None] + 2) * U32 * size * abs(s)
    if base is not None:
        want = want + base.double()
        bound = bound + 2 * U32 * (want.abs() + base.double().abs())
    return want, bound


def philox(counter, key):
    """Philox4x32-10 on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def numbers(rows, cols, seed, offset, first_row=0):
    """The elements' 16-bit numbers, [rows, cols] int64 on the CPU."""
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    out = torch.empty(rows, -(-cols // 8) * 8, dtype=torch.int64)
    for r in range(rows):
        for g in range(-(-cols // 8)):
            w = philox((g, first_row + r, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
            out[r, 8 * g:8 * g + 8] = torch.tensor([h for x in w for h in (x & 0xFFFF, x >> 16)])
    return out[:, :cols]


def numbers_fast(rows, cols, seed, offset, first_row=0):
    """The same with int64 tensors, whose products wrap modulo 2^64."""
    low = 0xFFFFFFFF
    groups = -(-cols // 8)
    c = [torch.arange(groups).repeat(rows), torch.arange(first_row, first_row + rows).repeat_interleave(groups),
         torch.full((rows * groups,), offset % (1 << 64) & low), torch.full((rows * groups,), offset % (1 << 64) >> 32)]
    k = [seed % (1 << 64) & low, seed % (1 << 64) >> 32]
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32 & low) ^ c[1] ^ k[0], q & low, (p >> 32 & low) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    halves = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1)
    return halves.view(rows, groups * 8)[:, :cols]


def limit_of(p):
    return int(math.floor(p * 65536 + 0.5))


def dropout(x, residual, p, nums):
    """out and its bound before the last rounding."""
    lim = limit_of(p)
    by = 0.0 if lim == 65536 else f32(65536 / (65536 - lim))
    kept = torch.where(nums.to(x.device) >= lim, x.double() * by, torch.zeros((), dtype=torch.float64, device=x.device))
    if residual is None:
        return kept, U32 * kept.abs()
    out = kept + residual.double()
    return out, U32 * (kept.abs() + out.abs())


def depth(vocab):
    """Additions in a row at most: a thread of 32 (vocab up to 2048) or 256 adds its columns
    in turn; then lanes, warps and blocks merge, three roundings each."""
    return max(min(vocab, 2048) / 32, vocab / 256) + 16 + 3 * (5 + 8 + 8)


def log_probs(logits, targets, scale):
    """logp, entropy, lse, all rows' log probabilities, and the bounds: of logp and lse before their
    last product and sum, of the entropy, and of lse's own rounding.

    t = (x - max) c, c = scale log2(e), is off by 3.25 U32 of itself; its power of two by 2
    ulps, 4 U32, more; the sum of them by depth() U32.  The mean of |t| ln2 over p is at most the entropy H, so
    log s is off by (4 H + 8 + depth) U32, logp by 4 U32 of z - max more.  The entropy's w / s is a mean of t: off by
    the mean of 4 U32 t^2, and by log s's errors of itself."""
    z = logits.double() * f32(scale)
    most = z.amax(1)
    dead = torch.isneginf(most)
    near = z - torch.where(dead, torch.zeros_like(most), most)[:, None]
    total = torch.log(torch.exp(near).sum(1))
    lse = most + torch.where(dead, torch.zeros_like(total), total)
    logs = torch.where(dead[:, None], z, near - total[:, None])  # apart from lse: a row of lowest values has no room for total
    p = torch.exp(logs)
    ent = -torch.where(p > 0, p * logs, torch.zeros_like(p)).sum(1)
    v = logits.shape[1]
    if targets is None:
        logp = None
    else:
        ok = valid(targets, v)
        logp = torch.where(ok, logs.gather(1, targets.long().clamp(0, v - 1)[:, None])[:, 0], torch.zeros_like(lse))
    far = torch.where(torch.isfinite(z) & (p > 0), near, torch.zeros_like(z))
    bound = U32 * (4 * ent + 8 + depth(v))
    ent_bound = (bound + 4 * U32) * (1 + 2 * ent) + 5 * U32 * (p * far * far).sum(1)
    return logp, ent, lse, logs, bound, ent_bound


def logp_bound(logp, bound):
    return bound + 6 * U32 * torch.where(torch.isfinite(logp), logp.abs(), torch.zeros_like(logp))


def top(logits, k):
    """Ids of the k largest logits: falling, equal ones by rising id, NaN last."""
    x = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits.double().to(logits.dtype))
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices
    nan = torch.isnan(logits).gather(1, order)
    order = order.gather(1, torch.sort(nan.int(), dim=1, stable=True).indices)
    return order[:, :k].to(torch.int32)


def log_probs_backward(logits, targets, scale, lse, entropy, dlogp, dentropy, dlse):
    """The gradient from the lse and entropy given, and its bound before the last rounding.
    p is off by the error of z - lse (3 U32 of itself) and 4 U32 for the power, its factor by a few
    U32 of its terms."""
    v = logits.shape[1]
    s = f32(scale)
    z = logits.double() * s
    none = lse <= -2.0 ** 100
    l = torch.where(none, torch.zeros_like(lse), lse).double()[:, None]
    logs = z - l
    p = torch.where(none[:, None], torch.zeros_like(z), torch.exp(logs))
    logs = torch.where(p > 0, logs, torch.zeros_like(logs))
    zero = torch.zeros_like(lse)
    d, e, q = (zero if t is None else t for t in (dlogp, dentropy, dlse))
    if targets is not None:
        d = torch.where(valid(targets, v), d, zero)
    d, e, q = (t.double()[:, None] for t in (d, e, q))
    h = (entropy if entropy is not None else zero).double()[:, None]
    want = s * p * (q - d - e * (logs + h))
    factor = abs(s) * (q.abs() + d.abs() + e.abs() * (logs.abs() + h.abs()))
    err = 4 * logs.abs() + 24
    # the power's results below 2^-126 are 0: p is off by as much, and the product by its factor more
    bound = U32 * err * p * factor + 2.0 ** -126 * (1 + factor)
    if targets is not None and dlogp is not None:
        hit = torch.zeros_like(z).scatter_(1, targets.long().clamp(0, v - 1)[:, None], 1.0) * s * d
        hit = torch.where(none[:, None], torch.zeros_like(hit), hit)
        want = want + hit
        bound = bound + 4 * U32 * hit.abs()
    return want, bound


def assert_close(got, want, bound, dt, what):
    """got, of type dt, is want within `bound` and one rounding (down to the smallest normal)."""
    limit = bound + U_OUT[dt] * (want.abs() + bound) + 2.0 ** -126
    err = (got.double() - want).abs()
    same = (got.double() == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | (err <= limit))
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{float(got[at])} for {float(want[at])}, bound {float(limit.expand_as(err)[at])}")
