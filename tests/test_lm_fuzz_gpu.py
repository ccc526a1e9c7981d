"""Seeded random calls of the language model operators: sizes, strides, offsets, types and options
together, against the formulas in 64 bits."""
import random

import pytest
import torch

import lm_ref as R
import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def size(rng, lo, hi):
    k = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, rng.choice([k, k | 1, -(-k // 64) * 64])))


def layout(rng, cols):
    """Row stride and offset."""
    return rng.choice([(cols, 0), (-(-cols // 16) * 16, 16), (cols + rng.randrange(9), rng.randrange(9))])


@pytest.mark.parametrize("seed", range(12))
def test_embedding(seed):
    rng, g = random.Random(seed), T.gen(seed)
    tokens, vocab, dim = size(rng, 1, 9000), size(rng, 1, 20000), size(rng, 1, 1500)
    while tokens * dim > 4 << 20 or vocab * dim > 4 << 20:
        dim = max(1, dim // 2)
    dt, out_dt, bits = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice([32, 64])
    scale = rng.choice([1.0, 0.37, -3.0])
    ids = T.skewed(g, tokens, vocab)
    if rng.random() < 0.5:
        ids[torch.rand(tokens, generator=g, device=DEV) < 0.2] = rng.choice([-1, vocab, -(2 ** 31)])
    ids = ids.to(torch.int32 if bits == 32 else torch.int64)
    lds = [layout(rng, dim) for _ in range(5)]
    table = T.place(T.normal(g, vocab, dim, dt=dt), *lds[0])
    out, buf = T.padded(tokens, dim, out_dt, *lds[1])
    cr.cr_embedding(table, vocab, ids, tokens, dim, dt, scale, out, out_dt)
    want = R.embedding(table, ids, scale)
    R.assert_close(out, want, R.U32 * want.abs(), out_dt, "embedding")
    T.untouched(out, buf, tokens, dim, *lds[1])
    dout = T.place(T.normal(g, tokens, dim, dt=dt), *lds[2])
    base = T.place(T.normal(g, vocab, dim, dt=out_dt), *lds[3]) if rng.random() < 0.6 else None
    where = base is not None and rng.random() < 0.5
    want, bound = R.embedding_backward(dout, ids, vocab, scale, base)
    dtable, buf = (base, None) if where else T.padded(vocab, dim, out_dt, *lds[4])
    T.back(dout, dt, ids, vocab, scale, base, dtable, out_dt)
    R.assert_close(dtable, want, bound, out_dt, "embedding backward")
    if not where:
        T.untouched(dtable, buf, vocab, dim, *lds[4])


@pytest.mark.parametrize("seed", range(12))
def test_dropout(seed):
    rng, g = random.Random(100 + seed), T.gen(seed)
    rows, cols, dt = size(rng, 1, 600), size(rng, 1, 3000), rng.choice(["bf16", "f32"])
    lds = [layout(rng, cols) for _ in range(3)]
    x = T.place(T.normal(g, rows, cols, dt=dt), *lds[0])
    res = T.place(T.normal(g, rows, cols, dt=dt), *lds[1]) if rng.random() < 0.5 else None
    p, key, off, call = rng.random(), rng.getrandbits(64), rng.getrandbits(64), rng.getrandbits(40)
    first = rng.choice([0, 17, 2 ** 32 - rows])
    out, buf = T.padded(rows, cols, dt, *lds[2])
    cr.cr_dropout(x, res, rows, cols, dt, p, T.rng_of(key, off), call, first, out)
    want, bound = R.dropout(x, res, p, R.numbers_fast(rows, cols, key, off + call, first))
    R.assert_close(out, want, bound, dt, "dropout")
    T.untouched(out, buf, rows, cols, *lds[2])


@pytest.mark.parametrize("seed", range(30))
def test_log_probs(seed):
    rng, g = random.Random(200 + seed), T.gen(seed)
    rows, vocab, dt = size(rng, 1, 1500), size(rng, 1, 150000), rng.choice(["bf16", "f32"])
    while rows * vocab > 8 << 20:
        rows = max(1, rows // 2)
    ld, off = layout(rng, vocab)
    logits = T.place(T.normal(g, rows, vocab, std=rng.choice([0.1, 2.0, 12.0]), dt=dt), ld, off)
    if rng.random() < 0.4:
        logits.masked_fill_(torch.rand(rows, vocab, generator=g, device=DEV) < rng.choice([0.5, 0.999]),
                            rng.choice([float("-inf"), torch.finfo(R.TORCH[dt]).min]))
    if rng.random() < 0.3:
        logits.copy_((logits.float() * 2).round() / 2)
    targets = torch.randint(-1, vocab + 1, (rows,), generator=g, device=DEV)
    scale = rng.choice([1.0, 0.5, 1.7])
    T.check_forward(logits, targets, dt, scale, rng.choice([0, 1, min(vocab, 7), min(vocab, 32)]))
    _, ent, lse, _, _ = T.forward(logits, targets, dt, scale)
    d, e, q = (T.normal(g, rows) if rng.random() < 0.6 else None for _ in range(3))
    ld, off = layout(rng, vocab)
    out, buf = T.padded(rows, vocab, dt, ld, off)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, scale, lse, ent, d, e, q, out)
    want, bound = R.log_probs_backward(logits, targets if d is not None else None, scale, lse, ent, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")
    T.untouched(out, buf, rows, vocab, ld, off)
