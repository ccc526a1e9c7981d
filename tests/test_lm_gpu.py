"""The language model operators of include/cr_lm.h on a GPU, against their formulas in 64 bits
(tests/lm_ref.py derives the bounds)."""
import math

import pytest
import torch

import lm_ref as R
from fsdp_emulated_ranks_gb300 import cr
from lm_ref import TORCH

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from fsdp_emulated_ranks_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, std=1.0, dt="f32"):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(TORCH[dt])


def padded(rows, cols, dt, ld=None, offset=0):
    """A matrix inside a larger buffer, NaN around it."""
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 64,), math.nan, dtype=TORCH[dt], device=DEV)
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols], buf


def place(x, ld=None, offset=0):
    """x's values in such a matrix."""
    dt = "bf16" if x.dtype == torch.bfloat16 else "f32"
    m, _ = padded(*x.shape, dt, ld, offset)
    m.copy_(x)
    return m


def untouched(m, buf, rows, cols, ld, offset):
    """Every value of buf outside the matrix is still NaN."""
    rest = buf.clone()
    rest[offset:offset + rows * ld].view(rows, ld)[:, :cols] = math.nan
    assert bool(torch.isnan(rest).all()), "written outside the matrix"


LAYOUTS = [(0, 0), (8, 16), (5, 1), (1, 3)]  # row stride beyond the columns, elements before the first


# ---- embedding -------------------------------------------------------------------------------

def ids_of(g, n, vocab, bits, bad=True):
    ids = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    if bad and n > 3:
        ids[0], ids[n // 2] = -1, vocab
        ids[n - 1] = 2 ** 31 - 1 if bits == 32 else 2 ** 40
    return ids.to(torch.int32 if bits == 32 else torch.int64)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,vocab,dim", [(1, 1, 1), (1, 100, 2048), (37, 50, 513), (300, 7, 1001), (5, 33, 4096)])
def test_embedding(tokens, vocab, dim, dt, out_dt, layout):
    extra, off = layout
    g = gen(tokens + dim)
    table = place(normal(g, vocab, dim, dt=dt), dim + extra, off)
    ids = ids_of(g, tokens, vocab, 32 if extra else 64)
    out, buf = padded(tokens, dim, out_dt, dim + extra, off)
    scale = math.sqrt(dim)
    cr.cr_embedding(table, vocab, ids, tokens, dim, dt, scale, out, out_dt)
    want = R.embedding(table, ids, scale)
    R.assert_close(out, want, R.U32 * want.abs(), out_dt, "embedding")
    untouched(out, buf, tokens, dim, dim + extra, off)


def test_embedding_without_a_table():
    out = torch.full((4, 8), 7.0, device=DEV)
    cr.cr_embedding(None, 0, torch.zeros(4, dtype=torch.int64, device=DEV), 4, 8, "f32", 1.0, out, "f32", ldt=8)
    assert bool((out == 0).all())


def back(dout, dt, ids, vocab, scale, base, dtable, out_dt, work=None):
    t, d = dout.shape
    need = cr.cr_embedding_backward_workspace_bytes(t, vocab, d)
    work = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV) if work is None else work
    cr.cr_embedding_backward(dout, dt, ids, t, vocab, d, scale, base, dtable, out_dt, work, work.numel())


def skewed(g, n, vocab):
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,vocab,dim", [(0, 9, 40), (1, 1, 1), (1, 300, 512), (31, 9, 77), (1024, 513, 64),
                                              (1025, 40, 520), (3000, 9000, 129), (5000, 3, 33)])
def test_embedding_backward(tokens, vocab, dim, dt, out_dt, layout):
    extra, off = layout
    g = gen(tokens + vocab + dim)
    dout = place(normal(g, tokens, dim, dt=dt), dim + extra, off)
    ids = skewed(g, tokens, vocab)
    if tokens > 30:
        ids[tokens // 3], ids[tokens - 1] = -5, vocab
    base = place(normal(g, vocab, dim, dt=out_dt), dim + extra, off) if extra != 8 else None
    dtable, buf = padded(vocab, dim, out_dt, dim + extra, off)
    back(dout, dt, ids, vocab, 1.7, base, dtable, out_dt)
    want, bound = R.embedding_backward(dout, ids, vocab, 1.7, base)
    R.assert_close(dtable, want, bound, out_dt, "embedding backward")
    untouched(dtable, buf, vocab, dim, dim + extra, off)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [256, 1111])
def test_embedding_backward_in_place(dt, dim):
    """Rows that no token names are not touched, NaN or not."""
    g = gen(5)
    tokens, vocab = 500, 4000
    dout, ids = normal(g, tokens, dim, dt=dt), skewed(g, tokens, vocab)
    dtable = normal(g, vocab, dim, dt=dt)
    free = torch.ones(vocab, dtype=torch.bool, device=DEV)
    free[ids] = False
    dtable[free] = math.nan
    base = dtable.clone()
    back(dout, dt, ids, vocab, 0.5, dtable, dtable, dt)
    want, bound = R.embedding_backward(dout, ids, vocab, 0.5, base)
    R.assert_close(dtable, want, bound, dt, "in place")


@pytest.mark.parametrize("tokens,vocab", [(2048, 1), (70000, 100), (20000, 2 ** 21)])
def test_embedding_backward_of_many_tokens(tokens, vocab):
    """Rows of one, of 64, 65, 128, 129 and of thousands of tokens; ids at both ends of
    the vocabulary; every token the same."""
    dim = 24
    g = gen(tokens)
    ids = skewed(g, tokens, vocab)
    at = 0
    for k, n in enumerate((64, 65, 128, 129)):
        if vocab > 100:
            ids[at:at + n] = vocab - 1 - k
            at += n
    ids = ids[torch.randperm(tokens, generator=g, device=DEV)].to(torch.int32)
    dout = normal(g, tokens, dim)
    dtable = torch.empty(vocab, dim, device=DEV)
    back(dout, "f32", ids, vocab, 1.0, None, dtable, "f32")
    want, bound = R.embedding_backward(dout, ids, vocab, 1.0, None)
    R.assert_close(dtable, want, bound, "f32", "many tokens")
    again = torch.empty_like(dtable)
    back(dout, "f32", ids, vocab, 1.0, None, again, "f32")
    assert torch.equal(dtable, again), "two calls differ"


def test_embedding_gradient_is_the_differences():
    """<dout, E(table + d) - E(table)> = <dtable, d>: the lookup is linear in the table."""
    g = gen(11)
    vocab, dim, tokens = 50, 48, 200
    table, step = normal(g, vocab, dim), normal(g, vocab, dim)
    ids, dout = ids_of(g, tokens, vocab, 64), normal(g, tokens, dim)
    one, two, dtable = torch.empty(tokens, dim, device=DEV), torch.empty(tokens, dim, device=DEV), torch.empty(vocab, dim, device=DEV)
    cr.cr_embedding(table, vocab, ids, tokens, dim, "f32", 3.0, one, "f32")
    cr.cr_embedding(table + step, vocab, ids, tokens, dim, "f32", 3.0, two, "f32")
    back(dout, "f32", ids, vocab, 3.0, None, dtable, "f32")
    left = float(((two.double() - one.double()) * dout.double()).sum())
    right = float((dtable.double() * step.double()).sum())
    # every product rounds by U32 a few times
    size = float((two.double().abs() + one.double().abs()).mul(dout.double().abs()).sum())
    assert abs(left - right) <= 64 * R.U32 * size


# ---- dropout ---------------------------------------------------------------------------------

def rng_of(seed, offset):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (5, 513), (2, 2048), (33, 257), (40, 1000)])
def test_dropout(rows, cols, residual, dt, layout):
    extra, off = layout
    g = gen(rows * cols)
    seed, offset, call = 0xFEDCBA9876543210, 0xFFFFFFFFFFFFFFFE, 5  # the sum wraps
    x = place(normal(g, rows, cols, dt=dt), cols + extra, off)
    res = place(normal(g, rows, cols, dt=dt), cols + extra, off) if residual else None
    out, buf = padded(rows, cols, dt, cols + extra, off)
    cr.cr_dropout(x, res, rows, cols, dt, 0.3, rng_of(seed, offset), call, 1000, out)
    want, bound = R.dropout(x, res, 0.3, R.numbers_fast(rows, cols, seed, offset + call, 1000))
    R.assert_close(out, want, bound, dt, "dropout")
    untouched(out, buf, rows, cols, cols + extra, off)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [512, 1001])
def test_dropout_in_place_and_slabs(dt, cols):
    """out on x, out on the residual, and slabs of rows give the same bits."""
    g = gen(3)
    rows, rng = 70, rng_of(9, 4)
    x, res = normal(g, rows, cols, dt=dt), normal(g, rows, cols, dt=dt)
    out = torch.empty_like(x)
    cr.cr_dropout(x, res, rows, cols, dt, 0.5, rng, 0, 0, out)
    a, b, c = x.clone(), res.clone(), torch.empty_like(x)
    cr.cr_dropout(a, res, rows, cols, dt, 0.5, rng, 0, 0, a)
    cr.cr_dropout(x, b, rows, cols, dt, 0.5, rng, 0, 0, b)
    for lo, hi in ((0, 1), (1, 33), (33, 70)):
        cr.cr_dropout(x[lo:hi], res[lo:hi], hi - lo, cols, dt, 0.5, rng, 0, lo, c[lo:hi])
    for t in (a, b, c):
        assert torch.equal(t, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 65])
def test_dropout_extremes(dt, cols):
    """p = 0 keeps and p = 1 drops everything; a dropped NaN or infinity leaves the residual."""
    g = gen(4)
    rows, rng = 9, rng_of(1, 2)
    x, res = normal(g, rows, cols, dt=dt), normal(g, rows, cols, dt=dt)
    out = torch.empty_like(x)
    cr.cr_dropout(x, None, rows, cols, dt, 0.0, rng, 0, 0, out)
    assert torch.equal(out, x)
    x[0], x[1] = math.nan, math.inf
    cr.cr_dropout(x, res, rows, cols, dt, 1.0, rng, 0, 0, out)
    assert torch.equal(out, res)
    cr.cr_dropout(x, res, rows, cols, dt, 0.5, rng, 0, 0, out)
    keep = R.numbers_fast(rows, cols, 1, 2).to(DEV) >= 32768
    assert torch.equal(torch.isnan(out[0]), keep[0]) and torch.equal(torch.isinf(out[1]), keep[1])
    assert torch.equal(out[~keep], res[~keep])


def test_dropout_share_and_gradient():
    """The share that is kept is binomial, and the call on a gradient is the transpose."""
    g = gen(8)
    rows, cols, p, rng = 400, 1000, 0.1, rng_of(77, 0)
    x, dout = normal(g, rows, cols), normal(g, rows, cols)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    cr.cr_dropout(x, None, rows, cols, "f32", p, rng, 1, 0, y)
    cr.cr_dropout(dout, None, rows, cols, "f32", p, rng, 1, 0, dx)
    n = rows * cols
    share = float((y != 0).sum()) / n
    assert abs(share - (1 - R.limit_of(p) / 65536)) < 6 * math.sqrt(p * (1 - p) / n)
    left, right = float((y.double() * dout.double()).sum()), float((x.double() * dx.double()).sum())
    assert abs(left - right) <= 4 * R.U32 * float((y.double() * dout.double()).abs().sum())
    other = torch.empty_like(x)
    cr.cr_dropout(x, None, rows, cols, "f32", p, rng, 2, 0, other)
    both = float(((y != 0) & (other != 0)).sum()) / n
    q = 1 - R.limit_of(p) / 65536
    assert abs(both - q * q) < 6 * math.sqrt(q * q * (1 - q * q) / n), "two calls' masks depend on each other"


# ---- log probabilities -----------------------------------------------------------------------

def forward(logits, targets, dt, scale, top=0, entropy=True):
    r, v = logits.shape
    logp, ent, lse = (torch.full((r,), 99.0, device=DEV) for _ in range(3))
    ids = torch.full((r, top), -7, dtype=torch.int32, device=DEV)
    tl = torch.full((r, top), 99.0, device=DEV)
    cr.cr_log_probs(logits, targets, r, v, dt, scale, logp if targets is not None else None,
                    ent if entropy else None, lse, top, ids if top else None, tl if top else None)
    return logp, ent, lse, ids, tl


def check_forward(logits, targets, dt, scale, top, what=""):
    logp, ent, lse, ids, tl = forward(logits, targets, dt, scale, top)
    w_logp, w_ent, w_lse, logs, bound, ent_bound = R.log_probs(logits, targets, scale)
    R.assert_close(logp, w_logp, R.logp_bound(w_logp, bound), "f32", what + " logp")
    R.assert_close(lse, w_lse, bound + 2 * R.U32 * torch.nan_to_num(w_lse.abs(), posinf=0), "f32", what + " lse")
    R.assert_close(ent, w_ent, ent_bound, "f32", what + " entropy")
    if top:
        want = R.top(logits, top)
        assert torch.equal(ids, want), f"{what} top ids: {(ids != want).sum()} differ"
        w_tl = logs.gather(1, want.long())
        R.assert_close(tl, w_tl, R.logp_bound(w_tl, bound[:, None]), "f32", what + " top logp")


VOCABS = [1, 2, 31, 257, 1000, 2048, 2049, 4099, 20000, 50257]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_log_probs(vocab, dt, layout):
    extra, off = layout
    g = gen(vocab)
    for rows, top in ((1, min(vocab, 20)), (7, min(vocab, 32)), (200, min(vocab, 5))):
        logits = place(normal(g, rows, vocab, std=3.0, dt=dt), vocab + extra, off)
        targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        if rows == 7:
            targets[1], targets[2] = -1, vocab
        check_forward(logits, targets.to(torch.int32) if extra else targets, dt, 1.0 if off else 0.7, top, f"rows {rows}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(3, 700), (400, 700), (2, 40000), (700, 5000)])
def test_log_probs_outputs_alone(rows, vocab, dt):
    """Each output without the others has the same bits."""
    g = gen(rows)
    logits = normal(g, rows, vocab, std=2.0, dt=dt)
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    logp, ent, lse, ids, tl = forward(logits, targets, dt, 1.0, 9)
    outs = {"logp": logp, "entropy": ent, "lse": lse}
    for name, want in outs.items():
        got = torch.empty(rows, device=DEV)
        cr.cr_log_probs(logits, targets if name == "logp" else None, rows, vocab, dt, 1.0,
                        **{"logp": None, name: got})
        assert torch.equal(got, want), name
    for name, want in (("top_ids", ids), ("top_logp", tl)):
        got = torch.empty_like(want)
        cr.cr_log_probs(logits, None, rows, vocab, dt, 1.0, None, top=9, **{name: got})
        assert torch.equal(got, want), name


def hard_rows(g, vocab, dt):
    """Rows on which a selection or a sum may go wrong."""
    rows = []
    base = torch.randn(vocab, generator=g, device=DEV)
    rows.append(torch.zeros(vocab, device=DEV))                              # all equal
    rows.append(torch.full((vocab,), -math.inf, device=DEV))                 # nothing left
    one = torch.full((vocab,), -math.inf, device=DEV)
    one[vocab // 2] = 2.0                                                    # one token left
    rows.append(one)
    few = torch.full((vocab,), -math.inf, device=DEV)
    few[vocab // 3::max(1, vocab // 4)] = base[vocab // 3::max(1, vocab // 4)]  # a few left
    rows.append(few)
    rows.append(torch.arange(vocab, device=DEV).float() * 1e-3)              # rising
    rows.append(-torch.arange(vocab, device=DEV).float() * 1e-3)             # falling
    lowest = torch.full((vocab,), -3.0e38, device=DEV)
    lowest[::7] = base[::7]                                                  # masked with the type's lowest value
    rows.append(lowest)
    rows.append(torch.full((vocab,), torch.finfo(TORCH[dt]).min, device=DEV))  # and nothing else
    rows.append((base * 2).round() / 2)                                      # few values, many ties
    sign = torch.zeros(vocab, device=DEV)
    sign[::2] = -0.0
    rows.append(sign)                                                        # zeros of both signs
    big = base.clone()
    big[vocab - 1] = 300.0                                                   # one far above
    rows.append(big)
    # the largest ones in the columns of few threads of 256 reading 16-byte vectors
    crowd = base - 50
    per = 8 if dt == "bf16" else 4
    col = torch.arange(vocab, device=DEV)
    crowd[(col // per) % 256 == 3] += 100
    rows.append(crowd)
    rows.append(base * 60)                                                   # sharp
    return torch.stack(rows).to(TORCH[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 300, 2048, 5003, 40000, 131072])
@pytest.mark.parametrize("copies", [1, 16])
def test_log_probs_of_hard_rows(vocab, dt, copies):
    g = gen(vocab)
    logits = hard_rows(g, vocab, dt).repeat(copies, 1)
    targets = torch.randint(0, vocab, (logits.shape[0],), generator=g, device=DEV)
    for top in (0, 1, 20, 32):
        check_forward(logits, targets, dt, 1.0, top, f"top {top}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,threads", [(3, 2048, 32), (2, 20000, 256), (2, 262144, 256), (700, 30000, 128)])
def test_log_probs_of_crowded_rows(rows, vocab, threads, dt):
    """The large logits of a row all in the columns of a few threads that read 16-byte vectors side by
    side: more of them than a list holds reach any bound that the threads' largest ones give."""
    g = gen(vocab)
    per = 8 if dt == "bf16" else 4
    col = torch.arange(vocab, device=DEV)
    logits = normal(g, rows, vocab)
    logits[:, (col // per) % threads < threads // 4] += 40.0
    logits = logits.to(TORCH[dt])
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    check_forward(logits, targets, dt, 1.0, 32, "crowded")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [50, 3001, 40000])
def test_log_probs_not_finite(vocab, dt):
    """NaN and +infinity make a row's numbers NaN, and no other row's; NaN ranks last."""
    g = gen(2)
    logits = normal(g, 5, vocab, dt=dt)
    logits[1, vocab // 2] = math.nan
    logits[2, 3] = math.inf
    logits[3] = math.nan
    targets = torch.zeros(5, dtype=torch.int64, device=DEV)
    logp, ent, lse, ids, tl = forward(logits, targets, dt, 1.0, 32)
    for t in (logp, ent, lse):
        assert torch.isnan(t).tolist() == [False, True, True, True, False]
    assert torch.equal(ids, R.top(logits, 32))
    few = torch.full((2, vocab), math.nan, device=DEV, dtype=TORCH[dt])
    few[0, 7], few[0, 9], few[1, 11] = -math.inf, 1.0, -math.inf
    assert torch.equal(forward(few, None, dt, 1.0, 20)[3], R.top(few, 20))


# ---- their gradient ----------------------------------------------------------------------------

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("parts", ["logp", "entropy", "lse", "all"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 31), (9, 1000), (2, 20001), (300, 513)])
def test_log_probs_backward(rows, vocab, parts, dt, layout):
    extra, off = layout
    g = gen(rows + vocab)
    logits = place(normal(g, rows, vocab, std=3.0, dt=dt), vocab + extra, off)
    if rows > 2:
        logits[1, :vocab // 2] = -math.inf
        logits[2] = -math.inf
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    if rows > 5:
        targets[4], targets[5] = -1, vocab
    _, ent, lse, _, _ = forward(logits, targets, dt, 0.8)
    d, e, q = (normal(g, rows) if parts in (name, "all") else None for name in ("logp", "entropy", "lse"))
    out, buf = padded(rows, vocab, dt, vocab + extra, off)
    cr.cr_log_probs_backward(logits, targets if d is not None else None, rows, vocab, dt, 0.8, lse,
                             ent if e is not None else None, d, e, q, out)
    want, bound = R.log_probs_backward(logits, targets, 0.8, lse, ent, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")
    untouched(out, buf, rows, vocab, vocab + extra, off)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, 0.8, lse, ent, d, e, q, logits)
    assert torch.equal(logits, out), "in place"


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 2048, 5003])
def test_log_probs_backward_of_hard_rows(vocab, dt):
    g = gen(vocab)
    logits = hard_rows(g, vocab, dt)
    rows = logits.shape[0]
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    _, ent, lse, _, _ = forward(logits, targets, dt, 1.0)
    d, e, q = (normal(g, rows) for _ in range(3))
    out = torch.empty_like(logits)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, 1.0, lse, ent, d, e, q, out)
    want, bound = R.log_probs_backward(logits, targets, 1.0, lse, ent, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")


def test_log_probs_gradient_is_the_differences():
    """Forward and backward calls against each other: the loss's change along a direction,
    from 64-bit differences of the formula at the point whose gradient the call gives, and
    from the call's own outputs at a step large enough for fp32."""
    g = gen(21)
    rows, vocab = 6, 500
    x, step = normal(g, rows, vocab), normal(g, rows, vocab)
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    d, e, q = (normal(g, rows) for _ in range(3))
    logp, ent, lse, _, _ = forward(x, targets, "f32", 1.3)
    dx = torch.empty_like(x)
    cr.cr_log_probs_backward(x, targets, rows, vocab, "f32", 1.3, lse, ent, d, e, q, dx)
    slope = float((dx.double() * step.double()).sum())

    def loss(t):
        lp, en, ls, _, _, _ = R.log_probs(t, targets, 1.3)
        return float((lp * d + en * e + ls * q).sum())
    h = 1e-5
    want = (loss(x.double() + h * step.double()) - loss(x.double() - h * step.double())) / (2 * h)
    assert abs(slope - want) <= 1e-5 * float((dx.double() * step.double()).abs().sum())
    h = 2.0 ** -6

    def measured(sign):
        lp, en, ls, _, _ = forward(x + sign * h * step, targets, "f32", 1.3)
        return float((lp.double() * d + en.double() * e + ls.double() * q).sum())
    # central differences are off by h^2/6 of the third derivative, a few units here
    assert abs((measured(1) - measured(-1)) / (2 * h) - slope) <= 64 * h * h


# ---- repeats, streams, graphs --------------------------------------------------------------------

def calls(g):
    """Every operator on fixed buffers: functions of no argument, and their outputs."""
    tokens, vocab, dim = 1500, 3000, 520
    table, ids = normal(g, vocab, dim, dt="bf16"), skewed(g, tokens, vocab)
    emb, drop = (torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dtable = torch.empty(vocab, dim, dtype=torch.bfloat16, device=DEV)
    work = torch.empty(cr.cr_embedding_backward_workspace_bytes(tokens, vocab, dim), dtype=torch.uint8, device=DEV)
    rng = rng_of(5, 6)
    logits = normal(g, tokens, vocab, std=2.0, dt="bf16")
    logp, ent, lse, tl = (torch.empty(n, device=DEV) for n in (tokens, tokens, tokens, tokens * 8))
    ti = torch.empty(tokens * 8, dtype=torch.int32, device=DEV)
    d = normal(g, tokens)
    dx = torch.empty_like(logits)
    # few rows, which clusters of blocks share
    wide = normal(g, 3, 70001, std=2.0, dt="f32")
    few, fi = torch.empty(3, device=DEV), torch.empty(3, 20, dtype=torch.int32, device=DEV)
    return [
        (cr.cr_log_probs, (wide, None, 3, 70001, "f32", 1.0, None, few, None, 20, fi)),
        (cr.cr_embedding, (table, vocab, ids, tokens, dim, "bf16", 2.0, emb, "bf16")),
        (cr.cr_dropout, (emb, emb, tokens, dim, "bf16", 0.2, rng, 1, 0, drop)),
        (cr.cr_embedding_backward, (drop, "bf16", ids, tokens, vocab, dim, 2.0, None, dtable, "bf16", work, work.numel())),
        (cr.cr_log_probs, (logits, ids, tokens, vocab, "bf16", 1.0, logp, ent, lse, 8, ti, tl)),
        (cr.cr_log_probs_backward, (logits, ids, tokens, vocab, "bf16", 1.0, lse, ent, d, d, None, dx)),
    ], (emb, drop, dtable, logp, ent, lse, ti, tl, dx, few, fi), rng


def test_two_streams_at_once():
    """Calls in flight on two streams, with a workspace each."""
    one, outs, _ = calls(gen(41))
    two, outs2, _ = calls(gen(42))
    want = []
    for cases, o in ((one, outs), (two, outs2)):
        for fn, args in cases:
            fn(*args)
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for fn, args in one:
            fn(*args, stream=streams[0])
        for fn, args in two:
            fn(*args, stream=streams[1])
    torch.cuda.synchronize()
    for o, w in zip((outs, outs2), want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_repeats_streams_graphs_prepared():
    cases, outs, rng = calls(gen(31))
    for fn, args in cases:
        fn(*args)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]

    def same(what):
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), what
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
    same("first")
    for _ in range(3):
        for fn, args in cases:
            fn(*args)
    same("repeats")
    side = torch.cuda.Stream()
    for fn, args in cases:
        fn(*args, stream=side)
    same("another stream")
    with torch.cuda.stream(side):
        prepared = [cr.prepare(fn, *args) for fn, args in cases]
    for p in prepared:
        p()
    same("prepared")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for fn, args in cases:
            fn(*args)
    graph.replay()
    graph.replay()
    same("graph")
    # a captured step's masks follow the offset in device memory
    rng[1] += 1
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(outs[1], want[1])
    emb = want[0]
    nums = R.numbers_fast(*emb.shape, 5, 8)
    w, bound = R.dropout(emb, emb, 0.2, nums)
    R.assert_close(outs[1], w, bound, "bf16", "moved offset")
