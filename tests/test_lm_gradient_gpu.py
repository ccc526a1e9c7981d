"""The gradient of log probabilities where the row's lse, rounded to fp32, says little of its
probabilities, against the formula from the logits alone (tests/lm_grad_ref.py derives the bound)."""
import math

import pytest
import torch

import lm_grad_ref as G
import lm_ref as R
import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import cr
from lm_ref import TORCH

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from fsdp_emulated_ranks_gb300 import build
    build.build()


def far_rows(g, vocab, dt):
    """Rows of a large lse, either sign, with ordinary ones between."""
    base = torch.randn(vocab, generator=g, device=DEV)
    some = torch.full((vocab,), -math.inf, device=DEV)
    some[vocab // 2:] = base[vocab // 2:] + 1e4
    masked = torch.full((vocab,), -1e9, device=DEV)
    masked[::3] = base[::3]
    rows = [torch.full((vocab,), c, device=DEV) for c in (-1e9, -1e4, 0.0, 1e4, 1e8, -1e30, 3e38)]
    rows += [base + c for c in (-300.0, 255.0, 300.0, -1e4, 1e6)]
    rows += [some, masked, base * 1000, base.abs() * 1e30, base * 1e3 - 1e9, base]
    return torch.stack(rows).to(TORCH[dt])


def check(logits, targets, dt, scale, d, e, q, layout=(0, 0)):
    rows, vocab = logits.shape
    extra, off = layout
    _, ent, lse, _, _ = T.forward(logits, targets, dt, scale)
    out, buf = T.padded(rows, vocab, dt, vocab + extra, off)
    cr.cr_log_probs_backward(logits, targets if d is not None else None, rows, vocab, dt, scale, lse,
                             ent if e is not None else None, d, e, q, out)
    want, bound = G.gradient(logits, targets, scale, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")
    T.untouched(out, buf, rows, vocab, vocab + extra, off)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, scale, lse, ent, d, e, q, logits)
    assert torch.equal(logits, out), "in place"


@pytest.mark.parametrize("layout", T.LAYOUTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("parts", ["logp", "entropy", "lse", "all"])
@pytest.mark.parametrize("vocab", [1, 31, 513, 5003])
def test_rows_of_a_large_lse(vocab, parts, dt, layout):
    g = T.gen(vocab)
    logits = far_rows(g, vocab, dt)
    rows = logits.shape[0]
    logits = T.place(logits, vocab + layout[0], layout[1])
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    targets[1], targets[7] = -1, vocab
    d, e, q = (T.normal(g, rows) if parts in (name, "all") else None for name in ("logp", "entropy", "lse"))
    check(logits, targets, dt, 1.0, d, e, q, layout)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.3, 2.0])
@pytest.mark.parametrize("copies,vocab", [(1, 40000), (1, 200001), (300, 700)])
def test_rows_of_a_large_lse_many_and_long(copies, vocab, scale, dt):
    """Rows more than the blocks that look for them, and longer than one reads at once; a scale that takes the
    logits past the type's end (an lse of infinity)."""
    g = T.gen(copies + vocab)
    logits = far_rows(g, vocab, dt).repeat(copies, 1)
    rows = logits.shape[0]
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    d, e, q = (T.normal(g, rows) for _ in range(3))
    check(logits, targets, dt, scale, d, e, q)


def test_rows_of_a_large_lse_in_a_graph():
    """A captured call follows the rows that it finds when it is replayed."""
    g = T.gen(5)
    rows, vocab = 40, 3000
    x = T.normal(g, rows, vocab)
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    d = T.normal(g, rows)
    logp, ent, lse = (torch.empty(rows, device=DEV) for _ in range(3))
    dx = torch.empty_like(x)

    def step():
        cr.cr_log_probs(x, targets, rows, vocab, "f32", 1.0, logp, ent, lse)
        cr.cr_log_probs_backward(x, targets, rows, vocab, "f32", 1.0, lse, ent, d, d, None, dx)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shift in (0.0, 1e4, -1e9):
        x[::3] += shift
        dx.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want, bound = G.gradient(x, targets, 1.0, d, d, None)
        R.assert_close(dx, want, bound, "f32", f"shift {shift}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 1001, 5003])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_without_tokens_get_zeros(bad, vocab, dt):
    """Whatever the gradients of their numbers: a z-loss gives such a row dlse = 2 c lse = -infinity, a ratio of
    its probabilities dlogp = NaN."""
    g = T.gen(vocab)
    rows = 6
    logits = T.normal(g, rows, vocab, dt=dt)
    logits[1], logits[4] = -math.inf, torch.finfo(TORCH[dt]).min
    targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    _, ent, lse, _, _ = T.forward(logits, targets, dt, 1.0)
    d, e, q = (T.normal(g, rows) for _ in range(3))
    want, bound = G.gradient(logits, targets, 1.0, d, e, q)
    for which in ((0,), (1,), (2,), (0, 1, 2)):
        terms = [t.clone() for t in (d, e, q)]
        for k in which:
            terms[k][1] = terms[k][4] = bad
        out = torch.full_like(logits, math.nan)
        cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, 1.0, lse, ent, *terms, out)
        assert bool((out[1] == 0).all()) and bool((out[4] == 0).all()), f"{which} {bad}"
        R.assert_close(out, want, bound, dt, "dlogits")
    dlse = 2e-4 * lse
    out = torch.full_like(logits, math.nan)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, 1.0, lse, None, d, None, dlse, out)
    dlse = torch.where(torch.isinf(dlse), torch.zeros_like(dlse), dlse)
    want, bound = G.gradient(logits, targets, 1.0, d, None, dlse)
    R.assert_close(out, want, bound, dt, "z-loss")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 1001, 5003])
def test_ruled_out_tokens_get_zeros(vocab, dt):
    """Also where the entropy's gradient is large: 0 log(0) is 0 times any finite number."""
    g = T.gen(vocab)
    rows = 6
    logits = T.normal(g, rows, vocab, dt=dt)
    logits[:, ::3] = -math.inf
    logits[2:4] += 1e4  # a large lse
    targets = 1 + 3 * torch.randint(0, vocab // 3, (rows,), generator=g, device=DEV)
    _, ent, lse, _, _ = T.forward(logits, targets, dt, 1.0)
    d, q = T.normal(g, rows), T.normal(g, rows)
    e = torch.tensor([1.0, 1e9, -1e10, 1e20, -1e30, 1e35], device=DEV)
    out = torch.full_like(logits, math.nan)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, 1.0, lse, ent, d, e, q, out)
    assert bool((out[:, ::3] == 0).all())
    want, bound = G.gradient(logits, targets, 1.0, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")
