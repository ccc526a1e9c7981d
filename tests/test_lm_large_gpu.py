"""Matrices of more than 2^32 elements in every language model operator: rows from the beginning,
either side of the offsets 2^31 and 2^32 and the end are compared with the formulas, or with the same
call on those rows alone."""
import pytest
import torch

import lm_ref as R
from fsdp_emulated_ranks_gb300 import cr
from test_ffn_large_gpu import filled, looked_at

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_embedding_of_a_large_table_and_its_gradient():
    vocab, dim = 2 ** 21, 2056
    table = filled(vocab, dim, BF16, 1)
    at = looked_at(vocab, dim)
    ids = at.repeat(3)
    out = torch.empty(len(ids), dim, dtype=BF16, device="cuda")
    cr.cr_embedding(table, vocab, ids, len(ids), dim, "bf16", 2.0, out, "bf16")
    assert torch.equal(out, table[ids] * 2)
    work = torch.empty(cr.cr_embedding_backward_workspace_bytes(len(ids), vocab, dim), dtype=torch.uint8, device="cuda")
    cr.cr_embedding_backward(out, "bf16", ids, len(ids), vocab, dim, 1.0, table, table, "bf16", work, work.numel())
    # base + 3 * (2 * base), rounded once: 7 base
    before = out[:len(at)].float() / 2
    assert torch.equal(table[at], (7 * before).to(BF16))
    near = (at[1:-1] + 7) % vocab
    assert torch.equal(table[near][:, 0], (near % 251).to(BF16)), "a row that no token names was touched"


def test_many_gradient_rows():
    tokens, dim, vocab = 2 ** 21 + 5, 2056, 3
    dout = filled(tokens, dim, BF16, 2)
    ids = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    at = looked_at(tokens, dim)
    ids[at] = (torch.arange(len(at), device="cuda") % vocab).to(torch.int32)
    dtable = torch.empty(vocab, dim, device="cuda")
    work = torch.empty(cr.cr_embedding_backward_workspace_bytes(tokens, vocab, dim), dtype=torch.uint8, device="cuda")
    cr.cr_embedding_backward(dout, "bf16", ids, tokens, vocab, dim, 1.0, None, dtable, "f32", work, work.numel())
    want, bound = R.embedding_backward(dout[at], ids[at], vocab, 1.0, None)
    R.assert_close(dtable, want, bound, "f32", "far rows")


def test_dropout_of_many_rows():
    rows, cols = 2 ** 21 + 3, 2056
    x = filled(rows, cols, BF16, 3)
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    want = {}
    at = looked_at(rows, cols).tolist()
    for r in at:
        row = torch.empty(1, cols, dtype=BF16, device="cuda")
        cr.cr_dropout(x[r:r + 1], x[r:r + 1], 1, cols, "bf16", 0.3, rng, 1, 7 + r, row)
        want[r] = row
    cr.cr_dropout(x, x, rows, cols, "bf16", 0.3, rng, 1, 7, x)
    for r in at:
        assert torch.equal(x[r:r + 1], want[r]), r


def test_log_probs_of_many_logits():
    """Rows with the same sums whatever is around them: each against a call on it alone."""
    rows, vocab = 2 ** 16 + 9, 66000
    x = filled(rows, vocab, BF16, 4)
    t = torch.arange(rows, device="cuda") % vocab
    lp, ent, lse = (torch.empty(rows, device="cuda") for _ in range(3))
    ti, tl = torch.empty(rows, 5, dtype=torch.int32, device="cuda"), torch.empty(rows, 5, device="cuda")
    cr.cr_log_probs(x, t, rows, vocab, "bf16", 1.0, lp, ent, lse, 5, ti, tl)
    at = looked_at(rows, vocab)
    some = x[at]
    w_lp, w_ent, w_lse, logs, bound, ent_bound = R.log_probs(some, t[at], 1.0)
    R.assert_close(lp[at], w_lp, R.logp_bound(w_lp, bound), "f32", "logp")
    R.assert_close(ent[at], w_ent, ent_bound, "f32", "entropy")
    R.assert_close(lse[at], w_lse, bound + 2 * R.U32 * w_lse.abs(), "f32", "lse")
    assert torch.equal(ti[at], R.top(some, 5))
    d = torch.full((rows,), 0.5, device="cuda")
    cr.cr_log_probs_backward(x, t, rows, vocab, "bf16", 1.0, lse, ent, d, d, None, x)
    want, bound = R.log_probs_backward(some, t[at], 1.0, lse[at], ent[at], d[at], d[at], None)
    R.assert_close(x[at], want, bound, "bf16", "dlogits")
