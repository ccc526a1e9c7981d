"""The scales of log probabilities: every one that the calls take, from fp32's smallest to 2^126."""
import pytest
import torch

import lm_grad_ref as G
import lm_ref as R
import test_lm_abi as A
import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import build as libbuild
from fsdp_emulated_ranks_gb300 import cr

MOST, LEAST = 2.0 ** 126, 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def test_scale_limits():
    above = float(torch.nextafter(torch.tensor(MOST), torch.tensor(float("inf"))))
    for fn in (A.logp, A.logp_back):
        for bad in (above, 2.0 ** 127, float("inf"), 0.0, LEAST / 4, -LEAST):
            A.expect(1, fn, scale=bad)
        for good in (MOST, LEAST):
            fn(rows=0, scale=good)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [33, 2049, 40000])
@pytest.mark.parametrize("scale", [LEAST, 1e-39, 2.0 ** -126, 1e20, MOST])
def test_extreme_scales(scale, vocab, dt):
    g = T.gen(vocab)
    rows = 5
    logits = (torch.rand(rows, vocab, generator=g, device="cuda") * 2 - 1).to(R.TORCH[dt])
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    T.check_forward(logits, targets, dt, scale, min(vocab, 9))
    _, ent, lse, _, _ = T.forward(logits, targets, dt, scale)
    d, e, q = (T.normal(g, rows) for _ in range(3))
    if scale == MOST:  # its products with the gradients stay finite
        d, e, q = d / 1024, e / 1024, q / 1024
    out = torch.empty_like(logits)
    cr.cr_log_probs_backward(logits, targets, rows, vocab, dt, scale, lse, ent, d, e, q, out)
    want, bound = G.gradient(logits, targets, scale, d, e, q)
    R.assert_close(out, want, bound, dt, "dlogits")


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [33, 40000])
def test_products_past_the_end(vocab):
    """lse and far tokens' logp become infinite; the others' logp, the entropy and the order do not."""
    g = T.gen(vocab)
    logits = (torch.rand(4, vocab, generator=g, device="cuda") * 2.0 ** -20 + 1).float()
    logits[:, 5], logits[:, 9] = 4.0, 4.0
    logits[1] *= -1
    logits[3] *= -1
    targets = torch.tensor([9, 20, 7, 5], device="cuda")
    logp, ent, lse, ids, tl = T.forward(logits, targets, "f32", MOST, 4)
    inf = float("inf")
    assert lse[[0, 2]].tolist() == [inf, inf] and bool((lse[[1, 3]] < -2.0 ** 125).all())
    half = torch.tensor(0.5).log()
    assert abs(float(logp[0]) - half) < 1e-6 and abs(float(ent[0]) + half) < 1e-6
    assert float(logp[3]) < -2.0 ** 127 and bool((logp[1:3] < -2.0 ** 100).all())
    assert torch.equal(ids, R.top(logits, 4))
    assert not bool(torch.isnan(torch.cat([logp, ent, lse, tl.flatten()])).any())
