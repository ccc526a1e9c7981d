"""The 64-bit gradient of tests/lm_grad_ref.py without a GPU: it is autograd's, and a constant added to a
row leaves it alone, however large."""
import math

import torch

import lm_grad_ref as G
import lm_ref as R


def case():
    g = torch.Generator().manual_seed(7)
    x = torch.randn(6, 50, generator=g, dtype=torch.float64) * 2
    x[1, ::3] = -math.inf
    t = torch.randint(0, 50, (6,), generator=g)
    t[1], t[4], t[5] = 1, -1, 50
    return x, t, *(torch.randn(6, generator=g, dtype=torch.float64) for _ in range(3))


def test_reference_is_autograds():
    x, t, d, e, q = case()
    x.requires_grad_()
    logs = torch.log_softmax(x * 0.5, 1)
    p = logs.exp()
    ent = -torch.where(p > 0, p * logs.clamp_min(-1e30), torch.zeros_like(p)).sum(1)
    chosen = torch.where(R.valid(t, 50), logs.gather(1, t.clamp(0, 49)[:, None])[:, 0], torch.zeros_like(ent))
    (chosen * d + ent * e + torch.logsumexp(x * 0.5, 1) * q).sum().backward()
    want, _ = G.gradient(x.detach(), t, 0.5, d, e, q)
    left = ~torch.isinf(x.detach())
    assert torch.allclose(x.grad[left], want[left], rtol=1e-10, atol=1e-12)
    assert bool((want[~left] == 0).all())


def test_reference_of_shifted_rows():
    x, t, d, e, q = case()
    x = (x * 64).round() / 64  # exact beside the shifts
    want, _ = G.gradient(x, t, 1.0, d, e, q)
    for c in (-2.0 ** 30, 300.0, 2.0 ** 40):
        assert torch.equal(G.gradient(x + c, t, 1.0, d, e, q)[0], want)
    alike, _ = G.gradient(torch.full((6, 50), -1e9), t, 1.0, d, None, None)
    d = torch.where(R.valid(t, 50), d, torch.zeros_like(d))
    assert torch.allclose(alike.sum(1), torch.zeros(6, dtype=torch.float64), atol=1e-15)
    assert torch.allclose(alike[:, 2], -d / 50 + torch.where(t == 2, d, torch.zeros_like(d)))
