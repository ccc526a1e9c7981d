"""examples/language_model_step.py: the language model operators, the feed-forward sublayer and the
FSDP step run together, and the model's gradients are those of torch's autograd on the same formulas
with the same dropout mask."""
import importlib.util
import math
import os

import pytest
import torch

import lm_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "language_model_step.py")
    spec = importlib.util.spec_from_file_location("language_model_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ranks,tokens,vocab,dim,ffn", [(4, 256, 300, 128, 256), (2, 100, 77, 72, 200)])
def test_training_runs_alike_on_all_ranks_and_twice(example, ranks, tokens, vocab, dim, ffn):
    losses, members = example.train(ranks, tokens, vocab, dim, ffn, steps=6)
    assert all(math.isfinite(x) for x in losses)
    for k in members[1:]:
        assert torch.equal(k.params, members[0].params)
    again, _ = example.train(ranks, tokens, vocab, dim, ffn, steps=6)
    assert again == losses


def test_gradients_are_autograds(example):
    """fp32 autograd on the same bf16 parameters.  The chain rounds activations and their
    gradients to bf16 (2^-8) about ten times over, and three checkpoints to e4m3, half a step of 2^-4 at most, about a
    third of that in the root mean square: 2^-4 of a gradient's norm holds both."""
    tokens, vocab, dim, ffn = 200, 150, 96, 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    flat = example.start(vocab, dim, ffn, gen).to(torch.bfloat16)
    rank = example.Rank(flat, tokens, vocab, dim, ffn, seed=77)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    ids[190:], targets[185:] = -1, -1
    dlogp = torch.randn(tokens, generator=gen, device="cuda") / tokens
    logp = rank.forward(ids, targets).clone()
    rank.backward(ids, targets, dlogp)

    leaf = flat.float().requires_grad_()
    p = example.views(leaf, vocab, dim, ffn)
    held = (ids >= 0)[:, None]
    x = p["table"][ids.clamp_min(0)] * held * dim ** 0.5
    norm = lambda h, w: h * torch.rsqrt(h.square().mean(1, keepdim=True) + example.EPS) * w
    y = norm(x, p["w1"])
    o = (torch.nn.functional.silu(y @ p["wg"].T) * (y @ p["wu"].T)) @ p["wd"].T
    limit = R.limit_of(example.DROP)
    keep = (R.numbers_fast(tokens, dim, 77, 0) >= limit).cuda()
    h = x + o * keep * (65536 / (65536 - limit))
    logs = torch.log_softmax(norm(h, p["w2"]) @ p["table"].T, 1)
    want = torch.where(targets >= 0, logs.gather(1, targets.clamp_min(0)[:, None])[:, 0], torch.zeros(tokens, device="cuda"))
    want.backward(dlogp)
    # logits of a few units carry about three roundings of 2^-8
    assert float((logp - want.detach()).abs().max()) < 16 * 2.0 ** -8
    assert float(logp[185:].abs().max()) == 0
    got, ref = example.views(rank.grads, vocab, dim, ffn), example.views(leaf.grad, vocab, dim, ffn)
    for name in got:
        off = float((got[name].float() - ref[name]).norm() / ref[name].norm())
        assert off < 2.0 ** -4, f"{name}: {off}"
