"""examples/feed_forward_step.py: the feed-forward operators and the FSDP step
run together, and the sublayer's gradients are those of torch's autograd on the
same formulas."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "feed_forward_step.py")
    spec = importlib.util.spec_from_file_location("feed_forward_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ranks,tokens,dim,ffn", [(4, 256, 128, 384), (3, 100, 72, 200)])
def test_training_lowers_the_loss_alike_on_all_ranks(example, ranks, tokens, dim, ffn):
    losses, members = example.train(ranks, tokens, dim, ffn, steps=15)
    assert losses[-1] < 0.8 * losses[0], losses
    for k in members[1:]:
        assert torch.equal(k.params, members[0].params)
    again, _ = example.train(ranks, tokens, dim, ffn, steps=15)
    assert again == losses


def test_gradients_are_autograds(example):
    """fp32 autograd on the same bf16 parameters.  The calls round activations to
    bf16 (2^-8) and the checkpoints to e4m3, half a step of 2^-4 at most, about a
    third of that in the root mean square of either factor of a gradient: 2^-4 of
    a gradient's norm holds both with room for bf16."""
    tokens, dim, ffn = 200, 96, 256
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std
    flat = torch.cat([1 + normal(dim, std=0.1), normal(2 * dim * ffn, std=dim ** -0.5),
                      normal(dim * ffn, std=ffn ** -0.5)]).to(torch.bfloat16)
    rank = example.Rank(flat, tokens, dim, ffn)
    x, r, dout = (normal(tokens, dim).to(torch.bfloat16) for _ in range(3))
    out = rank.forward(x, r)
    rank.backward(dout)
    leaf = flat.float().requires_grad_()
    xin = x.float().requires_grad_()
    p = example.views(leaf, dim, ffn)
    h = xin + r.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + example.EPS) * p["w"]
    a = torch.nn.functional.silu(y @ p["wg"].T) * (y @ p["wu"].T)
    want = h + a @ p["wd"].T
    want.backward(dout.float())
    want = want.detach()
    assert float((out - want).norm() / want.norm()) < 2.0 ** -7
    for got, ref in ((rank.grads, leaf.grad), (rank.dx, xin.grad)):
        assert float((got.float() - ref).norm() / ref.norm()) < 2.0 ** -4
