"""Data-parallel training steps of a small language model on one GPU.

N emulated ranks hold the same bf16 parameters and train on different tokens.  Every rank runs

    x = scale * table[ids];  y = rms_norm(x) w1;  a = act(y Wg^T) * (y Wu^T)
    h = x + dropout(a Wd^T);  logits = (rms_norm(h) w2) table^T
    loss = -mean over the targets of log softmax(logits)[target]

(no attention: a token predicts the next from itself), with the table at both ends: the head's
gradient of it comes from a matrix product, and the embedding's is added to that in place.  The last
places of each rank's batch hold no token.  One FSDP step then updates the parameters of all ranks.

    python examples/language_model_step.py [--ranks 4] [--tokens 512] [--vocab 1000] [--dim 256]
                                           [--ffn 512] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

from fsdp_emulated_ranks_gb300 import cr

EPS = 1e-6
DROP = 0.1
BF16 = {"device": "cuda", "dtype": torch.bfloat16}


def views(flat: torch.Tensor, vocab: int, dim: int, ffn: int) -> dict:
    """The model's parameters (or their gradients) inside a rank's flat buffer."""
    shapes = {"table": (vocab, dim), "wg": (ffn, dim), "wu": (ffn, dim), "wd": (dim, ffn), "w1": (dim,), "w2": (dim,)}
    out, at = {}, 0
    for name, shape in shapes.items():
        n = torch.Size(shape).numel()
        out[name] = flat[at:at + n].view(shape)
        at += n
    assert at == flat.numel()
    return out


class Rank:
    """One rank's parameters, gradients and activations."""

    def __init__(self, params: torch.Tensor, tokens: int, vocab: int, dim: int, ffn: int, seed: int):
        self.sizes = tokens, vocab, dim, ffn
        self.params, self.grads = params.clone(), torch.empty_like(params)
        self.p, self.g = views(self.params, vocab, dim, ffn), views(self.grads, vocab, dim, ffn)
        self.x, self.y, self.h, self.z, self.o, self.dx, self.dy, self.dz = (
            torch.empty(tokens, dim, **BF16) for _ in range(8))
        self.a, self.da = (torch.empty(tokens, ffn, **BF16) for _ in range(2))
        self.logits = torch.empty(tokens, vocab, **BF16)
        self.rstd1, self.rstd2, self.logp, self.lse = (torch.empty(tokens, device="cuda") for _ in range(4))
        q8 = lambda cols: cr.Q8(torch.empty(tokens, cols, dtype=torch.uint8, device="cuda"),
                                torch.empty(tokens, -(-cols // cr.Q8_GROUP), device="cuda"))
        self.y8, self.gate8, self.up8 = q8(dim), q8(ffn), q8(ffn)
        # dropout's seed, and an offset that moves by a step's dropout calls: one
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
        need = max(cr.cr_glu_workspace_bytes(tokens, dim, ffn), cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn),
                   cr.cr_rms_norm_backward_workspace_bytes(tokens, dim),
                   cr.cr_embedding_backward_workspace_bytes(tokens, vocab, dim))
        self.work = torch.empty(need, dtype=torch.uint8, device="cuda")

    def forward(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Log probabilities of the targets (0 where there is none)."""
        t, v, d, f = self.sizes
        p, work = self.p, self.work
        cr.cr_embedding(p["table"], v, ids, t, d, "bf16", d ** 0.5, self.x, "bf16")
        cr.cr_rms_norm(self.x, None, p["w1"], t, d, "bf16", EPS, None, self.y, self.y8, self.rstd1)
        cr.cr_glu(self.y, p["wg"], p["wu"], t, d, f, "bf16", "silu", self.a, self.gate8, self.up8, work, work.numel())
        torch.matmul(self.a, p["wd"].T, out=self.o)
        cr.cr_dropout(self.o, self.x, t, d, "bf16", DROP, self.rng, 0, 0, self.h)
        cr.cr_rms_norm(self.h, None, p["w2"], t, d, "bf16", EPS, None, self.z, None, self.rstd2)
        torch.matmul(self.z, p["table"].T, out=self.logits)
        cr.cr_log_probs(self.logits, targets, t, v, "bf16", 1.0, self.logp, None, self.lse)
        return self.logp

    def backward(self, ids: torch.Tensor, targets: torch.Tensor, dlogp: torch.Tensor) -> None:
        t, v, d, f = self.sizes
        p, g, work = self.p, self.g, self.work
        cr.cr_log_probs_backward(self.logits, targets, t, v, "bf16", 1.0, self.lse, None, dlogp, None, None,
                                 self.logits)  # in place
        torch.matmul(self.logits, p["table"], out=self.dz)
        torch.matmul(self.logits.T, self.z, out=g["table"])
        cr.cr_rms_norm_backward(self.dz, self.h, None, p["w2"], self.rstd2, None, t, d, "bf16", self.dz, g["w2"], "bf16",
                                work, work.numel())
        cr.cr_dropout(self.dz, None, t, d, "bf16", DROP, self.rng, 0, 0, self.o)  # the gradient of a Wd^T
        torch.matmul(self.o, p["wd"], out=self.da)
        cr.cr_glu_backward(self.da, self.gate8, self.up8, None, self.y8, p["wg"], p["wu"], t, d, f, "bf16", "silu",
                           self.dy, g["wg"], g["wu"], "bf16", self.a, work, work.numel())
        torch.matmul(self.o.T, self.a, out=g["wd"])
        cr.cr_rms_norm_backward(self.dy, self.x, None, p["w1"], self.rstd1, self.dz, t, d, "bf16", self.dx, g["w1"],
                                "bf16", work, work.numel())
        cr.cr_embedding_backward(self.dx, "bf16", ids, t, v, d, d ** 0.5, g["table"], g["table"], "bf16", work,
                                 work.numel())


def start(vocab: int, dim: int, ffn: int, gen: torch.Generator) -> torch.Tensor:
    """The fp32 parameters, flat."""
    normal = lambda n, std: torch.randn(n, generator=gen, device="cuda") * std
    return torch.cat([normal(vocab * dim, dim ** -0.5), normal(2 * dim * ffn, dim ** -0.5), normal(dim * ffn, ffn ** -0.5),
                      torch.ones(2 * dim, device="cuda")])


def train(ranks: int = 4, tokens: int = 512, vocab: int = 1000, dim: int = 256, ffn: int = 512, steps: int = 20,
          lr: float = 3e-3, seed: int = 0) -> tuple[list[float], list[Rank]]:
    """Mean loss of every step, and the ranks after the last one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    master = start(vocab, dim, ffn, gen)
    count = master.numel()
    members = [Rank(master.to(torch.bfloat16), tokens, vocab, dim, ffn, 1000 + r) for r in range(ranks)]
    shards = [cr.cr_shard_range(count, ranks, j) for j in range(ranks)]
    masters = [master[lo:hi].clone() for lo, hi in shards]
    m, v = ([torch.zeros(hi - lo, device="cuda") for lo, hi in shards] for _ in range(2))
    # every token has one successor: something to learn
    after = torch.randperm(vocab, generator=gen, device="cuda")
    used = tokens - tokens // 8
    data = []
    for _ in range(ranks):
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        targets = after[ids]
        ids[used:], targets[used:] = -1, -1
        data.append((ids, targets))
    dlogp = torch.full((tokens,), -1.0 / used, device="cuda")
    losses = []
    for step in range(1, steps + 1):
        total = torch.zeros((), device="cuda")
        for rank, (ids, targets) in zip(members, data):
            total -= rank.forward(ids, targets).sum() / used
            rank.backward(ids, targets, dlogp)
            rank.rng[1] += 1
        cr.cr_fsdp_step([k.grads for k in members], count, masters, m, v,
                        cr.adamw_cfg(lr=lr, weight_decay=0.0, step=step), [k.params for k in members])
        losses.append(float(total) / ranks)
        if cr.cr_glu_wait_word():
            raise RuntimeError(f"step {step}: a wait of the gated block ran out, its gradients are undefined")
    return losses, members


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("ranks", 4), ("tokens", 512), ("vocab", 1000), ("dim", 256), ("ffn", 512), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    losses, _ = train(args.ranks, args.tokens, args.vocab, args.dim, args.ffn, args.steps)
    for k, loss in enumerate(losses, 1):
        print(f"step {k:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
