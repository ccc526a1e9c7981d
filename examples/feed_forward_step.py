"""Data-parallel training steps of a feed-forward sublayer on one GPU.

N emulated ranks hold the same bf16 parameters and train on different tokens.
Every rank runs the sublayer

    h = x + r;  y = rms_norm(h) * w;  a = act(y Wg^T) * (y Wu^T);  out = h + a Wd^T

against a target, keeping y, gate and up as 8-bit checkpoints between forward
and backward, and leaves its bf16 gradients in its flat buffer.  One FSDP step
(reduce-scatter, AdamW on the fp32 shards, all-gather) then updates the
parameters of all ranks.

    python examples/feed_forward_step.py [--ranks 4] [--tokens 512] [--dim 256]
                                         [--ffn 1024] [--steps 20]
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
BF16 = {"device": "cuda", "dtype": torch.bfloat16}


def views(flat: torch.Tensor, dim: int, ffn: int) -> dict:
    """The sublayer's parameters (or their gradients) inside a rank's flat buffer."""
    sizes = {"w": (dim,), "wg": (ffn, dim), "wu": (ffn, dim), "wd": (dim, ffn)}
    out, at = {}, 0
    for name, shape in sizes.items():
        n = 1
        for s in shape:
            n *= s
        out[name] = flat[at:at + n].view(shape)
        at += n
    assert at == flat.numel()
    return out


def q8(rows: int, cols: int) -> cr.Q8:
    return cr.Q8(torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                 torch.empty(rows, -(-cols // cr.Q8_GROUP), device="cuda"))


class Rank:
    """One rank's parameters, gradients and activations."""

    def __init__(self, params: torch.Tensor, tokens: int, dim: int, ffn: int):
        self.tokens, self.dim, self.ffn = tokens, dim, ffn
        self.params, self.grads = params.clone(), torch.empty_like(params)
        self.p, self.g = views(self.params, dim, ffn), views(self.grads, dim, ffn)
        self.h, self.y = (torch.empty(tokens, dim, **BF16) for _ in range(2))
        self.a, self.da = (torch.empty(tokens, ffn, **BF16) for _ in range(2))
        self.dy, self.dx = (torch.empty(tokens, dim, **BF16) for _ in range(2))
        self.rstd = torch.empty(tokens, device="cuda")
        self.y8, self.gate8, self.up8 = q8(tokens, dim), q8(tokens, ffn), q8(tokens, ffn)
        need = max(cr.cr_glu_workspace_bytes(tokens, dim, ffn),
                   cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn),
                   cr.cr_rms_norm_backward_workspace_bytes(tokens, dim))
        self.work = torch.empty(need, dtype=torch.uint8, device="cuda")

    def forward(self, x: torch.Tensor, r: torch.Tensor) -> torch.Tensor:
        t, d, f, work = self.tokens, self.dim, self.ffn, self.work
        cr.cr_rms_norm(x, r, self.p["w"], t, d, "bf16", EPS, self.h, self.y, self.y8, self.rstd)
        # y lives on as its checkpoint only: backward does not read it
        cr.cr_glu(self.y, self.p["wg"], self.p["wu"], t, d, f, "bf16", "silu", self.a, self.gate8,
                  self.up8, work, work.numel())
        return self.h.float() + (self.a @ self.p["wd"].T).float()

    def backward(self, dout: torch.Tensor) -> None:
        """dout: the loss's gradient at the sublayer's output, bf16."""
        t, d, f, work = self.tokens, self.dim, self.ffn, self.work
        torch.matmul(dout, self.p["wd"], out=self.da)
        cr.cr_glu_backward(self.da, self.gate8, self.up8, None, self.y8, self.p["wg"], self.p["wu"],
                           t, d, f, "bf16", "silu", self.dy, self.g["wg"], self.g["wu"], "bf16",
                           self.a, work, work.numel())  # `a` recomputed from the checkpoints
        torch.matmul(dout.T, self.a, out=self.g["wd"])
        # dx: the gradient for the layer below, the residual stream's part added
        cr.cr_rms_norm_backward(self.dy, self.h, None, self.p["w"], self.rstd, dout, t, d, "bf16",
                                self.dx, self.g["w"], "bf16", work, work.numel())


def train(ranks: int = 4, tokens: int = 512, dim: int = 256, ffn: int = 1024, steps: int = 20,
          lr: float = 3e-3, seed: int = 0) -> tuple[list[float], list[Rank]]:
    """Mean loss of every step, and the ranks after the last one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    count = dim + 3 * dim * ffn
    master = torch.cat([torch.ones(dim, device="cuda"), normal(2 * dim * ffn, std=dim ** -0.5),
                        normal(dim * ffn, std=ffn ** -0.5)])
    params = master.to(torch.bfloat16)
    shards = [cr.cr_shard_range(count, ranks, j) for j in range(ranks)]
    masters = [master[lo:hi].clone() for lo, hi in shards]
    m, v = ([torch.zeros(hi - lo, device="cuda") for lo, hi in shards] for _ in range(2))
    members = [Rank(params, tokens, dim, ffn) for _ in range(ranks)]
    data = [[normal(tokens, dim).to(torch.bfloat16) for _ in range(3)] for _ in range(ranks)]
    losses = []
    for step in range(1, steps + 1):
        total = torch.zeros((), device="cuda")
        for rank, (x, r, target) in zip(members, data):
            diff = rank.forward(x, r) - target.float()
            total += diff.square().mean()
            rank.backward((2.0 / diff.numel() * diff).to(torch.bfloat16))
        cr.cr_fsdp_step([k.grads for k in members], count, masters, m, v,
                        cr.adamw_cfg(lr=lr, weight_decay=0.0, step=step),
                        [k.params for k in members])
        losses.append(float(total) / ranks)
        if cr.cr_glu_wait_word():
            raise RuntimeError(f"step {step}: a wait of the gated block ran out, its gradients are undefined")
    return losses, members


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("ranks", 4), ("tokens", 512), ("dim", 256), ("ffn", 1024), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    losses, _ = train(args.ranks, args.tokens, args.dim, args.ffn, args.steps)
    for k, loss in enumerate(losses, 1):
        print(f"step {k:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
