"""What include/cr_ffn.h says of the accuracy of cr_glu_backward's results: dg and du enter
the products as one bf16 number each (dx, and dwg and dwu of more than 64 tokens,
whatever dw_dtype) or as two (dwg and dwu of at most 64).

Rounding to bf16 is off by U16 / sqrt 3 in the root mean square at most, so one rounded
operand adds at most that part of a result's norm, however many terms a sum has, and a
result rounded to bf16 as much again.  Two parts leave U16^2 = 2^-16 of dg, of x's
checkpoint and of the product of what both left; the activation is within 2^-18 of its
terms and a sum of 64 within 2^-17: less than 2^-14 together."""
import math

import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

ONE = R.U16 / math.sqrt(3)  # a rounding to bf16


@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("dw_dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 16, 64, 65, 257, 2048])
def test_accuracy_of_the_blocks_gradients(tokens, dw_dt, held):
    dim, ffn, g = 264, 520, T.gen(tokens)
    x, da = T.rand(g, tokens, dim, "bf16"), T.rand(g, tokens, ffn, "bf16")
    wg, wu = (T.rand(g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    q, gv = T.store(T.rand(g, tokens, ffn, "f32"))
    p, uv = T.store(T.rand(g, tokens, ffn, "f32"))
    x8, xv = (None, x.double()) if held == "full" else T.store(x)
    work = torch.empty(cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    dwg, dwu = (torch.empty(ffn, dim, device="cuda", dtype=R.TORCH[dw_dt]) for _ in range(2))
    cr.cr_glu_backward(da, q, p, x if held == "full" else None, x8, wg, wu, tokens, dim, ffn, "bf16", "silu",
                       dx, dwg, dwu, dw_dt, None, work, work.numel())
    dg, du, _ = R.glu_act_backward(da, gv, uv, "silu")
    assert R.rel_norm(dx, dg @ wg.double() + du @ wu.double()) <= math.sqrt(2) * ONE
    operand, result = (ONE if tokens > 64 else 0), (ONE if dw_dt == "bf16" else 0)
    for got, want in ((dwg, dg.T @ xv), (dwu, du.T @ xv)):
        assert R.rel_norm(got, want) <= math.hypot(operand, result) + 2.0 ** -14
