"""The gradients of the whole feed-forward sublayer, as the calls leave them, against
torch's 64-bit autograd and against differences (tests/ffn_grad_ref.py) -- and,
without a GPU, mistakes planted in an emulation of the calls, which those two
tests have to find."""
import pytest
import torch

import ffn_grad_ref as G
import ffn_ref as R

SIZES = [(48, 136, 200), (130, 264, 328)]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("seed", range(5))
def test_emulated_gradients_pass(kind, seed):
    s = G.inputs(torch.Generator().manual_seed(seed))
    got, held = G.emulate(s, kind)
    assert not G.off_formula(got, G.reference(s, held, kind))
    assert not G.off_differences(s, got, held, kind)


FOUND = {"dx without the mean": "dx", "dx 1.2 times": "dx", "dwg 1.2 times": "dwg", "dw without 4 rows": "dw",
         "dwu without 4 tokens": "dwu", "slope without its second term": "dwg", "dx a row off": "dx",
         "dw without rstd": "dw"}


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("mutation", G.MUTATIONS)
@pytest.mark.parametrize("seed", range(5))
def test_planted_mistakes_are_found(mutation, kind, seed):
    s = G.inputs(torch.Generator().manual_seed(seed))
    got, held = G.emulate(s, kind, mutation)
    assert FOUND[mutation] in G.off_formula(got, G.reference(s, held, kind))
    # terms left out of a sum are no scale and no direction of it: differences need not show them
    if "without 4" not in mutation:
        assert FOUND[mutation] in G.off_differences(s, got, held, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,dim,ffn", SIZES)
def test_gradients_of_the_sublayer(rows, dim, ffn, kind):
    import test_ffn_gpu as T
    from fsdp_emulated_ranks_gb300 import cr
    s = G.inputs(T.gen(rows), rows, dim, ffn)
    dev = {"device": "cuda", "dtype": torch.bfloat16}
    h, y, a = torch.empty(rows, dim, **dev), torch.empty(rows, dim, **dev), torch.empty(rows, ffn, **dev)
    rstd = torch.empty(rows, device="cuda")
    held = [T.new_q8(rows, cols)[:3] for cols in (dim, ffn, ffn)]
    y8, g8, u8 = (q for q, _, _ in held)
    work = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    cr.cr_rms_norm(s["x"], s["r"], s["w"], rows, dim, "bf16", G.EPS, h, y, y8, rstd)
    cr.cr_glu(y, s["wg"], s["wu"], rows, dim, ffn, "bf16", kind, a, g8, u8, work, work.numel())
    dy, dx, dw = torch.empty(rows, dim, **dev), torch.empty(rows, dim, **dev), torch.empty(dim, **dev)
    dwg, dwu = torch.empty(ffn, dim, **dev), torch.empty(ffn, dim, **dev)
    cr.cr_glu_backward(s["k"], g8, u8, None, y8, s["wg"], s["wu"], rows, dim, ffn, "bf16", kind, dy, dwg, dwu,
                       "bf16", None, work, work.numel())
    cr.cr_rms_norm_backward(dy, h, None, s["w"], rstd, None, rows, dim, "bf16", dx, dw, "bf16", work,
                            work.numel())
    got = dict(zip(G.NAMES, (dx, dw, dwg, dwu)))
    kept = dict(zip("ygu", (R.decode(c, sc) for _, c, sc in held)), h=h.double())
    assert not G.off_formula(got, G.reference(s, kept, kind))
    assert not G.off_differences(s, got, kept, kind)
