"""Matrices of more than 2^32 elements: offsets that pass 32 bits in every feed-forward
operator.  Rows from the beginning, either side of the offsets 2^31 and 2^32 and the end
are compared with the same call on those rows alone, which reads and writes the same
values in the same order."""
import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

BF16 = {"dtype": torch.bfloat16, "device": "cuda"}


def looked_at(rows, cols):
    """Row numbers at which the offsets pass 2^31 and 2^32 elements, and the ends."""
    at = {0, 1, rows - 1}
    for k in (31, 32):
        r = (1 << k) // cols
        at |= {r - 1, r, r + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < rows), device="cuda")


def filled(rows, cols, dtype, seed):
    """Random rows, repeated with a period that is no divisor of the powers of two."""
    some = torch.randn(997, cols, generator=T.gen(seed), device="cuda").to(dtype)
    out = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for lo in range(0, rows, 997):
        n = min(997, rows - lo)
        out[lo:lo + n] = some[:n]
    out[:, 0] = (torch.arange(rows, device="cuda") % 251).to(dtype)
    return out


def q8(rows, cols):
    return (torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
            torch.empty(rows, R.groups(cols), device="cuda"))


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


# aligned rows in registers, odd rows staged, wide rows
@pytest.mark.parametrize("rows,cols", [(2_100_100, 2048), (2_100_100, 2049), (262_200, 16400)])
def test_norm_and_checkpoints(rows, cols):
    x = filled(rows, cols, torch.bfloat16, 1)
    w = torch.randn(cols, generator=T.gen(2), device="cuda").to(torch.bfloat16)
    at = looked_at(rows, cols)
    few, n = x[at].contiguous(), len(at)
    y, rstd, (codes, scales) = torch.empty_like(x), torch.empty(rows, device="cuda"), q8(rows, cols)
    cr.cr_rms_norm(x, None, w, rows, cols, "bf16", T.EPS, None, y, cr.Q8(codes, scales), rstd)
    y2, rstd2, (codes2, scales2) = torch.empty_like(few), torch.empty(n, device="cuda"), q8(n, cols)
    cr.cr_rms_norm(few, None, w, n, cols, "bf16", T.EPS, None, y2, cr.Q8(codes2, scales2), rstd2)
    for got, want in ((y, y2), (rstd, rstd2), (codes, codes2), (scales, scales2)):
        assert torch.equal(got[at], want)
    # the checkpoint's load and store, then the backward pass from it, over y
    cr.cr_q8_load(cr.Q8(codes, scales), rows, cols, y, "bf16")
    assert torch.equal(y[at].float(), R.decode(codes2, scales2).float().to(torch.bfloat16).float())
    cr.cr_q8_store(x, rows, cols, "bf16", cr.Q8(codes, scales))
    cr.cr_q8_store(few, n, cols, "bf16", cr.Q8(codes2, scales2))
    assert torch.equal(codes[at], codes2) and torch.equal(scales[at], scales2)
    work = torch.empty(cr.cr_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    dw = torch.empty(cols, device="cuda")
    cr.cr_rms_norm_backward(x, None, cr.Q8(codes, scales), w, rstd, None, rows, cols, "bf16", y, dw, "f32", work,
                            work.numel())
    cr.cr_rms_norm_backward(few, None, cr.Q8(codes2, scales2), w, rstd2, None, n, cols, "bf16", y2, None)
    assert torch.equal(y[at], y2) and torch.isfinite(dw).all()
    cr.cr_rms_norm_backward(x, x, None, w, rstd, None, rows, cols, "bf16", y, None)
    cr.cr_rms_norm_backward(few, few, None, w, rstd2, None, n, cols, "bf16", y2, None)
    assert torch.equal(y[at], y2)


@pytest.mark.parametrize("ffn", [8192, 8200, 8193])
def test_block(ffn):
    """Few values of K, so that the tokens' side is what is large; a token's results do not
    depend on the others' (the tiles differ, the order of the sums does not at one K block)."""
    tokens, dim = 525_000, 32
    x = filled(tokens, dim, torch.bfloat16, 3)
    g = T.gen(4)
    wg, wu = (T.rand(g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    at = looked_at(tokens, ffn)
    few, n = x[at].contiguous(), len(at)
    work = torch.empty(cr.cr_glu_workspace_bytes(tokens, dim, ffn), dtype=torch.uint8, device="cuda")
    a, gate, up = torch.empty(tokens, ffn, **BF16), q8(tokens, ffn), q8(tokens, ffn)
    cr.cr_glu(x, wg, wu, tokens, dim, ffn, "bf16", "silu", a, cr.Q8(*gate), cr.Q8(*up), work, work.numel())
    a2, gate2, up2 = torch.empty(n, ffn, **BF16), q8(n, ffn), q8(n, ffn)
    cr.cr_glu(few, wg, wu, n, dim, ffn, "bf16", "silu", a2, cr.Q8(*gate2), cr.Q8(*up2), work, work.numel())
    for got, want in zip((a, *gate, *up), (a2, *gate2, *up2)):
        assert torch.equal(got[at], want)
    del work
    # the gate's part, `a` as da
    dg, du = torch.empty_like(a), torch.empty_like(a)
    cr.cr_glu_act_backward(a, cr.Q8(*gate), cr.Q8(*up), tokens, ffn, "bf16", "gelu", dg, du)
    dg2, du2 = torch.empty_like(a2), torch.empty_like(a2)
    cr.cr_glu_act_backward(a2, cr.Q8(*gate2), cr.Q8(*up2), n, ffn, "bf16", "gelu", dg2, du2)
    assert torch.equal(dg[at], dg2) and torch.equal(du[at], du2)
    # the whole backward pass; dx against the formula on the rows looked at
    work = torch.empty(cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty(ffn, dim, device="cuda"), torch.empty(ffn, dim, device="cuda")
    cr.cr_glu_backward(a, cr.Q8(*gate), cr.Q8(*up), x, None, wg, wu, tokens, dim, ffn, "bf16", "gelu", dx, dwg,
                       dwu, "f32", None, work, work.numel())
    want = dg2.double() @ wg.double() + du2.double() @ wu.double()
    mag = dg2.double().abs() @ wg.double().abs() + du2.double().abs() @ wu.double().abs()
    # the products take the same bf16 dg and du: the sum and the result's rounding are left
    assert torch.all((dx[at].double() - want).abs() <= R.U16 * want.abs() + 2 * R.U32 * (2 * ffn + 2) * mag)
    for got, d in ((dwg, dg), (dwu, du)):
        want = torch.zeros(ffn, dim, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(want)
        for lo in range(0, tokens, 16384):
            dd, xx = d[lo:lo + 16384].double(), x[lo:lo + 16384].double()
            want += dd.T @ xx
            mag += dd.abs().T @ xx.abs()
        assert torch.all((got.double() - want).abs() <= 2 * R.U32 * (tokens + 2) * mag)
    assert cr.cr_glu_wait_word() == 0
