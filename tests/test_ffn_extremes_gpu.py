"""The gate's activation and its slope at magnitudes where they have saturated, up to
the largest finite ones: there act(g) is g or 0 and act'(g) is 1 or 0, to 64 bits."""
import math

import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

# |g|^2 passes fp32's range from 1.8e19 on, |g|^3 from 7e12 on
MAGNITUDES = [200.0, 1e4, 1e12, 1e13, 1e19, 2e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("left", [0, 3])  # vectors, and rows off the vector grid
def test_slope_of_saturated_gates(kind, left):
    """A row for each magnitude, of either sign; the checkpoint's own values are the gate's."""
    rows, cols, g = len(MAGNITUDES), 300, T.gen(1)
    sign = torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    gate = sign * torch.tensor(MAGNITUDES, device="cuda")[:, None]
    q, gv = T.store(gate)
    p, uv = T.store(torch.rand(rows, cols, generator=g, device="cuda") * 0.5)
    da = T.rand(g, rows, cols, "bf16", 1e-3)
    outs = [T.empty(rows, cols, "bf16", left, 0)[0] for _ in range(3)]
    cr.cr_glu_act_backward(T.strided(da, left, 0), q, p, rows, cols, "bf16", kind, *outs)
    on = gv > 0
    zero = torch.zeros_like(gv)
    d = da.double()
    want = (torch.where(on, d * uv, zero), torch.where(on, d * gv, zero), torch.where(on, gv * uv, zero))
    for got, ref in zip(outs, want):
        # bf16's rounding and a few fp32 ones
        assert torch.all((got.double() - ref).abs() <= (R.U16 + 2.0 ** -18) * ref.abs())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_slope_of_a_nan_gate(kind):
    codes = torch.tensor([[0x7F, 0xFF, 0x38]], device="cuda").to(torch.uint8)
    ones = torch.full((1, 3), 0x38, device="cuda").to(torch.uint8)  # 1.0
    scale = torch.ones(1, 1, device="cuda")
    outs = [torch.zeros(1, 3, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    cr.cr_glu_act_backward(torch.ones(1, 3, device="cuda", dtype=torch.bfloat16), cr.Q8(codes, scale),
                           cr.Q8(ones, scale), 1, 3, "bf16", kind, *outs)
    for out in outs:
        assert torch.isnan(out[0, :2]).all() and math.isfinite(float(out[0, 2]))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 200])
def test_block_of_saturated_gates(tokens, kind):
    """x = (magnitude, 1): the gate is +- the magnitude, up is 1/2, every sum exact."""
    mags = torch.tensor(MAGNITUDES, device="cuda").to(torch.bfloat16)
    for at in range(0, len(MAGNITUDES), tokens):
        m = mags[(torch.arange(tokens, device="cuda") + at) % len(MAGNITUDES)]
        x = torch.stack([m, torch.ones_like(m)], 1).contiguous()
        ffn = 130
        wg, wu = (torch.zeros(ffn, 2, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        wg[0::2, 0], wg[1::2, 0], wu[:, 1] = 1.0, -1.0, 0.5
        need = cr.cr_glu_workspace_bytes(tokens, 2, ffn)
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        a = torch.empty(tokens, ffn, device="cuda", dtype=torch.bfloat16)
        cr.cr_glu(x, wg, wu, tokens, 2, ffn, "bf16", kind, a, None, None, work, need)
        want = torch.zeros(tokens, ffn, dtype=torch.float64, device="cuda")
        want[:, 0::2] = 0.5 * m.double()[:, None]
        assert torch.all((a.double() - want).abs() <= (R.U16 + 2.0 ** -18) * want)
