"""Forms of the feed-forward kernels that tests/test_ffn_gpu.py does not reach: rows
above 8192 columns on the vector grid, and every operator on rows that start on 16
but not on 32 bytes."""
import math

import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

ES = {"bf16": 2, "f32": 4, "u8": 1}
NAME = {torch.bfloat16: "bf16", torch.float32: "f32", torch.uint8: "u8"}


def sides(cols, dt):
    """Columns left and right of a matrix in its buffer, so that it starts 16 bytes into
    a row and rows are a multiple of 16 bytes apart."""
    left = 16 // ES[dt]
    return left, -(left + cols) % left


def in16(t):
    return T.strided(t, *sides(t.shape[1], NAME[t.dtype]), 0 if t.dtype == torch.uint8 else math.nan)


def out16(rows, cols, dt):
    left, right = sides(cols, dt)
    out, wide = T.empty(rows, cols, dt, left, right)
    assert out.data_ptr() % 32 == 16 and wide.stride(0) * ES[dt] % 16 == 0
    return out, lambda: T.untouched(wide, left, cols)


def q16(rows, cols):
    codes, check = out16(rows, cols, "u8")
    scales = torch.full((rows, R.groups(cols)), math.nan, device="cuda")
    return cr.Q8(codes, scales), codes, scales, check


# ---- more than 8192 columns ---------------------------------------------------------------------

WIDE = [(1, 8208), (3, 12288), (130, 12288), (2, 12290), (2, 16384), (70, 20000)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", WIDE)
def test_rms_norm_wide(rows, cols, residual, dt):
    T.test_rms_norm(rows, cols, residual, dt)


@pytest.mark.parametrize("dt,dw_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("rows,cols", WIDE)
def test_rms_norm_backward_wide(rows, cols, held, dt, dw_dt):
    T.test_rms_norm_backward(rows, cols, held, dt, dw_dt)


@pytest.mark.parametrize("over", ["dy", "dres", "h"])
def test_rms_norm_backward_wide_in_place_and_alone(over):
    T.test_rms_norm_backward_in_place_and_alone(12288, over)


@pytest.mark.parametrize("over", ["x", "residual"])
def test_rms_norm_wide_in_place(over):
    T.test_rms_norm_in_place(12288, over)


# ---- rows on 16 bytes ---------------------------------------------------------------------------

SHAPES = [(3, 128), (7, 272), (5, 1000), (300, 384), (4, 2048), (33, 4097), (2, 8192), (3, 12288)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_q8_on_16_bytes(rows, cols, dt):
    g = T.gen(rows * 7 + cols)
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(
        torch.randint(-12, 12, (rows, cols), generator=g, device="cuda").float())
    v[torch.rand(rows, cols, generator=g, device="cuda") < 0.05] = 0
    v[rows // 2, :128] = 0
    if cols > 200:
        v[0, 5], v[0, 130], v[-1, 7] = math.inf, -math.inf, math.nan
    v = v.to(R.TORCH[dt])
    q, codes, scales, check = q16(rows, cols)
    cr.cr_q8_store(in16(v), rows, cols, dt, q)
    R.assert_q8(codes, scales, v.double())
    check()
    for out in ("bf16", "f32"):
        x, check = out16(rows, cols, out)
        cr.cr_q8_load(q, rows, cols, x, out)
        want = R.decode(codes, scales).float().to(R.TORCH[out])
        assert torch.equal(torch.nan_to_num(x, 1e9), torch.nan_to_num(want, 1e9))
        check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rms_norm_on_16_bytes(rows, cols, residual, dt):
    g = T.gen(rows + cols)
    x = T.rand(g, rows, cols, dt, 3.0)
    res = T.rand(g, rows, cols, dt) if residual else None
    w = (1 + T.rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])
    s, check_s = out16(rows, cols, dt)
    y, check_y = out16(rows, cols, dt)
    rstd = torch.empty(rows, device="cuda")
    q, codes, scales, check_q = q16(rows, cols)
    cr.cr_rms_norm(in16(x), in16(res) if residual else None, in16(w)[0], rows, cols, dt, T.EPS,
                   s if residual else None, y, q, rstd)
    T.check_norm(x, res, w[0], dt, T.EPS, {"y": y, "y8": (codes, scales), "rstd": rstd,
                                           **({"sum": s} if residual else {})})
    for check in (check_s, check_y, check_q):
        check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rms_norm_backward_on_16_bytes(rows, cols, held, dt):
    g = T.gen(rows * 3 + cols)
    h = T.rand(g, rows, cols, dt, 2.0)
    dy, dres = T.rand(g, rows, cols, dt, 1e-2), T.rand(g, rows, cols, dt, 1e-2)
    w = (1 + T.rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])
    rstd = R.norm(h, None, w[0], T.EPS)[1].float()
    q, hv = None, h
    if held == "q8":
        q, codes, scales, _ = q16(rows, cols)
        cr.cr_q8_store(h, rows, cols, dt, q)
        hv = R.decode(codes, scales)
    need = cr.cr_rms_norm_backward_workspace_bytes(rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    for res in (dres, None):
        dx, check = out16(rows, cols, dt)
        dw = torch.empty(cols, device="cuda")
        cr.cr_rms_norm_backward(in16(dy), in16(h) if held == "full" else None, q, in16(w)[0], rstd,
                                None if res is None else in16(res), rows, cols, dt, dx, dw, "f32",
                                work, need)
        want_dx, want_dw, mag, mag_dw = R.norm_backward(dy, hv, w[0], rstd, res)
        rel = (R.norm_depth(cols) + 8) * R.U32
        assert torch.all((dx.double() - want_dx).abs()
                         <= R.U_OUT[dt] * want_dx.abs() * (1 + rel) + rel * (mag + want_dx.abs()))
        rel_dw = (rows + 8) * R.U32
        assert torch.all((dw.double() - want_dw).abs()
                         <= R.U32 * want_dw.abs() * (1 + rel_dw) + rel_dw * mag_dw)
        check()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_act_backward_on_16_bytes(rows, cols, kind):
    g = T.gen(rows + 2 * cols)
    q, codes, scales, _ = q16(rows, cols)
    p, codes2, scales2, _ = q16(rows, cols)
    cr.cr_q8_store(T.rand(g, rows, cols, "f32", 3.0), rows, cols, "f32", q)
    cr.cr_q8_store(T.rand(g, rows, cols, "f32"), rows, cols, "f32", p)
    gv, uv = R.decode(codes, scales), R.decode(codes2, scales2)
    da = T.rand(g, rows, cols, "bf16")
    outs = [out16(rows, cols, "bf16") for _ in range(3)]
    cr.cr_glu_act_backward(in16(da), q, p, rows, cols, "bf16", kind, *[o for o, _ in outs])
    want = R.glu_act_backward(da, gv, uv, kind)
    # as in tests/test_ffn_gpu.py
    scale = [da.double().abs() * uv.abs() * (1 + gv.abs()), da.double().abs() * gv.abs(),
             gv.abs() * uv.abs()]
    for (out, check), ref, mag in zip(outs, want, scale):
        assert torch.all((out.double() - ref).abs() <= R.U16 * ref.abs() + 2.0 ** -18 * mag)
        check()


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("dim", [8, 512, 1000, 2056])
def test_few_tokens_on_16_bytes(tokens, dim):
    """The block that streams its weights: they start 16 bytes into a row."""
    T.check_glu(tokens, dim, 320, "silu", 8, -(8 + dim) % 8)
