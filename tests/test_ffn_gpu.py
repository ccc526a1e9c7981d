"""The feed-forward operators of include/cr_ffn.h against their formulas in
64 bits (tests/ffn_ref.py, where the error bounds are derived)."""
import math

import pytest
import torch

import ffn_ref as R
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rand(gen, rows, cols, dt, std=1.0):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(R.TORCH[dt])


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(t, left, right, fill=float("nan")):
    """The same matrix inside a wider one whose other columns are NaN."""
    rows, cols = t.shape
    wide = torch.full((rows, left + cols + right), fill, device=t.device).to(t.dtype)
    wide[:, left:left + cols] = t
    return wide[:, left:left + cols]


def empty(rows, cols, dt, left=0, right=0):
    """An output and the buffer around it, filled with a pattern."""
    dtype = {**R.TORCH, "u8": torch.uint8}[dt]
    wide = torch.full((rows, left + cols + right), 77, device="cuda").to(dtype)
    return wide[:, left:left + cols], wide


def untouched(wide, left, cols):
    assert torch.all(wide[:, :left] == 77) and torch.all(wide[:, left + cols:] == 77)


def new_q8(rows, cols, left=0, right=0):
    codes, around = empty(rows, cols, "u8", left, right)
    scales = torch.full((rows, R.groups(cols)), math.nan, device="cuda")
    return cr.Q8(codes, scales), codes, scales, around


def store(v):
    """v's 8-bit form through the library, and the values it stands for."""
    rows, cols = v.shape
    q, codes, scales, _ = new_q8(rows, cols)
    cr.cr_q8_store(v, rows, cols, "f32" if v.dtype == torch.float32 else "bf16", q)
    return q, R.decode(codes, scales)


# ---- 8-bit matrices ---------------------------------------------------------------------

Q8_SHAPES = [(1, 1), (1, 127), (3, 128), (5, 129), (2, 256), (7, 257), (300, 384), (33, 1000),
             (4, 4096), (1025, 2731)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", Q8_SHAPES)
@pytest.mark.parametrize("left,right", [(0, 0), (16, 16), (3, 2)])
def test_q8_store_and_load(rows, cols, dt, left, right):
    g = gen(rows * 7 + cols)
    # magnitudes over many binades, exact zeros, a group of zeros, values that are not finite
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(
        torch.randint(-12, 12, (rows, cols), generator=g, device="cuda").float())
    v[torch.rand(rows, cols, generator=g, device="cuda") < 0.05] = 0
    v[rows // 2, : min(cols, 128)] = 0
    if cols > 200:
        v[0, 5], v[0, 130], v[-1, 7] = math.inf, -math.inf, math.nan
    v = v.to(R.TORCH[dt])
    q, codes, scales, around = new_q8(rows, cols, left, right)
    cr.cr_q8_store(strided(v, left, right), rows, cols, dt, q)
    R.assert_q8(codes, scales, v.double())
    untouched(around, left, cols)
    for out in ("bf16", "f32"):
        x, wide = empty(rows, cols, out, left, right)
        cr.cr_q8_load(q, rows, cols, x, out)
        want = R.decode(codes, scales).float().to(R.TORCH[out])
        assert torch.equal(torch.nan_to_num(x, 1e9), torch.nan_to_num(want, 1e9))
        untouched(wide, left, cols)


def test_q8_every_code():
    """Every code loads as the value its bits mean."""
    codes = torch.arange(256, device="cuda").to(torch.uint8).reshape(2, 128).contiguous()
    scales = torch.tensor([[1.0], [0.5]], device="cuda")
    x = torch.empty(2, 128, device="cuda")
    cr.cr_q8_load(cr.Q8(codes, scales), 2, 128, x, "f32")
    want = R.decode(codes, scales)
    assert torch.equal(torch.isnan(x), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(x.double(), 0), torch.nan_to_num(want, 0))


def test_q8_extremes():
    """fp32's largest, smallest normal and subnormal values keep a finite, positive scale."""
    top = torch.finfo(torch.float32).max
    v = torch.zeros(5, 128, device="cuda")
    v[0, :2] = torch.tensor([top, -top / 3])
    v[1, :2] = torch.tensor([2.0 ** -126, 2.0 ** -130])
    v[2, 3] = 2.0 ** -149
    v[3, :] = math.inf
    q, codes, scales, _ = new_q8(5, 128)
    cr.cr_q8_store(v, 5, 128, "f32", q)
    R.assert_q8(codes, scales, v.double())
    assert torch.isfinite(scales).all() and (scales > 0).all()


# ---- RMS norm --------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 2048), (2, 7), (3, 255), (5, 256), (4, 257), (9, 1000), (1, 1024),
               (17, 1111), (6, 2049), (5, 4096), (3, 5001), (2, 8192), (3, 8193), (2, 20011),
               (700, 64), (1300, 384)]


def check_norm(x, res, w, dt, eps, out, slack_terms=8):
    h, rstd, v = R.norm(x, res, w, eps)
    rows, cols = x.shape
    rel = (R.norm_depth(cols) / 2 + slack_terms) * R.U32
    if "sum" in out:
        assert torch.all((out["sum"].double() - h).abs() <= (R.U_OUT[dt] + R.U32) * h.abs())
    if "y" in out:
        assert torch.all((out["y"].double() - v).abs() <= (R.U_OUT[dt] * (1 + rel) + rel) * v.abs())
    if "y8" in out:
        R.assert_q8(*out["y8"], v, slack=rel * v.abs())
    if "rstd" in out:
        assert torch.all((out["rstd"].double() - rstd).abs() <= rel * rstd)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_rms_norm(rows, cols, residual, dt):
    g = gen(rows + cols)
    x = rand(g, rows, cols, dt, 3.0)
    res = rand(g, rows, cols, dt) if residual else None
    w = (1 + rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])[0]
    s = torch.empty_like(x) if residual else None
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q, codes, scales, _ = new_q8(rows, cols)
    cr.cr_rms_norm(x, res, w, rows, cols, dt, EPS, s, y, q, rstd)
    out = {"y": y, "y8": (codes, scales), "rstd": rstd}
    if residual:
        out["sum"] = s
    check_norm(x, res, w, dt, EPS, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 1111, 2048, 9000])
@pytest.mark.parametrize("left,right", [(16, 8), (1, 2)])
def test_rms_norm_strided_and_optional(cols, left, right, dt):
    """Row strides off the vector grid, NaN beside the matrix, each output alone."""
    rows, g = 5, gen(cols)
    x, res = rand(g, rows, cols, dt), rand(g, rows, cols, dt)
    w = rand(g, 1, cols, dt)[0]
    xs, rs = strided(x, left, right), strided(res, right, left)
    for which in ("sum", "y", "y8", "rstd"):
        s, wide_s = empty(rows, cols, dt, left, right)
        y, wide_y = empty(rows, cols, dt, left, right)
        rstd = torch.empty(rows, device="cuda")
        q, codes, scales, around = new_q8(rows, cols, left, right)
        cr.cr_rms_norm(xs, rs, w, rows, cols, dt, EPS, s if which == "sum" else None,
                       y if which == "y" else None, q if which == "y8" else None,
                       rstd if which == "rstd" else None)
        out = {"sum": s, "y": y, "y8": (codes, scales), "rstd": rstd}
        check_norm(x, res, w, dt, EPS, {which: out[which]})
        for wide in (wide_s, wide_y, around):
            untouched(wide, left, cols)


@pytest.mark.parametrize("cols", [100, 2048, 9001])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_rms_norm_in_place(cols, over):
    rows, g = 6, gen(cols)
    x, res, w = rand(g, rows, cols, "bf16"), rand(g, rows, cols, "bf16"), rand(g, 1, cols, "bf16")[0]
    a, b = x.clone(), res.clone()
    target = a if over == "x" else b
    y = torch.empty_like(x)
    cr.cr_rms_norm(a, b, w, rows, cols, "bf16", EPS, target, y)
    check_norm(x, res, w, "bf16", EPS, {"sum": target, "y": y})
    a, b = x.clone(), res.clone()
    target = a if over == "x" else b
    cr.cr_rms_norm(a, b, w, rows, cols, "bf16", EPS, None, target)
    check_norm(x, res, w, "bf16", EPS, {"y": target})


def test_rms_norm_special_rows():
    """A row of zeros, of huge and of tiny values, of NaN and of infinities: no row touches another."""
    cols = 300
    x = torch.ones(6, cols, device="cuda")
    x[1] = 0
    x[2] = 1e18
    x[3] = 1e-18
    x[4, 7] = math.nan
    x[5, 7] = math.inf
    w = torch.full((cols,), 2.0, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    q, codes, scales, _ = new_q8(6, cols)
    cr.cr_rms_norm(x, None, w, 6, cols, "f32", EPS, None, y, q, rstd)
    check_norm(x[:4], None, w, "f32", EPS, {"y": y[:4], "rstd": rstd[:4]})
    assert torch.isnan(y[4]).all() and (codes[4] == 0x7F).all()
    assert torch.isnan(y[5, 7]) and (y[5, :7] == 0).all() and codes[5, 7] == 0x7F
    cr.cr_rms_norm(x, None, w, 2, cols, "f32", 0.0, None, y)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all()


# rows off the vector grid: both sides of each width at which the kernels change, and more
# rows than the blocks that run at once
APART = [(3, 256), (2500, 257), (700, 511), (650, 512), (640, 513), (1300, 1025), (700, 4099),
         (330, 8191), (320, 8192)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", APART)
def test_rms_norm_rows_that_start_apart(rows, cols, residual, dt):
    """Every matrix at an alignment of its own, NaN beside the inputs."""
    g = gen(rows + cols)
    x = rand(g, rows, cols, dt, 3.0)
    res = rand(g, rows, cols, dt) if residual else None
    w = (1 + rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])
    s, wide_s = empty(rows, cols, dt, 2, 3)
    y, wide_y = empty(rows, cols, dt, 5, 1)
    rstd = torch.empty(rows, device="cuda")
    q, codes, scales, around = new_q8(rows, cols, 7, 2)
    cr.cr_rms_norm(strided(x, 1, 4), strided(res, 3, 3) if residual else None, strided(w, 1, 1)[0],
                   rows, cols, dt, EPS, s if residual else None, y, q, rstd)
    check_norm(x, res, w[0], dt, EPS, {"y": y, "y8": (codes, scales), "rstd": rstd,
                                       **({"sum": s} if residual else {})})
    untouched(wide_s, 2, cols)
    untouched(wide_y, 5, cols)
    untouched(around, 7, cols)


@pytest.mark.parametrize("dt,dw_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_rms_norm_backward(rows, cols, held, dt, dw_dt):
    g = gen(rows * 3 + cols)
    h = rand(g, rows, cols, dt, 2.0)
    dy, dres = rand(g, rows, cols, dt, 1e-2), rand(g, rows, cols, dt, 1e-2)
    w = (1 + rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])[0]
    rstd = R.norm(h, None, w, EPS)[1].float()
    q, hv = (None, h) if held == "full" else store(h)
    need = cr.cr_rms_norm_backward_workspace_bytes(rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    for with_res in (True, False):
        dx, dw = torch.empty_like(h), torch.empty(cols, dtype=R.TORCH[dw_dt], device="cuda")
        cr.cr_rms_norm_backward(dy, h if held == "full" else None, q, w, rstd,
                                dres if with_res else None, rows, cols, dt, dx, dw, dw_dt, work, need)
        want_dx, want_dw, mag, mag_dw = R.norm_backward(dy, hv, w, rstd, dres if with_res else None)
        rel = (R.norm_depth(cols) + 8) * R.U32
        assert torch.all((dx.double() - want_dx).abs()
                         <= R.U_OUT[dt] * want_dx.abs() * (1 + rel) + rel * (mag + want_dx.abs()))
        # a column's terms: one after another in a block, then the blocks' sums
        rel_dw = (rows + 8) * R.U32
        assert torch.all((dw.double() - want_dw).abs()
                         <= R.U_OUT[dw_dt] * want_dw.abs() * (1 + rel_dw) + rel_dw * mag_dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("rows,cols", APART)
def test_rms_norm_backward_rows_that_start_apart(rows, cols, held, dt):
    g = gen(rows * 3 + cols)
    h = rand(g, rows, cols, dt, 2.0)
    dy, dres = rand(g, rows, cols, dt, 1e-2), rand(g, rows, cols, dt, 1e-2)
    w = (1 + rand(g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])
    rstd = R.norm(h, None, w[0], EPS)[1].float()
    q, hv = None, h
    if held == "q8":
        _, codes, scales, _ = new_q8(rows, cols)
        cr.cr_q8_store(h, rows, cols, dt, cr.Q8(codes, scales))
        hv = R.decode(codes, scales)
        q = cr.Q8(strided(codes, 3, 6, 0), strided(scales, 1, 1))
    need = cr.cr_rms_norm_backward_workspace_bytes(rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    dx, wide = empty(rows, cols, dt, 2, 5)
    dw = torch.empty(cols, device="cuda")
    for res in (strided(dres, 7, 2), None):
        cr.cr_rms_norm_backward(strided(dy, 1, 2), strided(h, 5, 4) if held == "full" else None, q,
                                strided(w, 1, 1)[0], rstd, res, rows, cols, dt, dx, dw, "f32", work,
                                need)
        want_dx, want_dw, mag, mag_dw = R.norm_backward(dy, hv, w[0], rstd,
                                                        None if res is None else dres)
        rel = (R.norm_depth(cols) + 8) * R.U32
        assert torch.all((dx.double() - want_dx).abs()
                         <= R.U_OUT[dt] * want_dx.abs() * (1 + rel) + rel * (mag + want_dx.abs()))
        rel_dw = (rows + 8) * R.U32
        assert torch.all((dw.double() - want_dw).abs()
                         <= R.U32 * want_dw.abs() * (1 + rel_dw) + rel_dw * mag_dw)
        untouched(wide, 2, cols)


@pytest.mark.parametrize("cols", [77, 2048, 9001])
@pytest.mark.parametrize("over", ["dy", "dres", "h"])
def test_rms_norm_backward_in_place_and_alone(cols, over):
    rows, dt, g = 7, "bf16", gen(cols)
    h, dy, dres = (rand(g, rows, cols, dt) for _ in range(3))
    w = rand(g, 1, cols, dt)[0]
    rstd = R.norm(h, None, w, EPS)[1].float()
    need = cr.cr_rms_norm_backward_workspace_bytes(rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    cr.cr_rms_norm_backward(dy, h, None, w, rstd, dres, rows, cols, dt, dx, dw, "f32", work, need)
    alone = torch.empty_like(dx)
    cr.cr_rms_norm_backward(dy, h, None, w, rstd, dres, rows, cols, dt, alone, None)
    assert torch.equal(dx, alone)
    only = torch.empty_like(dw)
    cr.cr_rms_norm_backward(dy, h, None, w, rstd, None, rows, cols, dt, None, only, "f32", work, need)
    assert torch.equal(dw, only)
    t = {"dy": dy.clone(), "dres": dres.clone(), "h": h.clone()}
    again = torch.empty_like(dw)
    cr.cr_rms_norm_backward(t["dy"], t["h"], None, w, rstd, t["dres"], rows, cols, dt, t[over], again,
                            "f32", work, need)
    assert torch.equal(t[over], dx) and torch.equal(again, dw)
    xs = [strided(t, 3, 4) for t in (dy, h, dres)]
    out, wide = empty(rows, cols, dt, 1, 6)
    cr.cr_rms_norm_backward(xs[0], xs[1], None, w, rstd, xs[2], rows, cols, dt, out, again, "f32",
                            work, need)
    untouched(wide, 1, cols)
    want_dx, _, mag, _ = R.norm_backward(dy, h, w, rstd, dres)
    rel = (R.norm_depth(cols) + 8) * R.U32
    assert torch.all((out.double() - want_dx).abs() <= R.U16 * want_dx.abs() * (1 + rel)
                     + rel * (mag + want_dx.abs()))


def test_norm_backward_of_no_rows_is_zero():
    dw = torch.full((300,), 5.0, device="cuda")
    need = cr.cr_rms_norm_backward_workspace_bytes(0, 300)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    w = torch.ones(300, device="cuda")
    cr.cr_rms_norm_backward(None, None, None, w, None, None, 0, 300, "f32", None, dw, "f32", work, need)
    assert (dw == 0).all()


# ---- the gate's backward pass -----------------------------------------------------------------

@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 127), (2, 128), (5, 129), (130, 300),
                                       (65, 1024), (1025, 2731)])
@pytest.mark.parametrize("left,right", [(0, 0), (5, 2)])
def test_act_backward(rows, cols, kind, left, right):
    g = gen(rows + 2 * cols)
    q, codes, scales, _ = new_q8(rows, cols, left, right)
    p, codes2, scales2, _ = new_q8(rows, cols, left, right)
    cr.cr_q8_store(rand(g, rows, cols, "f32", 3.0), rows, cols, "f32", q)
    cr.cr_q8_store(rand(g, rows, cols, "f32"), rows, cols, "f32", p)
    gv, uv = R.decode(codes, scales), R.decode(codes2, scales2)
    da = rand(g, rows, cols, "bf16")
    outs = [empty(rows, cols, "bf16", left, right) for _ in range(3)]
    cr.cr_glu_act_backward(strided(da, left, right), q, p, rows, cols, "bf16", kind,
                           *[o[0] for o in outs])
    want = R.glu_act_backward(da, gv, uv, kind)
    # exp's argument and result are off by a few ulps; 1 - p cancels for large g,
    # where the slope's terms are up to (1 + |g|) in magnitude
    scale = [da.double().abs() * uv.abs() * (1 + gv.abs()), da.double().abs() * gv.abs(),
             gv.abs() * uv.abs()]
    for (out, wide), ref, mag in zip(outs, want, scale):
        assert torch.all((out.double() - ref).abs() <= R.U16 * ref.abs() + 2.0 ** -18 * mag)
        untouched(wide, left, cols)
    # each output over da itself, alone
    for k in range(3):
        t = da.clone()
        cr.cr_glu_act_backward(t, q, p, rows, cols, "bf16", kind, *[t if i == k else None for i in range(3)])
        assert torch.equal(t, outs[k][0])


@pytest.mark.parametrize("rows,cols", [(7, 1), (9, 100), (5, 255), (12, 257), (33, 513), (40, 1111)])
@pytest.mark.parametrize("offs", [(0, 1, 2), (5, 0, 3), (4, 4, 7)])
@pytest.mark.parametrize("over", [None, 0, 1, 2])
def test_act_backward_rows_that_start_apart(rows, cols, offs, over):
    """Inputs and outputs each at an alignment of their own, one of them over da: the bits of
    the aligned call."""
    g = gen(rows + cols)
    q, codes, scales, _ = new_q8(rows, cols)
    p, codes2, scales2, _ = new_q8(rows, cols)
    cr.cr_q8_store(rand(g, rows, cols, "f32", 2.0), rows, cols, "f32", q)
    cr.cr_q8_store(rand(g, rows, cols, "f32"), rows, cols, "f32", p)
    da = rand(g, rows, cols, "bf16")
    pad = (-cols) % 16 + 16
    want = [empty(rows, cols, "bf16", 0, pad)[0] for _ in range(3)]
    q2 = cr.Q8(strided(codes, 0, pad, 0), scales)
    p2 = cr.Q8(strided(codes2, 0, pad, 0), scales2)
    cr.cr_glu_act_backward(strided(da, 0, pad), q2, p2, rows, cols, "bf16", "gelu", *want)
    outs = [empty(rows, cols, "bf16", off, 3 + k) for k, off in enumerate(offs)]
    src = strided(da, 3, 2)
    if over is not None:
        outs[over][0].copy_(da)
        src = outs[over][0]
    cr.cr_glu_act_backward(src, cr.Q8(strided(codes, 1, 4, 0), scales), p, rows, cols, "bf16", "gelu",
                           *[o[0] for o in outs])
    for (out, wide), ref, off in zip(outs, want, offs):
        assert torch.equal(out, ref)
        untouched(wide, off, cols)


# ---- the gated block --------------------------------------------------------------------------

GLU_SHAPES = [(1, 1, 1), (1, 2048, 512), (2, 64, 128), (7, 63, 127), (16, 128, 256), (17, 65, 129),
              (127, 200, 300), (128, 64, 128), (129, 8, 257), (300, 513, 64), (257, 512, 1024),
              (64, 1024, 72), (5, 72, 2056), (1000, 96, 40), (33, 1, 200), (70, 300, 1)]


def glu_slack(x, w, terms):
    """fp32 error of x w^T: 2 U32 an addition."""
    return 2 * R.U32 * (terms + 2) * (x.double().abs() @ w.double().abs().T)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,dim,ffn", GLU_SHAPES)
def test_glu(tokens, dim, ffn, kind):
    check_glu(tokens, dim, ffn, kind, 0, 0)


@pytest.mark.parametrize("tokens,dim,ffn", [(1, 128, 256), (9, 70, 130), (140, 64, 200), (130, 136, 264)])
@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (3, 5)])
def test_glu_strided(tokens, dim, ffn, left, right):
    check_glu(tokens, dim, ffn, "silu", left, right)


def check_glu(tokens, dim, ffn, kind, left, right):
    g = gen(tokens + dim + ffn)
    x = rand(g, tokens, dim, "bf16")
    wg, wu = (rand(g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    need = cr.cr_glu_workspace_bytes(tokens, dim, ffn)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    gv, uv, av = R.glu(x, wg, wu, kind)
    eg, eu = glu_slack(x, wg, dim), glu_slack(x, wu, dim)
    for keep in (False, True):
        a, wide = empty(tokens, ffn, "bf16", left, right)
        q, gc, gs, wide_g = new_q8(tokens, ffn, left, right)
        p, uc, us, wide_u = new_q8(tokens, ffn, left, right)
        cr.cr_glu(strided(x, left, right), strided(wg, left, right), strided(wu, right, left), tokens,
                  dim, ffn, "bf16", kind, a, q if keep else None, p if keep else None, work, need)
        # |act'| <= 1.2, |act(g)| <= |g|
        slack = 1.2 * uv.abs() * eg + (gv.abs() + 1.2 * eg) * eu + 2.0 ** -18 * av.abs()
        assert torch.all((a.double() - av).abs() <= R.U16 * (av.abs() + slack) + slack)
        assert R.rel_norm(a, av) <= R.U16
        untouched(wide, left, ffn)
        if keep:
            R.assert_q8(gc, gs, gv, slack=eg, what="gate")
            R.assert_q8(uc, us, uv, slack=eu, what="up")
            for wide in (wide_g, wide_u):
                untouched(wide, left, ffn)


@pytest.mark.parametrize("tokens,dim,ffn", [(1, 256, 128), (5, 40, 130), (200, 256, 384), (129, 72, 72)])
def test_glu_integers_are_exact(tokens, dim, ffn):
    """Small integers: every sum is exact in fp32, so the checkpoints must be those of the exact sums."""
    g = gen(dim)
    x = torch.randint(-4, 5, (tokens, dim), generator=g, device="cuda").to(torch.bfloat16)
    wg, wu = (torch.randint(-3, 4, (ffn, dim), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    need = cr.cr_glu_workspace_bytes(tokens, dim, ffn)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = torch.empty(tokens, ffn, dtype=torch.bfloat16, device="cuda")
    q, gc, gs, _ = new_q8(tokens, ffn)
    p, uc, us, _ = new_q8(tokens, ffn)
    cr.cr_glu(x, wg, wu, tokens, dim, ffn, "bf16", "silu", a, q, p, work, need)
    for codes, scales, w in ((gc, gs, wg), (uc, us, wu)):
        v = (x.double() @ w.double().T).float()
        q2, codes2, scales2, _ = new_q8(tokens, ffn)
        cr.cr_q8_store(v, tokens, ffn, "f32", q2)
        assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


# More tiles than SMs, with ragged edges, and (the last two) few in the last turn.
MANY_TILES = [(2600, 72, 3000), (1531, 1001, 2731), (1800, 4100, 1664), (2000, 2570, 2100)]


@pytest.mark.parametrize("tokens,dim,ffn", MANY_TILES)
def test_glu_many_tiles(tokens, dim, ffn):
    check_glu(tokens, dim, ffn, "silu", 0, 0)


@pytest.mark.parametrize("held,dw_dt", [("full", "f32"), ("q8", "bf16")])
@pytest.mark.parametrize("tokens,dim,ffn", MANY_TILES)
def test_glu_backward_many_tiles(tokens, dim, ffn, held, dw_dt):
    check_glu_backward(tokens, dim, ffn, held, dw_dt, "gelu", 0, 0)


# Tall tiles and, after them, halves of tall tiles; then operands whose rows are 128 bytes off.
@pytest.mark.parametrize("tokens,dim,ffn,side", [(2000, 3100, 2600, 0), (1900, 2056, 2600, 8)])
def test_glu_tall_tiles(tokens, dim, ffn, side):
    check_glu(tokens, dim, ffn, "silu", side, side)


@pytest.mark.parametrize("dw_dt", ["f32", "bf16"])
def test_glu_backward_tall_tiles(dw_dt):
    """dx: 168 tall tiles, 152 in a turn and 16 in halves on 152 SMs; dW: 252."""
    check_glu_backward(2900, 3330, 2270, "full", dw_dt, "silu", 0, 0)


def test_glu_integers_are_exact_with_many_tiles():
    test_glu_integers_are_exact(3000, 256, 1500)


def test_glu_rows_and_columns_stay_apart_with_many_tiles():
    test_glu_rows_and_columns_stay_apart(20000)


@pytest.mark.parametrize("tokens", [3, 130])
def test_glu_rows_and_columns_stay_apart(tokens):
    """NaN in one token reaches that token alone, NaN in one weight row that column alone."""
    dim, ffn, g = 96, 200, gen(5)
    x, wg, wu = rand(g, tokens, dim, "bf16"), rand(g, ffn, dim, "bf16"), rand(g, ffn, dim, "bf16")
    need = cr.cr_glu_workspace_bytes(tokens, dim, ffn)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    a, b = (torch.empty(tokens, ffn, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cr.cr_glu(x, wg, wu, tokens, dim, ffn, "bf16", "silu", a, None, None, work, need)
    x[1, 3] = math.nan
    wg[150, 5] = math.inf
    wu[7, 95] = math.nan
    q, gc, gs, _ = new_q8(tokens, ffn)
    cr.cr_glu(x, wg, wu, tokens, dim, ffn, "bf16", "silu", b, q, None, work, need)
    assert torch.isnan(b[1]).all() and torch.isnan(b[:, 7]).all()
    assert (gc[1] == 0x7F).all() and (gc[:, 150] & 0x7F == 0x7F).all() and torch.isfinite(gs).all()
    keep_r = [t for t in range(tokens) if t != 1]
    keep_c = [c for c in range(ffn) if c not in (7, 150)]
    assert torch.equal(a[keep_r][:, keep_c], b[keep_r][:, keep_c])
    assert (gc[keep_r][:, keep_c] & 0x7F != 0x7F).all()


@pytest.mark.parametrize("held", ["full", "q8"])
@pytest.mark.parametrize("dw_dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,dim,ffn", GLU_SHAPES)
def test_glu_backward(tokens, dim, ffn, held, dw_dt):
    check_glu_backward(tokens, dim, ffn, held, dw_dt, "silu" if dim % 2 else "gelu", 0, 0)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("tokens,dim,ffn", [(1, 128, 256), (9, 70, 130), (140, 64, 200), (130, 136, 264)])
def test_glu_backward_strided(tokens, dim, ffn, left, right):
    check_glu_backward(tokens, dim, ffn, "full", "bf16", "silu", left, right)


def check_glu_backward(tokens, dim, ffn, held, dw_dt, kind, left, right):
    g = gen(tokens * 3 + dim + ffn)
    x = rand(g, tokens, dim, "bf16")
    wg, wu = (rand(g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    da = rand(g, tokens, ffn, "bf16")
    q, gv = store(rand(g, tokens, ffn, "f32"))
    p, uv = store(rand(g, tokens, ffn, "f32"))
    x8, xv = (None, x.double()) if held == "full" else store(x)
    need = cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    dx, wide_dx = empty(tokens, dim, "bf16", left, right)
    a, wide_a = empty(tokens, ffn, "bf16", left, right)
    dwg, dwu = (torch.full((ffn, dim), math.nan, device="cuda").to(R.TORCH[dw_dt]) for _ in range(2))
    cr.cr_glu_backward(strided(da, left, right), q, p, strided(x, left, right) if held == "full" else None,
                       x8, strided(wg, left, right), strided(wu, right, left), tokens, dim, ffn, "bf16",
                       kind, dx, dwg, dwu, dw_dt, a, work, need)
    untouched(wide_dx, left, dim)
    untouched(wide_a, left, ffn)
    dg, du, av = R.glu_act_backward(da, gv, uv, kind)
    assert torch.all((a.double() - av).abs() <= R.U16 * av.abs() + 2.0 ** -18 * (gv * uv).abs())
    # exact operands against rounded ones: U16 of every term (dg and du; x is exact, or
    # within 2^-16 of its checkpoint's value), 2 U32 an addition
    edg = 2.0 ** -18 * da.double().abs() * uv.abs() * (1 + gv.abs())
    edu = 2.0 ** -18 * da.double().abs() * gv.abs()

    def check(got, pairs, terms, u_out, what, exact=False):
        want = sum(l @ r for l, r, _ in pairs)
        mag = sum((l.abs() + e) @ r.abs() for l, r, e in pairs)
        err = sum(e @ r.abs() for _, r, e in pairs)
        tol = u_out * want.abs() + (1 + u_out) * (R.U16 + 2 * R.U32 * (terms + 2)) * mag + 2 * err
        assert torch.all((got.double() - want).abs() <= tol), what
        # the operands' rounding taken into account, what is left is the result's own
        # rounding and, where fp32 and 64 bits round an operand apart, a rare U16
        near = sum((l if exact else R.bf16(l)) @ r for l, r, _ in pairs)
        if got.numel() > 500:
            assert R.rel_norm(got, near) <= max(u_out, 2.0 ** -12), what

    check(dx, [(dg, wg.double(), edg), (du, wu.double(), edu)], 2 * ffn, R.U16, "dx")
    # up to 64 tokens dW takes dg and du in two parts
    check(dwg, [(dg.T, xv, edg.T)], tokens, R.U_OUT[dw_dt], "dwg", tokens <= 64)
    check(dwu, [(du.T, xv, edu.T)], tokens, R.U_OUT[dw_dt], "dwu", tokens <= 64)


def test_glu_backward_outputs_alone():
    tokens, dim, ffn, g = 150, 136, 200, gen(2)
    x, da = rand(g, tokens, dim, "bf16"), rand(g, tokens, ffn, "bf16")
    wg, wu = rand(g, ffn, dim, "bf16"), rand(g, ffn, dim, "bf16")
    q, _ = store(rand(g, tokens, ffn, "f32"))
    p, _ = store(rand(g, tokens, ffn, "f32"))
    need = cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(which):
        out = {"dx": torch.zeros(tokens, dim, device="cuda", dtype=torch.bfloat16),
               "dwg": torch.zeros(ffn, dim, device="cuda", dtype=torch.bfloat16),
               "dwu": torch.zeros(ffn, dim, device="cuda", dtype=torch.bfloat16),
               "a": torch.zeros(tokens, ffn, device="cuda", dtype=torch.bfloat16)}
        out = {k: v if k in which else None for k, v in out.items()}
        dw = "dwg" in which or "dwu" in which
        cr.cr_glu_backward(da, q, p, x if dw else None, None, wg if "dx" in which else None,
                           wu if "dx" in which else None, tokens, dim, ffn, "bf16", "silu", out["dx"],
                           out["dwg"], out["dwu"], "bf16", out["a"], work, need)
        return out
    full = run(("dx", "dwg", "dwu", "a"))
    for k in full:
        assert torch.equal(run((k,))[k], full[k]), k


def test_block_of_nothing():
    """No tokens: dW = 0.  No hidden units: dx = 0.  No input dimension: a = act(0) * 0 = 0."""
    dev = {"device": "cuda", "dtype": torch.bfloat16}
    x, w = torch.ones(0, 64, **dev), torch.ones(40, 64, **dev)
    need = cr.cr_glu_backward_workspace_bytes(0, 64, 40)
    work = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    q, _ = store(torch.ones(1, 40, device="cuda"))
    dwg, dwu = torch.ones(40, 64, **dev), torch.ones(40, 64, **dev)
    cr.cr_glu_backward(None, q, q, None, None, w, w, 0, 64, 40, "bf16", "silu", None, dwg, dwu, "bf16",
                       None, work, need)
    assert (dwg == 0).all() and (dwu == 0).all()
    cr.cr_glu(x, w, w, 0, 64, 40, "bf16", "silu", torch.empty(0, 40, **dev))
    dx = torch.ones(5, 64, **dev)
    need = cr.cr_glu_backward_workspace_bytes(5, 64, 0)
    work = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    cr.cr_glu_backward(None, q, q, None, None, None, None, 5, 64, 0, "bf16", "silu", dx, None, None,
                       "bf16", None, work, need)
    assert (dx == 0).all()
    a = torch.ones(5, 40, **dev)
    need = cr.cr_glu_workspace_bytes(5, 0, 40)
    work = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    g8, codes, scales, _ = new_q8(5, 40)
    cr.cr_glu(None, None, None, 5, 0, 40, "bf16", "gelu", a, g8, None, work, need)
    assert (a == 0).all() and (codes & 0x7F == 0).all() and (scales == 2.0 ** -126).all()


# ---- gradients against differences of the forward pass ------------------------------------------

def test_gradients_against_differences():
    """The whole sublayer, a = glu(norm(x + r)), L = sum(a * k): the calls' gradients along a
    direction against central differences of the 64-bit forward pass.  The calls round their
    operands and results to bf16 and the checkpoints to e4m3 (half a step, 2^-4): each of the
    roughly 10^4 terms of the directional derivative carries an independent error of at most
    2^-4 + 4 U16 of its magnitude, so the sum is held to 4 * (2^-4 + 4 U16) times the terms'
    root of sum of squares."""
    rows, dim, ffn, g = 48, 136, 200, gen(9)
    x, r = rand(g, rows, dim, "bf16"), rand(g, rows, dim, "bf16")
    w = (1 + rand(g, 1, dim, "f32", 0.1)).to(torch.bfloat16)[0]
    wg, wu = (rand(g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    k = rand(g, rows, ffn, "bf16")
    dev = {"device": "cuda", "dtype": torch.bfloat16}
    s, y, rstd, a = torch.empty(rows, dim, **dev), torch.empty(rows, dim, **dev), torch.empty(rows, device="cuda"), torch.empty(rows, ffn, **dev)
    y8, yc, ys, _ = new_q8(rows, dim)
    g8, *_ = new_q8(rows, ffn)
    u8, *_ = new_q8(rows, ffn)
    work = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    cr.cr_rms_norm(x, r, w, rows, dim, "bf16", EPS, s, y, y8, rstd)
    cr.cr_glu(y, wg, wu, rows, dim, ffn, "bf16", "gelu", a, g8, u8, work, work.numel())
    dy, dx = torch.empty(rows, dim, **dev), torch.empty(rows, dim, **dev)
    dwg, dwu, dw = torch.empty(ffn, dim, **dev), torch.empty(ffn, dim, **dev), torch.empty(dim, **dev)
    cr.cr_glu_backward(k, g8, u8, None, y8, wg, wu, rows, dim, ffn, "bf16", "gelu", dy, dwg, dwu, "bf16",
                       None, work, work.numel())
    cr.cr_rms_norm_backward(dy, s, None, w, rstd, None, rows, dim, "bf16", dx, dw, "bf16", work, work.numel())

    def loss(x, w, wg, wu):
        y = R.norm(x, r, w, EPS)[2]
        return float((R.glu(y, wg, wu, "gelu")[2] * k.double()).sum())
    base = [t.double() for t in (x, w, wg, wu)]
    for n, grad in enumerate((dx, dw, dwg, dwu)):
        d = torch.randn(base[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up = [t + h * d if i == n else t for i, t in enumerate(base)]
        dn = [t - h * d if i == n else t for i, t in enumerate(base)]
        want = (loss(*up) - loss(*dn)) / (2 * h)
        terms = grad.double() * d
        assert abs(float(terms.sum()) - want) <= 4 * (2.0 ** -4 + 4 * R.U16) * float(terms.norm()), n


def test_no_wait_ran_out():
    """Runs after the tests of the block's kernels: none of their waits gave up."""
    assert cr.cr_glu_wait_word() == 0


# ---- streams, repeats, prepared calls and graphs ----------------------------------------------------

def block_state(seed, tokens=130, dim=200, ffn=264):
    g = gen(seed)
    return {"x": rand(g, tokens, dim, "bf16"), "wg": rand(g, ffn, dim, "bf16"),
            "wu": rand(g, ffn, dim, "bf16"), "da": rand(g, tokens, ffn, "bf16"),
            "w": rand(g, 1, dim, "bf16")[0]}


def sublayer(s, out, work, stream=None):
    tokens, dim = s["x"].shape
    ffn = s["wg"].shape[0]
    cr.cr_rms_norm(s["x"], None, s["w"], tokens, dim, "bf16", EPS, None, out["y"], out["y8"], out["rstd"], stream)
    cr.cr_glu(out["y"], s["wg"], s["wu"], tokens, dim, ffn, "bf16", "silu", out["a"], out["g8"], out["u8"],
              work, work.numel(), stream)
    cr.cr_glu_backward(s["da"], out["g8"], out["u8"], None, out["y8"], s["wg"], s["wu"], tokens, dim, ffn,
                       "bf16", "silu", out["dy"], out["dwg"], out["dwu"], "f32", None, work, work.numel(), stream)
    cr.cr_rms_norm_backward(out["dy"], s["x"], None, s["w"], out["rstd"], None, tokens, dim, "bf16", out["dx"],
                            out["dw"], "f32", work, work.numel(), stream)


def block_outputs(tokens=130, dim=200, ffn=264):
    b = {"device": "cuda", "dtype": torch.bfloat16}
    out = {"y": torch.zeros(tokens, dim, **b), "rstd": torch.zeros(tokens, device="cuda"),
           "a": torch.zeros(tokens, ffn, **b), "dy": torch.zeros(tokens, dim, **b),
           "dx": torch.zeros(tokens, dim, **b), "dwg": torch.zeros(ffn, dim, device="cuda"),
           "dwu": torch.zeros(ffn, dim, device="cuda"), "dw": torch.zeros(dim, device="cuda")}
    for name, cols in (("y8", dim), ("g8", ffn), ("u8", ffn)):
        out[name] = cr.Q8(torch.zeros(tokens, cols, dtype=torch.uint8, device="cuda"),
                          torch.zeros(tokens, R.groups(cols), device="cuda"))
    return out


def tensors(out):
    return {k: v.clone() for k, v in out.items() if torch.is_tensor(v)}


def test_repeats_are_bitwise_equal():
    s, work = block_state(1), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    out = block_outputs()
    sublayer(s, out, work)
    first = tensors(out)
    for fill in (0, 255):
        work.fill_(fill)
        out = block_outputs()
        sublayer(s, out, work)
        for k, v in tensors(out).items():
            assert torch.equal(v, first[k]), k


def test_streams():
    """Calls run on the stream they are given: two streams at once, inputs made on each."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    works = [torch.empty(1 << 26, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [block_outputs() for _ in range(2)]
    states = [block_state(10 + k) for k in range(2)]
    later = [block_state(20 + k) for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                for name in states[k]:
                    states[k][name].copy_(later[k][name])
            sublayer(states[k], outs[k], works[k], st)
    torch.cuda.synchronize()
    for k in range(2):
        want = block_outputs()
        sublayer(later[k], want, works[k])
        for name, v in tensors(outs[k]).items():
            assert torch.equal(v, want[name]), name


def test_prepared_and_captured():
    s, work, out = block_state(3), torch.empty(1 << 26, dtype=torch.uint8, device="cuda"), block_outputs()
    sublayer(s, out, work)
    want = tensors(out)
    out = block_outputs()
    p = cr.prepare(lambda: sublayer(s, out, work))
    p()
    for k, v in tensors(out).items():
        assert torch.equal(v, want[k]), k
    out = block_outputs()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sublayer(s, out, work)
    for name, v in block_state(4).items():
        s[name].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    got = tensors(out)
    out = block_outputs()
    sublayer(s, out, work)
    for k, v in tensors(out).items():
        assert torch.equal(v, got[k]), k
