"""The feed-forward operators of include/cr_ffn.h without a GPU: exported
symbols, argument checks (every call below fails one, or has nothing to do, so
no kernel is launched), workspace sizes, and the reference formulas' own
gradients against differences."""
import os
import re
import struct

import pytest
import torch

import ffn_ref as R
from fsdp_emulated_ranks_gb300 import build as libbuild
from fsdp_emulated_ranks_gb300 import cr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40  # an address never dereferenced
MIB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def L():
    libbuild.build()
    return cr.lib()


def at(k):
    return FAKE + k * 64 * MIB


def expect(status, fn, *args, **kw):
    with pytest.raises(cr.CRError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status, str(ei.value)
    return str(ei.value)


def header():
    text = open(os.path.join(ROOT, "include", "cr_ffn.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_exports_every_declared_symbol(L):
    declared = set(re.findall(r"\b(cr_[a-z0-9_]+)\s*\(", header()))
    assert declared == set(cr.FFN_EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def test_every_launching_call_is_preparable():
    decls = re.findall(r"\bcr_status\s+(cr_\w+)\s*\(([^;]*?)\);", header(), re.S)
    assert {n for n, params in decls if "cr_stream_t" in params} <= cr._PREPARABLE


def q8(k, cols=64, ld=None, lds=None):
    return cr.Q8(at(k), at(k + 1), cols if ld is None else ld, R.groups(cols) if lds is None else lds)


def test_q8_refusals():
    ok = dict(stream=0, ldx=64)
    expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", None, **ok)
    expect(1, cr.cr_q8_store, None, 4, 64, "bf16", q8(1), **ok)
    expect(1, cr.cr_q8_store, at(0), 4, 64, 9, q8(1), **ok)
    expect(2, cr.cr_q8_store, at(0), 4, 64, "i32", q8(1), **ok)
    expect(3, cr.cr_q8_store, at(0) + 1, 4, 64, "bf16", q8(1), **ok)
    expect(3, cr.cr_q8_store, at(0), 4, 64, "bf16", cr.Q8(at(1), at(2) + 2, 64, 1), **ok)
    expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", q8(1, ld=63), **ok)
    expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", q8(1, lds=0), **ok)
    expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", q8(1), stream=0, ldx=63)
    expect(2, cr.cr_q8_store, at(0), 1 << 31, 64, "bf16", q8(1), **ok)
    expect(2, cr.cr_q8_store, at(0), 4, 1 << 31, "bf16", q8(1), stream=0, ldx=1 << 31)
    expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", q8(1), stream=0, ldx=1 << 61)
    assert "overlaps" in expect(1, cr.cr_q8_store, at(0), 4, 64, "bf16", cr.Q8(at(0) + 64, at(1), 64, 1), **ok)
    assert "overlaps" in expect(1, cr.cr_q8_load, cr.Q8(at(0), at(1), 64, 1), 4, 64, at(1) - 4, "f32", **ok)
    expect(1, cr.cr_q8_load, None, 4, 64, at(0), "bf16", **ok)
    cr.cr_q8_store(None, 0, 64, "bf16", q8(1), **ok)
    cr.cr_q8_load(cr.Q8(0, 0, 0, 0), 4, 0, None, "f32", **ok)


def norm(x=at(0), res=at(1), w=at(2), rows=4, cols=64, dt="bf16", eps=1e-6, s=at(3), y=at(4), y8=None,
         rstd=at(7), **ld):
    ld = {"ldx": cols, "ldr": cols, "ldsum": cols, "ldy": cols, **ld}
    cr.cr_rms_norm(x, res, w, rows, cols, dt, eps, s, y, y8, rstd, 0, **ld)


def test_norm_refusals():
    for bad in ({"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}, {"x": None}, {"w": None},
                {"ldx": 63}, {"ldr": 1}, {"ldy": 63}, {"dt": 7}, {"y": at(3)}, {"rstd": at(0)},
                {"y8": cr.Q8(0, 0, 64, 1)}, {"s": at(2)}, {"y": at(0) + 128}, {"s": at(0), "ldsum": 72},
                {"y": at(0), "s": at(0)}):
        expect(1, norm, **bad)
    for bad in ({"x": at(0) + 1}, {"w": at(2) + 1}, {"rstd": at(7) + 2}, {"dt": "f32", "y": at(4) + 2}):
        expect(3, norm, **bad)
    for bad in ({"dt": "i32"}, {"cols": 1 << 31, "rows": 1}, {"rows": 1 << 31}):
        expect(2, norm, **bad)
    norm(rows=0)
    norm(cols=0)


def norm_back(dy=at(0), h=at(1), h8=None, w=at(2), rstd=at(3), dres=at(4), rows=4, cols=64, dt="bf16",
              dx=at(5), dw=at(6), dw_dt="bf16", ws=at(7), nbytes=MIB, **ld):
    ld = {"lddy": cols, "ldh": cols, "lddres": cols, "lddx": cols, **ld}
    cr.cr_rms_norm_backward(dy, h, h8, w, rstd, dres, rows, cols, dt, dx, dw, dw_dt, ws, nbytes, 0, **ld)


def test_norm_backward_refusals():
    for bad in ({"h": None}, {"h8": q8(8)}, {"dy": None}, {"rstd": None}, {"w": None}, {"ws": None},
                {"nbytes": 4 * 64 * 4 - 1}, {"dw": at(0)}, {"dx": at(2)}, {"dx": at(7)}, {"dw": at(7) + 64},
                {"dx": at(1), "lddx": 65}, {"lddy": 63}, {"dw_dt": 5}, {"dt": 5}):
        expect(1, norm_back, **bad)
    for bad in ({"ws": at(7) + 8}, {"dx": at(5) + 1}, {"rstd": at(3) + 1}, {"dw_dt": "f32", "dw": at(6) + 2}):
        expect(3, norm_back, **bad)
    for bad in ({"dt": "i32"}, {"dw_dt": "i32"}):
        expect(2, norm_back, **bad)
    norm_back(cols=0)
    norm_back(rows=0, dw=None)
    norm_back(dx=None, dw=None, ws=None)


def glu(x=at(0), wg=at(1), wu=at(2), t=4, d=64, f=64, dt="bf16", act="silu", a=at(3), g8=None, u8=None,
        ws=at(20), nbytes=64 * MIB, **ld):
    ld = {"ldx": d, "ldwg": d, "ldwu": d, "lda": f, **ld}
    cr.cr_glu(x, wg, wu, t, d, f, dt, act, a, g8, u8, ws, nbytes, 0, **ld)


def test_glu_refusals():
    for bad in ({"x": None}, {"wg": None}, {"wu": None}, {"a": None}, {"act": 2}, {"dt": 8}, {"ldx": 63},
                {"ldwg": 63}, {"lda": 63}, {"a": at(0)}, {"a": at(1) + 64}, {"g8": cr.Q8(0, 0, 64, 1)},
                {"g8": q8(4), "u8": q8(4)}, {"g8": cr.Q8(at(3) + 2, at(5), 64, 1)}, {"ldx": 1 << 60}):
        expect(1, glu, **bad)
    for bad in ({"x": at(0) + 1}, {"wu": at(2) + 1}, {"a": at(3) + 1}):
        expect(3, glu, **bad)
    for bad in ({"dt": "f32"}, {"dt": "i32"}, {"t": 1 << 31}, {"d": 1 << 31}, {"f": 1 << 31}):
        expect(2, glu, **bad)
    glu(t=0)
    glu(f=0)


def act_back(da=at(0), g8=None, u8=None, t=4, f=64, dt="bf16", act="silu", dg=at(5), du=at(6), a=at(7), **ld):
    ld = {"ldda": f, "lddg": f, "lddu": f, "lda": f, **ld}
    cr.cr_glu_act_backward(da, g8 or q8(1), u8 or q8(3), t, f, dt, act, dg, du, a, 0, **ld)


def test_act_backward_refusals():
    for bad in ({"da": None}, {"g8": cr.Q8(0, 0, 64, 1)}, {"dg": at(6)}, {"du": at(1)}, {"a": at(4)},
                {"act": -1}, {"lddg": 1}, {"dg": at(0), "lddg": 65}, {"dg": at(0) + 2}):
        expect(1, act_back, **bad)
    expect(1, cr.cr_glu_act_backward, at(0), None, q8(3), 4, 64, "bf16", "silu", at(5), at(6), stream=0, ldda=64)
    expect(3, act_back, a=at(7) + 1)
    expect(2, act_back, dt="f32")
    act_back(t=0)
    act_back(f=0)
    act_back(dg=None, du=None, a=None)


def glu_back(da=at(0), g8=q8(1), u8=q8(3), x=at(5), x8=None, wg=at(6), wu=at(7), t=4, d=64, f=64, dt="bf16",
             act="silu", dx=at(8), dwg=at(9), dwu=at(10), dw_dt="bf16", a=at(11), ws=at(20),
             nbytes=256 * MIB, **ld):
    ld = {"ldda": f, "ldx": d, "ldwg": d, "ldwu": d, "lddx": d, "lda": f, **ld}
    cr.cr_glu_backward(da, g8, u8, x, x8, wg, wu, t, d, f, dt, act, dx, dwg, dwu, dw_dt, a, ws, nbytes, 0, **ld)


def test_glu_backward_refusals():
    for bad in ({"da": None}, {"g8": None}, {"u8": None}, {"x": None}, {"x8": q8(12)}, {"wg": None}, {"wu": None},
                {"ws": None}, {"nbytes": 100}, {"dx": at(0)}, {"dwg": at(10)}, {"dwg": at(5)}, {"a": at(0)},
                {"a": at(20)}, {"act": 4}, {"dw_dt": 7}, {"ldda": 63}, {"ldx": 63}, {"lddx": 63}):
        expect(1, glu_back, **bad)
    for bad in ({"ws": at(20) + 8}, {"dx": at(8) + 1}, {"dwg": at(9) + 1}, {"dw_dt": "f32", "dwu": at(10) + 2}):
        expect(3, glu_back, **bad)
    for bad in ({"dt": "f32"}, {"dw_dt": "i32"}, {"t": 1 << 31}):
        expect(2, glu_back, **bad)


def test_packed_call_refusals(L):
    words = struct.pack("=4Qq2Q", at(0), 64, 4, 64, 1, 0, 0)
    assert L.cr_ffn_call(0, words) == 1 and b"q is NULL" in L.cr_last_error()
    assert L.cr_ffn_call(99, words) == 1 and b"unknown call" in L.cr_last_error()
    assert L.cr_ffn_call(0, None) == 1
    p = cr.prepare(norm, x=None)
    assert p._calls[0][0] == "cr_rms_norm"
    with pytest.raises(cr.CRError, match="cr_rms_norm: .*x is NULL"):
        p()


def test_columns_of_one_buffer_do_not_overlap():
    """Halves of a fused [rows, 2 * 64] buffer share no byte: the overlap check lets them
    pass and the next check refuses the call."""
    wide = dict(ldx=128, ldsum=128, ldr=128, ldy=128)
    msg = expect(1, norm, x=at(0), res=at(1), s=at(0) + 128, y=at(1) + 128, rstd=at(2), **wide)
    assert "rstd overlaps weight" in msg or "overlaps rstd" in msg
    assert "sum overlaps x" in expect(1, norm, s=at(0) + 126, **wide)
    assert "sum overlaps x" in expect(1, norm, s=at(0) - 126, **wide)
    assert "sum overlaps x" in expect(1, norm, s=at(0) - 128, **{**wide, "ldsum": 136})


def test_workspace_sizes():
    assert cr.cr_rms_norm_backward_workspace_bytes(0, 10) == 40
    for rows, cols in ((1, 7), (4, 64), (100000, 2048), (5, 20000)):
        assert 0 < cr.cr_rms_norm_backward_workspace_bytes(rows, cols) <= 1024 * cols * 4
    for t, d, f in ((1, 1, 1), (8192, 2048, 8192), (257, 1001, 2731)):
        assert cr.cr_glu_backward_workspace_bytes(t, d, f) >= 4 * t * f
        assert cr.cr_glu_backward_workspace_bytes(t, d, f) <= 2 * 2 * t * f + 2 * t * d + 6 * d * f \
            + 2 * (t + f) * 256 + (64 << 20)
        assert cr.cr_glu_workspace_bytes(t, d, f) <= 2 * t * d + 4 * d * f + 2 * (t + f) * 256 + (64 << 20)


def test_wrappers_refuse_strided_columns():
    x = torch.empty(64, 4, dtype=torch.bfloat16).T
    with pytest.raises(ValueError, match="contiguous"):
        cr.cr_q8_store(x, 4, 64, "bf16", q8(1), stream=0)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_reference_gradients_are_the_differences(kind):
    g = torch.Generator().manual_seed(3)
    x, r, dres = (torch.randn(6, 10, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(10, generator=g, dtype=torch.float64)
    wg, wu = (torch.randn(7, 10, generator=g, dtype=torch.float64) for _ in range(2))
    k = torch.randn(6, 7, generator=g, dtype=torch.float64)

    def loss(x, w, wg, wu):
        h, _, y = R.norm(x, r, w, 1e-3)
        return float((R.glu(y, wg, wu, kind)[2] * k).sum() + (h * dres).sum())
    h, rstd, y = R.norm(x, r, w, 1e-3)
    gate, up, _ = R.glu(y, wg, wu, kind)
    dg, du, _ = R.glu_act_backward(k, gate, up, kind)
    dx, dw, _, _ = R.norm_backward(dg @ wg + du @ wu, h, w, rstd, dres)
    grads = [dx, dw, dg.T @ y, du.T @ y]
    base = [x, w, wg, wu]
    for n, grad in enumerate(grads):
        for e in range(0, grad.numel(), 5):
            d = torch.zeros(grad.numel(), dtype=torch.float64)
            d[e] = 1e-5
            d = d.view(grad.shape)
            up_, dn = ([t + sign * d if i == n else t for i, t in enumerate(base)] for sign in (1, -1))
            want = (loss(*up_) - loss(*dn)) / 2e-5
            # central differences: truncation about h^2, cancellation 2^-53 |loss| / h
            assert abs(float(grad.flatten()[e]) - want) <= 1e-7 * (1 + abs(want))


def test_reference_decodes_every_code():
    codes = torch.arange(256).to(torch.uint8).reshape(2, 128)
    want = codes.view(torch.float8_e4m3fn).double()
    got = R.decode(codes, torch.ones(2, 1))
    assert torch.equal(torch.nan_to_num(got, 0), torch.nan_to_num(want, 0))
    assert torch.equal(torch.isnan(got), torch.isnan(want))
