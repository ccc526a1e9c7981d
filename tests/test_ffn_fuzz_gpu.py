"""Seeded random calls of the feed-forward operators: sizes from one up, each buffer at a
row stride and an alignment of its own, NaN beside the inputs and a pattern beside the
outputs, optional arguments there or not, in place or not, rows of zeros, infinities and
NaN -- against the formulas in 64 bits, with the bounds of tests/ffn_ref.py."""
import math
import random

import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed):
        self.rng, self.g = random.Random(seed), T.gen(seed)
        self.checks = []

    def size(self, hi):
        k = int(round(math.exp(self.rng.uniform(0, math.log(hi)))))
        return max(1, min(hi, k // 16 * 16 if self.rng.random() < 0.3 else k))

    def sides(self, cols, es):
        """Elements left and right of a matrix: none, whole 16 or 32 bytes, or any number."""
        kind = self.rng.randrange(4)
        if kind == 0:
            return 0, 0
        if kind == 1:
            return self.rng.randrange(9), self.rng.randrange(9)
        unit = (16 if kind == 2 else 32) // es
        left = unit * self.rng.randrange(3)
        return left, -(left + cols) % unit

    def put(self, t):
        """The same matrix (or vector, as one row) inside a buffer of its own."""
        if t is None:
            return None
        m = t if t.dim() == 2 else t[None]
        fill = 0 if t.dtype == torch.uint8 else math.nan
        out = T.strided(m, *self.sides(m.shape[1], t.element_size()), fill)
        return out if t.dim() == 2 else out[0]

    def out(self, rows, cols, dt):
        es = {"bf16": 2, "f32": 4, "u8": 1}[dt]
        left, right = self.sides(cols, es)
        m, wide = T.empty(rows, cols, dt, left, right)
        self.checks.append(lambda: T.untouched(wide, left, cols))
        return m

    def q8(self, rows, cols):
        codes = self.out(rows, cols, "u8")
        scales = self.out(rows, R.groups(cols), "f32")
        return cr.Q8(codes, scales), codes, scales

    def stored(self, v):
        rows, cols = v.shape
        q, codes, scales = self.q8(rows, cols)
        cr.cr_q8_store(v.contiguous(), rows, cols, "f32" if v.dtype == torch.float32 else "bf16", q)
        return q, R.decode(codes, scales)

    def maybe(self, v, p=0.5):
        return v if self.rng.random() < p else None

    def work(self, need):
        """A workspace of exactly the bytes asked for, 16-byte aligned, with a guard behind it."""
        buf = torch.full((need + 48,), 77, dtype=torch.uint8, device="cuda")
        self.checks.append(lambda: T.untouched(buf[None], 16, need))
        return buf[16:16 + need]

    def done(self):
        for check in self.checks:
            check()


@pytest.mark.parametrize("seed", range(120))
def test_fuzz_q8(seed):
    c = Case(1000 + seed)
    rows, cols, dt = c.size(300), c.size(3000), c.rng.choice(["bf16", "f32"])
    v = torch.randn(rows, cols, generator=c.g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (rows, cols), generator=c.g, device="cuda").float())
    v[torch.rand(rows, cols, generator=c.g, device="cuda") < 0.02] = math.inf * (1 - 2 * (seed % 2))
    v[torch.rand(rows, cols, generator=c.g, device="cuda") < 0.02] = math.nan
    v[torch.rand(rows, cols, generator=c.g, device="cuda") < 0.1] = 0
    v[c.rng.randrange(rows)] = 0
    v = v.to(R.TORCH[dt])
    q, codes, scales = c.q8(rows, cols)
    cr.cr_q8_store(c.put(v), rows, cols, dt, q)
    R.assert_q8(codes, scales, v.double())
    out = c.rng.choice(["bf16", "f32"])
    x = c.out(rows, cols, out)
    cr.cr_q8_load(q, rows, cols, x, out)
    want = R.decode(codes, scales).float().to(R.TORCH[out])
    assert torch.equal(torch.nan_to_num(x, 1e9), torch.nan_to_num(want, 1e9))
    c.done()


@pytest.mark.parametrize("seed", range(150))
def test_fuzz_rms_norm(seed):
    c = Case(2000 + seed)
    rows, cols, dt = c.size(600), c.size(12000 if seed % 3 else 700), c.rng.choice(["bf16", "f32"])
    x = T.rand(c.g, rows, cols, dt, 3.0)
    res = c.maybe(T.rand(c.g, rows, cols, dt))
    w = (1 + T.rand(c.g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])[0]
    if rows > 2:
        x[rows // 2] = 0
        if res is not None:
            res[rows // 2] = 0
    xin, rin = c.put(x), c.put(res)
    s, y = c.maybe(c.out(rows, cols, dt)), c.maybe(c.out(rows, cols, dt))
    if c.rng.random() < 0.3:
        (s, y) = (xin, y) if c.rng.random() < 0.5 else (s, xin)
    elif res is not None and c.rng.random() < 0.3:
        (s, y) = (rin, y) if c.rng.random() < 0.5 else (s, rin)
    q8 = c.maybe(c.q8(rows, cols))
    rstd = c.maybe(torch.empty(rows, device="cuda"), 0.8)
    cr.cr_rms_norm(xin, rin, c.put(w), rows, cols, dt, T.EPS, s, y, q8 and q8[0], rstd)
    got = {"sum": s, "y": y, "y8": q8 and q8[1:], "rstd": rstd}
    T.check_norm(x, res, w, dt, T.EPS, {k: v for k, v in got.items() if v is not None})
    c.done()


@pytest.mark.parametrize("seed", range(150))
def test_fuzz_rms_norm_backward(seed):
    c = Case(3000 + seed)
    rows, cols = c.size(900), c.size(12000 if seed % 3 else 700)
    dt, dw_dt = c.rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
    h = T.rand(c.g, rows, cols, dt, 2.0)
    dy, dres = T.rand(c.g, rows, cols, dt, 1e-2), c.maybe(T.rand(c.g, rows, cols, dt, 1e-2))
    w = (1 + T.rand(c.g, 1, cols, "f32", 0.2)).to(R.TORCH[dt])[0]
    rstd = R.norm(h, None, w, T.EPS)[1].float()
    hin, q, hv = c.put(h), None, h
    if c.rng.random() < 0.5:
        (q, hv), hin = c.stored(h), None
    dyin, rin = c.put(dy), c.put(dres)
    dx = c.out(rows, cols, dt)
    over = c.rng.choice([None, None, dyin, rin, hin])
    if over is not None:
        dx = over
    dx = c.maybe(dx, 0.8)
    dw = c.maybe(torch.empty(cols, device="cuda", dtype=R.TORCH[dw_dt]), 0.8)
    work = c.work(cr.cr_rms_norm_backward_workspace_bytes(rows, cols))
    cr.cr_rms_norm_backward(dyin, hin, q, c.put(w), rstd, rin, rows, cols, dt, dx, dw, dw_dt, work, work.numel())
    want_dx, want_dw, mag, mag_dw = R.norm_backward(dy, hv, w, rstd, dres)
    if dx is not None:
        rel = (R.norm_depth(cols) + 8) * R.U32
        assert torch.all((dx.double() - want_dx).abs()
                         <= R.U_OUT[dt] * want_dx.abs() * (1 + rel) + rel * (mag + want_dx.abs()))
    if dw is not None:
        rel = (rows + 8) * R.U32
        assert torch.all((dw.double() - want_dw).abs()
                         <= R.U_OUT[dw_dt] * want_dw.abs() * (1 + rel) + rel * mag_dw)
    c.done()


@pytest.mark.parametrize("seed", range(120))
def test_fuzz_act_backward(seed):
    c = Case(4000 + seed)
    rows, cols, kind = c.size(400), c.size(3000), c.rng.choice(["silu", "gelu"])
    q, gv = c.stored(T.rand(c.g, rows, cols, "f32", 3.0))
    p, uv = c.stored(T.rand(c.g, rows, cols, "f32"))
    da = T.rand(c.g, rows, cols, "bf16")
    din = c.put(da)
    outs = [c.maybe(c.out(rows, cols, "bf16"), 0.7) for _ in range(3)]
    if c.rng.random() < 0.4:
        outs[c.rng.randrange(3)] = din
    cr.cr_glu_act_backward(din, q, p, rows, cols, "bf16", kind, *outs)
    want = R.glu_act_backward(da, gv, uv, kind)
    # as in tests/test_ffn_gpu.py
    scale = [da.double().abs() * uv.abs() * (1 + gv.abs()), da.double().abs() * gv.abs(), gv.abs() * uv.abs()]
    for out, ref, mag in zip(outs, want, scale):
        if out is not None:
            assert torch.all((out.double() - ref).abs() <= R.U16 * ref.abs() + 2.0 ** -18 * mag)
    c.done()


@pytest.mark.parametrize("seed", range(120))
def test_fuzz_glu(seed):
    c = Case(5000 + seed)
    tokens, dim, ffn = c.size(5 if seed % 4 == 0 else 900), c.size(1500), c.size(1500)
    kind = c.rng.choice(["silu", "gelu"])
    x = T.rand(c.g, tokens, dim, "bf16")
    wg, wu = (T.rand(c.g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    a = c.out(tokens, ffn, "bf16")
    g8, u8 = c.maybe(c.q8(tokens, ffn)), c.maybe(c.q8(tokens, ffn))
    work = c.work(cr.cr_glu_workspace_bytes(tokens, dim, ffn))
    cr.cr_glu(c.put(x), c.put(wg), c.put(wu), tokens, dim, ffn, "bf16", kind, a, g8 and g8[0], u8 and u8[0],
              work, work.numel())
    gv, uv, av = R.glu(x, wg, wu, kind)
    eg, eu = T.glu_slack(x, wg, dim), T.glu_slack(x, wu, dim)
    slack = 1.2 * uv.abs() * eg + (gv.abs() + 1.2 * eg) * eu + 2.0 ** -18 * av.abs()
    assert torch.all((a.double() - av).abs() <= R.U16 * (av.abs() + slack) + slack)
    if g8:
        R.assert_q8(*g8[1:], gv, slack=eg, what="gate")
    if u8:
        R.assert_q8(*u8[1:], uv, slack=eu, what="up")
    c.done()


@pytest.mark.parametrize("seed", range(150))
def test_fuzz_glu_backward(seed):
    c = Case(6000 + seed)
    tokens, dim, ffn = c.size(900), c.size(1200), c.size(1200)
    kind, dw_dt = c.rng.choice(["silu", "gelu"]), c.rng.choice(["bf16", "f32"])
    x, da = T.rand(c.g, tokens, dim, "bf16"), T.rand(c.g, tokens, ffn, "bf16")
    wg, wu = (T.rand(c.g, ffn, dim, "bf16", dim ** -0.5) for _ in range(2))
    q, gv = c.stored(T.rand(c.g, tokens, ffn, "f32"))
    p, uv = c.stored(T.rand(c.g, tokens, ffn, "f32"))
    xin, x8, xv = c.put(x), None, x.double()
    if c.rng.random() < 0.5:
        (x8, xv), xin = c.stored(x), None
    dx, a = c.maybe(c.out(tokens, dim, "bf16"), 0.8), c.maybe(c.out(tokens, ffn, "bf16"))
    dwg, dwu = (c.maybe(torch.full((ffn * dim + 2,), 77.0, device="cuda").to(R.TORCH[dw_dt]), 0.8)
                for _ in range(2))
    packed = [None if t is None else t[1:1 + ffn * dim].view(ffn, dim) for t in (dwg, dwu)]
    work = c.work(cr.cr_glu_backward_workspace_bytes(tokens, dim, ffn))
    cr.cr_glu_backward(c.put(da), q, p, xin, x8, c.put(wg), c.put(wu), tokens, dim, ffn, "bf16", kind, dx,
                       *packed, dw_dt, a, work, work.numel())
    dg, du, av = R.glu_act_backward(da, gv, uv, kind)
    edg = 2.0 ** -18 * da.double().abs() * uv.abs() * (1 + gv.abs())
    edu = 2.0 ** -18 * da.double().abs() * gv.abs()

    def check(got, pairs, terms, u_out, what):  # as in tests/test_ffn_gpu.py
        want = sum(l @ r for l, r, _ in pairs)
        mag = sum((l.abs() + e) @ r.abs() for l, r, e in pairs)
        err = sum(e @ r.abs() for _, r, e in pairs)
        tol = u_out * want.abs() + (1 + u_out) * (R.U16 + 2 * R.U32 * (terms + 2)) * mag + 2 * err
        assert torch.all((got.double() - want).abs() <= tol), what
    if dx is not None:
        check(dx, [(dg, wg.double(), edg), (du, wu.double(), edu)], 2 * ffn, R.U16, "dx")
    for t, got, d, e in ((dwg, packed[0], dg, edg), (dwu, packed[1], du, edu)):
        if t is not None:
            check(got, [(d.T, xv, e.T)], tokens, R.U_OUT[dw_dt], "dw")
            assert float(t[0]) == 77 and float(t[-1]) == 77
    if a is not None:
        assert torch.all((a.double() - av).abs() <= R.U16 * av.abs() + 2.0 ** -18 * (gv * uv).abs())
    c.done()


def test_no_wait_ran_out_in_the_fuzz():
    assert cr.cr_glu_wait_word() == 0
