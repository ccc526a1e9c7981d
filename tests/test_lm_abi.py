"""The language model operators of include/cr_lm.h without a GPU: exported symbols, argument
checks (every call below fails one, or has nothing to do, so no kernel is launched), workspace
sizes, and the references' own gradients and random numbers."""
import os
import re
import struct

import pytest
import torch

import lm_ref as R
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
    text = open(os.path.join(ROOT, "include", "cr_lm.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_exports_every_declared_symbol(L):
    declared = set(re.findall(r"\b(cr_[a-z0-9_]+)\s*\(", header()))
    assert declared == set(cr.LM_EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def test_every_launching_call_is_preparable():
    decls = re.findall(r"\bcr_status\s+(cr_\w+)\s*\(([^;]*?)\);", header(), re.S)
    names = {n for n, params in decls if "cr_stream_t" in params}
    assert names == set(cr._LM_NAMES) and names <= cr._PREPARABLE


def embed(table=at(0), vocab=9, ids=at(1), tokens=4, dim=64, dt="bf16", scale=2.0, out=at(2), out_dt="bf16", bits=64, **ld):
    cr.cr_embedding(table, vocab, ids, tokens, dim, dt, scale, out, out_dt, 0, id_bits=bits,
                    **{"ldt": dim, "ldo": dim, **ld})


def test_embedding_refusals():
    for bad in ({"table": None}, {"ids": None}, {"out": None}, {"bits": 16}, {"bits": 0}, {"scale": float("nan")},
                {"scale": 1e39}, {"ldt": 63}, {"ldo": 63}, {"out": at(0)}, {"out": at(1)}, {"dt": 9}, {"out_dt": 9}):
        expect(1, embed, **bad)
    for bad in ({"table": at(0) + 1}, {"ids": at(1) + 4}, {"out_dt": "f32", "out": at(2) + 2}, {"bits": 32, "ids": at(1) + 2}):
        expect(3, embed, **bad)
    for bad in ({"dt": "i32"}, {"out_dt": "i32"}, {"vocab": 1 << 31}, {"tokens": 1 << 31}, {"dim": 1 << 31}):
        expect(2, embed, **bad)
    embed(tokens=0)
    embed(dim=0)


def embed_back(dout=at(0), dt="bf16", ids=at(1), tokens=4, vocab=9, dim=64, scale=1.0, base=at(2), dtable=at(3),
               out_dt="bf16", ws=at(4), nbytes=MIB, bits=64, **ld):
    cr.cr_embedding_backward(dout, dt, ids, tokens, vocab, dim, scale, base, dtable, out_dt, ws, nbytes, 0,
                             id_bits=bits, **{"lddo": dim, "ldb": dim, "ldt": dim, **ld})


def test_embedding_backward_refusals():
    need = cr.cr_embedding_backward_workspace_bytes(4, 9, 64)
    for bad in ({"dout": None}, {"ids": None}, {"dtable": None}, {"ws": None}, {"nbytes": need - 1}, {"bits": 8},
                {"scale": float("inf")}, {"lddo": 63}, {"ldb": 63}, {"ldt": 63}, {"dtable": at(0)}, {"dtable": at(1)},
                {"dtable": at(4)}, {"base": at(3), "ldb": 65}, {"base": at(3) + 64}, {"dt": 7}, {"out_dt": 7}):
        expect(1, embed_back, **bad)
    for bad in ({"dout": at(0) + 1}, {"ids": at(1) + 4}, {"ws": at(4) + 8}, {"out_dt": "f32", "dtable": at(3) + 2, "base": None}):
        expect(3, embed_back, **bad)
    for bad in ({"dt": "i32"}, {"out_dt": "i32"}, {"vocab": (1 << 21) + 1}, {"tokens": 1 << 31}, {"dim": 1 << 31}):
        expect(2, embed_back, **bad)
    embed_back(vocab=0)
    embed_back(dim=0)


def dropout(x=at(0), res=at(1), rows=4, cols=64, dt="bf16", p=0.1, rng=at(2), call=0, first=0, out=at(3), **ld):
    cr.cr_dropout(x, res, rows, cols, dt, p, rng, call, first, out, 0, **{"ldx": cols, "ldr": cols, "ldo": cols, **ld})


def test_dropout_refusals():
    for bad in ({"x": None}, {"rng": None}, {"out": None}, {"p": -0.1}, {"p": 1.1}, {"p": float("nan")},
                {"first": 1 << 33}, {"first": (1 << 32) - 3}, {"first": (1 << 64) - 2}, {"ldx": 63}, {"ldr": 63}, {"ldo": 63},
                {"out": at(2)}, {"out": at(0) + 2}, {"out": at(1), "ldo": 65}, {"dt": 5}):
        expect(1, dropout, **bad)
    for bad in ({"x": at(0) + 1}, {"rng": at(2) + 4}, {"out": at(3) + 1}, {"dt": "f32", "res": at(1) + 2}):
        expect(3, dropout, **bad)
    for bad in ({"dt": "i32"}, {"rows": 1 << 31}, {"cols": 1 << 31}):
        expect(2, dropout, **bad)
    dropout(rows=0)
    dropout(cols=0)


def logp(x=at(0), t=at(1), rows=4, vocab=64, dt="bf16", scale=1.0, lp=at(2), ent=at(3), lse=at(4), top=5, ids=at(5),
         tl=at(6), bits=64, **ld):
    cr.cr_log_probs(x, t, rows, vocab, dt, scale, lp, ent, lse, top, ids, tl, 0, id_bits=bits, **{"ldl": vocab, **ld})


def test_log_probs_refusals():
    for bad in ({"x": None}, {"t": None}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"scale": 1e38},
                {"scale": 1e-50}, {"top": -1}, {"top": 33}, {"vocab": 4}, {"vocab": 0, "top": 0}, {"bits": 63}, {"ldl": 63}, {"lp": at(0)},
                {"ent": at(2)}, {"lse": at(1)}, {"ids": at(6)}, {"tl": at(5) + 4}, {"dt": 4}):
        expect(1, logp, **bad)
    for bad in ({"x": at(0) + 1}, {"t": at(1) + 4}, {"lp": at(2) + 2}, {"ids": at(5) + 1}, {"tl": at(6) + 2}):
        expect(3, logp, **bad)
    for bad in ({"dt": "i32"}, {"rows": 1 << 31}, {"vocab": (1 << 31) - 65536}):
        expect(2, logp, **bad)
    logp(rows=0)
    logp(t=None, lp=None, ent=None, lse=None, ids=None, tl=None)
    logp(t=None, lp=None, ent=None, lse=None, top=0)


def logp_back(x=at(0), t=at(1), rows=4, vocab=64, dt="bf16", scale=1.0, lse=at(2), ent=at(3), d=at(4), e=at(5), q=at(6),
              dx=at(7), bits=64, **ld):
    cr.cr_log_probs_backward(x, t, rows, vocab, dt, scale, lse, ent, d, e, q, dx, 0, id_bits=bits,
                             **{"ldl": vocab, "lddl": vocab, **ld})


def test_log_probs_backward_refusals():
    for bad in ({"x": None}, {"t": None}, {"lse": None}, {"ent": None}, {"dx": None}, {"scale": 0.0}, {"vocab": 0}, {"bits": 1},
                {"ldl": 63}, {"lddl": 63}, {"dx": at(1)}, {"dx": at(2)}, {"dx": at(6)}, {"dx": at(0), "lddl": 65}, {"dt": 4}):
        expect(1, logp_back, **bad)
    for bad in ({"x": at(0) + 1}, {"t": at(1) + 4}, {"lse": at(2) + 2}, {"ent": at(3) + 1}, {"d": at(4) + 2}, {"e": at(5) + 2},
                {"q": at(6) + 2}, {"dx": at(7) + 1}):
        expect(3, logp_back, **bad)
    for bad in ({"dt": "i32"}, {"rows": 1 << 31}, {"vocab": 1 << 31}):
        expect(2, logp_back, **bad)
    logp_back(rows=0)


def test_packed_call_refusals(L):
    assert L.cr_lm_call(99, struct.pack("=16Q", *[0] * 16)) == 1 and b"unknown call" in L.cr_last_error()
    assert L.cr_lm_call(0, None) == 1
    p = cr.prepare(dropout, p=2.0)
    assert p._calls[0][0] == "cr_dropout"
    with pytest.raises(cr.CRError, match="cr_dropout: .*outside"):
        p()


def test_binding_takes_id_widths_from_tensors():
    assert cr._ids(torch.zeros(3, dtype=torch.int32), None)[1] == 32
    assert cr._ids(torch.zeros(3, dtype=torch.int64), None)[1] == 64
    assert cr._ids(at(0), None)[1] == 64 and cr._ids(at(0), 32)[1] == 32 and cr._ids(None, None) == (0, 64)
    for bad in (torch.zeros(3), torch.zeros(3, dtype=torch.int16)):
        with pytest.raises(ValueError, match="token ids"):
            cr._ids(bad, None)
    with pytest.raises(ValueError, match="contiguous"):
        cr._ids(torch.zeros(6, dtype=torch.int64)[::2], None)


def test_workspace_sizes():
    size = cr.cr_embedding_backward_workspace_bytes
    assert size(10, 0, 5) == size(10, 5, 0) == size(10, (1 << 21) + 1, 5) == size(1 << 31, 5, 5) == 0
    for t, v, d in ((0, 1, 1), (1, 1, 1), (8192, 32000, 2048), (65536, 131072, 4096), (1000, 1 << 21, 8)):
        parts = 2 * (t // 16 + 1)  # at most: two for every 16 tokens, an fp32 row and two counters a chunk each
        assert 8 * (t + v) < size(t, v, d) <= 8 * (t + v) + parts * (4 * (d + 519) + 8 * ((d + 7) // 256 + 1)) + 1024


def test_random_numbers_of_the_references_agree():
    """The published test vectors of Philox4x32-10, and the two references against each other."""
    assert R.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert R.philox((ones,) * 4, (ones,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert R.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) \
        == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    args = (3, 21, 0x123456789ABCDEF0, 0xFFFFFFFF00000001, 4294967290)
    assert torch.equal(R.numbers(*args), R.numbers_fast(*args))


def test_reference_gradients_are_autograds():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 40, generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.randint(0, 40, (5,), generator=g)
    t[3] = -1
    d, e, q = (torch.randn(5, generator=g, dtype=torch.float64) for _ in range(3))
    lp, ent, lse, _, _, _ = R.log_probs(x, t, 0.5)
    (lp * d + ent * e + lse * q).sum().backward()
    want, _ = R.log_probs_backward(x.detach(), t, 0.5, lse.detach(), ent.detach(), d, e, q)
    assert torch.allclose(x.grad, want, rtol=1e-10, atol=1e-12)
    table = torch.randn(7, 6, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.tensor([0, 3, 3, -1, 7, 6])
    dout = torch.randn(6, 6, generator=g, dtype=torch.float64)
    (R.embedding(table, ids, 2.0) * dout).sum().backward()
    want, _ = R.embedding_backward(dout, ids, 7, 2.0, None)
    assert torch.allclose(table.grad, want, rtol=1e-12, atol=0)
