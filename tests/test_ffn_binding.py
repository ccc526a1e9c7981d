"""The binding of the feed-forward operators: tensors whose layout a call cannot
express are refused, every other one gives its own address and row stride.  No
GPU: prepare() records the words of a call and launches nothing."""
import struct

import pytest
import torch

from fsdp_emulated_ranks_gb300 import build as libbuild
from fsdp_emulated_ranks_gb300 import cr

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def q8(rows, cols):
    return cr.Q8(t(rows, cols, dtype=torch.uint8), t(rows, -(-cols // cr.Q8_GROUP), dtype=torch.float32))


def words(p):
    raw = p._calls[0][2][1]
    return struct.unpack(f"={len(raw) // 8}Q", raw)


def norm(**kw):
    a = dict(x=t(4, 64), residual=None, weight=t(64), rows=4, cols=64, dtype="bf16", eps=1e-6, sum=None,
             y=t(4, 64), rstd=t(4, dtype=torch.float32), stream=0)
    a.update(kw)
    return cr.prepare(cr.cr_rms_norm, **a)


def norm_back(**kw):
    a = dict(dy=t(4, 64), h=t(4, 64), h8=None, weight=t(64), rstd=t(4, dtype=torch.float32), dres=None,
             rows=4, cols=64, dtype="bf16", dx=t(4, 64), dweight=t(64),
             workspace=t(4096, dtype=torch.uint8), workspace_bytes=4096, stream=0)
    a.update(kw)
    return cr.prepare(cr.cr_rms_norm_backward, **a)


def glu_back(**kw):
    a = dict(da=t(4, 32), g8=q8(4, 32), u8=q8(4, 32), x=t(4, 64), x8=None, wg=t(32, 64), wu=t(32, 64),
             tokens=4, dim=64, ffn=32, dtype="bf16", act="silu", dx=t(4, 64), dwg=t(32, 64), dwu=t(32, 64),
             workspace=t(1 << 16, dtype=torch.uint8), workspace_bytes=1 << 16, stream=0)
    a.update(kw)
    return cr.prepare(cr.cr_glu_backward, **a)


@pytest.mark.parametrize("call,name,view", [
    (glu_back, "dwg", lambda: t(32, 128)[:, :64]),       # half of a fused gradient
    (glu_back, "dwu", lambda: t(32, 128)[:, 64:]),
    (glu_back, "dwg", lambda: t(64, 32).T),
    (glu_back, "dwu", lambda: t(64, 64)[::2]),
    (glu_back, "workspace", lambda: t(1 << 17, dtype=torch.uint8)[::2]),
    (norm, "weight", lambda: t(128)[::2]),
    (norm, "weight", lambda: t(64, 3)[:, 1]),            # a column of a matrix
    (norm, "rstd", lambda: t(8, dtype=torch.float32)[::2]),
    (norm_back, "weight", lambda: t(128)[::2]),
    (norm_back, "rstd", lambda: t(4, 2, dtype=torch.float32)[:, 0]),
    (norm_back, "dweight", lambda: t(64, 2)[:, 0]),
    (norm_back, "workspace", lambda: t(8192, dtype=torch.uint8)[::2]),
    (norm, "weight", lambda: t(1).expand(64)),           # one value for all columns
])
def test_packed_arguments_refuse_strides(call, name, view):
    call()
    with pytest.raises(ValueError, match="contiguous"):
        call(**{name: view()})


@pytest.mark.parametrize("view", [lambda: t(128)[::2], lambda: t(1).expand(64)])
def test_a_row_given_as_a_vector_has_contiguous_columns(view):
    with pytest.raises(ValueError, match="contiguous"):
        norm(x=view(), y=t(1, 64), rows=1, rstd=None)
    x = t(64)
    assert words(norm(x=x, y=t(1, 64), rows=1, rstd=None))[0] == x.data_ptr()


def test_scales_refuse_strides():
    with pytest.raises(ValueError, match="contiguous"):
        cr.Q8(t(4, 256, dtype=torch.uint8), t(4, 4, dtype=torch.float32)[:, ::2])


def test_a_matrix_has_two_dimensions():
    """More are taken only where they add nothing: [batch, 1, columns], as the last token of
    each sequence comes."""
    last = t(4, 9, 64)[:, -1:]
    assert words(norm(x=last))[:2] == (last.data_ptr(), 9 * 64)
    for bad in (t(2, 2, 64), t(4, 64, 2).transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            norm(x=bad)


def test_row_strides_are_the_tensors():
    wide = t(4, 200)
    y = wide[:, 70:134]
    got = words(norm(y=y))
    assert got[11:13] == (y.data_ptr(), 200) and got[4] != 0
    dwg, dwu = t(64, 64)[:32], t(2, 32, 64)[1]           # contiguous parts of larger buffers
    got = words(glu_back(dwg=dwg, dwu=dwu))
    assert got[18:20] == (dwg.data_ptr(), dwu.data_ptr())
