"""Prepared feed-forward calls on the CPU: what they address stays alive and as it was at
preparation, also where the recorded function made it itself.  Nothing is launched:
the recorded words are looked at."""
import gc
import struct
import weakref

import pytest
import torch

from fsdp_emulated_ranks_gb300 import build as libbuild
from fsdp_emulated_ranks_gb300 import cr


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def words(p, k=0):
    raw = p._calls[k][2][1]
    return struct.unpack(f"={len(raw) // 8}Q", raw)


def parts(rows=4, cols=64):
    return torch.zeros(rows, cols, dtype=torch.uint8), torch.zeros(rows, 1)


def fields(address):
    q = cr.Q8.from_address(address)
    return q.codes, q.ld, q.scales, q.lds


def test_a_q8_made_while_recording_lives_as_long_as_the_prepared_call():
    x, (codes, scales) = torch.zeros(4, 64), parts()
    made = []

    def call():
        q = cr.Q8(codes, scales)
        made.append(weakref.ref(q))
        cr.cr_q8_store(x, 4, 64, "f32", q, stream=0)
        cr.cr_q8_load(q, 4, 64, x, "f32", stream=0)
    p = cr.prepare(call)
    gc.collect()
    assert made[0]() is None, "the function's own is gone"
    noise = [cr.Q8(1, 2, 3, 4) for _ in range(10000)]  # takes what was freed
    want = codes.data_ptr(), 64, scales.data_ptr(), 1
    assert fields(words(p, 0)[5]) == want and fields(words(p, 1)[0]) == want
    del noise


def test_a_prepared_call_keeps_the_q8_it_was_given():
    """Changed later, or its tensors dropped by everyone else."""
    x, (codes, scales) = torch.zeros(4, 64), parts()
    q = cr.Q8(codes, scales)
    p = cr.prepare(cr.cr_q8_store, x, 4, 64, "f32", q, stream=0)
    want = codes.data_ptr(), 64, scales.data_ptr(), 1
    refs = [weakref.ref(codes), weakref.ref(scales)]
    other = parts()
    q.__init__(*other)
    del codes, scales
    gc.collect()
    assert fields(words(p)[5]) == want
    assert all(r() is not None for r in refs)
    del p
    gc.collect()
    assert all(r() is None for r in refs)


def test_tensors_made_while_recording_are_held():
    made = []

    def call():
        x, w, y, rstd = torch.zeros(4, 64), torch.ones(64), torch.zeros(4, 64), torch.zeros(4)
        made.extend(weakref.ref(t) for t in (x, w, y, rstd))
        cr.cr_rms_norm(x, None, w, 4, 64, "f32", 1e-6, None, y, None, rstd, stream=0)
    p = cr.prepare(call)
    gc.collect()
    assert all(r() is not None for r in made)
    got = words(p)
    assert [got[0], got[4], got[11], got[14]] == [r().data_ptr() for r in made]


def test_calls_outside_prepare_hold_nothing():
    codes, scales = parts()
    q = cr.Q8(codes, scales)
    p = cr.prepare(cr.cr_q8_store, torch.zeros(4, 64), 4, 64, "f32", q, stream=0)
    n = len(p._keep[3])
    with pytest.raises(cr.CRError):
        cr.cr_q8_store(torch.zeros(4, 64), 4, 64, 9, q, stream=0)
    assert len(p._keep[3]) == n
