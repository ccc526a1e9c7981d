"""The bounded waits of the gated block's kernels, and the word that reports one
that ran out (cr_glu_wait_word)."""
import importlib.util
import os

import pytest
import torch

import ffn_ref as R
import test_ffn_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sums_longer_than_a_wait():
    """One tile whose K is ten million blocks, in four blocks of a cluster: 2.5 million each of
    at least 512 cycles, more than the 2^30 that any other wait may last.  Few
    values are not zero, so that every sum is exact."""
    dim, g = 640_000_000, T.gen(2)
    x = torch.zeros(1, dim, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, dim, dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, dim, (400,), generator=g, device="cuda")
    at[:4] = torch.tensor([0, dim - 1, dim // 2, dim // 4 * 3], device="cuda")
    x[0, at], w[0, at] = 1.0, 0.25
    want = float((x[0, at.unique()].double() * w[0, at.unique()].double()).sum())
    a = torch.zeros(1, 1, dtype=torch.bfloat16, device="cuda")
    q, gc, gs, _ = T.new_q8(1, 1)
    work = torch.empty(cr.cr_glu_workspace_bytes(1, dim, 1), dtype=torch.uint8, device="cuda")
    cr.cr_glu(x, w, w, 1, dim, 1, "bf16", "silu", a, q, None, work, work.numel())
    assert cr.cr_glu_wait_word() == 0
    R.assert_q8(gc, gs, torch.full((1, 1), want, dtype=torch.float64, device="cuda"))
    assert abs(float(a) - want * want) <= (R.U16 + 2.0 ** -18) * want * want  # silu(100) = 100


def test_example_stops_when_a_wait_ran_out(monkeypatch):
    spec = importlib.util.spec_from_file_location("feed_forward_step",
                                                  os.path.join(ROOT, "examples", "feed_forward_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    monkeypatch.setattr(example.cr, "cr_glu_wait_word", lambda clear=False: 1)
    with pytest.raises(RuntimeError, match="wait"):
        example.train(2, 40, 64, 72, steps=2)


def test_wait_word_waits_for_every_stream():
    """The word is read after what is still queued on a stream of the caller's own (which
    the default stream does not wait for): here some 0.2 s of work and an event behind it."""
    stream, done = torch.cuda.Stream(), torch.cuda.Event()
    assert cr.cr_glu_wait_word() == 0  # the library is loaded, its module too
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)
        done.record()
    assert cr.cr_glu_wait_word() == 0
    assert done.query()


def test_no_wait_ran_out_on_streams_or_in_graphs():
    """Read behind concurrent, prepared and captured calls."""
    T.test_streams()
    T.test_prepared_and_captured()
    assert cr.cr_glu_wait_word() == 0
