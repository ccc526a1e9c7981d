"""Calls of the language model operators on two streams at once write all of their outputs."""
import pytest
import torch

import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from fsdp_emulated_ranks_gb300 import build
    build.build()


def test_two_streams():
    """A workspace each; outputs and workspaces are cleared before every round."""
    one, outs, _ = T.calls(T.gen(41))
    two, outs2, _ = T.calls(T.gen(42))
    want = []
    for cases, o in ((one, outs), (two, outs2)):
        for fn, args in cases:
            fn(*args)
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for t in outs + outs2:
            t.fill_(-1 if t.dtype == torch.int32 else float("nan"))
        for cases in (one, two):
            for fn, args in cases:
                if fn is cr.cr_embedding_backward:
                    args[-2].fill_(0xA5)
        torch.cuda.synchronize()
        for (f, a), (h, b) in zip(one, two):
            f(*a, stream=streams[0])
            h(*b, stream=streams[1])
        torch.cuda.synchronize()
        for o, w in zip((outs, outs2), want):
            for a, b in zip(o, w):
                assert torch.equal(a, b)
