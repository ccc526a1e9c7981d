"""The embedding's gradient with one workspace for call after call, each of other ids: what a call finds
there is of the call before, and means nothing.  Nothing synchronises in between."""
import pytest
import torch

import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = 24


@pytest.fixture(scope="module", autouse=True)
def built():
    from fsdp_emulated_ranks_gb300 import build
    build.build()


def batches(tokens, vocab, dim, dt, based):
    """Ids, gradients and bases of different calls: of one call few rows have no token, of the next nearly all."""
    g = T.gen(tokens + vocab)
    out = []
    for k in range(CALLS):
        ids = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
        if k % 3 == 1:
            ids = T.skewed(g, tokens, vocab)
        if k % 3 == 2:
            ids[:] = k % vocab
        out.append((ids, T.normal(g, tokens, dim, dt=dt), T.normal(g, vocab, dim, dt=dt) if based else None))
    return out


@pytest.mark.parametrize("based", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,vocab,dim", [(700, 900, 512), (8192, 4000, 520), (64, 20000, 65)])
def test_a_workspace_for_call_after_call(tokens, vocab, dim, dt, based):
    calls = batches(tokens, vocab, dim, dt, based)
    need = cr.cr_embedding_backward_workspace_bytes(tokens, vocab, dim)
    alone = torch.empty(CALLS, vocab, dim, dtype=T.TORCH[dt], device=DEV)
    for (ids, dout, base), dtable in zip(calls, alone):
        work = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
        cr.cr_embedding_backward(dout, dt, ids, tokens, vocab, dim, 0.5, base, dtable, dt, work, need)
        torch.cuda.synchronize()
    work = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    got = torch.empty_like(alone)
    # a captured call reads what its ids and base hold when it is replayed
    ids, dout, out = calls[0][0].clone(), calls[0][1].clone(), torch.empty_like(alone[0])
    base = calls[0][2].clone() if based else None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.cr_embedding_backward(dout, dt, ids, tokens, vocab, dim, 0.5, base, out, dt, work, need)

    def replay(k):
        ids.copy_(calls[k][0])
        dout.copy_(calls[k][1])
        if based:
            base.copy_(calls[k][2])
        graph.replay()
        got[k].copy_(out)

    def call(k):
        i, d, b = calls[k]
        cr.cr_embedding_backward(d, dt, i, tokens, vocab, dim, 0.5, b, got[k], dt, work, need)

    def call_on_one_base(k):
        i, d, b = calls[k]
        if based:  # written by the kernel just before
            base.copy_(b)
            b = base
        cr.cr_embedding_backward(d, dt, i, tokens, vocab, dim, 0.5, b, got[k], dt, work, need)
    for one in (call, call_on_one_base, replay):
        got.fill_(7.0)
        for k in range(CALLS):
            one(k)
        torch.cuda.synchronize()
        assert torch.equal(got, alone), one.__name__
