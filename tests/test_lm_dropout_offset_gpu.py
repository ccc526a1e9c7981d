"""Dropout's masks over the steps of a model of several layers: no two calls share one where the offset moves by
the number of calls, and two would where it moved by less."""
import pytest
import torch

import test_lm_gpu as T
from fsdp_emulated_ranks_gb300 import cr

pytestmark = pytest.mark.gpu
LAYERS, STEPS = 3, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from fsdp_emulated_ranks_gb300 import build
    build.build()


def masks(move):
    x, rng = torch.ones(8, 512, device="cuda"), T.rng_of(7, 100)
    out = []
    for _ in range(STEPS):
        for layer in range(LAYERS):
            y = torch.empty_like(x)
            cr.cr_dropout(x, None, 8, 512, "f32", 0.5, rng, layer, 0, y)
            out.append((y != 0).flatten().tolist())
        rng[1] += move
    return {tuple(m) for m in out}


def test_masks_of_a_step_and_of_the_next():
    assert len(masks(LAYERS)) == LAYERS * STEPS
    assert len(masks(LAYERS + 2)) == LAYERS * STEPS
    assert len(masks(1)) == LAYERS + STEPS - 1  # call 1 of a step has call 0's of the next
