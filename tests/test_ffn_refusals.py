"""Arguments of the feed-forward calls that are in range as given but not in the type
a kernel computes in.  No GPU: every call is refused, or has nothing to do."""
import pytest

from fsdp_emulated_ranks_gb300 import build as libbuild
from fsdp_emulated_ranks_gb300 import cr

FAKE = 1 << 40  # an address never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def norm(eps, rows):
    cr.cr_rms_norm(FAKE, None, FAKE + (1 << 20), rows, 64, "f32", eps, None, FAKE + (1 << 21), None, None, 0,
                   ldx=64, ldy=64)


@pytest.mark.parametrize("eps", [1e39, 3.4028236e38, 1e300])
def test_eps_beyond_fp32_is_refused(eps):
    """It would be infinite in the kernel, and every rstd 0."""
    for rows in (0, 4):
        with pytest.raises(cr.CRError, match="finite in fp32") as ei:
            norm(eps, rows)
        assert ei.value.status == 1


@pytest.mark.parametrize("eps", [0.0, 1e-50, 1e-6, 3.4e38])
def test_eps_within_fp32_is_taken(eps):
    norm(eps, 0)
