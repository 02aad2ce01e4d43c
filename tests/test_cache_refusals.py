"""Host-side refusals of the cache's calls beside tests/test_cache_host.py's: no kernel is
launched."""
import pytest

import token_sampling_amd as sv
from tests.test_cache_host import FAKE, attention, built, compact, reserve, struct  # noqa: F401 (built: a fixture)


@pytest.mark.parametrize("call", [reserve, compact], ids=lambda f: f.__name__)
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_workspace_alignment(call, off):
    assert call(struct(), ws=FAKE + off) == sv.ERR_ARG


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scale_beyond_powers_of_two(scale):
    """Finite, but not once it counts powers of two: every score would be infinite or NaN."""
    assert attention(struct(), scale=scale, n=1 << 40) == sv.ERR_ARG
