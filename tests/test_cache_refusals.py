"""Host-side refusals of the cache's calls beside tests/test_cache_host.py's: no kernel is
launched."""
import pytest

import token_sampling_amd as sv
from tests.test_cache_host import FAKE, built, compact, reserve, struct  # noqa: F401 (built: a fixture)


@pytest.mark.parametrize("call", [reserve, compact], ids=lambda f: f.__name__)
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_workspace_alignment(call, off):
    assert call(struct(), ws=FAKE + off) == sv.ERR_ARG
