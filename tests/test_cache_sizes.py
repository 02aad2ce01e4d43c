"""Bytes of sv_cache_attention's workspace: what its rows' partial results take."""
import itertools

import pytest

import token_sampling_amd as sv
from tests.test_cache_host import built, struct  # noqa: F401 (built: a fixture)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("n_kv", [1, 2, 8])
def test_attention_bytes(n_kv, dim):
    """A binary32 result, its sum and its reference value (dim + 2 values) a row and head: once;
    once more where a key head's rows are too many for registers; two more where so many
    sessions can share enough.  And at most 64 rows (and 192 in the latter cases) for
    each of 512 pieces."""
    for B, R, G, pages in itertools.product((1, 2, 64, 4096), (1, 9, 65), (1, 4, 7), (1, 100, 1 << 14)):
        c = struct(n_kv=n_kv, head_dim=dim, max_pages=pages, n_slots=4096)
        many = R * G > (16 if dim == 256 else 64)
        share = B > 1 and pages * 64 >= 180000000 // (n_kv * dim * min(max(B, 20), 140))
        places = (1 + many + 2 * share) * B * R * G * n_kv + 512 * (64 + 192 * (many or share))
        got = sv.lib().sv_cache_attention_bytes(c, n_kv * G, B, R)
        assert 4 * (dim + 2) * B * R * G * n_kv < got <= 4 * (dim + 2) * places


def test_attention_bytes_of_one_row():
    """One session, one row, 32 heads of 128 in groups of 4."""
    c = struct(n_kv=8, max_pages=4096)
    assert sv.lib().sv_cache_attention_bytes(c, 32, 1, 1) <= 5 << 20
