"""sv_cache_write of a part of a line: the first session's rows begin anywhere in it, and the
rows before them and behind the last session's belong to nobody."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("before", [1, 7, 8, 15, 16, 17, 24, 100, 1000])
@pytest.mark.parametrize("start", [0, 5, 8, 16])
@pytest.mark.parametrize("first", ["session", "nobody", "empty"])
def test_write_behind_other_rows(before, start, first):
    """Page 0 belongs to two sessions that the call does not name: nothing of it changes."""
    rng = np.random.default_rng(before + start)
    n_kv, dim, page = 2, 64, 32
    cache = sv.make_cache(5, 40, 8, n_kv, dim, n_layers=2, page=page)
    # slot 4 has the pool's first pages, slots 1..3 those behind them
    ref = filled(cache, rng, [0, start, start, start, 70], order=[7, 8, 9, 0, 1, 2] if start else [0, 1, 2])
    n = np.array([20, 0 if first == "empty" else 9, 33])
    slots = np.array([1, 2, 3])
    if first == "empty":
        n = n[[1, 0, 2]]
    if first == "nobody":
        slots[0] = -1
    got = sv.cache_reserve(cache, dev(n), slots=dev(slots))
    assert got.tolist() == ref.reserve(list(slots), n).tolist() == [0, 0, 0]
    sv.cache_fork(cache, dev([4]), dev([0]))
    assert ref.fork([4], [0]).tolist() == [0]
    offsets = before + np.concatenate([[0], np.cumsum(n)])
    kv = rng.integers(-30000, 30000, (2, offsets[-1] + 13, n_kv, dim)).astype(np.int16)
    k, v = (torch.from_numpy(x).cuda().view(torch.bfloat16) for x in kv)
    sv.cache_write(cache, 1, k, v, slots=dev(slots), offsets=dev(offsets))
    ref.write(1, slots, [(kv[0][lo:hi], kv[1][lo:hi]) for lo, hi in zip(offsets, offsets[1:])])
    ref.same()
    assert 0 in ref.table[4]
