"""sv_cache_fork's refusals, place by place as include/specverify.h states them."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import Ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


NO = sv.S_BAD_CACHE


@pytest.mark.parametrize("src,dst,status,lens", [
    ([0, 3], [3, 5], [0, NO], {3: 40}),  # taken over and given on at once: only the second is refused
    ([3, 0], [5, 3], [NO, 0], {3: 40}),  # in either order
    ([0, 3], [3, 3], [NO, NO], {}),  # listed twice
    ([0, -1], [3, 3], [NO, 0], {}),  # also by a place that is left alone
    ([-1, 3], [3, 5], [0, NO], {}),
    ([0, 3], [3, -1], [0, 0], {3: 40}),  # no dst: nothing that src would be given on to
    ([0, 0, 1], [3, 4, 5], [0, 0, 0], {3: 40, 4: 40, 5: 70}),
    ([0, 4], [1, 5], [NO, 0], {}),  # not empty; an empty src
    ([0, 0], [0, 3], [NO, NO], {}),  # a src of its own, which is then a dst as well
    ([4, 4], [4, 5], [NO, NO], {}),
])
def test_places(src, dst, status, lens):
    cache = sv.make_cache(6, 12, 4, 1, 64, page=32)
    sv.cache_reserve(cache, dev([40, 70, 0, 0, 0, 0]))
    sv.cache_keep(cache, dev([40, 70, 0, 0, 0, 0]))
    assert sv.cache_fork(cache, dev(src), dev(dst)).tolist() == status
    want = [40, 70, 0, 0, 0, 0]
    for h, n in lens.items():
        want[h] = n
    assert cache.lens.tolist() == want
    Ref(cache).sound()
