"""A prompt of which a part is cached already: the rest goes through attention in rounds of rows,
each kept before the next."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import Ref
from tests.test_gpu_cache_attention import check, dev, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rest_of_a_prompt(dtype):
    """Two sessions go on from 100 cached tokens with 150 and 67 of their own."""
    rng = np.random.default_rng(1)
    Hkv, Hq, dim, R, rest = 2, 4, 64, 65, [150, 67]
    cache = sv.make_cache(3, 20, 5, Hkv, dim, page=64, dtype=dtype)
    cache.k.zero_(), cache.v.zero_()
    kv = torch.from_numpy(rng.standard_normal((2, 1, 100, Hkv, dim))).to(dtype).cuda()
    assert not sv.cache_reserve(cache, dev([100]), slots=dev([0])).any()
    sv.cache_write(cache, 0, kv[0], kv[1], slots=dev([0]))
    assert not sv.cache_keep(cache, dev([100]), slots=dev([0])).any()
    assert not sv.cache_fork(cache, dev([0, 0]), dev([1, 2])).any()
    line = torch.from_numpy(rng.standard_normal((2, sum(rest), Hkv, dim))).to(dtype).cuda()
    starts, done = [0, rest[0]], np.zeros(2, int)
    while (done < rest).any():
        rows = np.minimum(np.array(rest) - done, R)
        assert not sv.cache_reserve(cache, dev(rows), slots=dev([1, 2])).any()
        k, v = (torch.zeros((2, R, Hkv, dim), dtype=dtype, device="cuda") for _ in range(2))
        for b, (start, n) in enumerate(zip(starts + done, rows)):
            k[b, :n], v[b, :n] = line[0, start:start + n], line[1, start:start + n]
        sv.cache_write(cache, 0, k, v, slots=dev([1, 2]), rows=dev(rows))
        ref = Ref(cache)
        ref.sound()
        check(cache, ref, [1, 2], rows, queries(rng, (2, R, Hq, dim), dtype))
        assert not sv.cache_keep(cache, dev(rows), slots=dev([1, 2])).any()
        done += rows
    # what the rounds left is what one write of the whole line leaves
    assert cache.lens.tolist() == [100] + [100 + n for n in rest]
    keys, values = sv.cache_order(64, dim)
    for x, order, whole in ((cache.k, keys, line[0]), (cache.v, values, line[1])):
        for h, start, n in ((1, 0, rest[0]), (2, rest[0], rest[1])):
            pages = cache.table[h, :cache.held[h]].long()
            got = x[0, pages].flatten(2)[:, :, torch.from_numpy(order).cuda()].transpose(1, 2).reshape(-1, Hkv, dim)
            assert torch.equal(got[100:100 + n].view(torch.int16), whole[start:start + n].view(torch.int16))
