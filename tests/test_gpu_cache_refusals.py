"""Refusals of the cache's binding that need tensors on the GPU, beside those of
tests/test_gpu_cache_attention.py: the calls return before a kernel is launched."""
import pytest
import torch

import token_sampling_amd as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


@pytest.mark.parametrize("plane", ["k", "v"])
def test_out_in_the_cache(plane):
    """out may not lie in the pages that the call reads, nor reach into them; beside them
    it may."""
    pool = torch.zeros((2, 3, 2, 2, 32, 64), dtype=torch.bfloat16, device="cuda")
    cache = sv.make_cache(2, 2, 2, 2, 64, page=32)
    cache = cache._replace(**{plane: pool[:, 1:2][0]})
    assert not sv.cache_reserve(cache, torch.ones(2, dtype=torch.int32, device="cuda")).any()
    cache.k.zero_(), cache.v.zero_()
    plan = sv.cache_plan(cache, 4, 1)
    q = torch.ones((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    n, at = q.numel(), 2 * 2 * 32 * 64  # the plane is at .. 2 * at - 1 of the pool's elements
    for begin in (at, at + 64, 2 * at - n, at - n + 64, 2 * at - 64):
        with pytest.raises(ValueError, match="overlaps the cache"):
            sv.cache_attention(cache, 0, q, plan, out=pool.view(-1)[begin:begin + n].view(q.shape))
    for begin in (at - n, 2 * at):
        out = pool.view(-1)[begin:begin + n].view(q.shape)
        out.fill_(7)
        assert not sv.cache_attention(cache, 0, q, plan, out=out).any()


@pytest.mark.parametrize("other", [dict(page=64, max_pages=4), dict(n_slots=3), dict(max_pages=7)])
def test_plan_of_another_cache(other):
    """A plan names slots and places in their lists: of a cache with fewer or shorter ones it would
    lead behind the table."""
    sizes = dict(n_slots=5, n_pages=20, max_pages=8, n_kv=2, head_dim=64, page=32)
    cache, wrong = sv.make_cache(**sizes), sv.make_cache(**{**sizes, **other})
    assert not sv.cache_reserve(cache, torch.full((2,), 200, dtype=torch.int32, device="cuda")).any()
    plan = sv.cache_plan(cache, 4, 1, B=2)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="plan is of a cache of other pages"):
        sv.cache_attention(wrong, 0, q, plan)
    for x in cache[:2]:
        x.zero_()
    layer = cache._replace(k=cache.k.clone(), v=cache.v.clone())  # another layer's planes, the same lists
    assert not sv.cache_attention(layer, 0, q, plan).any()
