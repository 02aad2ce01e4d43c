"""The attention's workspace and plan: nothing behind their sizes is written, and nothing that they
held before the call counts."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.test_gpu_cache_attention import dev, queries
from tests.test_gpu_cache_sets import shared_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


@pytest.mark.parametrize("n,common,own,n_kv,G,dim,R", [
    (1, 0, 1, 1, 1, 64, 1), (1, 40, 30000, 2, 8, 128, 2), (7, 32, 3000, 2, 4, 64, 9), (7, 32, 900, 2, 4, 128, 33),
    (3, 64, 5000, 1, 7, 256, 5), (150, 1280, 200, 8, 2, 128, 3), (150, 1280, 200, 8, 4, 128, 17),
    (150, 2560, 300, 8, 1, 64, 2), (30, 4480, 700, 8, 1, 256, 9)])
def test_workspace_and_plan(n, common, own, n_kv, G, dim, R):
    rng = np.random.default_rng(n + dim + R)
    rows = rng.integers(0, R + 1, n)
    rows[0] = R
    cache, _ = shared_cache(n, common, [], rng.integers(own // 2, own + 1, n), n_kv, dim, 64, torch.bfloat16, rows)
    q = queries(rng, (n, R, n_kv * G, dim), torch.bfloat16).cuda()
    plan = sv.cache_plan(cache, n_kv * G, R, rows=dev(rows), slots=dev(range(n)))
    size, need, guard = plan.buffer.numel(), plan.workspace_bytes, 1 << 16
    outs = []
    for fill in (0x00, 0x7F, 0xFF):  # zeros, large values, NaN
        plan_bytes = torch.full((size + guard,), fill, dtype=torch.uint8, device="cuda")
        work = torch.full((need + guard,), fill, dtype=torch.uint8, device="cuda")
        plan = sv.cache_plan(cache, n_kv * G, R, rows=dev(rows), slots=dev(range(n)),
                             out=plan._replace(buffer=plan_bytes))
        assert plan.buffer is plan_bytes and plan.workspace_bytes == need
        outs.append(sv.cache_attention(cache, 0, q, plan, out=torch.zeros_like(q), workspace=work))
        assert (plan_bytes[size:] == fill).all() and (work[need:] == fill).all()
    assert outs[0].isfinite().all() and outs[0].any()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
