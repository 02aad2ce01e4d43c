"""sv_cache_attention where nearly all weight is on a few keys whose values are 0, so that the
output is what the many small weights carry."""
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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bits", [14, 21, 24.5, 26, 28])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("R", [1, 5, 9, 15, 33])
def test_small_weights(R, dim, bits, dtype):
    """Every 32nd key's score lies `bits` powers of two above the others', which are equal.
    4 query heads a key head: 4 to 60 rows in registers, 132 in wide sets."""
    Hkv, Hq, page, lens = 2, 8, 64, [300, 40]
    cache = sv.make_cache(2, 14, 7, Hkv, dim, page=page, dtype=dtype)
    rng = np.random.default_rng(R)
    ref = filled(cache, rng, [n + R for n in lens])
    as_bits = lambda x: torch.tensor(x).to(dtype).view(torch.int16).item()  # noqa: E731
    high = float(torch.tensor(bits * np.log(2) / dim ** 0.5).to(dtype))
    ref.k[:], ref.v[:] = 0, as_bits(4096.0)
    ref.k[..., ::32, :], ref.v[..., ::32, :] = as_bits(high), 0
    ref.lens[:] = lens
    ref.store()
    q = torch.ones((2, R, Hq, dim), dtype=dtype, device="cuda")
    plan = sv.cache_plan(cache, Hq, R)
    got = sv.cache_attention(cache, 0, q, plan).double().cpu().numpy()
    assert not plan.status.any()
    z = high * dim ** 0.5
    e = (dim + 8) * 2.0**-23 * abs(z)  # scores: products summed, scaled twice, put into exp2
    u = torch.finfo(dtype).eps / 2
    for b in range(2):
        for r in range(R):
            t = lens[b] + r + 1
            n_high = -(-t // 32)
            n_low = t - n_high
            small = np.exp(-z)
            want = 4096 * n_low * small / (n_high + n_low * small)
            # the output's rounding (halves below 2^-14: 2^-25), the weights', sums of t terms; and what
            # halves lose of small weights: 2^-25 each where the n_high largest are at least 2^7
            tol = 2 * u * want + want * ((t + 4) * 2.0**-23 + 2 * e)
            if dtype == torch.float16:
                tol += 2.0**-25 + 4096 * n_low * 2.0**-32 / n_high
            assert (np.abs(got[b, r] - want) <= tol).all(), (b, r, want, tol, np.abs(got[b, r] - want).max())


@pytest.mark.parametrize("dim,R", [(64, 1), (128, 9), (64, 12), (96, 15), (256, 1), (64, 33), (128, 33)])
@pytest.mark.parametrize("dtype,power", [(torch.float16, 23.2), (torch.float16, 24.4), (torch.float16, 25.7),
                                         (torch.float16, 26.8), (torch.bfloat16, 25.7), (torch.bfloat16, 29.5)])
def test_large_scores(dim, R, dtype, power):
    """Scores of about 2^power, whose last binary32 digit is worth one to many powers of two, rising
    from block to block of keys by steps of that size: outputs are means of what the keys
    hold, never NaN or infinite.  One session listed 64 times, so that a wave has many tiles."""
    Hkv, G, page, n, B = 8, 4, 64, 800, 64
    cache = sv.make_cache(1, 14, 14, Hkv, dim, page=page, dtype=dtype)
    rng = np.random.default_rng(R)
    ref = filled(cache, rng, [n + R])
    as_bits = lambda x: torch.from_numpy(np.asarray(x)).to(dtype).view(torch.int16).numpy()  # noqa: E731
    # half the dimensions make the scores' size, one the steps, which differ from row to row
    size = 2.0**power / np.log2(np.e) / (dim // 2)
    side = 2.0**np.floor(np.log2(size) / 2)
    k, q = np.zeros(dim), np.zeros((B, R, Hkv * G, dim))
    k[:dim // 2] = side
    q[..., :dim // 2] = size / side * rng.uniform(0.9, 1.1, (B, R, Hkv * G, 1))
    q[..., dim - 1] = rng.integers(2, 15, (B, R, Hkv * G))
    for t in range(n + R):
        p, u = ref.table[0, t // page], t % page
        k[dim - 1] = t // 128
        ref.k[0, p, :, u] = as_bits(k)
        ref.v[0, p, :, u] = as_bits(np.full(dim, 1.0 + t // 128))
    ref.lens[:] = n
    ref.store()
    slots = dev([0] * B)
    plan = sv.cache_plan(cache, Hkv * G, R, slots=slots)
    got = sv.cache_attention(cache, 0, torch.from_numpy(q).to(dtype).cuda(), plan, scale=1.0)
    assert not plan.status.any()
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    # between the smallest and the largest value, with the weights', the output's and the sums' roundings
    slack = 1 + 2 * torch.finfo(dtype).eps / 2 + (n + R + 4) * 2.0**-23
    assert (got >= 1 / slack).all() and (got <= (1 + (n + R) // 128) * slack).all()
