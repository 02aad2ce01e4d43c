"""sv_adjust_logits on batches that fill the card, where a wave takes several rows of
its session and starts after some, and the bound of the additions' rounding."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests import rules_ref as ref
from tests.test_gpu_adjust import Case, dev, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def repeated(case, n):
    """The batch of case's sessions n times over: its call's arguments."""
    tile = lambda a: dev(np.tile(a, (n,) + (1,) * (a.ndim - 1)))  # noqa: E731
    off, ids, val = case.bias
    offsets = np.concatenate([[0]] + [off[1:] + k * ids.size for k in range(n)]).astype(np.int32)
    return dict(tokens=tile(case.tokens), m=tile(case.m), penalties=tile(case.pen.view(np.uint8).reshape(case.B, 16)),
                history=sv.History(dev(case.counts), dev(case.seen)), slots=tile(case.slots),
                bias=sv.Bias(dev(offsets), dev(np.tile(ids, n)), dev(np.tile(val, n))), masks=dev(case.masks),
                mask_rows=tile(case.mask_rows))


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [110001, 110008])
@pytest.mark.parametrize("R", [9, 10, 17, 19])
def test_several_rows_a_wave(R, V, dtype):
    """40 sessions, 4 of them different: rows at odd addresses and at even ones, all of
    a session's in one wave or in two or three of up to 9."""
    case = Case(R, 4, R - 1, R, V, dtype, hist=2000, n_bias=200, ragged=R == 17)
    x = case.logits.cuda().repeat(10, 1, 1)
    args = repeated(case, 10)
    out = torch.full_like(x, 7.25)
    before = out[:4].clone()
    got = sv.adjust_logits(x, out=out, **args)
    torch.cuda.synchronize()
    assert (got["status"] == 0).all()
    case.check(out[:4], before)
    inside = sv.adjust_logits(x, out=x, **args)["logits"]
    torch.cuda.synchronize()
    case.check(inside[:4], case.logits)
    for y in (out, inside):
        assert torch.equal(bits(y[4:]), bits(y[:4].repeat(9, 1, 1)))


@pytest.mark.parametrize("B,M,V", [(1, 64, 700), (30, 64, 90), (500, 64, 33), (3, 5, 5003)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rounding(B, M, V, dtype):
    """However many drafted tokens are counted, a result is the same few roundings of u
    = 2^-24 away: with f the factor of the logit z, c the count, F and P the
    penalties, A the bias,
      the rounded reciprocal and the product, 2u |z f|,
      F c + P (rounded once), u (|F c| + |P|),
      its difference from A, u (|A| + |F c| + |P|), up to factors of 1 + u,
      the last sum, u (|z f| + |A| + |F c| + |P|), likewise,
    3u of the magnitudes' sum in all, the factors within 1 + 2^-20 and the
    product's underflow half of 2^-149; then half a step of the logits' type."""
    case = Case(77 + B, B, M, M + 1, V, dtype, rules="pb", hist=V, n_bias=V, ragged=False)
    case.tokens[:] = np.random.default_rng(B).choice([0, V // 2, V - 1], case.tokens.shape)
    case.bias[2][np.isinf(case.bias[2])] = 1e4  # cancels nothing that is finite
    exact, _, _, _ = case.reference()
    z, R = case.logits.double().numpy(), M + 1
    c, known = np.zeros(z.shape), np.zeros(z.shape, bool)
    for b in range(B):
        h = case.slots[b]
        if h >= 0:
            c[b] += case.counts[h]
            known[b] |= ref.unpack(case.seen[h, 0], V)
        for r in range(1, R):
            for t in case.tokens[b, :r]:
                c[b, r, t] += 1
    known |= c > 0
    rep, freq, pres = (case.pen[k].astype(np.float64)[:, None, None] for k in ("repetition", "frequency", "presence"))
    size = np.where(known, np.where(z > 0, z / rep, -z * rep), np.abs(z)) + np.abs(freq) * c + np.abs(pres) * (c > 0)
    off, ids, val = case.bias
    for b in range(B):
        size[b][:, ids[off[b]:off[b + 1]]] += np.abs(val[off[b]:off[b + 1]].astype(np.float64))
    err = 3 * 2.0**-24 * (1 + 2.0**-20) * size + 2.0**-149
    if dtype == "bf16":
        err = err + ref.HALF_STEP[dtype] * (np.abs(exact) + err) + 2.0**-134
    out = filled(case)
    case.run(out=out)
    x = case.logits.cuda()
    case.run(logits=x, out=x)
    torch.cuda.synchronize()
    for got in (out, x):
        over = np.abs(got.double().cpu().numpy() - exact) - err
        assert over.max() <= 0, (over.max(), int((over > 0).sum()))
