"""sv_adjust_logits: tokens that no rule changes keep their bits, signed zeros and
subnormals too, also where a rule looks at them and finds nothing to do."""
import numpy as np
import pytest
import torch

from tests import rules_ref as ref
from tests.test_gpu_adjust import Case, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


def quiet_case(seed, B, M, V, dtype, rules, repetition=1.0):
    """Zeros of both signs, subnormals and ordinary logits; penalties that change none
    of them (or zeros alone: a repetition penalty)."""
    case = Case(seed, B, M, M + 1, V, dtype, rules=rules, ragged=False)
    t = case.logits.dtype
    tiny = torch.finfo(t).tiny
    special = torch.tensor([0.0, -0.0, -0.0, tiny / 2, -tiny / 2, 1.0, -2.5] if repetition == 1.0 else [0.0, -0.0],
                           dtype=torch.float64).to(t)
    pick = torch.from_numpy(np.random.default_rng(seed).integers(0, special.numel(), case.logits.shape))
    case.logits = special[pick]
    case.pen["repetition"], case.pen["frequency"], case.pen["presence"] = repetition, 0, 0
    case.slots = np.arange(B, dtype=np.int32)
    return case


def results(case):
    out = filled(case)
    yield case.run(out=out)["logits"]
    x = case.logits.cuda()
    yield case.run(logits=x, out=x)["logits"]


# one row a wave (drafted tokens met before it), several rows a wave, and odd addresses
@pytest.mark.parametrize("B,M,V", [(1, 20, 1100), (2, 64, 515), (400, 6, 1099), (3, 0, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("repetition", [1.0, 1.3, 0.7])
def test_penalties_that_change_nothing(B, M, V, dtype, repetition):
    case = quiet_case(B + M, B, M, V, dtype, "p", repetition)
    for got in results(case):
        torch.cuda.synchronize()
        assert (bits(got) != bits(case.logits)).sum() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beside_biases_and_masks(dtype):
    case = quiet_case(5, 6, 9, 2050, dtype, "pbm")
    B, R, V = case.logits.shape
    same = np.ones((B, R, V), bool)
    off, ids, _ = case.bias
    for b in range(B):
        same[b][:, ids[off[b]:off[b + 1]]] = False
        for r in range(R):
            if case.mask_rows[b, r] >= 0:
                same[b, r] &= ref.unpack(case.masks[case.mask_rows[b, r]], V)
    for got in results(case):
        torch.cuda.synchronize()
        assert (bits(got)[same] != bits(case.logits)[same]).sum() == 0


@pytest.mark.parametrize("value,want", [(0.0, 0.0), (-0.0, -0.0)])
@pytest.mark.parametrize("B", [1, 300])
def test_zero_biases(value, want, B):
    """-0 plus a bias of either zero, by IEEE 754, in every row alike: met before a
    wave's first row, among its rows, or not at all."""
    case = quiet_case(9, B, 16, 700, "fp32", "p")
    case.logits[:] = -0.0
    case.tokens[:] = [3, 600, 3, 5] * 4
    case.bias = (np.arange(B + 1, dtype=np.int32) * 700, np.tile(np.arange(700, dtype=np.int32), B),
                 np.full(700 * B, value, np.float32))
    expect = bits(torch.full(case.logits.shape, want))
    for got in results(case):
        torch.cuda.synchronize()
        assert (bits(got) != expect).sum() == 0
