"""Rows that share logits are not adjusted in place: a failed session writes all its
rows, the unused ones too, so none may belong to another session."""
import itertools

import numpy as np
import pytest
import torch

import token_sampling_amd as sv

FAKE = 0x1000  # never dereferenced: the calls return first


def refused(ss, rs, B, R, V):
    """A call in place of B sessions of R target rows, known to overlap."""
    return sv.lib().sv_adjust_logits(FAKE, ss, rs, sv.BF16, FAKE, FAKE, FAKE, None, None, None, None, B, R - 1, R,
                                     V, FAKE, FAKE, None) == sv.ERR_ARG


def apart(ss, rs, B, R, V):
    at = sorted(b * ss + r * rs for b in range(B) for r in range(R))
    return all(y - x >= V for x, y in zip(at, at[1:]))


@pytest.mark.parametrize("ss,rs,B,R,V", [
    (30, 10, 2, 4, 10),    # three of four rows' room a session
    (39, 10, 2, 4, 10),    # one logit short
    (10, 20, 3, 3, 10),    # transposed, two of three sessions' room
    (0, 10, 2, 3, 10), (30, 0, 2, 3, 10), (9, 1000, 2, 1, 10), (1000, 9, 1, 2, 10),
    (1 << 40, 1 << 40, 2, 2, 10),
    (30, 19, 3, 3, 10)])   # rows between each other's, two of them in one place
def test_refuses_shared_rows(ss, rs, B, R, V):
    assert not apart(ss, rs, B, R, V)
    assert refused(ss, rs, B, R, V)


def test_refuses_what_overlaps():
    """Every small layout against the rows' places one by one: the binding's test,
    and the library's where it refuses."""
    for B, R, V in itertools.product((1, 2, 3, 5), (1, 2, 3, 6), (1, 3)):
        for ss, rs in itertools.product(range(0, 26), repeat=2):
            want = apart(ss, rs, B, R, V)
            assert sv._rows_apart(ss, rs, B, R, V) == want, (ss, rs, B, R, V)
            if not want:
                assert refused(ss, rs, B, R, V), (ss, rs, B, R, V)


@pytest.mark.gpu
@pytest.mark.parametrize("ss,rs", [(5, 1), (1, 3), (3, 2)], ids=["sessions", "transposed", "between"])
def test_layouts_in_place(ss, rs):
    """Rows side by side, transposed, and between each other's (strides of 3 and 2
    rows), with sessions that fail beside sound ones; what lies between them stays."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B, M, R, V = (3, 4, 5, 517) if ss != 3 else (4, 1, 2, 517)
    room = V + 3
    x = torch.full(((B - 1) * ss * room + (R - 1) * rs * room + V,), 9.0, device="cuda")
    rows = x.as_strided((B, R, V), (ss * room, rs * room, 1))
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows.copy_(torch.randn((B, R, V), device="cuda", generator=gen))
    before, logits = x.clone(), rows.clone()
    tokens = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    m = torch.full((B,), M - 1, dtype=torch.int32)
    m[1] = M + 1  # out of range
    pen = sv.make_penalties(B, 2.0)
    bias = sv.make_bias([{5: 1.5}] * B, V)
    got = sv.adjust_logits(rows, tokens, m.cuda(), penalties=pen, bias=bias, out=rows)
    torch.cuda.synchronize()
    assert got["status"].tolist() == [sv.S_LIMIT if b == 1 else 0 for b in range(B)]
    want = logits.clone()
    want[:, :M, 5] += 1.5
    z = want[:, 1:M, 0]
    want[:, 1:M, 0] = torch.where(z > 0, z / 2, z * 2)
    want[1] = float("nan")
    assert torch.equal(torch.nan_to_num(rows, 77.0), torch.nan_to_num(want, 77.0))
    used = np.zeros(x.numel(), bool)
    for b, r in itertools.product(range(B), range(R)):
        at = (b * ss + r * rs) * room
        used[at:at + V] = True
    between = torch.from_numpy(~used).cuda()
    assert torch.equal(x[between], before[between])
