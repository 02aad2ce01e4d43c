"""sv_count_tokens against a plain history (tests/rules_ref.py), exactly."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests import rules_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def start(rng, n, V):
    counts = np.where(rng.random((n, V)) < 0.2, rng.integers(1, 9, (n, V)), 0).astype(np.int32)
    seen = np.stack([ref.pack(rng.random((n, V)) < 0.1), ref.pack(counts > 0)], 1)
    return counts, seen


def same(history, counts, seen):
    torch.cuda.synchronize()
    assert np.array_equal(history.counts.cpu().numpy(), counts)
    assert np.array_equal(history.seen.cpu().numpy(), seen)


@pytest.mark.parametrize("prompt,clear", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("B,L,V", [(1, 1, 1), (1, 1, 33), (3, 9, 1000), (5, 65, 32), (4, 0, 50), (300, 5, 64),
                                   (2, 300, 31), (3, 4097, 5000), (2, 20000, 40001), (2, 1000, 300001)])
def test_rows_of_tokens(B, L, V, prompt, clear):
    rng = np.random.default_rng(B * 1000 + L)
    counts, seen = start(rng, B + 2, V)
    h = sv.History(dev(counts), dev(seen))
    slots = rng.permutation(B + 2)[:B].astype(np.int32)
    tokens = np.minimum((V * rng.random((B, L)) ** 3).astype(np.int32), V - 1)  # many repeats
    tokens[rng.random((B, L)) < 0.05] = -1
    tokens[rng.random((B, L)) < 0.02] = V
    lens = rng.integers(-1, L + 2, B).astype(np.int32)
    for use in (lens, None):
        sv.count_tokens(h, dev(tokens), slots=dev(slots), lens=dev(use), prompt=prompt, clear=clear)
        n = np.full(B, L) if use is None else use.clip(0, L)
        counts, seen = ref.note(counts, seen, slots, [tokens[b, :n[b]] for b in range(B)], 0 if prompt else 1, clear)
        same(h, counts, seen)


@pytest.mark.parametrize("L", [2, 2100])
def test_more_sessions_than_a_launch(L):
    rng = np.random.default_rng(2)
    B, V = 33000, 5
    h = sv.make_history(B, V)
    tokens = rng.integers(-1, V, (B, L)).astype(np.int32)
    sv.count_tokens(h, dev(tokens))
    torch.cuda.synchronize()
    want = np.stack([(tokens == v).sum(1) for v in range(V)], 1)
    assert np.array_equal(h.counts.cpu().numpy(), want)
    assert np.array_equal(ref.unpack(h.seen[:, 1].cpu().numpy(), V), want > 0)
    assert not h.seen[:, 0].any()
    sv.count_tokens(h, dev(tokens), prompt=True, clear=True)
    torch.cuda.synchronize()
    assert not h.counts.any() and not h.seen[:, 1].any()
    assert np.array_equal(ref.unpack(h.seen[:, 0].cpu().numpy(), V), want > 0)


@pytest.mark.parametrize("prompt", [True, False])
@pytest.mark.parametrize("lens", [[0], [1], [3, 0, 5], [0, 0, 0], [700, 1, 0, 12000], [40000]])
def test_line_of_tokens(lens, prompt):
    rng = np.random.default_rng(sum(lens))
    B, V = len(lens), 30011
    counts, seen = start(rng, B, V)
    h = sv.History(dev(counts), dev(seen))
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = np.minimum((V * rng.random(offsets[-1]) ** 4).astype(np.int32), V - 1)
    sv.count_tokens(h, dev(tokens), offsets=dev(offsets), prompt=prompt, clear=prompt)
    spans = [tokens[offsets[b]:offsets[b + 1]] for b in range(B)]
    same(h, *ref.note(counts, seen, None, spans, 0 if prompt else 1, prompt))


@pytest.mark.parametrize("L", [7, 9000])
def test_slots_shared_and_outside(L):
    """Sessions that name one slot add up; slots outside the pool are skipped."""
    rng = np.random.default_rng(L)
    V = 513
    counts, seen = start(rng, 4, V)
    h = sv.History(dev(counts), dev(seen))
    slots = np.array([2, -1, 2, 4, 0, 2], np.int32)
    tokens = rng.integers(0, V, (6, L)).astype(np.int32)
    tokens[:, 0] = 3
    for clear in (False, True):
        for prompt in (False, True):
            sv.count_tokens(h, dev(tokens), slots=dev(slots), prompt=prompt, clear=clear)
            counts, seen = ref.note(counts, seen, slots, list(tokens), 0 if prompt else 1, clear)
            same(h, counts, seen)


@pytest.mark.parametrize("offsets", [[-5, 3, 20], [0, 9, 4], [4, 4, 99]])
def test_offsets_are_cut_to_the_line(offsets):
    rng = np.random.default_rng(1)
    counts, seen = start(rng, 2, 40)
    h = sv.History(dev(counts), dev(seen))
    tokens = rng.integers(0, 40, 10).astype(np.int32)
    sv.count_tokens(h, dev(tokens), offsets=dev(np.array(offsets, np.int32)))
    spans = [tokens[max(0, offsets[b]):min(10, max(0, offsets[b + 1]))] for b in range(2)]
    same(h, *ref.note(counts, seen, None, spans, 1, False))


def test_one_token_many_times():
    h = sv.make_history(1, 100)
    sv.count_tokens(h, torch.full((1, 100000), 7, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert h.counts[0, 7] == 100000 and h.counts.sum() == 100000 and h.seen.count_nonzero() == 1


def test_captured_and_replayed():
    rng = np.random.default_rng(3)
    B, L, V = 40, 9, 2000
    counts, seen = start(rng, B, V)
    h = sv.History(dev(counts), dev(seen))
    tokens = torch.zeros((B, L), dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    sv.count_tokens(h, tokens, lens=lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.count_tokens(h, tokens, lens=lens)
    for _ in range(4):
        t, n = rng.integers(-1, 30, (B, L)).astype(np.int32), rng.integers(0, L + 1, B).astype(np.int32)
        tokens.copy_(dev(t)), lens.copy_(dev(n))
        g.replay()
        counts, seen = ref.note(counts, seen, None, [t[b, :n[b]] for b in range(B)], 1, False)
        same(h, counts, seen)
        sv.count_tokens(h, tokens, lens=lens, clear=True)  # eager, between replays
        counts, seen = ref.note(counts, seen, None, [t[b, :n[b]] for b in range(B)], 1, True)
        same(h, counts, seen)


def test_other_stream_and_refusals():
    h = sv.make_history(2, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sv.count_tokens(h, torch.tensor([[1, 1], [2, -1]], dtype=torch.int32, device="cuda"), stream=side)
    side.synchronize()
    assert h.counts[0, 1] == 2 and h.counts[1, 2] == 1 and h.counts.sum() == 3
    t = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        sv.count_tokens(h, t.long())
    with pytest.raises(ValueError):
        sv.count_tokens(h, t[:, 0])
    with pytest.raises(ValueError):
        sv.count_tokens(h, torch.zeros((3, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sv.count_tokens(h, t.view(-1), offsets=torch.zeros(2, dtype=torch.int32, device="cuda"), lens=t[0])
    with pytest.raises(ValueError):
        sv.count_tokens(sv.History(h.counts, h.seen[:, :, :1].contiguous()), t)
