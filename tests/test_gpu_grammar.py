"""sv_grammar_masks and sv_grammar_advance against plain walks, exactly."""
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
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def check_masks(nxt, accept, tokens, end, states, grammar=None):
    g, v = grammar or sv.make_grammar(nxt, accept), sv.make_vocab(tokens, end)
    got = sv.grammar_masks(g, v, dev(states))
    torch.cuda.synchronize()
    rows = {s: ref.allowed(nxt, accept, tokens, end, s) for s in set(states)}
    want = np.stack([ref.pack(rows[s]) for s in states])
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 63, 64, 65, 127, 500, 2049])
@pytest.mark.parametrize("S,C", [(1, 1), (5, 3), (40, 20)])
def test_masks(V, S, C):
    rng = np.random.default_rng(V * 10 + S)
    nxt, accept = ref.random_grammar(rng, S, C, live=0.7)
    tokens = ref.random_vocab(rng, V)
    end = rng.choice(V, min(V, 3), replace=False).tolist()
    states = [-1, S, 2**31 - 1, -2**31] + rng.integers(0, S, 20).tolist()
    check_masks(nxt, accept, tokens, end, states)


@pytest.mark.parametrize("S,C", [(700, 256), (70000, 3), (900, 90), (66000, 1), (17, 256)])
def test_masks_of_large_automata(S, C):
    rng = np.random.default_rng(S)
    nxt, accept = ref.random_grammar(rng, S, C, live=0.8)
    tokens = ref.random_vocab(rng, 700, longest=40)
    check_masks(nxt, accept, tokens, [5], rng.integers(0, S, 30).tolist())


@pytest.mark.parametrize("n", [1, 2, 3, 64, 65, 257, 5000])
def test_numbers_of_states(n):
    rng = np.random.default_rng(n)
    nxt, accept = ref.random_grammar(rng, 12, 9, live=0.6)
    tokens = ref.random_vocab(rng, 77)
    check_masks(nxt, accept, tokens, [], rng.integers(-1, 12, n).tolist())


@pytest.mark.parametrize("S,C", [(30, 11), (600, 90), (700, 256), (250, 256), (1500, 37)])
@pytest.mark.parametrize("V,n", [(77, 9000), (2500, 5000), (6200, 40)])
def test_tables_by_units(S, C, V, n):
    """Automata of every place (both sizes in LDS, global memory), with a few
    states a tile and with many."""
    rng = np.random.default_rng(S + V)
    nxt, accept = ref.random_grammar(rng, S, C, live=0.9)
    tokens = ref.random_vocab(rng, V, longest=20)
    used = rng.integers(0, S, 25)  # the reference walks each state once
    check_masks(nxt, accept, tokens, [7, 70], np.concatenate([[-1, S], rng.choice(used, n)]).tolist())


def test_more_states_than_a_workgroup_has_at_hand():
    rng = np.random.default_rng(9)
    nxt, accept = ref.random_grammar(rng, 10, 6, live=0.8)
    tokens = ref.random_vocab(rng, 70001, longest=3, control=40)
    check_masks(nxt, accept, tokens, [0, 70000], rng.integers(-1, 10, 9000).tolist())


def test_long_tokens():
    """Tokens much longer than a word, refused at their first and at their last byte."""
    nxt = np.full((3, 256), -1, np.int32)
    nxt[0, 32] = 0  # any run of spaces
    nxt[0, 97], nxt[1, 98], nxt[2, 99] = 1, 2, 0
    tokens = [b" " * k for k in (1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 128, 1000)]
    tokens += [b" " * k + b"x" for k in (0, 7, 8, 15, 16, 17, 128)] + [b"abc" * 50, b"abc" * 50 + b"b", b"x" + b" " * 99]
    check_masks(nxt, np.array([1, 0, 0]), tokens, [], [0, 1, 2, -1])
    check_advance(nxt, np.array([1, 0, 0]), tokens, [], np.array([0, 0, 1]),
                  np.array([[12, 20, 11], [19, 0, 0], [20, 0, 1]]), np.array([3, 3, 3]))


def test_bytes_at_the_ends_of_their_array():
    rng = np.random.default_rng(8)
    nxt, accept = ref.random_grammar(rng, 6, 256, live=0.95)
    for tokens in ([b"a"], [b"", b"ab"], [b"abc", b""], [b""], [b"", b""], [bytes(range(13))]):
        check_masks(nxt, accept, tokens, [], list(range(-1, 6)))


def test_tables_that_hold_nonsense():
    """Classes and states outside the table are refusals, offsets outside the bytes are cut."""
    nxt = torch.tensor([[0, 1], [7, -9]], dtype=torch.int32, device="cuda")
    classes = torch.zeros(256, dtype=torch.uint8, device="cuda")
    classes[98], classes[99] = 1, 200
    g = sv.Grammar(nxt, classes, torch.ones(2, dtype=torch.uint8, device="cuda"))
    plain = np.full((2, 256), 0, np.int32)
    plain[0, 98], plain[:, 99] = 1, -1
    plain[1] = -1
    tokens = [b"a", b"b", b"c", b"ab", b"ba", b"aab"]
    v = sv.make_vocab(tokens)
    got = sv.grammar_masks(g, v, dev([0, 1]))
    torch.cuda.synchronize()
    want = np.stack([ref.pack(ref.allowed(plain, np.ones(2), tokens, [], s)) for s in (0, 1)])
    assert np.array_equal(got.cpu().numpy(), want)
    v = sv.Vocab(v.bytes, torch.tensor([-3, 1, 1 << 30], dtype=torch.int32, device="cuda"), v.end)
    got = sv.grammar_masks(g, v, dev([0]))
    adv = sv.grammar_advance(g, v, dev([0, 0]), dev([[0], [1]]))
    torch.cuda.synchronize()
    assert got.shape == (1, 1)
    assert adv["states"][0].tolist() == [0, 0]


def check_advance(nxt, accept, tokens, end, state, drafts, lens, grammar=None):
    g, v = grammar or sv.make_grammar(nxt, accept), sv.make_vocab(tokens, end)
    got = sv.grammar_advance(g, v, dev(state), dev(drafts), lens=dev(lens))
    torch.cuda.synchronize()
    L = drafts.shape[1]
    want, last = ref.advance(nxt, tokens, end, state, drafts, np.full(len(state), L) if lens is None else lens)
    assert np.array_equal(got["states"].cpu().numpy(), want)
    assert np.array_equal(got["last"].cpu().numpy(), last)


@pytest.mark.parametrize("B,L", [(1, 0), (1, 1), (3, 4), (64, 8), (65, 9), (200, 65), (1000, 3)])
@pytest.mark.parametrize("S,C", [(4, 5), (900, 256)])
def test_advance(B, L, S, C):
    rng = np.random.default_rng(B + L)
    nxt, accept = ref.random_grammar(rng, S, C, live=0.97)
    V = 150
    tokens = ref.random_vocab(rng, V, longest=20)
    end = [3, 9]
    drafts = rng.integers(0, V, (B, L)).astype(np.int32)
    drafts[rng.random((B, L)) < 0.01] = -1
    drafts[rng.random((B, L)) < 0.01] = V
    state = rng.integers(-1, S + 1, B)
    check_advance(nxt, accept, tokens, end, state, drafts, rng.integers(-1, L + 2, B))
    check_advance(nxt, accept, tokens, end, state, drafts, None)


def test_advance_in_place():
    rng = np.random.default_rng(4)
    nxt, accept = ref.random_grammar(rng, 30, 12, live=0.95)
    tokens = ref.random_vocab(rng, 60)
    g, v = sv.make_grammar(nxt, accept), sv.make_vocab(tokens)
    state = rng.integers(-1, 30, 100).astype(np.int32)
    drafts = rng.integers(0, 60, (100, 5)).astype(np.int32)
    s = dev(state)
    sv.grammar_advance(g, v, s, dev(drafts), out={"states": torch.empty((100, 6), dtype=torch.int32, device="cuda"),
                                                  "last": s})
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), ref.advance(nxt, tokens, [], state, drafts, np.full(100, 5))[1])


def test_masks_agree_with_advance():
    """A token is allowed exactly where the walk over it goes on (end tokens aside)."""
    rng = np.random.default_rng(6)
    nxt, accept = ref.random_grammar(rng, 50, 30, live=0.8)
    V = 400
    g, v = sv.make_grammar(nxt, accept), sv.make_vocab(ref.random_vocab(rng, V))
    masks = sv.grammar_masks(g, v, dev(np.arange(50)))
    pairs = np.stack(np.meshgrid(np.arange(50), np.arange(V), indexing="ij"), -1).reshape(-1, 2)
    after = sv.grammar_advance(g, v, dev(pairs[:, 0]), dev(pairs[:, 1:]))["last"]
    torch.cuda.synchronize()
    assert np.array_equal(ref.unpack(masks.cpu().numpy(), V).reshape(-1), after.cpu().numpy() >= 0)


@pytest.mark.parametrize("S,C", [(20, 6), (900, 200)])
def test_captured_and_replayed(S, C):
    rng = np.random.default_rng(7)
    nxt, accept = ref.random_grammar(rng, S, C, live=0.9)
    tokens = ref.random_vocab(rng, 300)
    g, v = sv.make_grammar(nxt, accept), sv.make_vocab(tokens, [1])
    state, drafts = dev(np.zeros(9)), dev(np.zeros((9, 4)))
    call = lambda: (sv.grammar_masks(g, v, state), sv.grammar_advance(g, v, state, drafts))  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bits, adv = call()
    for _ in range(4):
        s, d = rng.integers(-1, S, 9), rng.integers(0, 300, (9, 4)).astype(np.int32)
        state.copy_(dev(s)), drafts.copy_(dev(d))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits.cpu().numpy(), np.stack([ref.pack(ref.allowed(nxt, accept, tokens, [1], k)) for k in s]))
        want, last = ref.advance(nxt, tokens, [1], s, d, np.full(9, 4))
        assert np.array_equal(adv["states"].cpu().numpy(), want) and np.array_equal(adv["last"].cpu().numpy(), last)
        eager, _ = call()
        torch.cuda.synchronize()
        assert torch.equal(eager, bits)


def test_binding_refusals():
    g = sv.make_grammar(np.zeros((2, 256), np.int32), [1, 0])
    v = sv.make_vocab([b"a", b"b"])
    t = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        sv.grammar_masks(g, v, t[0].long())
    with pytest.raises(ValueError):
        sv.grammar_masks(g, v, t)
    with pytest.raises(ValueError):
        sv.grammar_masks(g, v, t[0].contiguous(), out=torch.zeros((3, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(sv.SvError):
        sv.grammar_masks(g, v, t[0, :0].contiguous())
    with pytest.raises(ValueError):
        sv.grammar_advance(g, v, t[0].contiguous(), t[0].contiguous())
    with pytest.raises(sv.SvError):
        sv.grammar_advance(g, v, t[0].contiguous(), torch.zeros((2, 66), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sv.grammar_advance(sv.Grammar(g.next.cpu(), g.classes, g.accept), v, t[0].contiguous(), t)
