"""The cache's calls together, as a server's rounds make them: with the acceptance and
commit step, in a captured graph, on streams of their own."""
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


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


class Model:
    """A toy target: keys, values and queries of a token by table, layers side by side,
    logits from their attention's outputs."""

    def __init__(self, V, layers, Hq, Hkv, D, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, device="cuda", generator=g).to(dtype)  # noqa: E731
        self.k, self.v, self.q = rand(layers, V, Hkv, D), rand(layers, V, Hkv, D), rand(layers, V, Hq, D)
        self.head = torch.randn((layers * Hq * D, V), device="cuda", generator=g)

    def logits(self, outs):
        x = torch.cat([o.float().flatten(2) for o in outs], -1)
        return torch.matmul(x.flatten(0, 1), self.head).view(*x.shape[:2], -1)


def test_rounds_with_commit():
    """Prompts, forks, then rounds in which drafts are accepted in part: after every round
    the cache holds the keys and values of the committed tokens, and its logits are those
    of the tokens attended at once."""
    V, layers, Hq, Hkv, D, page, B, M = 300, 2, 6, 2, 64, 32, 6, 4
    rng = np.random.default_rng(1)
    model = Model(V, layers, Hq, Hkv, D, torch.bfloat16, 1)
    cache = sv.make_cache(9, 90, 12, Hkv, D, n_layers=layers, page=page)
    slots = np.array([3, 0, 8, 5, 6, 1])  # 8 and 5 go on from 0, 6 from 3
    prompts = {3: rng.integers(0, V, 50), 0: rng.integers(0, V, 300), 1: rng.integers(0, V, 1)}
    first = list(prompts)
    line = np.concatenate([prompts[h][:-1] for h in first])  # the last token comes with the first round
    offsets = np.concatenate([[0], np.cumsum([len(prompts[h]) - 1 for h in first])])
    n = dev(np.diff(offsets))
    assert not sv.cache_reserve(cache, n, slots=dev(first)).any()
    for layer in range(layers):
        t = dev(line).long()
        sv.cache_write(cache, layer, model.k[layer][t], model.v[layer][t], slots=dev(first), offsets=dev(offsets))
    assert not sv.cache_keep(cache, n, slots=dev(first)).any()
    assert not sv.cache_fork(cache, dev([0, 0, 3]), dev([8, 5, 6])).any()
    tokens = [list(prompts[{8: 0, 5: 0, 6: 3}.get(h, h)]) for h in slots]

    smp = sv.make_sampling(B, 1000, 0, 1000)
    rule = dev(np.full(B, sv.RULE_GREEDY))
    states = sv.make_states(B, m_cap=M)
    contracts = sv.make_contracts(B, m_max=M, max_new=1000)
    plan = None
    for round_ in range(1, 7):
        m = rng.integers(1, M + 1, B)
        last = dev([t[-1] for t in tokens])
        draft = rng.integers(0, V, (B, M))
        rows = dev(m + 1)
        d_slots = dev(slots)
        assert not sv.cache_reserve(cache, rows, slots=d_slots).any()
        plan = sv.cache_plan(cache, Hq, M + 1, rows=rows, slots=d_slots, out=plan)
        assert not plan.status.any()

        def forward(draft):
            t = torch.cat([last[:, None], dev(draft)], 1).long()
            outs = []
            for layer in range(layers):
                sv.cache_write(cache, layer, model.k[layer][t], model.v[layer][t], slots=d_slots, rows=rows)
                outs.append(sv.cache_attention(cache, layer, model.q[layer][t], plan,
                                               out=torch.zeros_like(model.q[layer][t])))
            return model.logits(outs)

        for i in range(M):  # drafts that the target agrees with, up to a place
            guess = forward(draft).argmax(-1).cpu().numpy()
            right = rng.random(B) < 0.7
            draft[right, i] = guess[right, i]
        logits = forward(draft)
        # the same rows against all tokens at once
        for b in range(B):
            whole = torch.tensor(list(tokens[b]) + list(draft[b]), device="cuda")
            for i in range(m[b] + 1):
                seen = whole[:len(tokens[b]) + i]
                outs = []
                for layer in range(layers):
                    k = model.k[layer][seen].double().repeat_interleave(Hq // Hkv, 1)
                    v = model.v[layer][seen].double().repeat_interleave(Hq // Hkv, 1)
                    z = (k * model.q[layer][seen[-1]].double()).sum(-1) * D ** -0.5
                    w = torch.softmax(z, 0)[..., None]
                    outs.append(((w * v).sum(0), (w * v.abs()).sum(0)))
                x = torch.cat([o.flatten() for o, _ in outs])
                # weights and output rounded to bfloat16 (2^-8 of |v|'s and the output's means),
                # sums and scores in binary32 (2^-14 together), then a product of that many terms
                tol = torch.cat([(2.0**-8 * (o.abs() + a) + 2.0**-14 * a).flatten() for o, a in outs])
                want, bound = x @ model.head.double(), (tol + 2.0**-14 * x.abs()) @ model.head.double().abs()
                assert ((logits[b, i].double() - want).abs() <= bound).all()
        got = sv.verify(logits, None, dev(draft), dev(m), rule, smp, 1, round_, commit=(contracts, states, None))
        assert not sv.cache_keep(cache, got["emitted_len"], slots=d_slots).any()
        emitted, out = got["emitted_len"].tolist(), got["out_tokens"].tolist()
        assert min(emitted) >= 1
        for b in range(B):
            tokens[b] += out[b][:emitted[b]]
        ref = Ref(cache)
        ref.sound()
        for b, h in enumerate(slots):
            t = torch.tensor(tokens[b][:-1])
            assert ref.lens[h] == len(t) and ref.held[h] == -(-len(t) // page)
            ids = ref.table[h, :ref.held[h]]
            for layer in range(layers):
                for pages, table in ((ref.k, model.k), (ref.v, model.v)):
                    have = pages[layer, ids].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:len(t)]
                    assert np.array_equal(have, table[layer].cpu()[t].view(torch.int16).numpy())
    sv.cache_keep(cache, dev([0] * 9), absolute=True)
    assert not cache.refs.any()


def session_round(cache, q, kv, rows, slots, base, plan=None, workspace=None):
    """A round that is taken back: pages, plan, rows, attention, pages again."""
    st = sv.cache_reserve(cache, rows, slots=slots)
    plan = sv.cache_plan(cache, q.shape[2], q.shape[1], rows=rows, slots=slots, out=plan)
    sv.cache_write(cache, 0, kv[0], kv[1], slots=slots, rows=rows)
    out = sv.cache_attention(cache, 0, q, plan, out=torch.zeros_like(q), workspace=workspace)
    return st, plan, out, sv.cache_keep(cache, base, slots=slots, absolute=True)


def filled_cache(rng, lens, fork, Hkv=2, D=64, page=32, R=5):
    n = len(lens) + fork
    cache = sv.make_cache(n, 400, 60, Hkv, D, page=page)
    add = dev(list(lens) + [0] * fork)
    sv.cache_reserve(cache, add)
    for x in cache[:2]:
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)))
    sv.cache_keep(cache, add)
    if fork:
        sv.cache_fork(cache, dev([0] * fork), dev(range(len(lens), n)))
    base = cache.lens.clone()
    make = lambda *shape: torch.from_numpy(rng.standard_normal(shape)).bfloat16().cuda()  # noqa: E731
    return cache, base, make(n, R, 6, D), make(2, n, R, Hkv, D), dev(rng.integers(1, R + 1, n)), dev(rng.permutation(n))


def test_captured_round():
    """A round captured once and replayed with other inputs, eager work in between."""
    rng = np.random.default_rng(2)
    cache, base, q, kv, rows, slots = filled_cache(rng, [700, 33, 64, 129], 5)
    count = base[slots.long()].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        session_round(cache, q, kv, rows, slots, count)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st, plan, out, st2 = session_round(cache, q, kv, rows, slots, count)
    for i in range(4):
        for x in (q, kv):
            x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        rows.copy_(dev(rng.integers(0, 6, len(rows))))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert not st.any() and not st2.any() and not plan.status.any()
        _, _, want, _ = session_round(cache, q, kv, rows, slots, count)  # eager
        assert torch.equal(got, want) and got.abs().sum() > 0
        Ref(cache).sound()


def test_two_graphs_in_turn():
    """Two captured rounds of different caches, replayed in turn."""
    rng = np.random.default_rng(3)
    rounds, graphs, outs = [], [], []
    for lens, fork in (([500, 20], 3), ([40, 41, 1000], 0)):
        cache, base, q, kv, rows, slots = filled_cache(rng, lens, fork)
        args = (cache, q, kv, rows, slots, base[slots.long()].contiguous())
        session_round(*args)
        rounds.append(args)
    torch.cuda.synchronize()
    for args in rounds:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(session_round(*args)[2])
        graphs.append(graph)
    want = [session_round(*args)[2] for args in rounds]
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()


def test_streams_side_by_side():
    """Rounds of two caches on two streams at once, many times over; and attention of one
    cache from two streams, each with its own outputs."""
    rng = np.random.default_rng(4)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    rounds = []
    for lens, fork in (([900, 200, 64], 4), ([1500, 7], 0)):
        cache, base, q, kv, rows, slots = filled_cache(rng, lens, fork)
        rounds.append((cache, q, kv, rows, slots, base[slots.long()].contiguous()))
    want = [session_round(*args)[2] for args in rounds]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, args in enumerate(rounds):
            with torch.cuda.stream(sides[i]):
                outs[i].append(session_round(*args)[2])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)
    cache, q, kv, rows, slots, _ = rounds[0]
    sv.cache_reserve(cache, rows, slots=slots)
    plan = sv.cache_plan(cache, q.shape[2], q.shape[1], rows=rows, slots=slots)
    sv.cache_write(cache, 0, kv[0], kv[1], slots=slots, rows=rows)
    torch.cuda.synchronize()
    got = [sv.cache_attention(cache, 0, q, plan, out=torch.zeros_like(q), stream=sides[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in got)


def test_stream_argument():
    """A call on a stream that is not current waits for that stream's work."""
    rng = np.random.default_rng(5)
    cache, base, q, kv, rows, slots = filled_cache(rng, [100, 50], 1)
    side = torch.cuda.Stream()
    add = torch.zeros(3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        add += 40
    st = sv.cache_reserve(cache, add, stream=side)
    side.synchronize()
    assert not st.any()
    assert cache.held.tolist() == [5, 3, 5]


def test_no_pages_means_no_commit():
    """A session for which the pool has no page gets NaN rows, which the acceptance step
    refuses, so nothing of it is kept; the others go on."""
    V, M = 64, 2
    cache = sv.make_cache(3, 5, 4, 1, 64, page=32)
    sv.cache_reserve(cache, dev([64, 32, 64]))
    sv.cache_keep(cache, dev([60, 32, 64]))
    for x in cache[:2]:
        x.normal_()
    rows = dev([3, 3, 3])
    st = sv.cache_reserve(cache, rows)
    assert st.tolist() == [0, sv.S_NO_PAGES, sv.S_NO_PAGES]
    plan = sv.cache_plan(cache, 2, M + 1, rows=rows)
    assert plan.status.tolist() == [0, sv.S_BAD_CACHE, sv.S_BAD_CACHE]
    kv = torch.randn((2, 3, 3, 1, 64), device="cuda").bfloat16()
    sv.cache_write(cache, 0, kv[0], kv[1])
    out = sv.cache_attention(cache, 0, torch.randn((3, 3, 2, 64), device="cuda").bfloat16(), plan)
    logits = torch.matmul(out.float().flatten(2), torch.randn((128, V), device="cuda"))
    got = sv.verify(logits, None, dev([[1, 2]] * 3), dev([2, 2, 2]), dev([1, 1, 1]), sv.make_sampling(3), 1, 1,
                    commit=(sv.make_contracts(3, m_max=M), sv.make_states(3), None))
    assert got["accepted_len"].tolist()[1:] == [sv.S_BAD_LOGITS] * 2 and got["accepted_len"][0] >= 0
    assert not sv.cache_keep(cache, got["emitted_len"]).any()
    assert cache.lens.tolist() == [60 + got["emitted_len"][0].item(), 32, 64]
    Ref(cache).sound()
