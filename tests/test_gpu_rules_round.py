"""The per-session rules as a server uses them: rounds of states, masks, adjusted
logits, the acceptance and commit step, the history and the states after the
committed tokens, all left on the device; every stage against its reference."""
import numpy as np
import pytest
import torch

import oracle
import token_sampling_amd as sv
from tests import parity
from tests import rules_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sentences():
    """Words of letters, numbers, separated by spaces, ended by a full stop: no
    state is without a next byte, the last one accepts."""
    nxt = np.full((5, 256), -1, np.int32)
    letters, digits = np.arange(97, 123), np.arange(48, 58)
    nxt[0, letters] = nxt[1, letters] = 1
    nxt[0, digits] = nxt[2, digits] = 2
    nxt[1, 32] = nxt[2, 32] = 0
    nxt[1, 46] = nxt[2, 46] = 3
    nxt[3, 32] = 0
    return nxt, np.array([0, 0, 0, 1, 0])


def vocabulary(rng, V):
    tokens = [bytes([c]) for c in range(256)]
    alphabet = np.frombuffer(b"abcdefghij0123 .", np.uint8)
    while len(tokens) < V - 3:
        tokens.append(bytes(rng.choice(alphabet, rng.integers(2, 6))))
    return tokens + [b""] * 3, [V - 2]  # the last but one token ends a text


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("in_place", [False, True])
def test_rounds(dtype, in_place):
    rng = np.random.default_rng(100 + in_place)
    B, M, V = 24, 4, 701
    kind = "bf16" if dtype == torch.bfloat16 else "fp32"
    nxt, accept = sentences()
    tokens, end = vocabulary(rng, V)
    g, v = sv.make_grammar(nxt, accept), sv.make_vocab(tokens, end)
    all_masks = sv.grammar_masks(g, v, dev(np.arange(5, dtype=np.int32)))
    allowed = {s: ref.allowed(nxt, accept, tokens, end, s) for s in range(-1, 5)}

    pen = np.zeros(B, sv.PENALTIES_DTYPE)
    pen["repetition"], pen["frequency"] = rng.choice([1.0, 1.2], B), rng.choice([0.0, 0.3], B)
    pen["presence"] = rng.choice([0.0, 0.4], B)
    penalties = dev(pen.view(np.uint8).reshape(B, 16))
    given = [{int(t): float(rng.uniform(-4, 4)) for t in rng.choice(V, 6, replace=False)} if b % 3 else None
             for b in range(B)]
    bias = sv.make_bias(given, V)
    bias_host = tuple(t.cpu().numpy() for t in bias)

    history = sv.make_history(B + 1, V)
    slots = rng.permutation(B + 1)[:B].astype(np.int32)
    prompts = [rng.integers(0, V, rng.integers(0, 30)).astype(np.int32) for _ in range(B)]
    offsets = np.concatenate([[0], np.cumsum([len(p) for p in prompts])]).astype(np.int32)
    sv.count_tokens(history, dev(np.concatenate(prompts)), slots=dev(slots), offsets=dev(offsets), prompt=True, clear=True)
    counts, seen = ref.note(np.zeros((B + 1, V), np.int32), np.zeros((B + 1, 2, (V + 31) // 32), np.int32), slots,
                            prompts, 0, True)

    contracts = oracle.make_contracts(B, m_max=M, max_new=60, stop=(end[0],))
    states = oracle.make_states(B, m_cap=M)
    c_dev, s_dev = dev(contracts.view(np.uint8).reshape(B, 64)), dev(states.view(np.uint8).reshape(B, 64))
    where = np.where(np.arange(B) % 4 == 0, -1, 0).astype(np.int32)  # a quarter has no grammar
    at = dev(where)
    smp = oracle.make_sampling(B)
    for b in range(B):
        smp[b]["temperature_milli"], smp[b]["top_k"], smp[b]["top_p_milli"] = [
            (1000, 0, 1000), (800, 20, 900), (1000, 0, 950), (0, 0, 1000)][b % 4]
    rule = np.array([2, 2, 1, 192])[np.arange(B) // 4 % 4].astype(np.int32)
    emitted_total = 0
    for r in range(1, 9):
        parity.log(f"[case] rules round {r} {kind} in_place={in_place}")
        raw = torch.from_numpy((2.5 * rng.standard_normal((B, M + 1, V))).astype(np.float32)).to(dtype)
        draft = torch.from_numpy((2.0 * rng.standard_normal((B, M, V))).astype(np.float32)).to(dtype)
        # the drafter knows no grammar: some of its tokens are refused; it draws
        # among the ids that every profile above leaves a positive q (rows of rule 2
        # sessions with a cut take its best token)
        x = draft.double().numpy()
        gumbel = x + np.where((np.arange(B) % 4 == 0)[:, None, None], -np.log(-np.log(rng.random(x.shape))), 0)
        drafts = gumbel.argmax(-1).astype(np.int32)
        m = rng.integers(1, M + 1, B).astype(np.int32)

        t_dev, m_dev = dev(drafts), dev(m)
        adv = sv.grammar_advance(g, v, at, t_dev, lens=m_dev)
        logits = raw.cuda()
        out = sv.adjust_logits(logits, tokens=t_dev, m=m_dev, penalties=penalties, history=history, slots=dev(slots),
                               bias=bias, masks=all_masks, mask_rows=adv["states"],
                               out=logits if in_place else torch.zeros_like(logits))
        got = sv.verify(out["logits"], draft.cuda(), t_dev, m_dev, dev(rule), parity.sampling_bytes(smp), 7, r,
                        commit=(c_dev, s_dev, None))
        sv.count_tokens(history, got["out_tokens"], slots=dev(slots), lens=got["emitted_len"])
        sv.grammar_advance(g, v, at, got["out_tokens"], lens=got["emitted_len"],
                           out={"states": torch.empty((B, M + 2), dtype=torch.int32, device="cuda"), "last": at})
        torch.cuda.synchronize()

        rows, _ = ref.advance(nxt, tokens, end, where, drafts, m)
        assert np.array_equal(adv["states"].cpu().numpy(), rows)
        assert (out["status"] == 0).all()
        exact, err, changed, used = ref.adjust(raw.double().numpy(), kind, drafts, m, pen, counts, seen, slots,
                                               bias_host, all_masks.cpu().numpy(), rows)
        adjusted = out["logits"].cpu()
        ref.check_adjusted(adjusted.double().numpy()[used], exact[used], err[used], kind)

        bits = lambda t: t.view(torch.int16).numpy().view(np.uint16) if kind == "bf16" else t.numpy()  # noqa: E731
        h = dict(target=bits(adjusted), draft=bits(draft), tokens=drafts, m=m, rule=rule, sampling=smp, seed=7, round=r)
        o = parity.run_oracle(h)
        assert (o["accepted_len"] >= 0).all()
        a = got["accepted_len"].cpu().numpy()
        assert np.array_equal(a, o["accepted_len"])
        before = states.copy()
        o_out, o_e, o_act = oracle.commit(contracts, states, m, a, o["out_tokens"])
        e, emitted = got["emitted_len"].cpu().numpy(), got["out_tokens"].cpu().numpy()
        assert np.array_equal(emitted, o_out) and np.array_equal(e, o_e)
        assert np.array_equal(got["action"].cpu().numpy(), o_act) and before["n"].sum() <= states["n"].sum()

        spans = [emitted[b, :e[b]] for b in range(B)]
        counts, seen = ref.note(counts, seen, slots, spans, 1, False)
        assert np.array_equal(history.counts.cpu().numpy(), counts)
        assert np.array_equal(history.seen.cpu().numpy(), seen)
        for b in range(B):  # every committed token is one its state allows
            s = where[b]
            for t in spans[b]:
                assert allowed[s][t], (r, b, s, t)
                s = ref.advance(nxt, tokens, end, np.array([s]), np.array([[t]]), [1])[1][0]
        _, where = ref.advance(nxt, tokens, end, where, emitted, e)
        assert np.array_equal(at.cpu().numpy(), where)
        emitted_total += int(e.sum())
    assert emitted_total > 4 * B


def test_a_mask_that_allows_nothing_fails_its_session():
    B, M, V = 3, 2, 300
    masks = sv.make_masks(np.stack([np.zeros(V, bool), np.ones(V, bool)]))
    rows = torch.ones((B, M + 1), dtype=torch.int32, device="cuda")
    rows[1, 2] = 0
    logits = torch.randn((B, M + 1, V), device="cuda")
    tokens = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    m = torch.full((B,), M, dtype=torch.int32, device="cuda")
    out = sv.adjust_logits(logits, tokens=tokens, masks=masks, mask_rows=rows, out=logits)["logits"]
    got = sv.verify(out, None, tokens, m, torch.ones_like(m), sv.make_sampling(B), 1, 1)
    torch.cuda.synchronize()
    assert got["accepted_len"][1] == sv.S_BAD_LOGITS
    assert (got["accepted_len"][[0, 2]] >= 0).all()


def test_a_failed_session_is_not_sampled():
    """Rows of a session whose controls are out of range are NaN: the acceptance
    step fails it and no other."""
    B, M, V = 4, 3, 500
    pen = sv.make_penalties(B, repetition=1.1)
    pen.view(torch.float32)[2, 0] = -1.0
    logits = torch.randn((B, M + 1, V), device="cuda").bfloat16()
    tokens = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    m = torch.full((B,), M, dtype=torch.int32, device="cuda")
    got = sv.adjust_logits(logits, tokens=tokens, m=m, penalties=pen, out=logits)
    res = sv.verify(got["logits"], None, tokens, m, torch.ones_like(m), sv.make_sampling(B), 1, 1)
    torch.cuda.synchronize()
    assert got["status"].tolist() == [0, 0, sv.S_BAD_CONTROL, 0]
    assert res["accepted_len"][2] == sv.S_BAD_LOGITS and (res["accepted_len"][[0, 1, 3]] >= 0).all()


def chain(seed, stream=None):
    """One batch's states, masks, adjusted rows and history; its results."""
    rng = np.random.default_rng(seed)
    B, M, V = 20, 6, 9000 + seed
    nxt, accept = ref.random_grammar(rng, 40, 25, live=0.9)
    tokens = ref.random_vocab(rng, V)
    g, v = sv.make_grammar(nxt, accept), sv.make_vocab(tokens, [3])
    at = dev(rng.integers(-1, 40, B).astype(np.int32))
    drafts = dev(rng.integers(0, V, (B, M)).astype(np.int32))
    m = dev(rng.integers(0, M + 1, B).astype(np.int32))
    logits = torch.randn((B, M + 1, V), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()
    history, pen = sv.make_history(B, V), sv.make_penalties(B, 1.2, 0.3, 0.1)
    out, status = torch.zeros_like(logits), torch.empty(B, dtype=torch.int32, device="cuda")
    states = {"states": torch.empty((B, M + 1), dtype=torch.int32, device="cuda"),
              "last": torch.empty(B, dtype=torch.int32, device="cuda")}
    bits = torch.empty((B * (M + 1), (V + 31) // 32), dtype=torch.int32, device="cuda")
    rows = torch.arange(B * (M + 1), dtype=torch.int32, device="cuda").view(B, M + 1)
    torch.cuda.synchronize()

    def go():
        sv.count_tokens(history, drafts, lens=m, clear=True, stream=stream)
        sv.grammar_advance(g, v, at, drafts, lens=m, out=states, stream=stream)
        sv.grammar_masks(g, v, states["states"].view(-1), out=bits, stream=stream)
        sv.adjust_logits(logits, tokens=drafts, m=m, penalties=pen, history=history, masks=bits, mask_rows=rows,
                         out=out, status=status, stream=stream)
        return [t.clone() for t in (out.view(torch.int16), status, states["states"], bits, history.counts, history.seen)]

    return go


def test_two_streams_at_once():
    want = [chain(s)() for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [chain(s, st) for s, st in zip((1, 2), streams)]
    torch.cuda.synchronize()
    for _ in range(5):
        for go, st in zip(runs, streams):
            with torch.cuda.stream(st):
                got = go()
            go.got = got
    torch.cuda.synchronize()
    for go, w in zip(runs, want):
        assert all(torch.equal(a, b) for a, b in zip(go.got, w))
        assert (w[1] == 0).all()


def test_two_graphs_in_turn():
    """Two captured batches replayed in turn and together with eager calls."""
    runs = [chain(s) for s in (3, 4)]
    want = [go() for go in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for go in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(go())
        graphs.append(g)
    for r in range(4):
        for g, o, go, w in zip(graphs, outs, runs, want):
            g.replay()
            eager = go()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, w)), r
            assert all(torch.equal(a, b) for a, b in zip(eager, w)), r
