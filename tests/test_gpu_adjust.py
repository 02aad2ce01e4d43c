"""sv_adjust_logits against the formula in 64 bits (tests/rules_ref.py): sizes,
types, strides, every rule alone and all together, rows left alone, values at
the ends of the range, failed sessions, streams and captured graphs."""
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


def dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype=dtype)


class Case:
    """One batch's inputs on the host, made from a seed."""

    def __init__(self, seed, B, M, R, V, dtype, rules="pbm", ragged=True, hist=60, n_bias=9, strict=None):
        rng = np.random.default_rng(seed)
        self.B, self.M, self.R, self.V, self.dtype = B, M, R, V, dtype
        x = torch.from_numpy((3 * rng.standard_normal((B, R, V))).astype(np.float32))
        self.logits = x.to(ref.torch_dtype(dtype))
        self.tokens = self.m = self.pen = self.counts = self.seen = self.slots = None
        self.bias = self.masks = self.mask_rows = None
        if M:
            # few distinct tokens: drafts repeat themselves and the history
            self.tokens = rng.integers(0, max(1, min(V, 12)), (B, M)).astype(np.int32)
            self.tokens[:, ::2] = rng.integers(0, V, self.tokens[:, ::2].shape)
            self.m = (rng.integers(0, M + 1, B) if ragged else np.full(B, M)).astype(np.int32)
        if "p" in rules:
            self.pen = np.zeros(B, sv.PENALTIES_DTYPE)
            self.pen["repetition"] = rng.choice([1.0, 1.1, 0.7, 3.0], B)
            self.pen["frequency"] = rng.choice([0, 0.25, -0.5, 1.7], B)
            self.pen["presence"] = rng.choice([0, 0.6, -1.1], B)
        if "p" in rules or "h" in rules:
            n = B + 2
            self.slots = rng.integers(-1, n, B).astype(np.int32)  # some shared, some without
            prompt = np.zeros((n, V), bool)
            self.counts = np.zeros((n, V), np.int32)
            for h in range(n):
                prompt[h, rng.integers(0, V, hist)] = True
                t = np.minimum((V * rng.random(hist) ** 2).astype(int), V - 1)
                self.counts[h] = np.bincount(t, minlength=V)
            self.seen = np.stack([ref.pack(prompt), ref.pack(self.counts > 0)], 1)
        if "b" in rules:
            lens = rng.integers(0, min(n_bias, V) + 1, B)
            lens[0] = min(n_bias, V)
            ids = [np.sort(rng.choice(V, k, replace=False)) for k in lens]
            val = rng.uniform(-6, 6, int(lens.sum())).astype(np.float32)
            val[rng.random(val.size) < 0.1] = -np.inf
            self.bias = (np.concatenate([[0], np.cumsum(lens)]).astype(np.int32),
                         np.concatenate(ids).astype(np.int32), val)
        if "m" in rules:
            share = np.array([0.0, 0.01, 0.5, 0.97, 1.0])  # the first mask allows nothing
            self.masks = ref.pack(rng.random((5, V)) < share[:, None])
            self.mask_rows = rng.integers(-1, 5, (B, R)).astype(np.int32)

    def run(self, logits=None, out=None, **kw):
        history = None if self.counts is None else sv.History(dev(self.counts), dev(self.seen))
        pen = None if self.pen is None else dev(self.pen.view(np.uint8).reshape(self.B, 16))
        bias = None if self.bias is None else sv.Bias(*map(dev, self.bias))
        return sv.adjust_logits(self.logits.cuda() if logits is None else logits, tokens=dev(self.tokens),
                                m=dev(self.m), penalties=pen, history=history, slots=dev(self.slots), bias=bias,
                                masks=dev(self.masks), mask_rows=dev(self.mask_rows), out=out, **kw)

    def reference(self):
        return ref.adjust(self.logits.double().numpy(), self.dtype, self.tokens, self.m, self.pen, self.counts,
                          self.seen, self.slots, self.bias, self.masks, self.mask_rows)

    def check(self, got, before):
        """got [B, R, V] after the call; before: what its memory held (rows that
        are not used keep it)."""
        exact, err, changed, used = self.reference()
        assert got.dtype == self.logits.dtype
        bits = lambda t: t.contiguous().view(torch.int16 if self.dtype == "bf16" else torch.int32).cpu().numpy()  # noqa: E731
        g, src, kept = bits(got), bits(self.logits), bits(before)
        assert np.array_equal(g[~used], kept[~used])
        same = used[:, :, None] & ~changed
        assert np.array_equal(g[same], src[same])  # tokens that no rule changes keep their bits
        x = got.double().cpu().numpy()
        ref.check_adjusted(x[used], exact[used], err[used], self.dtype)


def filled(case, value=7.25):
    return torch.full((case.B, case.R, case.V), value, dtype=case.logits.dtype, device="cuda")


def both_ways(case):
    out = filled(case)
    before = out.clone()
    got = case.run(out=out)
    torch.cuda.synchronize()
    assert got["logits"] is out and (got["status"] == 0).all()
    case.check(out, before)
    x = case.logits.cuda()
    got = case.run(logits=x, out=x)
    torch.cuda.synchronize()
    assert got["logits"] is x and (got["status"] == 0).all()
    case.check(x, case.logits)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 32, 33, 63, 64, 65, 255, 1000, 1023, 1024, 1025, 2047, 2048, 2049,
                               4095, 4097, 10007, 32000, 50257])
def test_sizes(V, dtype):
    both_ways(Case(V, 3, 4, 5, V, dtype))


@pytest.mark.parametrize("B,M,R", [(1, 0, 1), (5, 0, 1), (1, 1, 1), (1, 1, 2), (2, 8, 8), (2, 8, 9), (3, 64, 65),
                                   (1, 64, 64), (70, 3, 4), (300, 1, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows(B, M, R, dtype):
    both_ways(Case(B * 100 + M, B, M, R, 2100, dtype))


@pytest.mark.parametrize("rules", ["", "p", "b", "m", "pb", "pm", "bm", "h"])
@pytest.mark.parametrize("V", [999, 8192])
def test_rules_alone(rules, V):
    for dtype in ("bf16", "fp32"):
        both_ways(Case(17, 4, 5, 6, V, dtype, rules=rules))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_dense_rules(dtype):
    """Every token in the history, every token biased."""
    both_ways(Case(3, 3, 6, 7, 3001, dtype, hist=40000, n_bias=3001))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [110001, 110008])
def test_many_rows(V, dtype):
    """Enough rows for a wave a tile, at odd addresses and at even ones."""
    both_ways(Case(5, 40, 2, 3, V, dtype, hist=2000, n_bias=200))


@pytest.mark.parametrize("rules", ["p", "pb", "pbm"])
@pytest.mark.parametrize("B", [1, 40, 400])
def test_drafted_tokens_over_and_over(B, rules):
    """Every draft one of three tokens, biased and counted: met in each row, or
    before the first row of a wave."""
    case = Case(6, B, 20, 21, 1100, "fp32", rules=rules, n_bias=700)
    case.tokens = np.random.default_rng(1).choice([3, 600, 1099], case.tokens.shape).astype(np.int32)
    both_ways(case)


def test_more_sessions_than_a_launch():
    both_ways(Case(7, 33000, 1, 2, 9, "bf16", hist=5))


def test_no_history():
    """Penalties without a history count the drafted tokens alone."""
    case = Case(8, 4, 9, 10, 500, "fp32", rules="p", ragged=False)
    case.counts = case.seen = case.slots = None
    case.tokens[:] = case.tokens[:, :1]  # one token over and over
    both_ways(case)


def test_slot_of_each_session():
    case = Case(9, 4, 2, 3, 700, "bf16", rules="p")
    case.slots = None
    both_ways(case)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ends_of_the_range(dtype):
    """Infinities, the type's lowest and largest values, NaN and signed zeros,
    under every rule; masked NaN and infinities become -inf."""
    case = Case(21, 4, 3, 4, 777, dtype, ragged=False)
    t = case.logits.dtype
    special = torch.tensor([float("inf"), float("-inf"), float("nan"), torch.finfo(t).min, torch.finfo(t).max, 0.0,
                            -0.0, torch.finfo(t).tiny, -torch.finfo(t).tiny], dtype=torch.float64).to(t)
    pick = torch.from_numpy(np.random.default_rng(5).integers(0, 9, case.logits.shape))
    case.logits = special[pick]
    both_ways(case)


@pytest.mark.parametrize("layout", ["padded", "transposed", "shifted", "shared"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides(layout, dtype):
    case = Case(31, 3, 4, 5, 1003, dtype)
    B, R, V = case.logits.shape
    if layout == "padded":  # a vocabulary padded by the projection
        x = torch.full((B, R, V + 21), 9.0, dtype=case.logits.dtype, device="cuda")
        view = x[:, :, :V]
    elif layout == "transposed":
        x = torch.full((R, B, V), 9.0, dtype=case.logits.dtype, device="cuda")
        view = x.transpose(0, 1)
    elif layout == "shifted":  # rows at odd addresses
        x = torch.full((B * R * V + 3,), 9.0, dtype=case.logits.dtype, device="cuda")
        view = x[3:].view(B, R, V)
    else:  # one row for every session
        case.logits[:] = case.logits[:1]
        x = case.logits[:1].cuda()
        view = x.expand(B, R, V)
    if layout != "shared":
        view.copy_(case.logits)
    out = filled(case)
    before = out.clone()
    case.run(logits=view, out=out)
    torch.cuda.synchronize()
    case.check(out, before)
    if layout == "shared":
        with pytest.raises(ValueError):
            case.run(logits=view, out=view)
        return
    outside = x.clone()
    case.run(logits=view, out=view)
    torch.cuda.synchronize()
    case.check(view, case.logits)
    if layout == "padded":
        assert torch.equal(x[:, :, V:], outside[:, :, V:])
    if layout == "shifted":
        assert torch.equal(x[:3], outside[:3])


def test_failed_sessions():
    """Each fault fails its session alone: its rows become NaN."""
    B, M, V = 12, 3, 900
    case = Case(41, B, M, M + 1, V, "bf16", ragged=False)
    case.slots = np.zeros(B, np.int32)
    case.mask_rows[:] = 2
    want = np.zeros(B, np.int32)
    case.m[1], want[1] = M + 1, sv.S_LIMIT
    case.m[2], want[2] = -1, sv.S_LIMIT
    case.pen["repetition"][3], want[3] = 0.0, sv.S_BAD_CONTROL
    case.pen["frequency"][4], want[4] = np.nan, sv.S_BAD_CONTROL
    case.pen["reserved"][5], want[5] = 1, sv.S_BAD_CONTROL
    case.slots[6], want[6] = B + 2, sv.S_BAD_CONTROL
    case.mask_rows[7, 3], want[7] = 5, sv.S_BAD_CONTROL
    case.tokens[8, 2], want[8] = V, sv.S_BAD_PROPOSAL
    case.tokens[9, 0], want[9] = -1, sv.S_BAD_PROPOSAL
    case.m[10], case.mask_rows[10, 3], case.tokens[10, 2] = 2, 99, -1  # past the session's rows: not seen
    case.pen["repetition"][11], want[11] = np.inf, sv.S_BAD_CONTROL
    fine = want == 0
    for place in ("out", "in"):
        out = filled(case) if place == "out" else case.logits.cuda()
        before = out.clone()
        got = case.run(logits=out if place == "in" else None, out=out)
        torch.cuda.synchronize()
        assert got["status"].tolist() == want.tolist()
        bad = torch.from_numpy(~fine).cuda()
        assert torch.isnan(out[bad].float()).all()
        good = Case(41, B, M, M + 1, V, "bf16", ragged=False)  # the fine sessions, by themselves
        for f in ("m", "slots", "mask_rows", "tokens", "pen"):
            v = getattr(case, f).copy()
            v[~fine] = v[0]
            setattr(good, f, v)
        good.mask_rows[10, 3], good.tokens[10, 2] = -1, 0  # for the reference, which reads whole rows
        exact, err, changed, used = good.reference()
        ref.check_adjusted(out.double().cpu().numpy()[fine][used[fine]], exact[fine][used[fine]], err[fine][used[fine]],
                           "bf16")
        assert torch.equal(out[10, 3], before[10, 3])


def test_bias_offsets_out_of_range():
    case = Case(43, 4, 0, 1, 300, "fp32", rules="b")
    off, ids, val = case.bias
    n = ids.size
    for bad in ([-1, 1, 1, 1, 1], [0, 2, 1, 1, n], [0, 1, 1, 1, n + 1]):
        case.bias = (np.array(bad, np.int32), ids, val)
        got = case.run()
        torch.cuda.synchronize()
        want = [0 if 0 <= bad[b] <= bad[b + 1] <= n else sv.S_BAD_CONTROL for b in range(4)]
        assert got["status"].tolist() == want
    # ids outside the vocabulary have no effect
    case.bias = (np.array([0, 3, 3, 3, 3], np.int32), np.array([-7, 5, 300], np.int32), np.array([1, 2, 3], np.float32))
    both_ways(case)


@pytest.mark.parametrize("V", [301, 1022, 4093])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bits_past_the_vocabulary(V, dtype):
    """Bits at and past V of the history and of masks say nothing."""
    case = Case(45, 3, 2, 3, V, dtype)
    past = np.zeros((V + 31) // 32 * 32, bool)
    past[V:] = True
    junk = ref.pack(past[None])[0]
    case.seen |= junk
    case.masks |= junk
    B, R = 3, 3
    x = torch.full((B, R, V + 40), 9.0, dtype=case.logits.dtype, device="cuda")
    view = x[:, :, :V]
    view.copy_(case.logits)
    case.run(logits=view, out=view)
    torch.cuda.synchronize()
    case.check(view, case.logits)
    assert (x[:, :, V:] == 9.0).all()
    both_ways(case)


def test_binding_refusals():
    case = Case(44, 2, 2, 3, 64, "fp32")
    x = case.logits.cuda()
    with pytest.raises(TypeError):
        case.run(logits=x.half())
    with pytest.raises(ValueError):
        case.run(logits=x[0])
    with pytest.raises(ValueError):
        case.run(logits=x.transpose(1, 2))
    with pytest.raises(ValueError):
        case.run(out=torch.empty((2, 3, 65), device="cuda"))
    line = torch.empty(2 * 3 * 64 + 8, device="cuda")
    with pytest.raises(ValueError):
        case.run(logits=line[8:].view(2, 3, 64), out=line[:-8].view(2, 3, 64))
    with pytest.raises(ValueError):
        sv.adjust_logits(x)  # more than one row needs the drafted tokens
    with pytest.raises(ValueError):
        sv.adjust_logits(x[:, :1].contiguous(), masks=dev(case.masks))
    with pytest.raises(ValueError):
        sv.adjust_logits(x, tokens=dev(case.tokens), history=sv.make_history(1, 64),
                         penalties=sv.make_penalties(2))
    with pytest.raises(ValueError):
        sv.adjust_logits(x, tokens=dev(case.tokens), history=sv.make_history(2, 65),
                         penalties=sv.make_penalties(2))


def test_beyond_32_bit_offsets():
    """5.2e9 logits: the last sessions' rows lie past 2^32 elements."""
    B, M, V = 600, 64, 133001
    x = torch.empty((B, M + 1, V), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    case = Case(51, 2, M, M + 1, V, "bf16")  # sessions 0 and B - 1
    case.slots = np.zeros(2, np.int32)
    case.logits = x[[0, B - 1]].cpu()
    rep = lambda a: np.concatenate([a[:1].repeat(B - 1, 0), a[1:]])  # noqa: E731
    pen = dev(rep(case.pen).view(np.uint8).reshape(B, 16))
    m = np.concatenate([[case.m[0]], np.zeros(B - 2, np.int32), case.m[1:]]).astype(np.int32)
    off = case.bias[0]
    bias = sv.Bias(dev(np.concatenate([off[:1], np.full(B - 1, off[1]), off[2:]]).astype(np.int32)),
                   dev(case.bias[1]), dev(case.bias[2]))
    got = sv.adjust_logits(x, tokens=dev(rep(case.tokens)), m=dev(m), penalties=pen,
                           history=sv.History(dev(case.counts), dev(case.seen)), slots=dev(np.zeros(B, np.int32)),
                           bias=bias, masks=dev(case.masks), mask_rows=dev(rep(case.mask_rows)), out=x)
    torch.cuda.synchronize()
    assert (got["status"] == 0).all()
    case.check(x[[0, B - 1]], case.logits)


def test_other_stream():
    case = Case(61, 4, 5, 6, 5000, "bf16")
    side = torch.cuda.Stream()
    x = case.logits.cuda()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = case.run(logits=x)
    side.synchronize()
    before = filled(case)
    out = before.clone()
    torch.cuda.synchronize()
    b = case.run(logits=x, out=out, stream=side)
    side.synchronize()
    case.check(b["logits"], before)
    _, _, _, used = case.reference()
    u = torch.from_numpy(used).cuda()
    assert torch.equal(a["logits"][u].view(torch.int16), b["logits"][u].view(torch.int16))


def test_captured_and_replayed():
    case, other = (Case(s, 6, 4, 5, 4100, "bf16", ragged=False) for s in (71, 72))
    x = case.logits.cuda()
    tokens, m, slots = dev(case.tokens), dev(case.m), dev(case.slots)
    pen = dev(case.pen.view(np.uint8).reshape(6, 16))
    history = sv.History(dev(case.counts), dev(case.seen))
    masks, rows = dev(case.masks), dev(case.mask_rows)
    off, ids, val = case.bias
    bias = sv.Bias(dev(off), dev(ids), dev(val))
    other.bias = case.bias
    call = lambda out=None: sv.adjust_logits(x, tokens=tokens, m=m, penalties=pen, history=history,  # noqa: E731
                                             slots=slots, bias=bias, masks=masks, mask_rows=rows, out=out)
    out = filled(case)
    call(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(out)
    for c in (case, other, case, other):
        x.copy_(c.logits)
        tokens.copy_(dev(c.tokens)), slots.copy_(dev(c.slots))
        pen.copy_(dev(c.pen.view(np.uint8).reshape(6, 16)))
        history.counts.copy_(dev(c.counts)), history.seen.copy_(dev(c.seen))
        masks.copy_(dev(c.masks)), rows.copy_(dev(c.mask_rows))
        g.replay()
        torch.cuda.synchronize()
        assert (got["status"] == 0).all()
        c.check(out, out)
        eager = call()["logits"]
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int16), out.view(torch.int16))


def test_repeats_bit_for_bit():
    case = Case(81, 16, 8, 9, 30011, "bf16", hist=3000, n_bias=300)
    before = filled(case)
    outs = [case.run(out=before.clone())["logits"] for _ in range(4)]
    # and session by session: a row depends on its session alone
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    one = Case(81, 16, 8, 9, 30011, "bf16", hist=3000, n_bias=300)
    b = 5
    one.B, one.logits = 1, case.logits[b:b + 1]
    one.tokens, one.m, one.pen, one.slots = case.tokens[b:b + 1], case.m[b:b + 1], case.pen[b:b + 1], case.slots[b:b + 1]
    lo, hi = case.bias[0][b], case.bias[0][b + 1]
    one.bias = (np.array([0, hi - lo], np.int32), case.bias[1][lo:hi], case.bias[2][lo:hi])
    one.mask_rows = case.mask_rows[b:b + 1]
    alone = one.run(out=before[:1].clone())["logits"]
    torch.cuda.synchronize()
    assert torch.equal(alone[0].view(torch.int16), outs[0][b].view(torch.int16))
