"""Host-side refusals of the per-session rules (no kernel is launched): the C
ABI's argument checks, and the binding's."""
import ctypes
import os

import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests import rules_ref as ref

FAKE = 0x1000  # never dereferenced: the calls return first


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(sv.LIB_PATH):
        from token_sampling_amd import build
        build.build()


def test_records():
    assert sv.PENALTIES_DTYPE.itemsize == 16
    assert sv.status_str(sv.S_BAD_CONTROL) not in (sv.status_str(-99), sv.status_str(sv.S_BAD_LOGITS))
    p = sv.make_penalties(3, repetition=[1, 1.1, 2], frequency=0.5, device="cpu")
    r = p.numpy().view(sv.PENALTIES_DTYPE).reshape(-1)
    assert np.allclose(r["repetition"], [1, 1.1, 2]) and (r["frequency"] == 0.5).all()
    for bad in (dict(repetition=0.0), dict(repetition=-1.0), dict(frequency=float("nan")),
                dict(presence=float("inf"))):
        with pytest.raises(ValueError):
            sv.make_penalties(2, device="cpu", **bad)


def test_makers():
    h = sv.make_history(2, 33, device="cpu")
    assert h.counts.shape == (2, 33) and h.seen.shape == (2, 2, 2)
    b = sv.make_bias([{5: 1.0, 2: -3.0}, None, {}, {0: float("-inf")}], 8, device="cpu")
    assert b.offsets.tolist() == [0, 2, 2, 2, 3] and b.ids.tolist() == [2, 5, 0]
    for bad in ({8: 1.0}, {-1: 1.0}, {1: float("inf")}, {1: float("nan")}):
        with pytest.raises(ValueError):
            sv.make_bias([bad], 8, device="cpu")
    rng = np.random.default_rng(1)
    a = rng.random((3, 70)) < 0.5
    m = sv.make_masks(a, device="cpu")
    assert m.shape == (3, 3) and np.array_equal(ref.unpack(m.numpy(), 70), a)
    nxt, accept = ref.random_grammar(rng, 9, 7)
    g = sv.make_grammar(nxt, accept, device="cpu")
    assert g.next.shape[1] <= 7
    assert np.array_equal(g.next.numpy()[:, g.classes.numpy()], nxt)
    with pytest.raises(ValueError):
        sv.make_grammar(np.full((2, 256), 2), [0, 1], device="cpu")
    v = sv.make_vocab([b"ab", b"", b"\xff"], end=[1], device="cpu")
    assert v.offsets.tolist() == [0, 2, 2, 3] and v.bytes.tolist() == [97, 98, 255]
    with pytest.raises(ValueError):
        sv.make_vocab([b"a"], end=[1], device="cpu")


def adjust(logits=FAKE, ss=30, rs=10, dtype=0, tokens=FAKE, m=FAKE, pen=FAKE, hist="ok", slots=FAKE,
           bias="ok", masks="ok", B=2, M=2, R=3, V=10, out=FAKE, status=FAKE):
    h = {"ok": sv._History(FAKE, FAKE, 2), "null": sv._History(None, FAKE, 2),
         "none": sv._History(FAKE, FAKE, 0), "few": sv._History(FAKE, FAKE, 1)}.get(hist, hist)
    b = {"ok": sv._Bias(FAKE, FAKE, FAKE, 3), "null": sv._Bias(None, FAKE, FAKE, 3),
         "ids": sv._Bias(FAKE, None, FAKE, 3), "neg": sv._Bias(FAKE, FAKE, FAKE, -1),
         "long": sv._Bias(FAKE, FAKE, FAKE, (1 << 30) + 1)}.get(bias, bias)
    k = {"ok": sv._Masks(FAKE, FAKE, 1), "null": sv._Masks(FAKE, None, 1),
         "none": sv._Masks(FAKE, FAKE, 0)}.get(masks, masks)
    ptr = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return sv.lib().sv_adjust_logits(logits, ss, rs, dtype, tokens, m, pen, ptr(h), slots, ptr(b),
                                     ptr(k), B, M, R, V, out, status, None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(out=None), dict(dtype=2), dict(B=0), dict(B=(1 << 21) + 1),
    dict(M=-1, R=1), dict(M=65, R=65), dict(R=0, M=0), dict(R=4), dict(R=1), dict(V=0),
    dict(V=(1 << 24) + 1), dict(ss=-1), dict(rs=-1), dict(ss=(1 << 40) + 1), dict(tokens=None),
    dict(hist="null"), dict(hist="none"), dict(hist="few", slots=None), dict(bias="null"),
    dict(bias="ids"), dict(bias="neg"), dict(bias="long"), dict(masks="null"), dict(masks="none")],
    ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_adjust_refuses(bad):
    assert adjust(**bad) == sv.ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(hist=None), dict(counts=None), dict(n_slots=0), dict(tokens=None), dict(B=0), dict(L=-1),
    dict(V=0), dict(V=(1 << 24) + 1), dict(plane=2), dict(plane=-1), dict(offsets=FAKE, lens=FAKE),
    dict(slots=None, n_slots=1)], ids=str)
def test_count_refuses(bad):
    a = dict(hist=True, counts=FAKE, n_slots=2, slots=FAKE, tokens=FAKE, offsets=None, lens=None, B=2,
             L=4, V=10, plane=1)
    a.update(bad)
    h = ctypes.byref(sv._History(a["counts"], FAKE, a["n_slots"])) if a["hist"] else None
    assert sv.lib().sv_count_tokens(h, a["slots"], a["tokens"], a["offsets"], a["lens"], a["B"], a["L"],
                                    a["V"], a["plane"], 0, None) == sv.ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(next=None), dict(classes=None), dict(accept=None), dict(S=0), dict(C=0), dict(C=257),
    dict(offsets=None), dict(bytes=None), dict(n_bytes=-1), dict(n_bytes=(1 << 30) + 1), dict(n_end=9), dict(n_end=-1),
    dict(end=None), dict(V=0), dict(V=(1 << 24) + 1), dict(states=None), dict(out=None), dict(n=0), dict(n=(1 << 30) + 1)], ids=str)
def test_grammar_refuses(bad):
    a = dict(next=FAKE, classes=FAKE, accept=FAKE, S=2, C=3, bytes=FAKE, offsets=FAKE, end=FAKE, n_bytes=9,
             n_end=1, V=4, states=FAKE, out=FAKE, n=2)
    a.update(bad)
    g = ctypes.byref(sv._Grammar(a["next"], a["classes"], a["accept"], a["S"], a["C"]))
    v = ctypes.byref(sv._Vocab(a["bytes"], a["offsets"], a["end"], a["n_bytes"], a["n_end"], a["V"]))
    L = sv.lib()
    assert L.sv_grammar_masks(g, v, a["states"], a["n"], a["out"], None) == sv.ERR_ARG
    assert L.sv_grammar_advance(g, v, a["states"], FAKE, None, a["n"], 4, a["out"], None, None) == sv.ERR_ARG


def test_grammar_refuses_lengths():
    g, v = sv._Grammar(FAKE, FAKE, FAKE, 2, 3), sv._Vocab(FAKE, FAKE, FAKE, 9, 1, 4)
    call = lambda g_, v_, tokens, B, L: sv.lib().sv_grammar_advance(  # noqa: E731
        g_, v_, FAKE, tokens, None, B, L, FAKE, None, None)
    ok = ctypes.byref(g), ctypes.byref(v)
    assert call(*ok, None, 2, 4) == sv.ERR_ARG
    assert call(*ok, FAKE, 2, 66) == sv.ERR_ARG
    assert call(*ok, FAKE, 2, -1) == sv.ERR_ARG
    assert call(*ok, FAKE, (1 << 21) + 1, 4) == sv.ERR_ARG
    assert call(None, ok[1], FAKE, 2, 4) == sv.ERR_ARG
    assert call(ok[0], None, FAKE, 2, 4) == sv.ERR_ARG


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        sv.adjust_logits(torch.zeros(1, 1, 4))
    with pytest.raises(TypeError):
        sv.adjust_logits([1.0])
    with pytest.raises(ValueError):
        sv.count_tokens(sv.make_history(1, 4, device="cpu"), torch.zeros((1, 2), dtype=torch.int32))
    g = sv.make_grammar(np.full((1, 256), 0), [1], device="cpu")
    v = sv.make_vocab([b"a"], device="cpu")
    with pytest.raises(ValueError):
        sv.grammar_masks(g, v, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.grammar_advance(g, v, torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32))
