"""Plain references of the per-session rules, in numpy: adjusted logits in 64
bits with the bound of their rounding, the history, automaton masks and
states."""
import numpy as np
import torch

HALF_STEP = {"bf16": 2.0**-8, "fp32": 2.0**-24}


def torch_dtype(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def unpack(words, V):
    b = np.ascontiguousarray(words).view(np.uint8)
    return np.unpackbits(b, axis=-1, bitorder="little")[..., :V].astype(bool)


def pack(bits):
    V = bits.shape[-1]
    full = np.zeros(bits.shape[:-1] + ((V + 31) // 32 * 32,), np.uint8)
    full[..., :V] = bits
    return np.packbits(full, axis=-1, bitorder="little").view("<i4")


def adjust(logits, dtype, tokens=None, m=None, pen=None, counts=None, seen=None, slots=None,
           bias=None, masks=None, mask_rows=None):
    """(exact, err, changed, used): [B, R, V] float64 results and the bound of what
    binary32 arithmetic and one rounding to dtype may be off by; whether a rule
    changes the element; [B, R] rows used.

    Each binary32 operation is off by at most 2^-24 of its result: 2 for the
    product with a reciprocal, 1 for frequency * count and 1 for its
    difference, 1 for the presence, 1 for the bias, and 2 for each drafted
    token counted on its own.  Their results are all within the sum of the
    terms' magnitudes, which bounds the whole; the last rounding is off by at
    most half a step of dtype."""
    z = logits.astype(np.float64)
    B, R, V = z.shape
    M = 0 if tokens is None else tokens.shape[1]
    used = np.ones((B, R), bool)
    if m is not None:
        used = np.arange(R)[None, :] < (m + R - M)[:, None]
    size = np.abs(z)
    changed = np.zeros(z.shape, bool)
    with np.errstate(invalid="ignore", over="ignore"):
        if pen is not None:
            rep, freq, pres = (pen[f].astype(np.float64)[:, None, None]
                               for f in ("repetition", "frequency", "presence"))
            c = np.zeros((B, R, V))
            known = np.zeros((B, R, V), bool)
            for b in range(B):
                h = -1 if counts is None else (b if slots is None else slots[b])
                if h >= 0:
                    c[b] += counts[h]
                    known[b] |= unpack(seen[h, 0], V)
                for r in range(R):
                    for j in range(min(r, M if m is None else m[b])):
                        c[b, r, tokens[b, j]] += 1
            known |= c > 0
            z = np.where(known, np.where(z > 0, z / rep, z * rep), z)
            z = np.where(known, z - freq * c - pres * (c > 0), z)
            size = size * np.maximum(rep, 1 / rep) + np.abs(freq) * c + np.abs(pres)
            changed |= known
        if bias is not None:
            off, ids, val = bias
            for b in range(B):
                for e in range(off[b], off[b + 1]):
                    if 0 <= ids[e] < V:
                        z[b, :, ids[e]] += np.float64(val[e])
                        size[b, :, ids[e]] += abs(np.float64(val[e]))
                        changed[b, :, ids[e]] = True
        err32 = (8 + 2 * M) * 2.0**-24 * size
    if masks is not None:
        for b in range(B):
            for r in range(R):
                if used[b, r] and mask_rows[b, r] >= 0:
                    out = ~unpack(masks[mask_rows[b, r]], V)
                    z[b, r, out] = -np.inf
                    changed[b, r, out] = True
    with np.errstate(invalid="ignore"):
        err = np.where(changed, HALF_STEP[dtype] * (np.abs(z) + err32) + err32, 0)
    return z, err, changed, used


def check_adjusted(got, exact, err, dtype):
    """got against exact: infinities where exact, rounded to dtype, has them (or,
    within the bound of overflow, the largest value), NaN where it has NaN."""
    got = got.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        rounded = torch.from_numpy(np.ascontiguousarray(exact)).to(torch_dtype(dtype)).double().numpy()
        nan = np.isnan(exact)
        assert np.array_equal(np.isnan(got), nan)
        inf = np.isinf(rounded) & ~nan
        assert np.array_equal(got[inf], rounded[inf])
        fine = ~nan & ~inf
        off = np.abs(got[fine] - exact[fine]) - err[fine]
    assert (off <= 0).all(), (off.max(), int((off > 0).sum()))


def note(counts, seen, slots, spans, plane, clear):
    """The history after sv_count_tokens; spans: each session's tokens."""
    counts, bits = counts.copy(), unpack(seen, counts.shape[1])
    V, n = counts.shape[1], counts.shape[0]
    for b in range(len(spans)):
        h = b if slots is None else slots[b]
        if clear and 0 <= h < n:
            counts[h] = 0
            bits[h] = False
    for b, span in enumerate(spans):
        h = b if slots is None else slots[b]
        if not 0 <= h < n:
            continue
        for t in span:
            if 0 <= t < V:
                bits[h, plane, t] = True
                if plane == 1:
                    counts[h, t] += 1
    return counts, pack(bits)


def walk(nxt, s, text):
    for c in text:
        s = nxt[s, c]
        if s < 0:
            return -1
    return s


def allowed(nxt, accept, tokens, end, s):
    if s < 0 or s >= nxt.shape[0]:
        return np.ones(len(tokens), bool)
    return np.array([bool(accept[s]) if t in end else len(x) > 0 and walk(nxt, s, x) >= 0
                     for t, x in enumerate(tokens)])


def advance(nxt, tokens, end, state, drafts, lens):
    B, L = drafts.shape
    out = np.full((B, L + 1), -1, np.int32)
    last = np.full(B, -1, np.int32)
    for b in range(B):
        s = state[b] if 0 <= state[b] < nxt.shape[0] else -1
        out[b, 0] = s
        for i in range(min(max(lens[b], 0), L)):
            t = drafts[b, i]
            ok = s >= 0 and 0 <= t < len(tokens) and t not in end and len(tokens[t]) > 0
            s = walk(nxt, s, tokens[t]) if ok else -1
            out[b, i + 1] = s
        last[b] = s
    return out, last


def random_grammar(rng, S, C, live=0.3):
    """A random automaton of S states whose bytes fall into C kinds."""
    kind = rng.integers(0, C, 256)
    table = np.where(rng.random((S, C)) < live, rng.integers(0, S, (S, C)), -1)
    return table[:, kind].astype(np.int32), (rng.random(S) < 0.3).astype(np.uint8)


def random_vocab(rng, V, longest=12, control=3):
    tokens = [bytes(rng.integers(0, 256, rng.integers(1, longest + 1), dtype=np.uint8).tolist()) for _ in range(V)]
    for t in rng.choice(V, min(control, V), replace=False):
        tokens[t] = b""
    return tokens
