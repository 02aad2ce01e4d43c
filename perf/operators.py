"""The logits operators and the state they keep, as measured calls.

A serving round with per-session rules runs, around the acceptance step:
  advance   the automaton's state before every row of the round, from the drafted tokens
  masks     the vocabulary masks of automaton states, as bits
  adjust    penalties for repeated tokens, biases and masks on the rows' logits
  count     the committed tokens (or a new session's prompt) into the history that penalties read

``prepare`` makes what a server holds on the GPU before the call; ``run`` is the call: with ``own`` the
library's operator, otherwise its formula in elementary torch operations.

Sizes are those of the acceptance step's workloads (batch, drafts, vocabulary) or generic ones.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
MAX_BYTES = 32  # longest token of the synthetic vocabularies


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one small batch, every rule on: latency
        dict(name="adjust_tiny", op="adjust", B=4, M=4, bonus=1, V=1024, dtype="fp32", hist=200, pen=True, bias=8,
             mask=True, ragged=False, place="out"),
        # a chat batch with penalties only, target rows of four drafts
        dict(name="adjust_b64", op="adjust", B=64, M=4, bonus=1, V=32000, dtype="bf16", hist=1500, pen=True, bias=0,
             mask=False, ragged=False, place="out"),
        # the headline batch, every rule on
        dict(name="adjust_b256", op="adjust", B=256, M=8, bonus=1, V=128256, dtype="bf16", hist=2000, pen=True,
             bias=300, mask=True, ragged=False, place="out"),
        # ragged proposals, a vocabulary whose rows start at odd addresses, structured output
        dict(name="adjust_ragged_odd", op="adjust", B=192, M=16, bonus=1, V=151935, dtype="bf16", hist=6000, pen=True,
             bias=0, mask=True, ragged=True, place="out"),
        # plain decoding: one binary32 row a session, long histories
        dict(name="adjust_decode_fp32", op="adjust", B=256, M=0, bonus=1, V=129280, dtype="fp32", hist=16000, pen=True,
             bias=40, mask=False, ragged=False, place="out"),
        # the headline batch without structured output, in place: what changes is a few thousand tokens a row
        dict(name="adjust_in_place", op="adjust", B=256, M=8, bonus=1, V=128256, dtype="bf16", hist=2000, pen=True,
             bias=300, mask=False, ragged=False, place="in"),
        # a round's committed tokens
        dict(name="count_commit", op="count", B=256, L=9, V=128256, prompts=False),
        # new sessions: their slots cleared, their prompts of up to 32k tokens noted
        dict(name="count_prompts", op="count", B=64, L=32768, V=128256, prompts=True),
        # the masks of one round's states of a small batch
        dict(name="masks_step", op="masks", V=32000, fields=12, n=20, every=False),
        # every state of a large schema, when a grammar is admitted
        dict(name="masks_schema", op="masks", V=128256, fields=80, n=1500, every=True),
        # the headline batch's drafted tokens
        dict(name="advance_b256", op="advance", B=256, M=8, V=128256, fields=80),
        # the largest batch, 64 drafts a session
        dict(name="advance_large", op="advance", B=1024, M=64, V=129280, fields=80),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["adjust", "adjust", "adjust", "count", "masks", "advance"])
    V = spread(600, 152000)
    if op == "adjust":
        M, bonus = rng.choice([0, 1, 2, 3, 5, 8, 16, 33, 64]), rng.choice([0, 1, 1])
        bonus = 1 if M == 0 else bonus
        B = min(spread(1, 512), max(1, 400_000_000 // ((M + bonus) * V)))
        return dict(op=op, B=B, M=M, bonus=bonus, V=V, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    hist=spread(10, 20000), pen=rng.random() < 0.8, bias=rng.choice([0, spread(1, 400)]),
                    mask=rng.random() < 0.5, ragged=rng.random() < 0.5, place=rng.choice(["out", "out", "in"]))
    if op == "count":
        if rng.random() < 0.5:
            return dict(op=op, B=spread(1, 512), L=rng.randint(1, 65), V=V, prompts=False)
        L = spread(2, 32000)
        return dict(op=op, B=min(spread(1, 64), 2_000_000 // L), L=L, V=V, prompts=True)
    if op == "masks":
        if rng.random() < 0.4:
            fields = spread(1, 70)
            return dict(op=op, V=V, fields=fields, n=20 * fields, every=True)
        return dict(op=op, V=V, fields=spread(1, 400), n=spread(1, 900), every=False)
    return dict(op=op, B=spread(1, 1000), M=rng.randint(1, 64), V=V, fields=spread(1, 400))


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    V = case["V"]
    W = (V + 31) // 32

    def dev(a, dtype=None):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype=dtype)

    def zipf(n):  # token ids: frequent ones low, as in a vocabulary sorted by merges
        return np.minimum((V * rs.random_sample(n) ** 3).astype(np.int32), V - 1)

    def pack(bits):  # [rows, V] bool on the host -> [rows, W] int32
        full = np.zeros((bits.shape[0], W * 32), np.uint8)
        full[:, :V] = bits
        return np.packbits(full, axis=1, bitorder="little").view(np.int32)

    if case["op"] == "adjust":
        B, M, R = case["B"], case["M"], case["M"] + case["bonus"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        logits = torch.empty((B, R, V), dtype=dtype, device=DEV).normal_(0, 2, generator=gen)
        logits += 8 * (torch.rand((R, V), device=DEV, generator=gen) < 0.005).to(dtype)  # a heavy tail
        s = {"case": case, "logits": logits, "tokens": None, "m": None, "pen": None, "counts": None, "seen": None,
             "slots": None, "bias": None, "masks": None, "mask_rows": None}
        # rows that a session does not use keep what they held
        s["out"] = logits if case["place"] == "in" else torch.zeros_like(logits)
        if M:
            s["tokens"] = dev(zipf(B * M).reshape(B, M))
            s["m"] = dev(rs.randint(1, M + 1, B).astype(np.int32) if case["ragged"] else np.full(B, M, np.int32))
        if case["pen"]:
            p = np.zeros((B, 4), np.float32)
            p[:, 0] = rs.choice([1.0, 1.05, 1.1, 1.3], B)
            p[:, 1], p[:, 2] = rs.choice([0, 0.2, 0.5], B), rs.choice([0, 0.3, 0.6], B)
            s["pen"] = dev(p.view(np.uint8))
            slots = rs.permutation(B + 3)[:B].astype(np.int32)  # a pool with free slots
            counts, bits = np.zeros((B + 3, V), np.int32), np.zeros(((B + 3) * 2, V), bool)
            n = max(1, case["hist"] // 2)
            for b in range(B + 3):
                bits[2 * b, zipf(rs.randint(0, n + 1))] = True
                counts[b] = np.bincount(zipf(rs.randint(0, n + 1)), minlength=V)
                bits[2 * b + 1] = counts[b] > 0
            s["counts"], s["slots"] = dev(counts), dev(slots)
            s["seen"] = dev(pack(bits).reshape(B + 3, 2, W))
        if case["bias"]:
            k = min(case["bias"], V)
            ids = [np.unique(rs.randint(0, V, q)).astype(np.int32) for q in rs.randint(0, k + 1, B)]
            lens = np.array([i.size for i in ids])
            val = rs.uniform(-5, 5, int(lens.sum())).astype(np.float32)
            val[rs.random_sample(val.size) < 0.2] = -100.0  # tokens banned the usual way
            s["bias"] = (dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)), dev(np.concatenate(ids)), dev(val))
        if case["mask"]:
            n = 48  # half strict states, a quarter inside strings, the rest between
            share = np.concatenate([np.full(24, 20 / V), np.full(12, 0.9), np.linspace(0.02, 0.6, 12)])
            s["masks"] = dev(pack(rs.random_sample((n, V)) < share[:, None]))
            s["mask_rows"] = dev(rs.randint(-1, n, (B, R)).astype(np.int32))
        return s

    if case["op"] == "count":
        B, L = case["B"], case["L"]
        n = B + 3
        s = {"case": case, "slots": dev(rs.permutation(n)[:B].astype(np.int32)), "lens": None, "offsets": None}
        old = zipf(n * 500).reshape(n, 500)
        s["counts"] = torch.zeros((n, V), dtype=torch.int32, device=DEV)
        s["counts"].scatter_add_(1, dev(old, torch.int64), torch.ones((n, 500), dtype=torch.int32, device=DEV))
        bits = np.zeros((n, 2, V), bool)
        np.put_along_axis(bits[:, 0], zipf(n * 300).reshape(n, 300), True, 1)
        np.put_along_axis(bits[:, 1], old, True, 1)
        s["seen"] = dev(pack(bits.reshape(n * 2, V)).reshape(n, 2, W))
        if case["prompts"]:
            lens = np.maximum(1, (L * rs.random_sample(B)).astype(np.int64))
            lens[0] = L
            s["offsets"] = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
            s["tokens"] = dev(zipf(int(lens.sum())))
        else:
            lens = rs.randint(0, L + 1, B).astype(np.int32)
            t = zipf(B * L).reshape(B, L)
            t[np.arange(L)[None, :] >= lens[:, None]] = -1  # as the commit step leaves them
            s["tokens"], s["lens"] = dev(t), dev(lens)
        return s

    # --- a byte automaton for objects of `fields` members, and a vocabulary ---
    letters = np.frombuffer(b"etaoinshrdlcumwfgypbvkjxqz", np.uint8)
    freq = np.exp(-0.12 * np.arange(26))
    freq /= freq.sum()
    rows = []  # next state of each byte

    def state():
        rows.append(np.full(256, -1, np.int32))
        return len(rows) - 1

    def literal(at, text):
        for c in text:
            to = state()
            rows[at][c] = to
            at = to
        return at

    digits, printable = np.arange(48, 58), np.arange(32, 256)
    at = literal(state(), b"{")
    for f in range(case["fields"]):
        name = bytes(rs.choice(letters, rs.randint(3, 11), p=freq))
        at = literal(at, b'"' + name + b'": ')
        done, kind = state(), f % 3
        if kind == 0:  # a string, with escapes
            body, esc = state(), state()
            rows[at][34] = body
            rows[body][printable] = body
            rows[body][34], rows[body][92] = done, esc
            rows[esc][[34, 92, 110, 116]] = body
        elif kind == 1:  # a number
            whole, point, frac = state(), state(), state()
            rows[at][digits] = rows[whole][digits] = whole
            rows[whole][46] = point
            rows[point][digits] = rows[frac][digits] = frac
            rows[whole][32] = rows[frac][32] = done
        else:  # a choice
            for word in (b"true", b"false", b"null"):
                rows[literal(at, word[:-1])][word[-1]] = done
        last = f + 1 == case["fields"]
        at = literal(done, b"}" if last else b", ")
    nxt = np.stack(rows)
    S = nxt.shape[0]
    accept = np.zeros(S, np.uint8)
    accept[at] = 1
    kinds, classes = np.unique(nxt, axis=1, return_inverse=True)  # bytes that no state tells apart

    n_end, n_free = 2, 14  # control tokens: two that end a text, others never allowed
    words = V - 256 - n_end - n_free
    lens = np.clip(rs.geometric(0.18, words) + 1, 2, 14)
    lens[rs.random_sample(words) < 0.002] = MAX_BYTES
    text = rs.choice(letters, int(lens.sum()), p=freq)
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    lead = rs.random_sample(words)
    text[starts[lead < 0.5]] = 32
    marks = np.frombuffer(b'",:{}.0123456789\\', np.uint8)
    special = np.nonzero(lead > 0.88)[0]
    text[starts[special]] = rs.choice(marks, special.size)
    text[starts[special] + 1] = rs.choice(marks, special.size)
    flat = np.concatenate([np.arange(256, dtype=np.uint8), text])
    lens = np.concatenate([np.ones(256, np.int64), lens, np.zeros(n_end + n_free, np.int64)])
    offsets = np.concatenate([[0], np.cumsum(lens)])
    s = {"case": case, "next": dev(np.ascontiguousarray(kinds)), "classes": dev(classes.reshape(-1).astype(np.uint8)),
         "accept": dev(accept), "bytes": dev(flat), "offsets": dev(offsets.astype(np.int32)),
         "end": dev(np.arange(V - n_free - n_end, V - n_free, dtype=np.int32)), "longest": int(lens.max())}
    if case["op"] == "masks":
        n = case["n"]
        s["states"] = dev((np.arange(n) % S if case["every"] else rs.randint(-1, S, n)).astype(np.int32))
        return s

    # drafted tokens: a text of the automaton, cut into the longest tokens that fit it
    B, M = case["B"], case["M"]
    ids = {}
    for t in range(V - n_end - n_free):
        ids[bytes(flat[offsets[t]:offsets[t + 1]])] = t
    where, chain, before = 0, [], []
    while where != at or not chain:
        live = np.nonzero(nxt[where] >= 0)[0]
        text, q = b"", where
        while len(text) < 14 and q != at:
            live = np.nonzero(nxt[q] >= 0)[0]
            inside = live.size > 100  # a string: letters mostly, then its end
            c = int(letters[rs.randint(26)]) if inside and rs.random_sample() < 0.93 else int(34 if inside else rs.choice(live))
            text += bytes([c])
            q = nxt[q][c]
        k = next(k for k in range(len(text), 0, -1) if text[:k] in ids)
        before.append(where)
        chain.append(ids[text[:k]])
        for c in text[:k]:
            where = nxt[where][c]
    chain, before = np.array(chain + [V - n_free - n_end]), np.array(before + [at])
    pos = rs.randint(0, len(chain), B)
    take = pos[:, None] + np.arange(M)[None, :]
    tokens = np.where(take < len(chain), chain[np.minimum(take, len(chain) - 1)], V - 1).astype(np.int32)
    wrong = rs.random_sample((B, M)) < 0.02  # drafts that the automaton may refuse
    tokens[wrong] = rs.randint(0, V, int(wrong.sum()))
    state0 = before[pos].astype(np.int32)
    state0[rs.random_sample(B) < 0.1] = -1  # sessions without a grammar
    m = rs.randint(1, M + 1, B).astype(np.int32)
    sizes = np.where(np.arange(M)[None, :] < m[:, None], np.maximum(lens[tokens], 1), 0)
    s.update(tokens=dev(tokens), state=dev(state0), lens=dev(m), steps=int(sizes.sum(1).max()))
    return s


# ---------------------------------------------------------------------------------------- plain forms
def unpack(words, V):
    """[..., W] int32 words -> [..., V] bool."""
    bits = (words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return bits.flatten(-2)[..., :V].bool()


def pack_bits(bits):
    """[..., V] bool -> [..., W] int32 words."""
    V = bits.shape[-1]
    full = torch.nn.functional.pad(bits, (0, -V % 32)).unflatten(-1, (-1, 32)).to(torch.int64)
    words = (full << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def plain_adjust(s):
    logits, tokens, m = s["logits"], s["tokens"], s["m"]
    B, R, V = logits.shape
    z = logits.float()
    if s["pen"] is not None:
        rep, freq, pres = s["pen"].view(torch.float32)[:, :3].reshape(B, 3, 1, 1).unbind(1)
        slots = s["slots"].long()
        count = s["counts"][slots].float().unsqueeze(1).expand(B, R, V)
        if tokens is not None:  # the drafted tokens before each row
            M = tokens.shape[1]
            before = (torch.arange(M, device=DEV) < torch.arange(R, device=DEV)[:, None]).float()
            count = count.scatter_add(2, tokens.long()[:, None, :].expand(B, R, M), before.expand(B, R, M))
        seen = unpack(s["seen"][slots, 0], V).unsqueeze(1) | (count > 0)
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - freq * count - pres * (count > 0)
    if s["bias"] is not None:
        offsets, ids, values = s["bias"]
        whose = torch.searchsorted(offsets, torch.arange(ids.numel(), device=DEV, dtype=torch.int32), right=True) - 1
        z = z + torch.zeros((B, V), device=DEV).index_put((whose, ids.long()), values).unsqueeze(1)
    if s["masks"] is not None:
        rows = s["mask_rows"].long()
        allowed = unpack(s["masks"], V)[rows.clamp(min=0)] | (rows < 0).unsqueeze(-1)
        z = torch.where(allowed, z, -math.inf)
    z = z.to(logits.dtype)
    if m is not None and s["case"]["ragged"]:
        used = torch.arange(R, device=DEV) < (m + (R - tokens.shape[1]))[:, None]
        z = torch.where(used.unsqueeze(-1), z, s["out"])
    s["out"].copy_(z)
    return s["out"]


def plain_count(s):
    counts, seen, tokens, slots = s["counts"], s["seen"], s["tokens"].long(), s["slots"].long()
    V = counts.shape[1]
    if s["offsets"] is not None:  # slots cleared, the prompts' tokens noted
        at = torch.arange(tokens.numel(), device=DEV, dtype=torch.int32)
        whose = torch.searchsorted(s["offsets"], at, right=True) - 1
        bits = torch.zeros((slots.numel(), V), dtype=torch.bool, device=DEV)
        bits[whose, tokens] = True
        counts[slots] = 0
        seen[slots, 1] = 0
        seen[slots, 0] = pack_bits(bits)
        return {"counts": counts, "seen": seen}
    L = tokens.shape[1]
    used = (torch.arange(L, device=DEV) < s["lens"][:, None]) & (tokens >= 0)
    tokens = tokens.clamp(min=0)
    rows = slots[:, None].expand_as(tokens)
    counts.index_put_((rows, tokens), used.int(), accumulate=True)
    same = (tokens[:, :, None] == tokens[:, None, :]) & used[:, None, :]
    first = used & ~(same & torch.ones((L, L), dtype=torch.bool, device=DEV).tril(-1)).any(-1)
    words = seen[rows, 1, tokens >> 5]
    new = first & ((words >> (tokens & 31).int()) & 1 == 0)
    add = torch.where(new, torch.ones_like(words) << (tokens & 31).int(), 0)
    seen[:, 1].index_put_((rows, tokens >> 5), add, accumulate=True)  # bits of their own: adding sets them
    return {"counts": counts, "seen": seen}


def plain_masks(s):
    nxt, S = s["next"].long(), s["next"].shape[0]
    offsets = s["offsets"].long()
    V = offsets.numel() - 1
    size = offsets[1:] - offsets[:-1]
    table = torch.cat([torch.where(nxt < 0, S, nxt), torch.full_like(nxt[:1], S)])  # row S: refused
    start = s["states"].long()
    at = torch.where(start < 0, S, start)[:, None].expand(-1, V)
    for k in range(s["longest"]):  # a byte's state depends on the one before it
        byte = s["bytes"][(offsets[:-1] + k).clamp(max=s["bytes"].numel() - 1)].long()
        at = torch.where(k < size, table[at, s["classes"].long()[byte]], at)
    allowed = (at < S) & (size > 0)
    allowed[:, s["end"].long()] = (s["accept"].bool()[start.clamp(min=0)])[:, None]
    return pack_bits(allowed | (start < 0)[:, None])


def plain_advance(s):
    nxt, S = s["next"].long(), s["next"].shape[0]
    tokens, lens, offsets = s["tokens"].long(), s["lens"].long(), s["offsets"].long()
    B, L = tokens.shape
    C = nxt.shape[1]
    # the sessions' tokens as one line of symbols each: bytes' classes, or C for a token without bytes or one that ends
    table = torch.cat([torch.where(nxt < 0, S, nxt), torch.full_like(nxt[:1], S)])
    table = torch.cat([table, torch.full_like(table[:, :1], S)], 1)
    used = torch.arange(L, device=DEV) < lens[:, None]
    size = offsets[1:] - offsets[:-1]
    ends = (tokens[:, :, None] == s["end"]).any(-1) | (size[tokens] == 0)
    stop = torch.where(used, size[tokens].clamp(min=1), 0).cumsum(1)
    step = torch.arange(s["steps"], device=DEV).expand(B, -1)
    which = torch.searchsorted(stop, step.contiguous(), right=True).clamp(max=L - 1)
    begin = torch.cat([torch.zeros_like(stop[:, :1]), stop[:, :-1]], 1)
    place = offsets[tokens.gather(1, which)] + step - begin.gather(1, which)
    symbol = s["classes"].long()[s["bytes"][place.clamp(min=0, max=s["bytes"].numel() - 1)].long()]
    symbol = torch.where(ends.gather(1, which), C, symbol)
    start = s["state"].long()
    at = torch.where(start < 0, S, start)
    line = torch.empty((B, s["steps"] + 1), dtype=torch.int64, device=DEV)
    line[:, 0] = at
    for k in range(s["steps"]):  # a byte's state depends on the one before it
        at = table[at, symbol[:, k]]
        line[:, k + 1] = at
    states = torch.cat([line[:, :1], line.gather(1, stop)], 1)
    states = torch.where(torch.cat([torch.ones_like(used[:, :1]), used], 1) & (states < S), states, -1)
    return {"last": states.gather(1, lens[:, None])[:, 0].int(), "states": states.int()}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"adjust": plain_adjust, "count": plain_count, "masks": plain_masks, "advance": plain_advance}[op](s)
    import token_sampling_amd as sv

    if op == "adjust":
        history = None if s["counts"] is None else sv.History(s["counts"], s["seen"])
        bias = None if s["bias"] is None else sv.Bias(*s["bias"])
        return sv.adjust_logits(s["logits"], tokens=s["tokens"], m=s["m"], penalties=s["pen"], history=history,
                                slots=s["slots"], bias=bias, masks=s["masks"], mask_rows=s["mask_rows"],
                                out=s["out"])["logits"]
    if op == "count":
        sv.count_tokens(sv.History(s["counts"], s["seen"]), s["tokens"], slots=s["slots"], lens=s["lens"],
                        offsets=s["offsets"], prompt=s["offsets"] is not None, clear=s["offsets"] is not None)
        return {"counts": s["counts"], "seen": s["seen"]}
    grammar = sv.Grammar(s["next"], s["classes"], s["accept"])
    vocab = sv.Vocab(s["bytes"], s["offsets"], s["end"])
    if op == "masks":
        return sv.grammar_masks(grammar, vocab, s["states"])
    return sv.grammar_advance(grammar, vocab, s["state"], s["tokens"], lens=s["lens"])


# ------------------------------------------------------------------------------------------- the floor
def work(case):
    V = case["V"]
    W = (V + 31) // 32
    if case["op"] == "adjust":
        B, M, R = case["B"], case["M"], case["M"] + case["bonus"]
        rows = B * ((M + 1) / 2 + case["bonus"]) if case["ragged"] and M else B * R
        size = 2 if case["dtype"] == "bf16" else 4
        touched = 0  # elements of a row that penalties and biases change
        byte = rows * W * 4 if case["mask"] else 0
        if case["pen"]:
            # distinct tokens of n drawn with density V^(-1/3) v^(-2/3) / 3, half prompt, half output
            n = case["hist"] / 4
            v = np.arange(V)
            p = ((v + 1) / V) ** (1 / 3) - (v / V) ** (1 / 3)
            out = float((1 - np.exp(-n * p)).sum())
            touched += float((1 - np.exp(-2 * n * p)).sum())
            byte += B * (2 * W * 4 + 4 * out + 16)
        touched += min(case["bias"], V) / 2
        byte += B * 8 * min(case["bias"], V) / 2 + B * M * 4
        moved = rows * V if case["place"] == "out" else rows * (touched + (0.55 * V if case["mask"] else 0))
        return {"bytes": 2 * size * moved + byte, "flops": 6 * rows * touched}
    if case["op"] == "count":
        if case["prompts"]:
            return {"bytes": case["B"] * (case["L"] / 2 * 4 + V * 4 + 2 * W * 4), "flops": 0}
        return {"bytes": case["B"] * (case["L"] / 2 * (4 + 8 + 8) + 8), "flops": 0}
    S = 18 * case["fields"] + 2
    if case["op"] == "masks":
        n = case["n"]
        return {"bytes": n * W * 4 + V * 11 + S * 40 * 4, "flops": n * V * 2}
    return {"bytes": case["B"] * (case["M"] / 2 * (4 + 4 + 14 + 24) + 12), "flops": case["B"] * case["M"] * 8}


# ----------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The adjusted logits in 64 bits, session by session; the other operators' outputs are whole numbers."""
    if case["op"] != "adjust":
        return None
    s = prepare(case, seed)
    logits = s["logits"]
    B, R, V = logits.shape
    out = s["out"].double()
    bits = 1 << np.arange(8, dtype=np.uint8)
    pen = None if s["pen"] is None else s["pen"].cpu().numpy().view(np.float32).astype(np.float64)

    def flags(words):  # a [W] word row -> [V] bool
        b = words.cpu().numpy().view(np.uint8)
        return torch.from_numpy(((b[:, None] & bits) != 0).reshape(-1)[:V]).to(DEV)

    table = None if s["masks"] is None else [flags(s["masks"][k]) for k in range(s["masks"].shape[0])]
    pick = None if table is None else s["mask_rows"].tolist()
    tokens = None if s["tokens"] is None else s["tokens"].tolist()
    m = None if s["m"] is None else s["m"].tolist()
    starts = None if s["bias"] is None else s["bias"][0].tolist()
    for b in range(B):
        z = logits[b].double()
        rows = R if m is None else m[b] + R - len(tokens[b])
        if pen is not None:
            h = int(s["slots"][b])
            c = s["counts"][h].double().repeat(R, 1)
            for j in range(0 if tokens is None else min(len(tokens[b]), R - 1)):
                c[j + 1:, tokens[b][j]] += 1
            known = flags(s["seen"][h, 0]) | (c >= 1)
            z = torch.where(known, torch.where(z > 0, z / pen[b, 0], z * pen[b, 0]), z)
            z = z - (pen[b, 1] * c + pen[b, 2] * c.clamp(max=1))
        if starts is not None:
            at = slice(starts[b], starts[b + 1])
            z[:, s["bias"][1][at].long()] += s["bias"][2][at].double()
        for r in range(rows):
            if table is not None and pick[b][r] >= 0:
                z[r][~table[pick[b][r]]] = -math.inf
        out[b, :rows] = z[:rows]
    return out
