"""A paged cache of keys and values and the attention that reads it, as measured calls.

A verifying round of a target model over a paged cache runs, around the acceptance step:
  reserve  pages for the round's rows, private ones where a session shares its last page
  write    the rows' keys and values into the pages, in each layer
  attend   the rows' attention over the pages, in each layer; what sessions share is read once
  keep     the committed tokens kept, the pages behind them freed
and, between rounds, fork (sessions that go on from one) and compact (used pages to the pool's front).
``prepare`` makes what a server holds on the GPU before the call; ``run`` is the call: with ``own`` the
library's operator, otherwise its formula in elementary torch operations.

A page holds ``page`` tokens of a layer's head as blocks of 32 tokens, in the order in which the matrix
instructions read them: with token t = (T, a, b, c) of sizes (page / 32, 4, 2, 4) and dimension d = (C, g, e) of
sizes (D / 32, 4, 8), keys are laid out as (T, b, C, g, a, c, e); with t = (T, g, e) of sizes (page / 32, 4, 8) and
d = (n, m) of sizes (D / 16, 16), values as (T, n, g, m, e).

Batches, drafts and rows are those of the acceptance step's workloads; heads, lengths and pages are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------------------------- cases
def listed():
    head8 = dict(Hq=32, Hkv=8, D=128, page=64)
    return [
        # one session, one token: latency
        dict(name="attend_one", op="attend", B=1, R=1, **head8, dtype="bf16", prefix=0, fam=0, famlen=0, ctx=700,
             ragged=False, fused=True),
        # the headline batch, eight drafts, conversations of up to 4096 tokens
        dict(name="attend_b256", op="attend", B=256, R=9, **head8, dtype="bf16", prefix=0, fam=0, famlen=0, ctx=4096,
             ragged=True, fused=True),
        # two sessions over whole books, four drafts
        dict(name="attend_long", op="attend", B=2, R=5, Hq=64, Hkv=8, D=128, page=128, dtype="fp16", prefix=0, fam=0,
             famlen=0, ctx=131072, ragged=False, fused=False),
        # the headline batch behind one prompt of 8192 tokens
        dict(name="attend_prefix", op="attend", B=256, R=9, **head8, dtype="bf16", prefix=8192, fam=0, famlen=0,
             ctx=500, ragged=True, fused=True),
        # ragged proposals and idle places, small pages, samples of one question behind a short prompt
        dict(name="attend_odd", op="attend", B=45, R=17, Hq=21, Hkv=3, D=64, page=32, dtype="fp16", prefix=480, fam=5,
             famlen=1504, ctx=777, ragged=True, fused=False),
        # a round's rows
        dict(name="write_round", op="write", B=256, R=9, **head8, dtype="bf16", prompts=False, ctx=2000),
        # new sessions' prompts
        dict(name="write_prompts", op="write", B=48, R=5000, **head8, dtype="bf16", prompts=True, ctx=0),
        # the pages of a round of the largest batch
        dict(name="round_b1024", op="round", B=1024, R=65, page=32, ctx=6000),
        # samples of one question: forked, and their own last pages; few of a small model's, and many
        dict(name="fork_small", op="fork", B=4, ways=2, Hq=12, Hkv=2, D=64, page=32, dtype="fp16", layers=2, ctx=300),
        dict(name="fork_samples", op="fork", B=24, ways=4, **head8, dtype="bf16", layers=16, ctx=2500),
        # a pool after sessions have left: small, and one of many gigabytes
        dict(name="compact_small", op="compact", pages=300, held=0.5, Hkv=2, D=64, page=32, dtype="fp16", layers=2),
        dict(name="compact_large", op="compact", pages=1600, held=0.6, Hkv=8, D=128, page=64, dtype="bf16", layers=32),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "attend", "attend", "write", "round", "fork", "compact"])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (64, 8), (28, 4), (40, 8), (16, 16), (5, 5), (8, 1), (12, 2), (71, 1)])
    D, page = rng.choice([64, 96, 128, 128, 256]), rng.choice([32, 64, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attend":
        R = rng.choice([1, 1, 2, 4, 5, 6, 9, 9, 17, 33, 65])
        shared = rng.choice([0, 0, 1, 2])
        prefix = spread(32, 8192) // page * page if shared else 0
        fam = rng.randint(2, 9) if shared == 2 else 0
        famlen = spread(32, 4000) // page * page if fam else 0
        ctx = spread(1, 100000)
        # bytes read once, and products, of at most the largest cases
        ctx = min(ctx, 150_000_000_000 // (4 * Hq * D * R))
        B = min(spread(1, 256), max(1, 2_000_000_000 // (ctx * Hkv * D * 4)),
                max(1, 150_000_000_000 // (4 * Hq * D * R * (ctx + prefix + famlen))))
        return dict(op=op, B=B, R=R, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, prefix=prefix, fam=fam,
                    famlen=famlen, ctx=ctx, ragged=rng.random() < 0.6, fused=rng.random() < 0.5)
    if op == "write":
        if rng.random() < 0.5:
            return dict(op=op, B=spread(1, 256), R=rng.randint(1, 33), Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                        prompts=False, ctx=spread(1, 2000))
        R = spread(2, 16000)
        return dict(op=op, B=max(1, min(spread(1, 64), 100_000_000 // (R * Hkv * D))), R=R, Hq=Hq, Hkv=Hkv, D=D,
                    page=page, dtype=dtype, prompts=True, ctx=0)
    if op == "round":
        return dict(op=op, B=spread(1, 1000), R=rng.randint(1, 65), page=page, ctx=spread(1, 6000))
    layers = rng.randint(1, 24)
    byte = layers * Hkv * D * page * 4  # of a page
    if op == "fork":
        ways, B = rng.randint(1, 8), spread(1, 64)
        B = max(1, min(B, 300_000_000 // (byte * (ways + 1))))
        return dict(op=op, B=B, ways=ways, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, layers=layers,
                    ctx=spread(1, max(2, min(4000, page * (6_000_000_000 // (byte * B * 2))))))
    return dict(op=op, pages=max(9, min(spread(50, 20000), 10_000_000_000 // byte)), held=rng.uniform(0.1, 0.9),
                Hkv=Hkv, D=D, page=page, dtype=dtype, layers=layers)


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, page = case["op"], case["page"]

    def dev(a, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)

    def normal(*shape):
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, 1, generator=gen)

    s = {"case": case}

    def pool(n_pages, layers, Hkv, D, tables, lens, extra=2):
        """Sessions' page lists on scattered slots of a pool."""
        B, n_slots = len(tables), len(tables) + extra
        slots = rs.permutation(n_slots)[:B]
        table = np.full((n_slots, s["max_pages"]), -1, np.int32)
        held, length, refs = np.zeros(n_slots, np.int32), np.zeros(n_slots, np.int32), np.zeros(n_pages, np.int32)
        for b, t in enumerate(tables):
            table[slots[b], :len(t)] = t
            held[slots[b]], length[slots[b]] = len(t), lens[b]
            refs[t] += 1
        if op == "round":
            s["k"], s["v"] = torch.zeros((2, 1, n_pages, 1, page, 64), dtype=torch.bfloat16, device=DEV)
        else:
            s["k"], s["v"] = normal(layers, n_pages, Hkv, page, D), normal(layers, n_pages, Hkv, page, D)
        s.update(table=dev(table), held=dev(held), lens=dev(length), refs=dev(refs))
        return slots

    def pages_for(n):
        return -(-n // page)

    if op in ("attend", "write"):
        B, R, Hq, Hkv, D = (case[k] for k in ("B", "R", "Hq", "Hkv", "D"))
        rows = np.full(B, R)
        if op == "attend":
            own_len = rs.randint(max(1, case["ctx"] // 4), case["ctx"] + 1, B) if case["ragged"] else np.full(B, case["ctx"])
            if case["ragged"]:
                rows = rs.randint(1, R + 1, B)
            common, family = pages_for(case["prefix"]), pages_for(case["famlen"])
        else:
            own_len = rs.randint(0, case["ctx"] + 1, B)
            rows = np.maximum(1, (R * rs.random_sample(B)).astype(np.int64)) if case["prompts"] else rs.randint(1, R + 1, B)
            common = family = 0
        fam = case.get("fam", 0)
        base = case.get("prefix", 0) + case.get("famlen", 0)
        tables, lens = [], base + own_len
        need = [pages_for(lens[b] + rows[b]) - common - family for b in range(B)]
        n_fam = -(-B // fam) if fam else 0
        longest = pages_for(base + case["ctx"] + R) - common - family  # a pool of one size, whatever the lengths
        n_pages = common + family * max(1, n_fam) + B * longest + 7
        order = rs.permutation(n_pages)
        take = iter(order)
        first = [next(take) for _ in range(common)]
        for b in range(B):
            if b == 0 or (fam and b % fam == 0):
                mine = [next(take) for _ in range(family)]
            tables.append(first + mine + [next(take) for _ in range(need[b])])
        s["max_pages"] = common + family + longest + 3
        slots = pool(n_pages, 1, Hkv, D, tables, lens)
        s["host"] = [(int(slots[b]), int(lens[b]), int(rows[b])) for b in range(B)]
        if op == "attend":
            if case["ragged"] and B > 8:
                for b in rs.permutation(B)[:B // 16 + 1]:
                    s["host"][b] = (-1, 0, int(rows[b]))  # a place that no session has
            qkv = normal(B, R, Hq + 2 * Hkv, D) if case["fused"] else normal(B, R, Hq, D)
            s["q"] = qkv[:, :, :Hq]
            s["out"] = torch.zeros((B, R, Hq, D), dtype=qkv.dtype, device=DEV)
        elif case["prompts"]:
            s["offsets"] = dev(np.concatenate([[0], np.cumsum(rows)]))
            kv = normal(int(rows.sum()), 2 * Hkv, D)
            s["new_k"], s["new_v"] = kv[:, :Hkv], kv[:, Hkv:]
        else:
            qkv = normal(B, R, Hq + 2 * Hkv, D)
            s["new_k"], s["new_v"] = qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["slots"] = dev([h for h, _, _ in s["host"]])
        s["rows"] = dev(rows)
        s["N"] = int(rows.sum())
        if own and op == "attend":
            import token_sampling_amd as sv
            s["plan"] = sv.cache_plan(cache_of(s), n_heads=Hq, R=R, rows=s["rows"], slots=s["slots"])
        return s

    if op == "round":
        B, R = case["B"], case["R"]
        lens = rs.randint(case["ctx"] // 8, case["ctx"] + 1, B)
        need = [pages_for(n + R) for n in lens]
        n_pages = B * pages_for(case["ctx"] + R) + 5
        take = iter(rs.permutation(n_pages))
        tables = [[next(take) for _ in range(n)] for n in need]
        s["max_pages"] = pages_for(case["ctx"] + R) + 3
        slots = pool(n_pages, 1, 1, 64, tables, lens)
        s["slots"], s["rows"], s["base"] = dev(slots), dev(rs.randint(1, R + 1, B)), dev(lens)
        return s

    if op == "fork":
        B, ways = case["B"], case["ways"]
        lens = rs.randint(max(1, case["ctx"] // 2), case["ctx"] + 1, B)
        need = [pages_for(n) for n in lens]
        n_pages = B * (pages_for(case["ctx"]) + ways * 2) + 3
        order = rs.permutation(n_pages)
        take = iter(order)
        tables = [[next(take) for _ in range(n)] for n in need]
        s["max_pages"] = pages_for(case["ctx"]) + 3
        slots = pool(n_pages, case["layers"], case["Hkv"], case["D"], tables, lens, extra=B * ways)
        free = np.setdiff1d(np.arange(B * (ways + 1)), slots)
        s["src"], s["dst"] = dev(np.repeat(slots, ways)), dev(rs.permutation(free))
        s["zero"], s["rows"] = dev(np.zeros(B * ways)), dev(np.full(B * ways, 9))
        return s

    # compact: sessions of a few pages each, some gone
    n, sizes = case["pages"], []
    while sum(sizes) < n:
        sizes.append(min(1 + 7 * len(sizes) % 23, n - sum(sizes)))
    ends = np.cumsum(rs.permutation(sizes))
    parts = np.split(rs.permutation(n), ends[:-1])
    tables = parts[:max(1, round(len(parts) * case["held"]))]
    for i in range(1, len(tables), 5):  # sessions that share their first page
        tables[i][0] = tables[i - 1][0]
    s["max_pages"] = 24
    pool(n, case["layers"], case["Hkv"], case["D"], tables, [len(t) * page - 1 for t in tables])
    s["old"] = {k: s[k].clone() for k in ("table", "refs")}
    return s


def cache_of(s):
    import token_sampling_amd as sv
    return sv.Cache(s["k"], s["v"], s["table"], s["lens"], s["held"], s["refs"])


# ---------------------------------------------------------------------------------------- plain forms
def token_rows(pages, keys):
    """Pages [n, Hkv, page, D] as they are held -> [Hkv, n * page, D] in token order."""
    n, H, page, D = pages.shape
    if keys:
        x = pages.view(n, H, page // 32, 2, D // 32, 4, 4, 4, 8).permute(1, 0, 2, 6, 3, 7, 4, 5, 8)
    else:
        x = pages.view(n, H, page // 32, D // 16, 4, 16, 8).permute(1, 0, 2, 4, 6, 3, 5)
    return x.reshape(H, n * page, D)


def plain_attend(s):
    case = s["case"]
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    for b, (slot, length, rows) in enumerate(s["host"]):
        if slot < 0:
            continue
        n = length + rows
        ids = s["table"][slot, :-(-n // page)].long()
        k = token_rows(s["k"][0][ids], True)[:, :n].float()
        v = token_rows(s["v"][0][ids], False)[:, :n].float()
        q = s["q"][b, :rows].float().view(rows, Hkv, G, D).transpose(0, 1).reshape(Hkv, rows * G, D)
        z = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
        z = z.view(Hkv, rows, G, n)
        hidden = torch.arange(n, device=DEV) > (length + torch.arange(rows, device=DEV))[:, None]
        z = z.masked_fill(hidden[None, :, None], -math.inf)
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = (p / p.sum(-1, keepdim=True)).view(Hkv, rows * G, n)
        o = torch.matmul(p, v).view(Hkv, rows, G, D).transpose(0, 1).reshape(rows, Hq, D)
        s["out"][b, :rows] = o.to(s["out"].dtype)
    return s["out"]


def plain_write(s):
    case = s["case"]
    Hkv, D, page = (case[k] for k in ("Hkv", "D", "page"))
    at = torch.arange(s["N"], device=DEV)
    starts = s["offsets"][:-1].long() if case["prompts"] else s["rows"].long().cumsum(0) - s["rows"]
    whose = torch.searchsorted(starts, at, right=True) - 1
    i = at - starts[whose]
    k, v = (s["new_k"], s["new_v"]) if case["prompts"] else (s["new_k"][whose, i], s["new_v"][whose, i])
    slot = s["slots"].long()[whose]
    pos = s["lens"].long()[slot] + i
    held = s["table"].long()[slot, pos // page]
    u, d = (pos % page)[:, None, None], torch.arange(D, device=DEV)
    block = ((held[:, None] * Hkv + torch.arange(Hkv, device=DEV)) * page * D)[:, :, None]
    t = u % 32
    row, half = t // 8 * 4 + t % 4, t // 4 % 2
    k_at = ((u // 32 * 2 + half) * (D // 32) + d // 32) * 512 + (d // 8 % 4 * 16 + row) * 8 + d % 8
    v_at = (u // 32 * (D // 16) + d // 16) * 512 + (t // 8 * 16 + d % 16) * 8 + t % 8
    s["k"].view(-1)[block + k_at] = k
    s["v"].view(-1)[block + v_at] = v
    return {"k": s["k"], "v": s["v"]}


def plain_keep(s, slots, count):
    """The slots' first count tokens stay."""
    slots, page = slots.long(), s["case"]["page"]
    stay = (count + page - 1) // page
    rows = s["table"][slots]
    gone = (torch.arange(rows.shape[1], device=DEV) >= stay[:, None]) & (rows >= 0)
    s["refs"].index_add_(0, rows.clamp(min=0).view(-1).long(), -gone.view(-1).int())
    s["table"][slots] = torch.where(gone, -1, rows)
    s["lens"][slots] = count
    s["held"][slots] = torch.minimum(s["held"][slots], stay)


def plain_reserve(s, slots, add):
    """Pages for add more tokens, the lowest free ones in the sessions' order; a shared last page is copied first."""
    slots, page = slots.long(), s["case"]["page"]
    table, refs = s["table"], s["refs"]
    length, held = s["lens"][slots], s["held"][slots]
    more = ((length + add + page - 1) // page - held).clamp(min=0)
    last = length // page
    old = table[slots, last.clamp(max=table.shape[1] - 1).long()].long()
    copy = (last < held) & (add > 0) & (refs[old.clamp(min=0)] > 1)
    want = more + copy
    upto = want.cumsum(0)
    n_pages = refs.numel()
    is_free = refs == 0
    rank = is_free.cumsum(0)
    served = (upto <= rank[-1]) | (want == 0)
    free = torch.full((n_pages + 1,), 0, dtype=torch.int64, device=DEV)
    free.scatter_(0, torch.where(is_free, rank - 1, n_pages), torch.arange(n_pages, device=DEV))
    copy, more = copy & served, torch.where(served, more, 0)
    col = torch.arange(table.shape[1], device=DEV)
    before = (upto - want)[:, None]
    nth = torch.where(col == last[:, None], 0, copy[:, None] + col - held[:, None])
    fresh = ((col >= held[:, None]) & (col < (held + more)[:, None])) | (copy[:, None] & (col == last[:, None]))
    new = free[(before + nth).clamp(min=0, max=n_pages)]
    nth0 = free[before[:, 0].clamp(max=n_pages)]
    flat = torch.where(fresh, new, n_pages).view(-1)
    refs_more = torch.cat([refs, refs.new_zeros(1)])
    refs_more.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    refs_more.index_add_(0, torch.where(copy, old, n_pages), -torch.ones_like(old, dtype=torch.int32))
    refs.copy_(refs_more[:n_pages])
    table[slots] = torch.where(fresh, new.int(), table[slots])
    s["held"][slots] = held + more
    return torch.where(copy, old, nth0), nth0


def plain_compact(s):
    refs, table = s["refs"], s["table"]
    n = refs.numel()
    at = torch.arange(n, device=DEV)
    used = refs > 0
    count = used.sum()
    hole, mover = ~used & (at < count), used & (at >= count)
    spare = torch.full((n + 1,), n, dtype=torch.int64, device=DEV)
    spare.scatter_(0, torch.where(hole, hole.cumsum(0) - 1, n), at)
    to = torch.where(mover, spare[(mover.cumsum(0) - 1).clamp(min=0)], at)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    src = mover.nonzero()[:, 0]
    dst = to[src]
    for x in (s["k"], s["v"]):
        x[:, dst] = x[:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    return count.int().view(1)


def run(s):
    op = s["case"]["op"]
    if own:
        import token_sampling_amd as sv
        cache = cache_of(s)
    if op == "attend":
        if not own:
            return plain_attend(s)
        return sv.cache_attention(cache, 0, s["q"], s["plan"], out=s["out"])
    if op == "write":
        if not own:
            return plain_write(s)
        if s["case"]["prompts"]:
            sv.cache_write(cache, 0, s["new_k"], s["new_v"], slots=s["slots"], offsets=s["offsets"])
        else:
            sv.cache_write(cache, 0, s["new_k"], s["new_v"], slots=s["slots"], rows=s["rows"])
        return {"k": s["k"], "v": s["v"]}
    if op == "round":
        # a round of which nothing was committed, and the next one's pages; with the library also the plan that all
        # layers' attention of the round shares
        if own:
            sv.cache_keep(cache, s["base"], slots=s["slots"], absolute=True)
            sv.cache_reserve(cache, s["rows"], slots=s["slots"])
            sv.cache_plan(cache, n_heads=1, R=s["case"]["R"], rows=s["rows"], slots=s["slots"])
        else:
            plain_keep(s, s["slots"], s["base"])
            plain_reserve(s, s["slots"], s["rows"])
    elif op == "fork":
        # the last forks end, new ones begin, each with a last page of its own
        if own:
            sv.cache_keep(cache, s["zero"], slots=s["dst"], absolute=True)
            sv.cache_fork(cache, s["src"], s["dst"])
            sv.cache_reserve(cache, s["rows"], slots=s["dst"])
        else:
            plain_keep(s, s["dst"], s["zero"])
            src, dst = s["src"].long(), s["dst"].long()
            page = s["case"]["page"]
            have = (s["lens"][src] + page - 1) // page
            rows = torch.where(torch.arange(s["max_pages"], device=DEV) < have[:, None], s["table"][src], -1)
            s["table"][dst], s["lens"][dst], s["held"][dst] = rows, s["lens"][src], have
            s["refs"].index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).view(-1).int())
            old, new = plain_reserve(s, s["dst"], s["rows"])
            tokens = torch.arange(page, device=DEV) // 32 * 32 < (s["lens"][dst] % page)[:, None]  # blocks in use
            part = tokens[None, :, None, :, None]
            for x in (s["k"], s["v"]):
                x[:, new] = torch.where(part & (old != new)[None, :, None, None, None], x[:, old], x[:, new])
        return {"k": s["k"], "v": s["v"], **{k: s[k] for k in ("table", "lens", "held", "refs")}}
    else:
        # a fragmented pool's tables, as they are found again before every pass
        for k, x in s["old"].items():
            s[k].copy_(x)
        used = sv.cache_compact(cache) if own else plain_compact(s)
        return {"used": used, "k": s["k"], "v": s["v"], "table": s["table"], "refs": s["refs"]}
    return {k: s[k] for k in ("table", "lens", "held", "refs")}


# ------------------------------------------------------------------------------------------- the floor
def work(case):
    op, page = case["op"], case["page"]
    if op == "attend":
        B, R, Hq, Hkv, D = (case[k] for k in ("B", "R", "Hq", "Hkv", "D"))
        rows = (R + 1) / 2 if case["ragged"] else R
        ctx = case["ctx"] * 5 / 8 if case["ragged"] else case["ctx"]
        live = B - (B // 16 + 1 if case["ragged"] and B > 8 else 0)
        shared = case["prefix"] + case["famlen"]
        fams = -(-B // case["fam"]) if case["fam"] else 0
        tokens = live * (ctx + rows) + case["prefix"] + case["famlen"] * fams
        return {"bytes": 4 * Hkv * D * tokens + 4 * live * rows * Hq * D,
                "flops": 4 * D * Hq * live * rows * (shared + ctx + (rows + 1) / 2)}
    if op == "write":
        rows = case["B"] * (case["R"] / 2 if case["prompts"] else (case["R"] + 1) / 2)
        return {"bytes": 8 * case["Hkv"] * case["D"] * rows, "flops": 0}
    if op == "round":
        # refs read, freed and taken pages' entries written, the sessions' numbers read and written
        pages = case["B"] * ((case["ctx"] + case["R"]) / page + 0.5)
        return {"bytes": 4 * pages + case["B"] * (32 + 16 * (case["R"] / 2 / page + 0.5)), "flops": 0}
    byte = case["layers"] * case["Hkv"] * case["D"] * 4  # of a token
    if op == "fork":
        n = case["B"] * case["ways"]
        part = sum(-(-u // 32) * 32 for u in range(page)) / page  # blocks in use of the last page
        return {"bytes": 2 * n * byte * part + 16 * n * case["ctx"] * 3 / 4 / page, "flops": 0}
    moved = case["pages"] * case["held"] * (1 - case["held"])
    return {"bytes": 2 * moved * page * byte + 8 * case["pages"], "flops": 0}


# ----------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The attention's rows in 64 bits, head by head; the other operators copy and count."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    # where a token's dimensions stand in a page's block, by the layout's definition
    t = torch.arange(page).view(-1, 4, 2, 4)
    k_at = torch.empty(page, D, dtype=torch.int64)
    v_at = torch.empty(page, D, dtype=torch.int64)
    place = torch.arange(page * D).view(page // 32, 2, D // 32, 4, 4, 4, 8)  # T, b, C, g, a, c, e
    for T in range(page // 32):
        for a in range(4):
            for b in range(2):
                for c in range(4):
                    k_at[t[T, a, b, c]] = place[T, b, :, :, a, c, :].reshape(-1)
    place = torch.arange(page * D).view(page // 32, D // 16, 4, 16, 8)  # T, n, g, m, e
    for x in range(page):
        v_at[x] = place[x // 32, :, x % 32 // 8, :, x % 8].reshape(-1)
    k_at, v_at = k_at.to(DEV), v_at.to(DEV)
    out = s["out"].double()
    for b, (slot, length, rows) in enumerate(s["host"]):
        if slot < 0:
            continue
        n = length + rows
        ids = s["table"][slot, :(n - 1) // page + 1].long()
        for h in range(Hkv):
            k = s["k"][0, ids, h].reshape(len(ids), -1)[:, k_at].view(-1, D)[:n].double()
            v = s["v"][0, ids, h].reshape(len(ids), -1)[:, v_at].view(-1, D)[:n].double()
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            q = s["q"][b, :rows, heads].double()
            z = torch.mm(q.reshape(-1, D), k.t().contiguous()).view(rows, -1, n) * D ** -0.5
            for r in range(rows):
                z[r, :, length + r + 1:] = -math.inf
            w = torch.softmax(z, -1)
            out[b, :rows, heads] = torch.mm(w.view(-1, n), v).view(rows, -1, D)
    return out
