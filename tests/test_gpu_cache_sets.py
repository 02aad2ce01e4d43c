"""sv_cache_attention's kinds of sets against attention in 64 bits: rows in registers of every
size, rows in wide sets, keys that many sessions share.  A plan's counts show that a case is of
the kind that it is meant for."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import Ref
from tests.test_gpu_cache_attention import check, dev, make, queries

pytestmark = pytest.mark.gpu
BOTH = [torch.bfloat16, torch.float16]
NARROW, WIDE = 0, 1
BLOCK = 128


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def counts(plan):
    """(blocks, sets) of the narrow and the wide line, of a key head, where a plan begins."""
    raw = plan.buffer[:56].cpu().numpy().tobytes()
    return np.frombuffer(raw[:16], np.int64).tolist(), np.frombuffer(raw[48:56], np.int32).tolist()


def blocks(lo, hi):
    return -(-(hi - lo) // BLOCK)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("R,Hq,Hkv", [(5, 8, 2), (9, 8, 2), (12, 8, 2), (7, 14, 2), (9, 14, 2), (16, 8, 2), (1, 64, 1)])
def test_rows_in_registers(R, Hq, Hkv, dim, dtype):
    """17 to 64 rows a key head: two to four tiles of 16 rows a wave."""
    assert 16 < R * Hq // Hkv <= 64
    rng = np.random.default_rng(R * Hq + dim)
    lens, rows = [40, 0, 1000, 128, 333], [R, R, max(1, R // 2), R, 1]
    cache, ref = make(rng, lens, rows, Hkv, dim, dtype=dtype)
    q = queries(rng, (5, R, Hq, dim), dtype)
    plan = sv.cache_plan(cache, Hq, R, rows=dev(rows), slots=dev(range(5)))
    assert counts(plan) == ([sum(blocks(0, a + b) for a, b in zip(lens, rows)), 0], [5, 0])
    check(cache, ref, range(5), rows, q, plan=plan)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("dim,R,Hq", [(64, 17, 8), (64, 65, 14), (96, 17, 8), (128, 33, 6), (128, 65, 8), (256, 5, 8), (256, 65, 4)])
def test_rows_in_wide_sets(dim, R, Hq, dtype):
    """Too many rows for registers: whole blocks of keys in wide sets, the rest in narrow ones."""
    rng = np.random.default_rng(R + dim)
    Hkv, lens, rows = 2, [300, 1024, 127, 128], [R, R, R, 1]
    cache, ref = make(rng, lens, rows, Hkv, dim, dtype=dtype)
    plan = sv.cache_plan(cache, Hq, R, rows=dev(rows), slots=dev(range(4)))
    assert counts(plan)[1][WIDE] > 0
    check(cache, ref, range(4), rows, queries(rng, (4, R, Hq, dim), dtype), plan=plan)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_largest_scores_move_in_wide_sets(dim, dtype):
    """Scores that rise by more than 2^8 from tile to tile, for some rows at one tile and for
    others at another, and fall again: the reference value follows within the inner loop."""
    rng = np.random.default_rng(dim)
    R, Hq, Hkv, lens = 33, 8, 2, [896, 640]
    cache, ref = make(rng, lens, [R, R], Hkv, dim, dtype=dtype)
    as_bits = lambda x: torch.from_numpy(x).to(dtype).view(torch.int16).numpy()  # noqa: E731
    half = dim // 2
    for h in range(2):
        for t in range(lens[h] + R):
            p, u = ref.table[h, t // 64], t % 64
            k = rng.standard_normal((Hkv, dim)) * 0.1
            k[:, :half] += t // 32 * 0.5  # rises all the way
            k[:, half:] += 6 * np.sin(t // 32)  # rises and falls
            ref.k[0, p, :, u] = as_bits(k)
    ref.store()
    q = rng.standard_normal((2, R, Hq, dim)) * 0.1
    for r in range(R):  # a row looks at either half, or at both, up or down
        q[:, r, :, :half] += (r % 3 - 1) * 24 / dim
        q[:, r, :, half:] += (r // 3 % 3 - 1) * 24 / dim
    plan = sv.cache_plan(cache, Hq, R, rows=dev([R, R]), slots=dev([0, 1]))
    assert counts(plan)[1][WIDE] > 0
    for scale in (1.0, 0.2, 3.0):
        check(cache, ref, [0, 1], [R, R], torch.from_numpy(q).to(dtype), scale=scale, plan=plan)


def shared_cache(n, common, families, own, n_kv, dim, page, dtype, rows):
    """n sessions on slots 0 .. n - 1 that go on from one prompt of `common` tokens; families
    (first, last, tokens) of them share more; then own[b] tokens and rows[b] rows each."""
    pages = lambda x: -(-x // page)  # noqa: E731
    n_pages = pages(common) + sum(pages(t) for _, _, t in families) + sum(pages(o + r) + 1 for o, r in zip(own, rows))
    most = common + max([t for _, _, t in families], default=0) + max(o + r for o, r in zip(own, rows))
    cache = sv.make_cache(n + 1, n_pages, pages(most) + 1, n_kv, dim, page=page, dtype=dtype)

    def grow(slots, add):
        assert not sv.cache_reserve(cache, dev(add), slots=dev(slots)).any()
        assert not sv.cache_keep(cache, dev(add), slots=dev(slots)).any()

    grow([n], [common])
    for first, last, tokens in families:
        sv.cache_fork(cache, dev([n]), dev([first]))
        grow([first], [tokens])
        if last > first:
            sv.cache_fork(cache, dev([first] * (last - first)), dev(range(first + 1, last + 1)))
    rest = [b for b in range(n) if not any(f <= b <= g for f, g, _ in families)]
    if rest:
        sv.cache_fork(cache, dev([n] * len(rest)), dev(rest))
    grow(range(n), own)
    assert not sv.cache_reserve(cache, dev(rows), slots=dev(range(n))).any()
    for x in cache[:2]:
        x.normal_()
    ref = Ref(cache)
    ref.sound()
    return cache, ref


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("dim,n_kv,common", [(64, 8, 2560), (96, 8, 1792), (128, 8, 1280), (256, 4, 1280)])
@pytest.mark.parametrize("R,G,live", [(1, 1, 3), (3, 2, 9), (1, 2, 150), (33, 2, 5)])
def test_shared_prompt(dim, n_kv, common, R, G, live, dtype):
    """150 sessions behind one prompt, of which some have rows: few enough for a narrow set over
    the shared keys, or wide ones; a place without a session among them."""
    rng = np.random.default_rng(dim + R + live)
    n, page = 150, 64
    own = rng.integers(0, 150, n)
    rows = np.zeros(n, int)
    rows[np.sort(rng.permutation(n)[:live])] = rng.integers(1, R + 1, live)
    rows[np.nonzero(rows)[0][0]] = R
    cache, ref = shared_cache(n, common, [], own, n_kv, dim, page, dtype, rows)
    slots = np.arange(n)
    idle = np.nonzero(rows == 0)[0]
    if len(idle):
        slots[idle[len(idle) // 2]] = -1
    plan = sv.cache_plan(cache, n_kv * G, R, rows=dev(rows), slots=dev(slots))
    all_rows = int(rows.sum()) * G
    registers = 16 if R * G <= 16 or dim == 256 else 32 if R * G <= 32 else 48 if R * G <= 48 or R * G > 64 else 64
    got_blocks, got_sets = counts(plan)
    if R * G <= registers:  # every session's own keys in one narrow set
        mine = sum(blocks(0, o + r) for o, r in zip(own, rows) if r)
        if all_rows <= registers:
            assert got_blocks == [mine + common // BLOCK, 0] and got_sets == [(rows > 0).sum() + 1, 0]
        else:
            assert got_blocks[NARROW] == mine and got_blocks[WIDE] == got_sets[WIDE] * common // BLOCK > 0
    else:  # fewer blocks than without sharing
        assert sum(got_blocks) < blocks(0, common) * (rows > 0).sum()
    check(cache, ref, slots, rows, queries(rng, (n, R, n_kv * G, dim), dtype), plan=plan)


@pytest.mark.parametrize("G,live", [(1, 10), (3, 60)])
def test_two_levels_of_many(G, live):
    """More sessions than the plan's workgroup has threads: one prompt of all, families that
    share as much again and lie across places 1023 and 1024, one too short for that."""
    rng = np.random.default_rng(live)
    n, n_kv, dim, page, R, common = 1400, 8, 64, 32, 2, 2560
    families = [(0, 399, 2688), (400, 599, 96), (600, 1199, 2560), (1200, 1399, 2816)]
    own = rng.integers(0, 60, n)
    rows = np.zeros(n, int)
    rows[rng.permutation(n)[:live]] = rng.integers(1, R + 1, live)
    rows[[30, 450, 1023, 1024, 1300]] = 1, 2, 2, 1, 2
    cache, ref = shared_cache(n, common, families, own, n_kv, dim, page, torch.bfloat16, rows)
    slots = np.arange(n)
    for b in (0, 600, 1022, 1025, 1399):
        if rows[b] == 0:
            slots[b] = -1
    q = queries(rng, (n, R, n_kv * G, dim), torch.bfloat16)
    plan = sv.cache_plan(cache, n_kv * G, R, rows=dev(rows), slots=dev(slots))

    def sets(some):  # (line, number) of the rows' sets over shared keys
        x = int(some.sum()) * G
        return (NARROW, 1) if 0 < x <= 16 else (WIDE, -(-x // 192))

    want_blocks, want_sets = [0, 0], [0, 0]
    for where, tokens in [(slice(0, n), common)] + [(slice(f, g + 1), t) for f, g, t in families if t >= 2560]:
        line, k = sets(rows[where])
        want_sets[line] += k
        want_blocks[line] += k * (tokens // BLOCK)
    for b in np.nonzero(rows)[0]:
        family = [t for f, g, t in families if f <= b <= g][0]
        want_sets[NARROW] += 1
        want_blocks[NARROW] += blocks(0, (96 if family < 2560 else 0) + own[b] + rows[b])
    assert counts(plan) == (want_blocks, want_sets)
    check(cache, ref, slots, rows, q, plan=plan)
    # the same sessions in an order in which no neighbours belong together beyond the prompt
    order = rng.permutation(n)
    check(cache, ref, slots[order], rows[order], q[order])


@pytest.mark.parametrize("dtype", BOTH)
def test_shared_layers_strides_and_bits(dtype):
    """Shared keys in another layer, a slice of a wider projection, and the same bits again."""
    rng = np.random.default_rng(3)
    n, n_kv, dim, R = 150, 8, 128, 2
    rows = np.where(rng.random(n) < 0.1, R, 0)
    rows[[0, 149]] = R
    cache, ref = shared_cache(n, 1280, [], np.zeros(n, int), n_kv, dim, 64, dtype, rows)
    wide = queries(rng, (n, R, 3 * n_kv, dim), dtype).cuda()
    plan = sv.cache_plan(cache, 2 * n_kv, R, rows=dev(rows), slots=dev(range(n)))
    assert counts(plan)[1][WIDE] > 0
    one = check(cache, ref, range(n), rows, wide[:, :, n_kv:], plan=plan)
    again = sv.cache_attention(cache, 0, wide[:, :, n_kv:], plan, out=torch.full_like(one, 7))
    assert torch.equal(one, again)


def test_shared_captured_and_side_by_side():
    """Rounds behind a shared prompt, captured and replayed with other rows and queries, eager
    work in between; then from two streams at once, each call with a workspace of its own."""
    rng = np.random.default_rng(4)
    n, n_kv, dim, R = 150, 8, 128, 3
    full = np.full(n, R)
    cache, _ = shared_cache(n, 1280, [], rng.integers(0, 90, n), n_kv, dim, 64, torch.bfloat16, full)
    rows, slots = dev(rng.integers(0, R + 1, n)), dev(range(n))
    q = queries(rng, (n, R, 2 * n_kv, dim), torch.bfloat16).cuda()

    def attend(out):
        plan = sv.cache_plan(cache, 2 * n_kv, R, rows=rows, slots=slots)
        return plan, sv.cache_attention(cache, 0, q, plan, out=out)

    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, _ = attend(out)
    for _ in range(4):
        q.copy_(queries(rng, q.shape, torch.bfloat16))
        rows.copy_(dev(rng.integers(0, R + 1, n)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert counts(plan)[1][WIDE] > 0
        assert torch.equal(attend(torch.zeros_like(q))[1], out)
    torch.cuda.synchronize()
    want = out.clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(q) for _ in range(8)]
    torch.cuda.synchronize()
    for i, x in enumerate(outs):
        with torch.cuda.stream(streams[i % 2]):
            attend(x)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
