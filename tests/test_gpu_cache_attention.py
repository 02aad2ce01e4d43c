"""sv_cache_plan and sv_cache_attention against attention in 64 bits
(tests/cache_ref.py), within the bound that Ref.attention derives."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a, dtype=np.int32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def queries(rng, shape, dtype, factor=2.0):
    return torch.from_numpy(factor * rng.standard_normal(shape)).to(dtype)


def check(cache, ref, slots, rows, q, scale=None, layer=0, status=None, out=None, plan=None):
    """One call, compared where rows are in use; the rest must keep what it held."""
    B, R, Hq, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    failed = status if status is not None else [0] * B
    want, tol = ref.attention(layer, slots, [0 if f else n for f, n in zip(failed, rows)], q.double().cpu().numpy(), sc, cache.k.dtype)
    if plan is None:
        plan = sv.cache_plan(cache, Hq, R, rows=dev(rows), slots=dev(slots))
    if out is None:
        out = torch.full((B, R, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    got = sv.cache_attention(cache, layer, q.cuda() if not q.is_cuda else q, plan, scale=scale, out=out)
    assert got is out
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    st = plan.status.tolist()
    assert st == ([0] * B if status is None else status)
    for b in range(B):
        n = 0 if slots[b] == -1 else rows[b]
        if st[b] < 0:
            assert np.isnan(got[b]).all(), b
            continue
        assert (got[b, n:] == 7.0).all(), b
        assert np.array_equal(np.isnan(got[b, :n]), np.isnan(want[b, :n])), b
        with np.errstate(invalid="ignore"):
            err = np.abs(got[b, :n] - want[b, :n])
        same = (got[b, :n] == want[b, :n]) | np.isnan(want[b, :n])
        assert (same | (err <= tol[b, :n])).all(), (b, float((err / tol[b, :n])[~same].max()))
    return out


def make(rng, lens, rows, n_kv, dim, page=64, dtype=torch.bfloat16, layers=1, extra=3, garbage=None):
    """Sessions of lens tokens and their rows written, garbage behind them."""
    n = [int(a + b) for a, b in zip(lens, rows)]
    pages = sum(-(-x // page) for x in n) + extra
    cache = sv.make_cache(len(lens), pages, max(-(-x // page) for x in n) + 2, n_kv, dim, n_layers=layers, page=page,
                          dtype=dtype)
    ref = filled(cache, rng, n, garbage=garbage)
    ref.lens[:] = lens
    cache.lens.copy_(torch.from_numpy(ref.lens))
    return cache, ref


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_shapes(dim, page, dtype):
    rng = np.random.default_rng(dim + page)
    lens = [0, 1, 31, 32, 127, 128, 200, 300]
    rows = [1, 3, 3, 2, 1, 3, 0, 3]
    cache, ref = make(rng, lens, rows, 2, dim, page, dtype)
    check(cache, ref, range(8), rows, queries(rng, (8, 3, 6, dim), dtype))


@pytest.mark.parametrize("R,Hq,Hkv", [(1, 1, 1), (1, 71, 1), (1, 16, 16), (5, 5, 5), (9, 32, 8), (2, 17, 1), (8, 8, 4),
                                      (4, 8, 1), (11, 3, 1), (65, 2, 2), (65, 12, 1), (17, 28, 4)])
def test_heads(R, Hq, Hkv):
    rng = np.random.default_rng(R * Hq)
    lens, rows = [40, 0, 333, 128], [R, R, max(1, R // 2), R]
    cache, ref = make(rng, lens, rows, Hkv, 64)
    check(cache, ref, range(4), rows, queries(rng, (4, R, Hq, 64), torch.bfloat16))


@pytest.mark.parametrize("dim,dtype", [(128, torch.bfloat16), (256, torch.float16)])
def test_long(dim, dtype):
    """Many pieces a session, and a short one beside it."""
    rng = np.random.default_rng(3)
    lens, rows = [20000, 5, 7001], [2, 1, 2]
    cache, ref = make(rng, lens, rows, 2, dim, dtype=dtype)
    check(cache, ref, range(3), rows, queries(rng, (3, 2, 8, dim), dtype, 4.0))


def test_idle_and_empty():
    rng = np.random.default_rng(4)
    lens, rows = [50, 60, 70, 80], [2, 2, 2, 2]
    cache, ref = make(rng, lens, rows, 2, 64)
    q = queries(rng, (6, 4, 4, 64), torch.bfloat16)
    check(cache, ref, [-1, 2, -1, 0, 3, -1], [2, 2, 4, 0, 1, 9], q)  # 9 rows of nobody
    check(cache, ref, [-1] * 6, [1] * 6, q)
    check(cache, ref, [2, 2, 1, 1, 2, 0], [1, 2, 2, 2, 0, 2], q)  # a slot may be read twice


def test_failed():
    rng = np.random.default_rng(5)
    lens, rows = [50, 60, 64, 30, 10], [2, 2, 2, 2, 2]
    cache, ref = make(rng, lens, rows, 2, 64)
    q = queries(rng, (7, 4, 4, 64), torch.bfloat16)
    L, C = sv.S_LIMIT, sv.S_BAD_CACHE
    check(cache, ref, [0, 1, 5, -2, 2, 3, 4], [2, 5, 1, 1, 2, -1, 2], q, status=[0, L, C, C, 0, L, 0])
    # rows behind the pages; a page that another list holds
    ref.lens[0] = 63
    ref.refs[ref.table[1, 0]] = 2
    ref.store()
    check(cache, ref, [0, 1, 2, 3, 4, 0, 0], [2, 2, 2, 2, 2, 1, 0], q, status=[C, C, 0, 0, 0, 0, 0])


def test_masked_infinities():
    """What a row does not see has no part in it: values that are not finite in later
    rows' places and behind them; the rows that see them get what the formula gives."""
    rng = np.random.default_rng(6)
    lens, rows = [30, 61, 5, 64, 126], [5, 5, 5, 5, 5]
    for dtype in (torch.bfloat16, torch.float16):
        cache, ref = make(rng, lens, rows, 2, 64, dtype=dtype)
        bits = lambda x: torch.tensor(x).to(dtype).view(torch.int16).item()  # noqa: E731
        for h, (n, where, value) in enumerate([(30, 2, np.nan), (61, 3, np.inf), (5, 4, -np.inf), (64, 1, np.nan),
                                               (126, 2, np.inf)]):
            at = n + where
            p = ref.table[h, at // 64]
            for x in ((ref.k, ref.v) if value != value else (ref.v,)):
                x[0, p, :, at % 64, 7::16] = bits(value)
        ref.store()
        check(cache, ref, range(5), rows, queries(rng, (5, 5, 4, 64), dtype))


def test_scores_far_apart():
    """Scores whose largest comes first, last and in between; equal scores; a large scale."""
    rng = np.random.default_rng(7)
    lens, rows = [700, 700, 700, 1000], [3] * 4
    cache, ref = make(rng, lens, rows, 1, 128)
    for h, at in enumerate((0, 699, 350)):
        p = ref.table[h, at // 64]
        ref.k[0, p, :, at % 64] = torch.full((128,), 3.0, dtype=torch.bfloat16).view(torch.int16).numpy()
    ref.k[0, ref.table[3, :16]] = 0
    ref.store()
    q = queries(rng, (4, 3, 8, 128), torch.bfloat16)
    q[:, :, ::2] = q[:, :, ::2].abs()
    check(cache, ref, range(4), rows, q)
    check(cache, ref, range(4), rows, q, scale=1.0)
    check(cache, ref, range(4), rows, q, scale=1e-30)


@pytest.mark.parametrize("R", [1, 3, 9])
@pytest.mark.parametrize("common,families,members", [(512, 1, 5), (256, 3, 4), (640, 2, 3), (64, 2, 2), (2048, 1, 20)])
def test_shared(common, families, members, R):
    """Sessions forked from one prompt, families of them forked further on; the same
    rows in another order give the same outputs within the bound."""
    rng = np.random.default_rng(common + R)
    page, Hkv, Hq, dim = 64, 2, 8, 64
    n = families * members
    cache = sv.make_cache(n + 1, 600, 60, Hkv, dim, page=page)
    filled(cache, rng, [common] + [0] * n)
    grow = lambda slots, add: (sv.cache_reserve(cache, dev(add), slots=dev(slots)),  # noqa: E731
                               sv.cache_keep(cache, dev(add), slots=dev(slots)))
    for f in range(families):
        head = 1 + f * members
        sv.cache_fork(cache, dev([0]), dev([head]))
        grow([head], [384 + 13 * f])
        sv.cache_fork(cache, dev([head] * (members - 1)), dev(range(head + 1, head + members)))
    slots = np.arange(1, n + 1)
    grow(slots, rng.integers(0, 200, n))
    rows = rng.integers(0, R + 1, n)
    rows[0] = R
    sv.cache_reserve(cache, dev(rows), slots=dev(slots))
    torch.cuda.synchronize()
    # the tokens so far stand in shared pages; now all pages in use get values
    for x in cache[:2]:
        x.copy_(torch.randn(x.shape, device="cuda"))
    from tests.cache_ref import Ref
    ref = Ref(cache)
    ref.sound()
    q = queries(rng, (n, R, Hq, dim), torch.bfloat16)
    check(cache, ref, slots, rows, q)
    order = rng.permutation(n)
    check(cache, ref, slots[order], rows[order], q)
    some = slots.copy()
    some[rng.random(n) < 0.4] = -1
    check(cache, ref, some, rows, q)


def test_strides_and_layers():
    rng = np.random.default_rng(9)
    lens, rows = [100, 3, 64], [4, 4, 4]
    cache, ref = make(rng, lens, rows, 2, 64, layers=3)
    wide = queries(rng, (3, 4, 4 + 4 + 1, 64), torch.bfloat16).cuda()
    for layer in range(3):
        check(cache, ref, range(3), rows, wide[:, :, 2:6], layer=layer)
    check(cache, ref, range(3), rows, wide[:, :1, 2:6].expand(3, 4, 4, 64))  # one row's queries for all
    turned = queries(rng, (4, 4, 3, 64), torch.bfloat16).cuda().permute(2, 0, 1, 3)
    check(cache, ref, range(3), rows, turned)
    other = queries(rng, (4, 3, 4, 64), torch.bfloat16).cuda().transpose(0, 1)
    check(cache, ref, range(3), rows, other)


def test_slot_order_and_all_slots():
    rng = np.random.default_rng(10)
    lens, rows = [100, 3, 64, 0], [2, 2, 2, 2]
    cache, ref = make(rng, lens, rows, 1, 128)
    q = queries(rng, (4, 2, 4, 128), torch.bfloat16).cuda()
    one = check(cache, ref, range(4), rows, q)
    plan = sv.cache_plan(cache, 4, 2)  # every slot, every row
    assert plan.B == 4
    assert torch.equal(one, sv.cache_attention(cache, 0, q, plan))
    order = [2, 0, 3, 1]
    plan = sv.cache_plan(cache, 4, 2, slots=dev(order), out=plan)
    assert torch.equal(one[order], sv.cache_attention(cache, 0, q[order].contiguous(), plan))


@pytest.mark.parametrize("B", [1, 1023, 1025, 4096])
def test_many_sessions(B):
    """Short sessions, one row each; many places name the same slots."""
    rng = np.random.default_rng(B)
    lens = [0, 31, 32, 100]
    cache, ref = make(rng, lens, [1] * 4, 1, 64, page=32)
    slots = rng.integers(-1, 4, B)
    slots[0] = 3
    check(cache, ref, slots, [1] * B, queries(rng, (B, 1, 2, 64), torch.bfloat16))


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(11)
    lens, rows = [3000, 100, 64, 900], [5, 5, 5, 5]
    cache, ref = make(rng, lens, rows, 2, 128)
    q = queries(rng, (4, 5, 16, 128), torch.bfloat16).cuda()
    plan = sv.cache_plan(cache, 16, 5)
    first = sv.cache_attention(cache, 0, q, plan)
    for _ in range(3):
        assert torch.equal(first, sv.cache_attention(cache, 0, q, plan))


def test_far_pages():
    """A layer that begins behind 2^32 bytes of its plane."""
    page, Hkv, dim, n_pages = 128, 8, 128, 8400
    cache = sv.make_cache(1, n_pages, 4, Hkv, dim, n_layers=3, page=page)
    assert 2 * cache.k[:2].numel() > 2**32
    cache.refs[:n_pages - 2] = 1
    sv.cache_reserve(cache, dev([200]))
    assert cache.table[0].tolist() == [n_pages - 2, n_pages - 1, -1, -1]
    kv = torch.randn((2, 1, 200, Hkv, dim), device="cuda").bfloat16()
    sv.cache_write(cache, 2, kv[0], kv[1])
    sv.cache_keep(cache, dev([199]))
    q = torch.randn((1, 1, 16, dim), device="cuda").bfloat16()
    sv.cache_reserve(cache, dev([1]))
    out = sv.cache_attention(cache, 2, q, sv.cache_plan(cache, 16, 1))
    k, v, x = kv[0, 0].double().cpu(), kv[1, 0].double().cpu(), q[0, 0].double().cpu()
    for h in range(16):
        w = torch.softmax(k[:, h // 2] @ x[h] * dim ** -0.5, 0)
        A = w @ v[:, h // 2].abs()
        # as in Ref.attention: the output's and the weights' rounding, and 2^-14 for scores and sums
        err = (out[0, 0, h].double().cpu() - w @ v[:, h // 2]).abs()
        assert (err <= 2.0**-8 * (w @ v[:, h // 2]).abs() + (2.0**-8 + 2.0**-14) * A).all()


def test_binding_checks():
    rng = np.random.default_rng(12)
    cache, _ = make(rng, [10, 20], [2, 2], 2, 64)
    q = queries(rng, (2, 2, 4, 64), torch.bfloat16).cuda()
    plan = sv.cache_plan(cache, 4, 2)
    with pytest.raises(sv.SvError):
        sv.cache_plan(cache, 3, 2)
    with pytest.raises(sv.SvError):
        sv.cache_plan(cache, 4, 66)
    with pytest.raises(ValueError):
        sv.cache_plan(cache, 4, 2, rows=dev([1, 1]), slots=dev([1]))
    with pytest.raises(ValueError):
        sv.cache_plan(cache, 4, 2, B=3)
    with pytest.raises(ValueError):
        sv.cache_plan(cache, 4, 1, out=plan)
    with pytest.raises(TypeError):
        sv.cache_attention(cache, 0, q.half(), plan)
    with pytest.raises(ValueError):
        sv.cache_attention(cache, 0, q[:1], plan)
    with pytest.raises(ValueError):
        sv.cache_attention(cache, 0, q, plan, out=q)
    with pytest.raises(ValueError):
        sv.cache_attention(cache, 0, q, plan, out=q[:, :1])
    for bad in (dict(layer=1), dict(layer=-1), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(sv.SvError):
            sv.cache_attention(cache, bad.get("layer", 0), q, plan, scale=bad.get("scale"))
    with pytest.raises(sv.SvError):
        sv.cache_attention(cache, 0, q, plan, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def test_many_sessions_share():
    """More sessions than a plan's workgroup has threads, behind one prompt, rows of one
    and of several tokens, a few idle places among them."""
    rng = np.random.default_rng(13)
    n, page = 1300, 64
    cache = sv.make_cache(n + 1, 9 + 2 * n, 8, 1, 64, page=page)
    sv.cache_reserve(cache, dev([300]), slots=dev([n]))
    sv.cache_keep(cache, dev([300]), slots=dev([n]))
    sv.cache_fork(cache, dev([n] * n), dev(range(n)))
    rows = rng.integers(1, 4, n)
    assert not sv.cache_reserve(cache, dev(rows), slots=dev(range(n))).any()
    for x in cache[:2]:
        x.normal_()
    from tests.cache_ref import Ref
    ref = Ref(cache)
    ref.sound()
    slots = np.arange(n)
    slots[rng.random(n) < 0.1] = -1
    check(cache, ref, slots, rows, queries(rng, (n, 3, 2, 64), torch.bfloat16))


@pytest.mark.parametrize("dim,dtype,Hq,R", [(128, torch.bfloat16, 16, 2), (256, torch.float16, 8, 3), (96, torch.bfloat16, 8, 65)])
def test_long_shared(dim, dtype, Hq, R):
    """Many sessions behind a prompt long enough to be read once for all, most of them
    without rows this round; the first row block of the prompt's sets is partly filled, and
    with 65 rows a session it takes several."""
    rng = np.random.default_rng(dim)
    n, common, page, Hkv = 150, 2304, 64, 8
    cache = sv.make_cache(n + 1, 40 + 4 * n, 50, Hkv, dim, page=page, dtype=dtype)
    sv.cache_reserve(cache, dev([common + 17]), slots=dev([n]))
    sv.cache_keep(cache, dev([common + 17]), slots=dev([n]))
    sv.cache_fork(cache, dev([n] * n), dev(range(n)))
    rows = np.where(rng.random(n) < 0.06, rng.integers(1, R + 1, n), 0)
    rows[[3, 77]] = R
    assert not sv.cache_reserve(cache, dev(rows), slots=dev(range(n))).any()
    for x in cache[:2]:
        x.normal_()
    from tests.cache_ref import Ref
    slots = np.arange(n)
    slots[10:13] = -1
    check(cache, Ref(cache), slots, rows, queries(rng, (n, R, Hq, dim), dtype))


def test_two_levels():
    """Families within a batch: what all share and what a family shares beyond it, each long
    enough to be read once."""
    rng = np.random.default_rng(14)
    fams, members, page, Hkv, dim, R = 3, 24, 256, 8, 256, 3
    n = fams * members
    cache = sv.make_cache(n + 1, 60 + 25 * fams + 2 * n, 40, Hkv, dim, page=page)
    grow = lambda slots, add: (sv.cache_reserve(cache, dev(add), slots=dev(slots)),  # noqa: E731
                               sv.cache_keep(cache, dev(add), slots=dev(slots)))
    grow([n], [2048])
    for f in range(fams):
        head = f * members
        sv.cache_fork(cache, dev([n]), dev([head]))
        grow([head], [4700 if f else 100])  # the first family is too short for a level of its own
        sv.cache_fork(cache, dev([head] * (members - 1)), dev(range(head + 1, head + members)))
    rows = np.where(rng.random(n) < 0.1, rng.integers(1, R + 1, n), 0)
    rows[[0, 30, 31, 60]] = R
    assert not sv.cache_reserve(cache, dev(rows), slots=dev(range(n))).any()
    for x in cache[:2]:
        x.normal_()
    from tests.cache_ref import Ref
    ref = Ref(cache)
    ref.sound()
    check(cache, ref, np.arange(n), rows, queries(rng, (n, R, 16, dim), torch.bfloat16))
