"""sv_cache_reserve, _keep, _fork, _compact and _write against a plain cache
(tests/cache_ref.py), exactly."""
import numpy as np
import pytest
import torch

import token_sampling_amd as sv
from tests.cache_ref import Ref, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sv.lib()
    yield


def dev(a, dtype=np.int32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def small(rng, n_slots=7, n_pages=60, max_pages=9, n_kv=2, dim=64, page=32, layers=2, dtype=torch.bfloat16, lens=None):
    cache = sv.make_cache(n_slots, n_pages, max_pages, n_kv, dim, n_layers=layers, page=page, dtype=dtype)
    if lens is None:
        lens = rng.integers(0, max_pages * page // 2, n_slots)
    return cache, filled(cache, rng, lens)


def reserve(cache, ref, slots, add):
    got = sv.cache_reserve(cache, dev(add), slots=dev(slots))
    want = ref.reserve(range(len(add)) if slots is None else list(slots), add)
    assert got.cpu().tolist() == want.tolist()
    ref.same()


def keep(cache, ref, slots, count, absolute=False):
    got = sv.cache_keep(cache, dev(count), slots=dev(slots), absolute=absolute)
    want = ref.keep(range(len(count)) if slots is None else list(slots), count, absolute)
    assert got.cpu().tolist() == want.tolist()
    ref.same()


def fork(cache, ref, src, dst):
    got = sv.cache_fork(cache, dev(src), dev(dst))
    assert got.cpu().tolist() == ref.fork(list(src), list(dst)).tolist()
    ref.same()


@pytest.mark.parametrize("page,dim,layers", [(32, 64, 1), (64, 96, 2), (128, 128, 3), (256, 256, 1)])
def test_rounds(page, dim, layers):
    """Rounds of reserve and keep on listed slots, then on all."""
    rng = np.random.default_rng(page)
    cache, ref = small(rng, page=page, dim=dim, layers=layers)
    for i in range(4):
        slots = rng.permutation(7)[:5]
        slots[rng.integers(5)] = -1
        add = rng.integers(0, 66, 5)
        reserve(cache, ref, slots, add)
        keep(cache, ref, slots, (add * rng.random(5)).astype(int))
    reserve(cache, ref, None, rng.integers(0, 20, 7))
    keep(cache, ref, None, rng.integers(0, 40, 7), absolute=True)
    keep(cache, ref, None, np.zeros(7), absolute=True)
    assert not ref.refs.any()


def test_limits_and_bad_slots():
    rng = np.random.default_rng(5)
    cache, ref = small(rng, lens=[0, 1, 31, 32, 33, 200, 288])
    reserve(cache, ref, [0, 3, 3, 7, -2, -1, 6, 5], [5, 5, 5, 5, 5, 5, 1, -1])  # 3 twice; 6 has all its pages full
    reserve(cache, ref, [6, 5, 4, 0], [0, 88, 89 + 200, 288])
    keep(cache, ref, [0, 3, 3, 7, -2, -1, 6, 5], [2, 0, 0, 0, 0, 99, 1, -1])
    keep(cache, ref, [0, 1, 2], [286, 32, 33], absolute=True)
    keep(cache, ref, [0, 1, 2], [287, 31, 1], absolute=True)
    big = [2**31 - 1] * 3
    reserve(cache, ref, [0, 1, 2], big)
    keep(cache, ref, [0, 1, 2], big)


def test_pool_runs_out():
    """Pages go in the sessions' order; the first that does not fit stops those behind it."""
    rng = np.random.default_rng(6)
    cache, ref = small(rng, n_pages=10, lens=[30, 0, 64, 0, 0, 5, 0])  # 4 in use
    reserve(cache, ref, [0, 1, 2, 3, 4, 5, 6], [3, 64, 0, 64, 32, 20, 1])  # 1+2+0+2+1+0+1 of 6
    reserve(cache, ref, [1, 2, 4, 5], [1, 0, 0, 27])
    keep(cache, ref, [3], [0], absolute=True)
    reserve(cache, ref, [6, 0], [64, 40])


def test_empty_pool_and_all_pages():
    rng = np.random.default_rng(7)
    cache, ref = small(rng, n_slots=2, n_pages=1, max_pages=1, lens=[0, 0])
    reserve(cache, ref, None, [0, 0])
    reserve(cache, ref, None, [32, 1])
    reserve(cache, ref, None, [1, 1])
    keep(cache, ref, None, [32, 0])


@pytest.mark.parametrize("n_pages", [31, 33, 1000, 32768, 70001])
def test_long_lists(n_pages):
    """Prompts of many pages, in a pool that is fragmented."""
    rng = np.random.default_rng(n_pages)
    cache = sv.make_cache(40, n_pages, n_pages, 1, 64, page=32)
    ref = Ref(cache, pages=False)
    ref.refs[rng.random(n_pages) < 0.6] = 1  # pages that other lists of the program hold
    ref.sound = lambda: None
    ref.store()
    free = int((ref.refs == 0).sum())
    add = np.minimum(free * 32 // 8 * rng.random(40) ** 2, n_pages * 32).astype(int)
    reserve(cache, ref, rng.permutation(40), add)
    keep(cache, ref, None, np.zeros(40), absolute=True)


def test_many_sessions():
    rng = np.random.default_rng(8)
    n = 4096
    cache = sv.make_cache(n + 5, 9000, 3, 1, 64, page=32)
    ref = Ref(cache, pages=False)
    slots = rng.permutation(n + 5)[:n]
    slots[10] = slots[4000]
    reserve(cache, ref, slots, rng.integers(0, 97, n))
    keep(cache, ref, slots, rng.integers(0, 64, n))
    reserve(cache, ref, slots, rng.integers(0, 65, n))
    keep(cache, ref, slots, rng.integers(-1, 64, n), absolute=True)


def test_the_most_slots():
    cache = sv.make_cache(1 << 16, 4, 1, 1, 64, page=32)
    ref = Ref(cache)
    reserve(cache, ref, [65535, 65536, 0, 65535], [1, 1, 1, 1])
    reserve(cache, ref, [65535, 31, 32], [1, 32, 1])
    keep(cache, ref, [65535, 65536, 31], [1, 1, 1])


@pytest.mark.parametrize("page,dim,dtype", [(32, 64, torch.float16), (64, 128, torch.bfloat16), (256, 96, torch.bfloat16),
                                            (128, 256, torch.float16)])
def test_forks(page, dim, dtype):
    """Forks, then rows of their own: a last page that others hold is copied."""
    rng = np.random.default_rng(dim)
    lens = [2 * page + 1, 3 * page, 0, page - 1, 0, 0, 0, 0, 0, 0]
    cache, ref = small(rng, n_slots=10, n_pages=40, page=page, dim=dim, layers=3, dtype=dtype, lens=lens)
    fork(cache, ref, [0, 0, 1, 3, 2, -1, 0], [4, 5, 6, 7, 8, 9, -1])
    reserve(cache, ref, [0, 4, 5, 6, 7], [1, 1, 1, 1, 1])  # 0, 4 and 5 all want the page they share
    reserve(cache, ref, [1, 3, 2], [9, 1, 3])
    keep(cache, ref, [4, 6], [1, 1])
    keep(cache, ref, [0], [page // 2], absolute=True)  # into pages that 5 holds too
    reserve(cache, ref, [0, 5], [0, 0])
    reserve(cache, ref, [0, 5], [page, page])
    keep(cache, ref, [0, 5, 1, 4, 6, 7], [0] * 6, absolute=True)


def test_forks_refused():
    rng = np.random.default_rng(11)
    cache, ref = small(rng, n_slots=8, lens=[40, 50, 60, 0, 0, 0, 0, 0])
    fork(cache, ref, [0, 1, 2, 0, 3, 8, 0, 0, 5], [3, 3, 1, 0, 4, 4, -2, 8, 5])
    fork(cache, ref, [0, 3, 4], [3, 5, 6])  # 3 is taken over and given on at once
    fork(cache, ref, [0, 0], [6, 7])
    fork(cache, ref, [0], [6])


def test_copies_without_pages():
    """A session whose copy finds no page keeps sharing, and its rows are not written."""
    rng = np.random.default_rng(12)
    cache, ref = small(rng, n_slots=4, n_pages=3, lens=[40, 0, 0, 0], dim=64)
    fork(cache, ref, [0], [1])
    reserve(cache, ref, [0, 1], [1, 1])  # one page for two copies
    assert ref.refs[ref.table[1, 1]] == 1
    kv = rng.integers(0, 1000, (2, 2, 2, 2, 64)).astype(np.int16)
    k, v = (torch.from_numpy(x).cuda().view(torch.bfloat16) for x in kv)
    sv.cache_write(cache, 1, k, v)
    ref.write(1, [0, 1], [(kv[0][b], kv[1][b]) for b in range(2)])
    ref.same()
    fork(cache, ref, [0], [2])
    reserve(cache, ref, [2], [1])  # none left: 0 and 2 share
    sv.cache_write(cache, 0, k, v, slots=dev([0, 2]))
    ref.same()


@pytest.mark.parametrize("n_pages,share", [(9, 0.5), (64, 0.1), (64, 0.9), (500, 0.5), (9000, 0.1), (40, 0.0), (40, 1.0)])
def test_compact(n_pages, share):
    rng = np.random.default_rng(n_pages)
    n_slots = 12
    cache = sv.make_cache(n_slots, n_pages, 200, 1, 64, n_layers=2, page=32)
    ref = Ref(cache)
    for x in (ref.k, ref.v):
        x[:] = rng.integers(0, 30000, x.shape)
    pages = rng.permutation(n_pages)[:min(int(n_pages * share), n_slots * 100)]
    for i, part in enumerate(np.array_split(pages, n_slots)):
        ref.table[i, :len(part)] = part
        ref.held[i] = len(part)
        ref.lens[i] = max(0, len(part) * 32 - 5)
        ref.refs[part] += 1
    for i in range(1, n_slots, 3):  # first pages that two hold
        if ref.held[i] and ref.held[i - 1]:
            ref.refs[ref.table[i, 0]] -= 1
            ref.table[i, 0] = ref.table[i - 1, 0]
            ref.refs[ref.table[i, 0]] += 1
    ref.store()
    for _ in range(2):  # the second time nothing moves
        moved = torch.full((n_pages,), 7, dtype=torch.int32, device="cuda")
        used = sv.cache_compact(cache, moved=moved)
        want, where = ref.compact()
        ref.same()
        assert used.tolist() == [want]
        assert np.array_equal(moved.cpu().numpy(), where)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,dim,R", [(32, 64, 1), (32, 128, 9), (64, 96, 33), (128, 128, 17), (256, 256, 65), (64, 64, 200)])
def test_write(page, dim, R, dtype):
    rng = np.random.default_rng(R)
    n, Hkv = 6, 3
    lens = rng.integers(0, 3 * page, n)
    lens[:3] = 0, page - 1, 2 * page
    cache = sv.make_cache(n + 2, 80, 12, Hkv, dim, n_layers=2, page=page, dtype=dtype)
    ref = filled(cache, rng, list(lens) + [0, 0])
    slots = rng.permutation(n + 2)[:n]
    slots[4] = -1
    reserve(cache, ref, slots, np.minimum(rng.integers(0, R + 1, n) + R // 2, 12 * page - 3 * page))
    rows = rng.integers(-1, R + 2, n)  # cut to [0, R]; some have fewer pages than rows
    wide = rng.integers(-30000, 30000, (n, R, 2 * Hkv + 3, dim)).astype(np.int16)
    t = torch.from_numpy(wide).cuda().view(dtype)
    for use in (rows, None):
        sv.cache_write(cache, 1, t[:, :, 2:2 + Hkv], t[:, :, 3 + Hkv:], slots=dev(slots), rows=dev(use))
        cut = np.full(n, R) if use is None else use.clip(0, R)
        ref.write(1, slots, [(wide[b, :cut[b], 2:2 + Hkv], wide[b, :cut[b], 3 + Hkv:]) for b in range(n)])
        ref.same()


@pytest.mark.parametrize("lens", [[0], [1], [7, 0, 9], [100, 1, 0, 33], [8, 8, 8, 8, 8, 8], [3000], [0, 0, 0]])
@pytest.mark.parametrize("start", [0, 5, 8])
def test_write_line(lens, start):
    """Prompts in one line, behind `start` tokens of each session."""
    rng = np.random.default_rng(sum(lens) + start)
    B, Hkv, dim = len(lens), 2, 64
    cache = sv.make_cache(B + 1, 200, 100, Hkv, dim, page=32)
    ref = filled(cache, rng, [start] * (B + 1))
    slots = rng.permutation(B + 1)[:B]
    reserve(cache, ref, slots, np.array(lens))
    offsets = np.concatenate([[0], np.cumsum(lens)])
    kv = rng.integers(-30000, 30000, (2, offsets[-1], Hkv, dim)).astype(np.int16)
    k, v = (torch.from_numpy(x).cuda().view(torch.bfloat16) for x in kv)
    sv.cache_write(cache, 0, k, v, slots=dev(slots), offsets=dev(offsets))
    ref.write(0, slots, [(kv[0][lo:hi], kv[1][lo:hi]) for lo, hi in zip(offsets, offsets[1:])])
    ref.same()


def test_write_line_cut():
    """Offsets that leave the line are cut to it."""
    rng = np.random.default_rng(3)
    cache = sv.make_cache(3, 30, 10, 1, 64, page=32)
    ref = filled(cache, rng, [0, 0, 0])
    reserve(cache, ref, None, [40, 40, 40])
    kv = rng.integers(-30000, 30000, (2, 50, 1, 64)).astype(np.int16)
    k, v = (torch.from_numpy(x).cuda().view(torch.bfloat16) for x in kv)
    sv.cache_write(cache, 0, k, v, offsets=dev([-3, 20, 45, 90]))
    ref.write(0, [0, 1, 2], [(kv[0][lo:hi], kv[1][lo:hi]) for lo, hi in ((0, 20), (20, 45), (45, 50))])
    ref.same()


def test_far_pages():
    """A pool of more than 2^32 bytes a plane: the last pages of the last layer."""
    layers, n_pages, Hkv, dim, page = 3, 5600, 8, 128, 128
    cache = sv.make_cache(2, n_pages, 4, Hkv, dim, n_layers=layers, page=page)
    assert 2 * cache.k.numel() > 2**32
    cache.refs[:n_pages - 3] = 1
    add = dev([130, 0])
    assert sv.cache_reserve(cache, add).tolist() == [0, 0]
    assert cache.table[0].tolist() == [n_pages - 3, n_pages - 2, -1, -1]
    rng = np.random.default_rng(4)
    kv = rng.integers(-30000, 30000, (2, 1, 130, Hkv, dim)).astype(np.int16)
    k, v = (torch.from_numpy(x).cuda().view(torch.bfloat16) for x in kv)
    sv.cache_write(cache, 2, k, v, slots=dev([0]))
    sv.cache_keep(cache, dev([130]), slots=dev([0]))
    sv.cache_fork(cache, dev([0]), dev([1]))
    sv.cache_reserve(cache, dev([1]), slots=dev([1]))
    assert cache.table[1].tolist() == [n_pages - 3, n_pages - 1, -1, -1]
    orders = sv.cache_order(page, dim)
    for x, order, want in zip(cache[:2], orders, kv):
        got = x[2, cache.table[1, :2].long()].view(torch.int16).cpu().numpy().reshape(2, Hkv, -1)[..., order]
        got = got.transpose(0, 2, 1, 3).reshape(2 * page, Hkv, dim)[:130]
        assert np.array_equal(got, want[0])


def test_binding_checks():
    cache = sv.make_cache(3, 10, 4, 2, 64, page=32)
    i = dev([0, 0, 0])
    x = torch.zeros((3, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sv.cache_reserve(cache, dev([0] * 4))  # more sessions than slots
    with pytest.raises(TypeError):
        sv.cache_reserve(cache, i.long())
    with pytest.raises(ValueError):
        sv.cache_keep(cache, i, slots=i[:2])
    with pytest.raises(ValueError):
        sv.cache_fork(cache, i, i[:2])
    with pytest.raises(sv.SvError):
        sv.cache_reserve(cache, i, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sv.cache_write(cache, 0, x, x[:, :1])
    with pytest.raises(TypeError):
        sv.cache_write(cache, 0, x.half(), x.half())
    with pytest.raises(ValueError):
        sv.cache_write(cache, 0, x, x, rows=i, offsets=dev([0, 1, 2, 3]))
    with pytest.raises(sv.SvError):
        sv.cache_write(cache, 1, x, x)
    odd = torch.zeros((3, 2, 2, 65), dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(ValueError):
        sv.cache_write(cache, 0, odd, x)
    with pytest.raises(ValueError):
        sv.cache_write(cache, 0, x.transpose(2, 3).contiguous().transpose(2, 3), x)
    with pytest.raises(ValueError):
        sv.cache_compact(cache, moved=i)
    with pytest.raises(ValueError):
        sv.cache_reserve(cache._replace(lens=cache.lens[:2]), i)
    torch.cuda.synchronize()
