"""Host-side refusals of the cache's calls (no kernel is launched): the C ABI's
argument checks, and the binding's; the order of a page's elements."""
import ctypes
import os

import numpy as np
import pytest
import torch

import token_sampling_amd as sv

FAKE = 0x1000  # never dereferenced: the calls return first


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(sv.LIB_PATH):
        from token_sampling_amd import build
        build.build()


def struct(**bad):
    a = dict(k=FAKE, v=FAKE, table=FAKE, lens=FAKE, held=FAKE, refs=FAKE, dtype=0, n_layers=2, n_pages=50, n_kv=2,
             page=64, head_dim=128, n_slots=8, max_pages=6)
    a.update(bad)
    return ctypes.byref(sv._Cache(**a))


BAD = [dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(held=None), dict(refs=None),
       dict(k=FAKE + 8), dict(v=FAKE + 2), dict(refs=FAKE + 4), dict(dtype=1), dict(dtype=3), dict(n_layers=0),
       dict(n_layers=4097), dict(n_pages=0), dict(n_pages=(1 << 20) + 1), dict(n_kv=0), dict(n_kv=1025), dict(page=16),
       dict(page=48), dict(page=512), dict(head_dim=32), dict(head_dim=80), dict(head_dim=192), dict(n_slots=0),
       dict(n_slots=(1 << 16) + 1), dict(max_pages=0), dict(max_pages=(1 << 20) + 1)]


def reserve(c, slots=FAKE, add=FAKE, B=4, ws=FAKE, n=1 << 20):
    return sv.lib().sv_cache_reserve(c, slots, add, B, None, ws, n, None)


def keep(c, slots=FAKE, count=FAKE, B=4):
    return sv.lib().sv_cache_keep(c, slots, count, 0, B, None, None)


def fork(c, src=FAKE, dst=FAKE, n=4):
    return sv.lib().sv_cache_fork(c, src, dst, n, None, None)


def compact(c, used=FAKE, ws=FAKE, n=1 << 20):
    return sv.lib().sv_cache_compact(c, used, None, ws, n, None)


def write(c, layer=0, frm="ok", k=FAKE, v=FAKE, strides=(1024, 256, 128) * 2, slots=FAKE, rows=None, offsets=None, B=4,
          R=3):
    r = ctypes.byref(sv._Rows(k, v, *strides)) if frm else None
    return sv.lib().sv_cache_write(c, layer, r, slots, rows, offsets, B, R, None)


def plan(c, slots=FAKE, heads=8, B=4, R=3, buf=FAKE, n=1 << 20):
    return sv.lib().sv_cache_plan(c, slots, None, heads, B, R, None, buf, n, None)


def attention(c, layer=0, q=FAKE, strides=(3 * 1024, 1024, 128), scale=0.1, buf=FAKE, heads=8, B=4, R=3, out=FAKE, ws=FAKE,
              n=1 << 28):
    return sv.lib().sv_cache_attention(c, layer, q, *strides, scale, buf, heads, B, R, out, ws, n, None)


@pytest.mark.parametrize("call", [reserve, keep, fork, compact, write, plan, attention], ids=lambda f: f.__name__)
@pytest.mark.parametrize("bad", [None] + BAD, ids=str)
def test_bad_caches(call, bad):
    assert call(None if bad is None else struct(**bad)) == sv.ERR_ARG
    L = sv.lib()
    c = None if bad is None else struct(**bad)
    assert L.sv_cache_workspace_bytes(c, 4) == 0
    assert L.sv_cache_plan_bytes(c, 8, 4, 3) == 0
    assert L.sv_cache_attention_bytes(c, 8, 4, 3) == 0


@pytest.mark.parametrize("call,bad", [
    (reserve, dict(add=None)), (reserve, dict(ws=None)), (reserve, dict(B=0)), (reserve, dict(B=4097)),
    (reserve, dict(slots=None, B=9)), (keep, dict(count=None)), (keep, dict(B=0)), (keep, dict(B=4097)),
    (keep, dict(slots=None, B=9)), (fork, dict(src=None)), (fork, dict(dst=None)), (fork, dict(n=0)), (fork, dict(n=4097)),
    (compact, dict(used=None)), (compact, dict(ws=None)), (write, dict(layer=-1)), (write, dict(layer=2)),
    (write, dict(frm=None)), (write, dict(k=None)), (write, dict(v=None)), (write, dict(k=FAKE + 8)),
    (write, dict(strides=(1024, 256, -8) * 2)), (write, dict(strides=(1024, 256, 4) * 2)),
    (write, dict(strides=((1 << 40) + 8, 256, 128) * 2)), (write, dict(R=-1)), (write, dict(B=0)), (write, dict(B=4097)),
    (write, dict(slots=None, B=9)), (write, dict(rows=FAKE, offsets=FAKE)), (plan, dict(heads=0)), (plan, dict(heads=7)),
    (plan, dict(heads=1026)), (plan, dict(B=0)), (plan, dict(B=4097)), (plan, dict(R=0)), (plan, dict(R=66)),
    (plan, dict(buf=None)), (plan, dict(buf=FAKE + 8)), (plan, dict(slots=None, B=9)), (attention, dict(layer=-1)),
    (attention, dict(layer=2)), (attention, dict(q=None)), (attention, dict(out=None)), (attention, dict(ws=None)),
    (attention, dict(buf=None)), (attention, dict(q=FAKE + 2)), (attention, dict(out=FAKE + 8)),
    (attention, dict(ws=FAKE + 8)), (attention, dict(strides=(-8, 1024, 128))), (attention, dict(strides=(8, 1020, 128))),
    (attention, dict(scale=0.0)), (attention, dict(scale=-1.0)), (attention, dict(scale=float("inf"))),
    (attention, dict(scale=float("nan"))), (attention, dict(heads=7)), (attention, dict(B=0)), (attention, dict(R=66))],
    ids=lambda x: x.__name__ if callable(x) else str(x))
def test_bad_arguments(call, bad):
    assert call(struct(), **bad) == sv.ERR_ARG


def test_small_workspaces():
    L = sv.lib()
    c = struct()
    assert reserve(c, n=L.sv_cache_workspace_bytes(c, 4) - 1) == sv.ERR_WORKSPACE
    assert compact(c, n=L.sv_cache_workspace_bytes(c, 1) - 1) == sv.ERR_WORKSPACE
    assert plan(c, n=L.sv_cache_plan_bytes(c, 8, 4, 3) - 1) == sv.ERR_WORKSPACE
    assert attention(c, n=L.sv_cache_attention_bytes(c, 8, 4, 3) - 1) == sv.ERR_WORKSPACE
    assert L.sv_cache_workspace_bytes(c, 4097) == 0 and L.sv_cache_plan_bytes(c, 8, 4, 66) == 0
    assert write(c, R=0, k=None, v=None) == sv.OK  # no rows: nothing to do


@pytest.mark.parametrize("page,dim", [(32, 64), (64, 96), (128, 128), (256, 256)])
def test_order(page, dim):
    """The order of a page's elements, place by place from the header's definition."""
    keys, values = sv.cache_order(page, dim)
    for order in (keys, values):
        assert np.array_equal(np.sort(order.reshape(-1)), np.arange(page * dim))
    rng = np.random.default_rng(page + dim)
    for t, d in zip(rng.integers(0, page, 200), rng.integers(0, dim, 200)):
        c, b, a, T = t % 4, t // 4 % 2, t // 8 % 4, t // 32
        e, g, C = d % 8, d // 8 % 4, d // 32
        assert keys[t, d] == ((((((T * 2 + b) * (dim // 32) + C) * 4 + g) * 4 + a) * 4 + c) * 8 + e)
        e, g = t % 8, t // 8 % 4
        m, n = d % 16, d // 16
        assert values[t, d] == (((T * (dim // 16) + n) * 4 + g) * 16 + m) * 8 + e


def test_makers():
    c = sv.make_cache(3, 10, 4, 2, 64, n_layers=5, page=32, device="cpu")
    assert c.k.shape == c.v.shape == (5, 10, 2, 32, 64) and c.k.dtype == torch.bfloat16
    assert c.table.shape == (3, 4) and (c.table == -1).all()
    for x, n in ((c.lens, 3), (c.held, 3), (c.refs, 10)):
        assert x.shape == (n,) and not x.any()
    for bad in (dict(page=16), dict(page=100)):
        with pytest.raises(ValueError):
            sv.make_cache(3, 10, 4, 2, 64, device="cpu", **bad)
    with pytest.raises(ValueError):
        sv.make_cache(3, 10, 4, 2, 72, device="cpu")
    with pytest.raises(TypeError):
        sv.make_cache(3, 10, 4, 2, 64, dtype=torch.float32, device="cpu")


def test_binding_refuses_host_tensors():
    c = sv.make_cache(3, 10, 4, 2, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: sv.cache_reserve(c, i), lambda: sv.cache_keep(c, i), lambda: sv.cache_fork(c, i, i),
                 lambda: sv.cache_compact(c), lambda: sv.cache_write(c, 0, x, x), lambda: sv.cache_plan(c, 2, 1, rows=i),
                 lambda: sv.cache_attention(c, 0, x, sv.CachePlan(i, i, 2, 2, 1, 2, 64, 64))):
        with pytest.raises(ValueError):
            call()


def test_statuses():
    texts = {sv.status_str(s) for s in (sv.S_NO_PAGES, sv.S_BAD_CACHE, sv.S_LIMIT, sv.S_BAD_CONTROL, -99)}
    assert len(texts) == 5
