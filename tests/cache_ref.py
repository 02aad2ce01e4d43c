"""A plain paged cache on the host: the page calls with whole numbers, attention in
64 bits, written from the definitions in include/specverify.h."""
import numpy as np
import torch

import token_sampling_amd as sv


class Ref:
    """table, lens, held, refs and the pages' bits k, v [n_layers, n_pages, n_kv, page,
    head_dim] by token (int16)."""

    def __init__(self, cache, pages=True):
        self.cache, self.pages = cache, pages  # pages=False: only the lists
        self.page, self.dim = cache.k.shape[3:]
        self.orders = sv.cache_order(self.page, self.dim)
        self.load()

    def load(self):
        torch.cuda.synchronize()
        c = self.cache
        self.table, self.lens, self.held, self.refs = (x.cpu().numpy().copy() for x in c[2:])
        self.k, self.v = self.by_token() if self.pages else (np.zeros((1, len(self.refs), 1, 32, 1), np.int16),) * 2

    def by_token(self):
        out = []
        for x, order in zip(self.cache[:2], self.orders):
            x = x.view(torch.int16).cpu().numpy()
            out.append(x.reshape(*x.shape[:3], -1)[..., order].copy())
        return out

    def store(self):
        """The reference's state into the cache."""
        for x, order, mine in zip(self.cache[:2] if self.pages else (), self.orders, (self.k, self.v)):
            flat = np.empty((*mine.shape[:3], self.page * self.dim), np.int16)
            flat[..., order.reshape(-1)] = mine.reshape(*mine.shape[:3], -1)
            x.view(torch.int16).copy_(torch.from_numpy(flat.reshape(mine.shape)))
        for x, mine in zip(self.cache[2:], (self.table, self.lens, self.held, self.refs)):
            x.copy_(torch.from_numpy(mine))

    def same(self):
        torch.cuda.synchronize()
        c = self.cache
        for x, mine, name in zip(c[2:], (self.table, self.lens, self.held, self.refs),
                                 ("table", "lens", "held", "refs")):
            assert np.array_equal(x.cpu().numpy(), mine), name
        for x, mine, name in zip(self.by_token() if self.pages else (), (self.k, self.v), "kv"):
            assert np.array_equal(x, mine), name
        self.sound()

    def sound(self):
        """Every list's pages counted once, nothing behind them."""
        refs = np.zeros_like(self.refs)
        for h, row in enumerate(self.table):
            assert (row[self.held[h]:] == -1).all()
            assert self.lens[h] <= self.held[h] * self.page
            np.add.at(refs, row[:self.held[h]], 1)
        assert np.array_equal(refs, self.refs)

    def pages_of(self, n):
        return -(-n // self.page)

    def bad(self, slots, b):
        h = slots[b]
        return not -1 <= h < len(self.lens) or (h >= 0 and (np.asarray(slots) == h).sum() > 1)

    def reserve(self, slots, add):
        status = np.zeros(len(slots), np.int32)
        free = list(np.nonzero(self.refs == 0)[0])
        n_free, want, plan = len(free), 0, []
        refs0 = self.refs.copy()
        for b, h in enumerate(slots):
            if self.bad(slots, b):
                status[b] = sv.S_BAD_CACHE
                continue
            if h < 0:
                continue
            total = self.pages_of(int(self.lens[h]) + int(add[b]))
            if add[b] < 0 or total > self.table.shape[1]:
                status[b] = sv.S_LIMIT
                continue
            more = max(0, total - self.held[h])
            last = self.lens[h] // self.page
            copy = add[b] > 0 and last < self.held[h] and refs0[self.table[h, last]] > 1
            want += more + copy
            if more + copy and want > n_free:
                status[b] = sv.S_NO_PAGES
                continue
            if copy:
                old, new = self.table[h, last], free.pop(0)
                part = self.lens[h] % self.page
                part = -(-part // 32) * 32
                for x in (self.k, self.v):
                    x[:, new, :, :part] = x[:, old, :, :part]
                self.table[h, last] = new
                self.refs[new] = 1
                self.refs[old] -= 1
            for _ in range(more):
                new = free.pop(0)
                self.table[h, self.held[h]] = new
                self.held[h] += 1
                self.refs[new] = 1
        return status

    def keep(self, slots, count, absolute):
        status = np.zeros(len(slots), np.int32)
        for b, h in enumerate(slots):
            if self.bad(slots, b):
                status[b] = sv.S_BAD_CACHE
            elif h >= 0:
                n = int(count[b]) + (0 if absolute else int(self.lens[h]))
                if count[b] < 0 or n > self.held[h] * self.page:
                    status[b] = sv.S_LIMIT
                    continue
                while self.held[h] > self.pages_of(n):
                    self.held[h] -= 1
                    self.refs[self.table[h, self.held[h]]] -= 1
                    self.table[h, self.held[h]] = -1
                self.lens[h] = n
        return status

    def fork(self, src, dst):
        status = np.zeros(len(src), np.int32)
        n_slots = len(self.lens)
        todo = []
        for i, (s, d) in enumerate(zip(src, dst)):
            if s == -1 or d == -1:
                continue
            if not (0 <= s < n_slots and 0 <= d < n_slots) or (np.asarray(dst) == d).sum() > 1 \
                    or s in dst or self.held[d] != 0:
                status[i] = sv.S_BAD_CACHE
            else:
                todo.append((s, d))
        for s, d in todo:
            n = self.pages_of(self.lens[s])
            self.table[d, :n] = self.table[s, :n]
            self.refs[self.table[s, :n]] += 1
            self.lens[d], self.held[d] = self.lens[s], n
        return status

    def compact(self):
        used = int((self.refs > 0).sum())
        moved = np.where(self.refs > 0, np.arange(len(self.refs)), -1)
        holes = [p for p in range(used) if self.refs[p] == 0]
        for old in range(used, len(self.refs)):
            if self.refs[old] == 0:
                continue
            new = holes.pop(0)
            moved[old] = new
            self.table[self.table == old] = new
            self.refs[new], self.refs[old] = self.refs[old], 0
            for x in (self.k, self.v):
                x[:, new] = x[:, old]
        return used, moved

    def write(self, layer, slots, spans):
        """spans: per session (k, v) [n, n_kv, head_dim] int16."""
        for h, (k, v) in zip(slots, spans):
            if not 0 <= h < len(self.lens):
                continue
            for i in range(len(k)):
                at = int(self.lens[h]) + i
                if at // self.page >= self.held[h] or self.refs[self.table[h, at // self.page]] != 1:
                    continue
                p = self.table[h, at // self.page]
                self.k[layer, p, :, at % self.page] = k[i]
                self.v[layer, p, :, at % self.page] = v[i]

    def attention(self, layer, slots, rows, q, scale, dtype):
        """Outputs [B, R, Hq, D] in 64 bits (NaN where not defined) and their bounds.

        The bound, with u the relative rounding of dtype: u |o| for the output, u A for
        the weights (A = sum_t w_t |v_t|; fp16 weights, whose sum is at least 1
        before it is divided out, are off by 2^-25 where they are subnormal), and in binary32
        (n + 4) 2^-23 A for sums of n terms that join in any order, and for the scores,
        D products summed, scaled twice and put into exp2, 2 A max_t e_t with e_t =
        (D + 8) 2^-23 scale sum_d |q_d k_td|."""
        B, R, Hq, D = q.shape
        Hkv = self.k.shape[2]
        G = Hq // Hkv
        u = torch.finfo(dtype).eps / 2
        out, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
        as_float = lambda x: torch.from_numpy(np.ascontiguousarray(x)).view(dtype).double().numpy()  # noqa: E731
        for b, h in enumerate(slots):
            if not 0 <= h < len(self.lens) or rows[b] < 1:
                continue
            n = int(self.lens[h]) + int(rows[b])
            ids = self.table[h, :self.pages_of(n)]
            k = as_float(self.k[layer, ids].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n])
            v = as_float(self.v[layer, ids].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n])
            for r in range(rows[b]):
                t = int(self.lens[h]) + r + 1
                for hq in range(Hq):
                    kk, vv, x = k[hq // G, :t], v[hq // G, :t], q[b, r, hq]
                    z = kk @ x * scale
                    with np.errstate(all="ignore"):
                        w = np.exp(z - z.max())
                        w /= w.sum()
                        o = w @ vv
                        A = w @ np.abs(vv)
                        e = (D + 8) * 2.0**-23 * scale * (np.abs(kk) @ np.abs(x)).max()
                        tiny = 2.0**-25 * np.abs(vv).sum(0) if dtype == torch.float16 else 0
                        out[b, r, hq] = o
                        tol[b, r, hq] = u * np.abs(o) + A * (u + (t + 4) * 2.0**-23 + 2 * e) + tiny
        return out, tol


def filled(cache, rng, lens, order=None, garbage=None):
    """Gives slot h lens[h] tokens in pages of a random order; all pages hold normal
    values, those of no token the bits of garbage (NaN by default)."""
    r = Ref(cache)
    dtype = cache.k.dtype
    shape = r.k.shape
    take = iter(rng.permutation(shape[1]) if order is None else order)
    bits = lambda x: torch.from_numpy(x).to(dtype).view(torch.int16).numpy()  # noqa: E731
    nan = bits(np.array([np.nan if garbage is None else garbage]))[0]
    for x in (r.k, r.v):
        x[:] = nan
    for h, n in enumerate(lens):
        for i in range(r.pages_of(n)):
            p = next(take)
            r.table[h, i] = p
            r.refs[p] = 1
            m = min(r.page, n - i * r.page)
            for x in (r.k, r.v):
                x[:, p, :, :m] = bits(rng.standard_normal((shape[0], shape[2], m, r.dim)))
        r.lens[h], r.held[h] = n, r.pages_of(n)
    r.store()
    return r
