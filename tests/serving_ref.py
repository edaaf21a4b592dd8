"""Plain 64-bit implementations of the serving operators, written from their definitions in
include/energon_rce.h: numpy on the host, loops over sequences and heads, no shared code with
the library.  What the definitions hold in fp32 (scales, quotients of codes) is fp32 here."""
from __future__ import annotations

import numpy as np


def spans(lens):
    ends = np.cumsum(lens)
    return [(int(e - n), int(e)) for n, e in zip(lens, ends)]


def prompt(q, k, v, lens, scale):
    """o [T, heads, d], lse [heads, T], mag [T, heads, d] = sum p |v|, smag [heads, T] = the largest
    scale sum_d |q_d k_d| among a query's keys (both size the rounding errors)."""
    T, H, d = q.shape
    g = H // k.shape[1]
    o, mag = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, smag = np.zeros((H, T)), np.zeros((H, T))
    for a, b in spans(lens):
        n = b - a
        if n == 0:
            continue
        after = np.triu(np.ones((n, n), bool), 1)
        for j in range(H):
            kk, vv = k[a:b, j // g], v[a:b, j // g]
            x = np.where(after, -np.inf, q[a:b, j] @ kk.T * scale)
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            l = e.sum(1, keepdims=True)
            o[a:b, j], mag[a:b, j] = (e / l) @ vv, (e / l) @ np.abs(vv)
            lse[j, a:b] = (m + np.log(l))[:, 0]
            smag[j, a:b] = np.where(after, 0.0, np.abs(q[a:b, j]) @ np.abs(kk).T * scale).max(1)
    return o, lse, mag, smag


def key_weights(q, k, lse, lens, scale, window):
    T, H, _ = q.shape
    kv = k.shape[1]
    g = H // kv
    w = np.zeros((kv, T))
    for a, b in spans(lens):
        n = b - a
        first = max(0, n - window)
        for j in range(H):
            x = q[a + first:b, j] @ k[a:b, j // g].T * scale
            p = np.exp(x - lse[j, a + first:b, None])
            p[np.arange(n)[None, :] > np.arange(first, n)[:, None]] = 0.0
            w[j // g, a:b] += p.sum(0)
    return w


F32_MIN = np.float32(2.0 ** -126)


class Cache:
    """The paged cache on the host."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, weight):
        self.codes = {"k": k_codes.copy(), "v": v_codes.copy()}
        self.scale = {"k": k_scale.copy(), "v": v_scale.copy()}
        self.weight = None if weight is None else weight.copy()
        self.n_pages, self.kv, self.P, self.d = k_codes.shape

    def held(self, name, pages, j, n):
        """Tokens 0 .. n-1 of one head as values in 64 bits."""
        rows = [self.codes[name][p, j].astype(np.float64) * float(self.scale[name][p, j]) for p in pages]
        return np.concatenate(rows)[:n] if rows else np.zeros((0, self.d))


def encode(x, scale):
    """Codes of fp32 values for an fp32 scale."""
    if scale > 0:
        with np.errstate(over="ignore", invalid="ignore"):
            q = np.clip(np.rint(x.astype(np.float32) / np.float32(scale)), -127, 127)
    else:
        q = np.zeros_like(x, dtype=np.float32)
    q = np.where(np.isinf(x), np.sign(x) * 127, q)
    return np.where(np.isnan(x), 0, q).astype(np.int8)


def append(cache, table, cache_lens, k, v, weights, new):
    """new[b] rows per sequence, packed in k and v (fp32 values)."""
    for b, (a, e) in enumerate(spans(new)):
        at, row = int(cache_lens[b]) - new[b], a
        while row < e:
            P = cache.P
            take = min(e - row, P - at % P)
            p, s0 = int(table[b, at // P]), at % P
            for j in range(cache.kv):
                for name, x in (("k", k), ("v", v)):
                    y = x[row:row + take, j].astype(np.float32)
                    fin = np.abs(y[np.isfinite(y)])
                    need = np.float32(fin.max() if fin.size else 0) * np.float32(1.0 / 127.0)
                    need = need if need >= F32_MIN else np.float32(0)
                    scale = need
                    if s0 > 0:
                        old, times = cache.scale[name][p, j], 1.0
                        if old > 0:
                            while float(old) * times < float(need):
                                times *= 2.0
                            scale = np.float32(float(old) * times)
                            c = cache.codes[name][p, j]
                            c[:] = np.rint(c.astype(np.float64) / times).astype(np.int8)
                    cache.scale[name][p, j] = scale
                    cache.codes[name][p, j, s0:s0 + take] = encode(y, scale)
                if cache.weight is not None:
                    cache.weight[p, j, s0:s0 + take] = 0.0 if weights is None else weights[j, row:row + take]
            at, row = at + take, row + take


def decode(cache, table, cache_lens, q, scale, good=None):
    """o [B, heads, d], lse [B, heads], probabilities per (b, head), sum p |V|, largest scale sum |q K|.
    good(b, t): whether token t counts."""
    B, H, d = q.shape
    g = H // cache.kv
    o, mag = np.zeros((B, H, d)), np.zeros((B, H, d))
    lse, smag, probs = np.full((B, H), -np.inf), np.zeros((B, H)), {}
    for b in range(B):
        n = int(cache_lens[b])
        pages = [int(p) for p in table[b, :-(-n // cache.P)]]
        ok = np.array([good is None or good(b, t) for t in range(n)], bool)
        pages = [p if 0 <= p < cache.n_pages else 0 for p in pages]
        for j in range(cache.kv):
            K, V = cache.held("k", pages, j, n), cache.held("v", pages, j, n)
            for h in range(j * g, (j + 1) * g):
                x = np.where(ok, K @ q[b, h] * scale, -np.inf)
                probs[b, h] = np.zeros(n)
                if not ok.any():
                    continue
                m = x.max()
                e = np.exp(x - m)
                p = e / e.sum()
                o[b, h], mag[b, h] = p @ V, p @ np.abs(V)
                lse[b, h], probs[b, h] = m + np.log(e.sum()), p
                smag[b, h] = (np.abs(K) @ np.abs(q[b, h]) * scale)[ok].max()
    return o, lse, probs, mag, smag


def evict(cache, table, cache_lens, new_table, budget, recent):
    """Works on a copy of the old cache, so that in place and out of place are the same."""
    src = Cache(cache.codes["k"], cache.codes["v"], cache.scale["k"], cache.scale["v"], cache.weight)
    P, lens = cache.P, []
    for b, n in enumerate(int(x) for x in cache_lens):
        keep = min(n, budget)
        lens.append(keep)
        in_place = keep > 0 and table[b, 0] == new_table[b, 0]
        if in_place and n <= budget:
            continue
        for j in range(cache.kv):
            w = np.array([src.weight[table[b, t // P], j, t % P] for t in range(n)], np.float32)
            if n > budget:
                m = n - recent
                key = np.where(np.isnan(w[:m]), -np.inf, w[:m].astype(np.float64))
                order = sorted(range(m), key=lambda t: (np.isnan(w[t]), -key[t], t))
                pos = sorted(order[:budget - recent]) + list(range(m, n))
            else:
                pos = list(range(n))
            for at in range(0, keep, P):
                part, to = pos[at:at + P], int(new_table[b, at // P])
                cache.weight[to, j, :len(part)] = w[part]
                for name in ("k", "v"):
                    s = np.array([src.scale[name][table[b, t // P], j] for t in part], np.float32)
                    big = s.max()
                    for i, t in enumerate(part):
                        ratio = s[i] / big if s[i] > 0 else np.float32(0)
                        c = src.codes[name][table[b, t // P], j, t % P].astype(np.float32) * np.float32(ratio)
                        cache.codes[name][to, j, i] = np.rint(c).astype(np.int8)
                    cache.scale[name][to, j] = big
    return lens
