"""The paged 8-bit cache in float64 (NumPy): e4m3 codes, appending, attention, token weights, eviction.

Test infrastructure only (see the package docstring).

Written from the definitions in include/lix_kv8.h, one sequence and head at a
time; caches are dicts of uint8 codes k, v [num_pages, Hkv, page, D] and
float64 scales k_scale, v_scale [num_pages, Hkv].
"""

import numpy as np


def _e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), c >> 3 & 15, c & 7
        t[c] = sign * (np.ldexp(m, -9) if e == 0 else np.ldexp(8 + m, e - 10))
    t[0x7F] = t[0xFF] = np.nan
    return t


E4M3 = _e4m3_table()


def e4m3_encode(x):
    """Codes of the nearest e4m3 values, ties to the even code, saturating at 448; NaN becomes 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, np.nan_to_num(mag), side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code |= np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def page_scale(top):
    """The smallest power of two >= top / 448, at least 2^-60."""
    e = -60
    while np.ldexp(448.0, e) < top:
        e += 1
    return np.ldexp(1.0, e)


def finite_top(x):
    x = np.abs(x[np.isfinite(x)])
    return float(x.max()) if x.size else 0.0


def _page(cache, table_row, nth):
    if nth >= len(table_row):
        return -1
    pid = int(table_row[nth])
    return pid if 0 <= pid < cache["k"].shape[0] else -1


def _length(table, lens, b, page):
    return int(min(max(int(lens[b]), 0), table.shape[1] * page))


def append(cache, k, v, table, lens, new_lens=None):
    """k, v float64 [B, S, Hkv, D]; the cache is changed in place."""
    B, S, H, _ = k.shape
    page = cache["k"].shape[2]
    for b in range(B):
        n = _length(table, lens, b, page)
        m = S if new_lens is None else int(min(max(int(new_lens[b]), 0), S))
        for nth in range(n // page, (n + m - 1) // page + 1 if m else 0):
            pid = _page(cache, table[b], nth)
            if pid < 0:
                continue
            lo, hi = max(n, nth * page), min(n + m, (nth + 1) * page)
            old = lo - nth * page
            for name, x in (("k", k), ("v", v)):
                for h in range(H):
                    rows = x[b, lo - n:hi - n, h]
                    before = cache[name + "_scale"][pid, h]
                    scale = page_scale(finite_top(rows))
                    if old:
                        scale = max(scale, before)
                        if scale != before:
                            # products of the library are in fp32
                            kept = np.float32(E4M3[cache[name][pid, h, :old]]) * np.float32(before)
                            cache[name][pid, h, :old] = e4m3_encode(np.float32(kept / np.float32(scale)))
                    cache[name + "_scale"][pid, h] = scale
                    cache[name][pid, h, old:old + hi - lo] = e4m3_encode(np.float32(np.float32(rows) / np.float32(scale)))


def _tokens(cache, name, table, b, h, n):
    """Values of the n tokens of a sequence and which of them are on a page."""
    page = cache["k"].shape[2]
    x = np.zeros((n, cache["k"].shape[3]))
    there = np.zeros(n, dtype=bool)
    for s in range(n):
        pid = _page(cache, table[b], s // page)
        if pid >= 0:
            x[s] = E4M3[cache[name][pid, h, s % page]] * cache[name + "_scale"][pid, h]
            there[s] = True
    return x, there


def _seen(n, t, b, q_start, q_lens, ratio):
    if q_lens is not None and t >= q_lens[b]:
        return 0
    if q_start is None:
        return n
    return max(0, min(n, (int(q_start[b]) + t + 1) // ratio))


def attention(q, cache, table, lens, scale, q_start=None, q_lens=None, ratio=1, indices=None):
    """q float64 [B, S, Hq, D].  Returns out, lse, and for error bounds: mag = sum p |v|, top = the largest
    scale * sum |q k| of a row's scores."""
    B, S, Hq, D = q.shape
    H = cache["k"].shape[1]
    G = Hq // H
    page = cache["k"].shape[2]
    out = np.zeros(q.shape)
    mag = np.zeros(q.shape)
    lse = np.full((B, S, Hq), -np.inf)
    top = np.zeros((B, S, Hq))
    for b in range(B):
        n = _length(table, lens, b, page)
        for h in range(H):
            k, there = _tokens(cache, "k", table, b, h, n)
            v, _ = _tokens(cache, "v", table, b, h, n)
            for t in range(S):
                seen = _seen(n, t, b, q_start, q_lens, ratio)
                if indices is None:
                    at = np.arange(seen)
                else:
                    at = indices[b, t].astype(np.int64)
                    at = at[(at >= 0) & (at < seen)]
                at = at[there[at]]
                if at.size == 0:
                    continue
                for g in range(G):
                    x = scale * (k[at] @ q[b, t, h * G + g])
                    top[b, t, h * G + g] = scale * (np.abs(np.nan_to_num(k[at])) @ np.abs(q[b, t, h * G + g])).max()
                    m = x.max()
                    p = np.exp(x - m)
                    lse[b, t, h * G + g] = m + np.log(p.sum())
                    p = p / p.sum()
                    out[b, t, h * G + g] = p @ v[at]
                    mag[b, t, h * G + g] = p @ np.abs(np.nan_to_num(v[at]))
    return out, lse, mag, top


def token_weights(q, cache, table, lens, lse, scale, q_start=None, q_lens=None, ratio=1):
    """float64 [B, Hkv, max_pages * page]; NaN for tokens behind the sequence (not written)."""
    B, S, Hq, D = q.shape
    H, page = cache["k"].shape[1], cache["k"].shape[2]
    G = Hq // H
    w = np.full((B, H, table.shape[1] * page), np.nan)
    for b in range(B):
        n = _length(table, lens, b, page)
        for h in range(H):
            k, there = _tokens(cache, "k", table, b, h, n)
            w[b, h, :n] = 0.0
            for t in range(S):
                seen = _seen(n, t, b, q_start, q_lens, ratio)
                for g in range(G):
                    ref = lse[b, t, h * G + g]
                    if seen == 0 or ref == -np.inf:
                        continue
                    p = np.exp(scale * (k[:seen] @ q[b, t, h * G + g]) - ref)
                    w[b, h, :seen] += np.where(there[:seen], p, 0.0)
    return w


def evict(cache, table, lens, weights, new_table, keep, recent=0, sinks=0):
    """The cache is changed in place; returns new_lens, kept, new_weights."""
    H, page = cache["k"].shape[1], cache["k"].shape[2]
    B = len(lens)
    new_lens = np.zeros(B, dtype=np.int32)
    kept = np.full((B, H, keep), -1, dtype=np.int32)
    new_w = np.zeros((B, H, keep), dtype=weights.dtype)
    for b in range(B):
        n = _length(table, lens, b, page)
        count = new_lens[b] = min(n, keep)
        for h in range(H):
            if n <= keep:
                chosen = list(range(n))
            else:
                rest = sorted(range(sinks, n - recent), key=lambda s: (-weights[b, h, s], s))
                chosen = sorted(list(range(sinks)) + rest[:keep - recent - sinks] + list(range(n - recent, n)))
            kept[b, h, :count] = chosen
            new_w[b, h, :count] = weights[b, h, chosen]
            for first in range(0, count, page):
                pid = _page(cache, new_table[b], first // page)
                if pid < 0:
                    continue
                for name in ("k", "v"):
                    rows = []
                    for s in chosen[first:first + page]:
                        src = _page(cache, table[b], s // page)
                        rows.append(np.zeros(cache["k"].shape[3]) if src < 0 else
                                    np.float32(E4M3[cache[name][src, h, s % page]]) *
                                    np.float32(cache[name + "_scale"][src, h]))
                    rows = np.array(rows, dtype=np.float32)
                    scale = page_scale(finite_top(rows.astype(np.float64)))
                    cache[name + "_scale"][pid, h] = scale
                    cache[name][pid, h, :len(rows)] = e4m3_encode(rows / np.float32(scale))
    return new_lens, kept, new_w
