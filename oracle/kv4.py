"""Plain definitions of the 4-bit key/value cache, its attention and its page keeping.

numpy and Python only, in fp64 and whole numbers, written from the format and rules that
include/nm_spmv.h states; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def page_bytes(ps: int, H: int, D: int) -> int:
    return H * 2 * ps * (D // 2 + D // 32)


def quantize(x: np.ndarray):
    """fp64 [..., D] -> codes uint8 [..., D], scale bytes uint8 [..., D/32]: for every value the nearest of
    the fifteen numbers, by looking at all of them; of two equally near ones the even code."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    byte = np.zeros(top.shape, dtype=np.int64)
    nz = top > 0
    m, e = np.frexp(top[nz])  # top = m 2^e, m in [0.5, 1): biased exponent e - 1 + 127, significand 2 m
    byte[nz] = e - 1 + 127 - 2 + (2 * m > 1.75)
    byte = np.clip(byte, 16, 252)
    y = b / np.exp2(byte - 127.0)[..., None]
    d = np.abs(np.abs(y)[..., None] - E2M1)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: argmin takes the first of equals
    code = order[np.argmin(d[..., order], -1)] | (np.signbit(b).astype(np.int64) << 3)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def dequantize(code: np.ndarray, byte: np.ndarray) -> np.ndarray:
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(np.exp2(byte.astype(np.float64) - 127.0), 32, -1)


def places(ps: int, D: int, values: bool):
    """Byte index [ps][D] of every channel and [ps][D/32] of every scale within a head's block."""
    t, c, b = np.arange(ps)[:, None], np.arange(D)[None, :], np.arange(D // 32)[None, :]
    if values:
        at = ps * D // 2 + ((t // 4 * (D // 8) + c // 8) * 4 + t % 4) * 4 + c % 8 // 2
        sc = ps * D + ps * D // 32 + (t // 4 * (D // 32) + b) * 4 + t % 4
    else:
        at = t * (D // 2) + c // 2
        sc = ps * D + ((t // 64 * 16 + t % 16) * (D // 32) + b) * 4 + t % 64 // 16
    return at, sc


def _place(s, i, n, kv_len, table, num_pages, ps):
    pos = int(kv_len[s]) - n + i
    if pos < 0 or pos // ps >= table.shape[1]:
        return None
    page = int(table[s, pos // ps])
    return (page, pos % ps) if 0 <= page < num_pages else None


def append(cache, k, v, table, kv_len, q_start, ps):
    """cache uint8 [N, page_bytes], k and v fp64 [T, H, D]: stores the rows in place."""
    T, H, D = k.shape
    block = page_bytes(ps, 1, D)
    codes = [quantize(k), quantize(v)]
    at = [places(ps, D, False), places(ps, D, True)]
    odd = np.arange(D) % 2
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        for i in range(n):
            t = int(q_start[s]) + i
            where = _place(s, i, n, kv_len, table, len(cache), ps)
            if where is None or t >= T:
                continue
            page, tok = where
            for h in range(H):
                for (code, byte), (pl, sc) in zip(codes, at):
                    c = code[t, h]
                    cache[page, h * block + pl[tok, ::2]] = c[odd == 0] | (c[odd == 1] << 4)
                    cache[page, h * block + sc[tok]] = byte[t, h]


def unpack_pages(cache, ps, H, D):
    """cache uint8 [N, page_bytes] -> K, V fp64 [N, H, ps, D]."""
    x = cache.reshape(len(cache), H, -1)
    out = []
    for values in (False, True):
        at, sc = places(ps, D, values)
        c = x[:, :, at.reshape(-1)].reshape(len(cache), H, ps, D)
        c = np.where(np.arange(D) % 2, c >> 4, c & 15)
        with np.errstate(over="ignore"):
            out.append(dequantize(c, x[:, :, sc.reshape(-1)].reshape(len(cache), H, ps, D // 32)))
    return out


def rows_of(cache, table, kv_len, q_start, ps, H, D, T):
    """What unpack gives: K, V fp64 [T, H, D], zeros where a row has no place, NaN behind the last sequence."""
    K, V = unpack_pages(cache, ps, H, D)
    k, v = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan)
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        for i in range(n):
            t = int(q_start[s]) + i
            if t >= T:
                continue
            where = _place(s, i, n, kv_len, table, len(cache), ps)
            k[t] = v[t] = 0.0
            if where is not None:
                k[t], v[t] = K[where[0], :, where[1]], V[where[0], :, where[1]]
    return k, v


def attention(q, cache, table, kv_len, q_start, ps, n_kv, scale, window):
    """q fp64 [T, Hq, D] -> dict of fp64 arrays over the rows of the sequences (NaN behind them):
    out [T, Hq, D], lse [T, Hq]; absum = sum_j p_j |V_j| [T, Hq, D], and over the seen keys of a row the largest
    scale * sum |q K| (smax) and scale * max |q| * sum |K| (srow), the largest |V|
    (vmax) and their number (keys)."""
    T, Hq, D = q.shape
    K, V = unpack_pages(cache, ps, n_kv, D)
    r = {"out": np.full((T, Hq, D), np.nan), "absum": np.full((T, Hq, D), np.nan)}
    for n in ("lse", "smax", "srow", "vmax", "keys"):
        r[n] = np.full((T, Hq), np.nan)
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        end = int(kv_len[s])
        cols = min(table.shape[1], max(0, -(-end // ps)))
        pages = table[s, :cols].astype(np.int64)
        good = (pages >= 0) & (pages < len(cache))
        pages = np.where(good, pages, 0)
        j = np.arange(cols * ps)
        for h in range(Hq):
            kh = h // (Hq // n_kv)
            Ks = K[pages, kh].reshape(-1, D)
            Vs = V[pages, kh].reshape(-1, D)
            for i in range(n):
                t = int(q_start[s]) + i
                if t >= T:
                    continue
                p = end - n + i
                see = (j <= p) & np.repeat(good, ps)
                if window:
                    see &= j > p - window
                r["keys"][t, h] = see.sum()
                if not see.any():
                    r["out"][t, h] = r["absum"][t, h] = r["smax"][t, h] = r["srow"][t, h] = r["vmax"][t, h] = 0.0
                    r["lse"][t, h] = -np.inf
                    continue
                k, v = Ks[see], Vs[see]
                x = scale * (k @ q[t, h])
                m = x.max()
                w = np.exp(x - m)
                l = w.sum()
                r["out"][t, h] = w @ v / l
                r["absum"][t, h] = w @ np.abs(v) / l
                r["lse"][t, h] = m + np.log(l)
                r["vmax"][t, h] = np.abs(v).max()
                r["smax"][t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
                r["srow"][t, h] = abs(scale) * np.abs(k).sum(-1).max() * np.abs(q[t, h]).max()
    return r


# ---- page keeping, request by request ----

def _pages(n, ps, cols):
    return min(max(0, -(-int(n) // ps)), cols)


def _give_back(table, refs, row, keep, have):
    for c in range(keep, have):
        page = table[row, c]
        if 0 <= page < len(refs):
            refs[page] -= 1
        table[row, c] = -1


def resize(new_len, table, kv_len, refs, ps):
    """In place; -> (moves [S, 2], missing)."""
    S, cols = table.shape
    moves = np.full((S, 2), -1, dtype=np.int32)
    for s in range(S):
        if new_len[s] >= 0:
            _give_back(table, refs, s, _pages(new_len[s], ps, cols), _pages(kv_len[s], ps, cols))
    before = refs.copy()
    free = [p for p in range(len(refs)) if before[p] <= 0]
    asked = 0
    for s in range(S):
        want, old = int(new_len[s]), max(0, int(kv_len[s]))
        if want < 0 or want > cols * ps:
            continue
        if want <= old:
            kv_len[s] = want
            continue
        have, need = _pages(old, ps, cols), _pages(want, ps, cols)
        first, tail = have, -1
        if old % ps and have:
            page = table[s, have - 1]
            if 0 <= page < len(refs) and before[page] > 1:
                first, tail = have - 1, page
        at = asked
        asked += max(0, need - first)
        if asked > len(free) and need > first:
            continue
        for c in range(first, need):
            page = free[at + c - first]
            table[s, c] = page
            refs[page] = 1
        if tail >= 0:
            refs[tail] -= 1
            moves[s] = tail, table[s, first]
        kv_len[s] = want
    return moves, max(0, asked - len(free))


def fork(parent, child, table, kv_len, refs, ps):
    """In place; -> (moves [n, 2], missing)."""
    S, cols = table.shape
    n = len(parent)
    moves = np.full((n, 2), -1, dtype=np.int32)
    children = set(int(c) for c in child)
    ok = []
    for i in range(n):
        p, c = int(parent[i]), int(child[i])
        ok.append(0 <= p < S and 0 <= c < S and p != c and p not in children and c not in [int(x) for x in child[:i]])
    for i in range(n):
        if ok[i]:
            _give_back(table, refs, int(child[i]), 0, _pages(kv_len[child[i]], ps, cols))
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    asked = 0
    for i in range(n):
        if not ok[i]:
            continue
        p, c = int(parent[i]), int(child[i])
        table[c] = -1
        length = int(kv_len[p])
        kv_len[c] = 0
        if length <= 0 or length > cols * ps:
            continue
        full = length // ps
        if length % ps:
            asked += 1
            if asked > len(free):
                continue
            table[c, full] = free[asked - 1]
            refs[free[asked - 1]] = 1
            if 0 <= table[p, full] < len(refs):
                moves[i] = table[p, full], free[asked - 1]
        for col in range(full):
            table[c, col] = table[p, col]
            if 0 <= table[p, col] < len(refs):
                refs[table[p, col]] += 1
        kv_len[c] = length
    return moves, max(0, asked - len(free))


def compact(table, kv_len, refs, ps, max_moves):
    """In place; -> (moves [max_moves, 2], used)."""
    S, cols = table.shape
    used = [p for p in range(len(refs)) if refs[p] > 0]
    U = len(used)
    movers = [p for p in used if p >= U][:max_moves]
    holes = [p for p in range(U) if refs[p] <= 0][:max_moves]
    moves = np.full((max_moves, 2), -1, dtype=np.int32)
    to = dict(zip(movers, holes))
    for s in range(S):
        for c in range(_pages(kv_len[s], ps, cols)):
            table[s, c] = to.get(int(table[s, c]), table[s, c])
    for j, (a, b) in enumerate(zip(movers, holes)):
        moves[j] = a, b
        refs[b], refs[a] = refs[a], 0
    return moves, U
