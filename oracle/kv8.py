"""Plain definitions of the 8-bit key/value cache: rotated tokens in, attention over all keys and over selected blocks, and the choice of
blocks.

numpy and Python only, in fp64 and whole numbers, written from the format and rules that include/nm_spmv.h states;
shares no code with the library.
"""
from __future__ import annotations

import numpy as np

E4M3 = np.array([m / 8 * 2.0**-6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])  # 127 numbers
NAN = 0x7F
LOW, HIGH = 63, 182


def page_bytes(ps: int, H: int, D: int) -> int:
    return -(-H * (ps // 64) * (130 * D + 4) // 128) * 128


def scale_byte(top: float) -> int:
    if top == 0:
        return LOW
    m, e = np.frexp(top)  # top = m 2^e, m in [0.5, 1): biased exponent e - 1 + 127, significand 2 m
    return int(np.clip(e - 1 + 127 - 8 + (2 * m > 1.75), LOW, HIGH))


def encode(x: np.ndarray) -> np.ndarray:
    """fp64 -> the nearest code; of two equally near ones the even one; above 448 that; NaN its own."""
    a = np.minimum(np.abs(x), 448.0)
    up = np.clip(np.searchsorted(E4M3, a), 1, 126)
    low = up - 1
    d_low, d_up = a - E4M3[low], E4M3[up] - a
    code = np.where((d_low < d_up) | ((d_low == d_up) & (low % 2 == 0)), low, up)
    code = np.where(np.isnan(x), NAN, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def decode(code: np.ndarray) -> np.ndarray:
    v = np.append(E4M3, np.nan)[code & 127]
    return np.where(code & 128, -v, v)


def power(byte) -> np.ndarray:
    return np.exp2(np.asarray(byte, dtype=np.float64) - 127)


def places(D: int):
    """Byte index [64][D] of every key and value within the 128 D bytes of a block of one head."""
    t, c = np.arange(64)[:, None], np.arange(D)[None, :]
    return (c // 16 * 64 + t) * 16 + c % 16, 64 * D + ((t // 4 % 4) * D + c) * 16 + t // 16 * 4 + t % 4


def offsets(ps: int, H: int, D: int, h: int, block: int):
    """Byte places in a page of a block's values, bounds and scales."""
    B = ps // 64
    i = h * B + block
    return i * 128 * D, H * B * 128 * D + i * 2 * D, H * B * 130 * D + i * 4


def rotate(x, place, turn, interleaved):
    """x fp64 [heads, D] of one row; turn fp32 [positions, pairs, 2]."""
    if turn is None:
        return x
    P = turn.shape[1]
    c, s = turn[place, :, 0].astype(np.float64), turn[place, :, 1].astype(np.float64)
    a, b = (np.arange(0, 2 * P, 2), np.arange(1, 2 * P, 2)) if interleaved else (np.arange(P), np.arange(P, 2 * P))
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def _page(s, pos, table, num_pages, ps):
    if pos < 0 or pos // ps >= table.shape[1]:
        return None
    page = int(table[s, pos // ps])
    return page if 0 <= page < num_pages else None


def append(cache, k, v, table, kv_len, q_start, ps, turn=None, interleaved=False):
    """cache uint8 [N, page_bytes], k and v fp64 [T, H, D]: stores the rows in place."""
    T, H, D = k.shape
    kat, vat = places(D)
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        begin = int(kv_len[s]) - n
        rows = {begin + i: int(q_start[s]) + i for i in range(n) if int(q_start[s]) + i < T}
        for block in sorted({p // 64 for p in rows}):
            page = _page(s, block * 64, table, len(cache), ps) if block >= 0 else None
            if page is None:
                continue
            new = [p for p in range(block * 64, block * 64 + 64) if p in rows]
            had = new[0] % 64
            tok = np.array([p % 64 for p in new])
            for h in range(H):
                at, bounds, scales = offsets(ps, H, D, h, block % (ps // 64))
                b = cache[page]
                x = np.stack([rotate(k[rows[p]], p, turn, interleaved)[h] for p in new])
                y = np.stack([v[rows[p], h] for p in new])
                x = np.where(np.isfinite(x) & (np.abs(x) < 2.0**128), x, np.nan)
                lost = ~np.isfinite(y).all(-1)
                y = np.where(np.isfinite(y), y, 0.0)
                for i, (z, where) in enumerate(((x, kat), (y, vat))):
                    byte = scale_byte(np.abs(np.nan_to_num(z)).max())
                    if had:
                        was = min(int(b[scales + i]), HIGH)
                        byte = max(byte, was)
                        if byte > was:
                            old = at + where[:had]
                            b[old] = encode(decode(b[old]) * power(was) / power(byte))
                            if i == 0:
                                b[bounds : bounds + 2 * D] = encode(decode(b[bounds : bounds + 2 * D]) * power(was) / power(byte))
                    code = encode(z / power(byte))
                    if i == 0:
                        code[lost, 0] = NAN
                        kept = np.nan_to_num(decode(encode(np.nan_to_num(x) / power(byte))))
                        most, least = kept.max(0), kept.min(0)
                        if had:
                            most = np.maximum(most, decode(b[bounds : bounds + D]))
                            least = np.minimum(least, decode(b[bounds + D : bounds + 2 * D]))
                        b[bounds : bounds + D], b[bounds + D : bounds + 2 * D] = encode(most), encode(least)
                    b[at + where[tok]] = code
                    b[scales + i] = byte
                b[scales + 2 : scales + 4] = 0


def unpack_pages(cache, ps, H, D):
    """cache uint8 [N, page_bytes] -> K, V fp64 [N, H, ps, D] and bounds fp64 [N, H, ps / 64, 2, D]."""
    N, B = len(cache), ps // 64
    kat, vat = places(D)
    x = cache[:, : H * B * 128 * D].reshape(N, H, B, 128 * D)
    bounds = cache[:, H * B * 128 * D : H * B * 130 * D].reshape(N, H, B, 2, D)
    scales = cache[:, H * B * 130 * D : H * B * (130 * D + 4)].reshape(N, H, B, 4)
    with np.errstate(over="ignore", invalid="ignore"):
        K = decode(x[..., kat.reshape(-1)]).reshape(N, H, B, 64, D) * power(scales[..., 0])[..., None, None]
        V = decode(x[..., vat.reshape(-1)]).reshape(N, H, B, 64, D) * power(scales[..., 1])[..., None, None]
        b = decode(bounds) * power(scales[..., 0])[..., None, None]
    return K.reshape(N, H, ps, D), V.reshape(N, H, ps, D), b


def rows_of(cache, table, kv_len, q_start, ps, H, D, T):
    """What unpack gives: K, V fp64 [T, H, D], zeros where a row has no place, NaN behind the last sequence."""
    K, V, _ = unpack_pages(cache, ps, H, D)
    k, v = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan)
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        for i in range(n):
            t, pos = int(q_start[s]) + i, int(kv_len[s]) - n + i
            if t >= T:
                continue
            page = _page(s, pos, table, len(cache), ps)
            k[t] = v[t] = 0.0
            if page is not None:
                k[t], v[t] = K[page, :, pos % ps], V[page, :, pos % ps]
    return k, v


def _sequence(X, table, s, length, ps, N):
    """[cols * ps ...] rows of a sequence and which of them have a page."""
    cols = min(table.shape[1], max(0, -(-int(length) // ps)))
    pages = table[s, :cols].astype(np.int64)
    good = (pages >= 0) & (pages < N)
    return np.where(good, pages, 0), good


def select(q, cache, table, kv_len, q_start, ps, n_kv, top, first, last):
    """q fp64 [T, Hq, D] -> int32 [T, n_kv, top]; -2 in the rows behind the last sequence."""
    T, Hq, D = q.shape
    _, _, bounds = unpack_pages(cache, ps, n_kv, D)
    out = np.full((T, n_kv, top), -2, dtype=np.int32)
    B, group = ps // 64, Hq // n_kv
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        for i in range(n):
            t, p = int(q_start[s]) + i, int(kv_len[s]) - n + i
            if t >= T:
                continue
            blocks = [b for b in range(0, p // 64 + 1) if p >= 0 and _page(s, b * 64, table, len(cache), ps) is not None]
            for h in range(n_kv):
                x = q[t, h * group : (h + 1) * group]
                rank = []
                for b in blocks:
                    most, least = bounds[int(table[s, b // B]), h, b % B]
                    score = sum(np.maximum(x[g] * most, x[g] * least).sum() for g in range(group)) if np.isfinite(x).all() else 0.0
                    forced = b < first or b > p // 64 - last
                    rank.append((not forced, -score if not forced else 0.0, b))
                got = sorted(b for _, _, b in sorted(rank)[:top])
                out[t, h] = got + [-1] * (top - len(got))
    return out


def attention(q, cache, table, kv_len, q_start, ps, n_kv, scale, window=0, selected=None):
    """q fp64 [T, Hq, D] -> dict of fp64 arrays over the rows of the sequences (NaN behind them):
    out [T, Hq, D], lse [T, Hq]; absum = sum_j p_j |V_j| [T, Hq, D], and over the seen keys of a row the largest
    scale * sum |q K| (smax), the largest |V| (vmax) and their number (keys, -1 behind the last sequence)."""
    T, Hq, D = q.shape
    K, V, _ = unpack_pages(cache, ps, n_kv, D)
    r = {"out": np.full((T, Hq, D), np.nan), "absum": np.full((T, Hq, D), np.nan), "keys": np.full((T, Hq), -1.0)}
    for n in ("lse", "smax", "vmax"):
        r[n] = np.full((T, Hq), np.nan)
    group = Hq // n_kv
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        end = int(kv_len[s])
        pages, good = _sequence(K, table, s, end, ps, len(cache))
        j, has = np.arange(len(pages) * ps), np.repeat(good, ps)
        for h in range(Hq):
            Ks, Vs = K[pages, h // group].reshape(-1, D), V[pages, h // group].reshape(-1, D)
            for i in range(n):
                t, p = int(q_start[s]) + i, end - n + i
                if t >= T:
                    continue
                see = np.flatnonzero((j <= p) & has & ((j > p - window) if window else True))
                if selected is not None:
                    named = [see[see // 64 == b] for b in selected[t, h // group] if b >= 0]
                    see = np.concatenate(named) if named else see[:0]
                r["keys"][t, h] = len(see)
                if not len(see):
                    r["out"][t, h] = r["absum"][t, h] = r["smax"][t, h] = r["vmax"][t, h] = 0.0
                    r["lse"][t, h] = -np.inf
                    continue
                k, v = Ks[see], Vs[see]
                with np.errstate(invalid="ignore"):
                    x = scale * (k @ q[t, h])
                    m = x.max()
                    w = np.exp(x - m)
                    l = w.sum()
                    r["out"][t, h] = w @ v / l
                    r["absum"][t, h] = w @ np.abs(v) / l
                    r["lse"][t, h] = m + np.log(l)
                    r["vmax"][t, h] = np.abs(v).max()
                    r["smax"][t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
    return r
