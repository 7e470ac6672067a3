"""Inputs for the tests of the 4-bit key/value cache, and the bounds its results are held to."""
from __future__ import annotations

import numpy as np

import synth
from oracle import kv4


def bf16(a) -> np.ndarray:
    """Rounded to bf16, as fp64."""
    return synth.bf16_bits_to_f32(synth.to_bf16_bits(np.asarray(a, dtype=np.float32))).astype(np.float64)


def bits(a) -> np.ndarray:
    return synth.to_bf16_bits(np.asarray(a, dtype=np.float32))


def batch(g, rows, lens, ps, extra_cols=1, spare=3):
    """(table int32 [S, cols], kv_len, q_start, num_pages): pages in random order, -1 behind the last ones."""
    counts = [max(0, -(-n // ps)) for n in lens]
    cols = max(counts + [1]) + extra_cols
    N = sum(counts) + spare
    order = g.permutation(N)
    table = np.full((len(lens), cols), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at : at + n]
        at += n
    return table, np.array(lens, dtype=np.int32), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32), N


def filled_cache(g, N, ps, H, D, low=118, high=132, junk=None):
    """Random codes; scale bytes in [low, high), so magnitudes reach 6 * 2^(high - 128)."""
    cache = g.integers(0, 256, size=(N, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    x = cache.reshape(N, H, -1)
    x[:, :, ps * D :] = g.integers(low, high, size=x[:, :, ps * D :].shape, dtype=np.uint8)
    return cache


def poison(cache, table, kv_len, ps, H, D):
    """0xFF (scales that are no number) in every place that no sequence holds."""
    held = np.zeros((len(cache), ps), dtype=bool)
    for s in range(len(kv_len)):
        for j in range(int(kv_len[s])):
            page = table[s, j // ps] if j // ps < table.shape[1] else -1
            if 0 <= page < len(cache):
                held[page, j % ps] = True
    x = cache.reshape(len(cache), H, -1)
    for values in (False, True):
        at, sc = kv4.places(ps, D, values)
        for p, t in zip(*np.nonzero(~held)):
            x[p][:, at[t]] = 255
            x[p][:, sc[t]] = 255


def attention_bounds(r):
    """Largest differences of (out, lse) from the fp64 results r that the arithmetic allows.

    Scores: 32 channels of a query are held as four 6-bit pieces, at most 2^-20 of their largest magnitude off
    (four_pieces goes through every number they can hold); the products
    are exact and their 128 sums, the scale and log2(e) round in fp32: 136 steps of 2^-24 of sum |q K|; the
    exponent's argument and exp2 itself: 4 steps of the largest score.  exp(x) is off by the score's
    difference, for weight and for sum, hence 2 delta.  Weights are rounded to bf16 for the products, 2^-8 (half
    a step, relative); n products and joined parts are summed in fp32, as is the sum itself.  The result is
    rounded once to bf16.  The largest weight of a row is kept between 2^-8 and 1.  Weights and products below
    2^-126 are not normal fp32 numbers and may count as 0: each key then lacks at most 2^-126 (|V| + 1) of a sum
    that is divided by at least 2^-8."""
    keys = r["keys"]
    delta = 2.0**-20 * r["srow"] + 140 * 2.0**-24 * r["smax"] + 2.0**-22
    fp32 = 2.0**-24 * (keys + 64)
    lse = delta + fp32 + 2.0**-22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0))
    rel = (2.0**-8 + 2 * delta + 2 * fp32)[..., None]
    out = 2.0**-8 * np.abs(r["out"]) + rel * r["absum"] * (1 + 2.0**-8)
    out = out + 2.0**-118 * (1 + keys * (r["vmax"] + 1))[..., None]
    return out, lse


E2M3 = np.array([m / 8 for m in range(8)] + [(1 + m / 8) * 2.0**e for e in range(3) for m in range(8)])


def four_pieces(q):
    """What four E2M3 pieces with scales of 2^-2, 2^-6, 2^-11 and 2^-16 leave of numbers of a block whose
    largest magnitude is in [1, 2): rounding to nearest, a tie to the even code, 7.5 the largest."""
    rest = np.asarray(q, dtype=np.float64)
    order = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    for s in (2, 6, 11, 16):
        a = np.abs(rest) * 2.0**s
        near = E2M3[order[np.argmin(np.abs(a[..., None] - E2M3[order]), -1)]]
        rest = rest - np.sign(rest) * near * 2.0**-s
    return rest
