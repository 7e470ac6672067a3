"""Inputs for the tests of the 8-bit key/value cache, and the bounds its results are held to."""
from __future__ import annotations

import numpy as np

from oracle import kv8


def filled_cache(g, N, ps, H, D, low=118, high=128):
    """Random codes that are numbers, scale bytes in [low, high), bounds of what is there."""
    B = ps // 64
    cache = g.integers(0, 256, size=(N, kv8.page_bytes(ps, H, D)), dtype=np.uint8)
    v, b, s = sections(cache, ps, H, D)
    v[(v & 127) == 127] ^= 1
    s[..., :2] = g.integers(low, high, size=s[..., :2].shape, dtype=np.uint8)
    K = kv8.decode(v[..., kv8.places(D)[0].reshape(-1)]).reshape(N, H, B, 64, D)
    b[..., 0, :], b[..., 1, :] = kv8.encode(K.max(-2)), kv8.encode(K.min(-2))
    return cache


def sections(cache, ps, H, D):
    """Views: values [N, H, B, 128 D], bounds [N, H, B, 2, D], scales [N, H, B, 4]."""
    N, B = len(cache), ps // 64
    a, c, e = H * B * 128 * D, H * B * 130 * D, H * B * (130 * D + 4)
    return cache[:, :a].reshape(N, H, B, 128 * D), cache[:, a:c].reshape(N, H, B, 2, D), cache[:, c:e].reshape(N, H, B, 4)


def poison(cache, table, kv_len, ps, H, D):
    """NaN in every place that no sequence holds."""
    held = np.zeros((len(cache), ps), dtype=bool)
    for s in range(len(kv_len)):
        for j in range(int(kv_len[s])):
            page = table[s, j // ps] if j // ps < table.shape[1] else -1
            if 0 <= page < len(cache):
                held[page, j % ps] = True
    v, b, sc = sections(cache, ps, H, D)
    kat, vat = kv8.places(D)
    for p, blk in np.ndindex(len(cache), ps // 64):
        empty = np.flatnonzero(~held[p, 64 * blk : 64 * blk + 64])
        for at in (kat, vat):
            v[p, :, blk, at[empty].reshape(-1)] = 255
        if len(empty) == 64:
            b[p, :, blk], sc[p, :, blk] = 255, 255


def attention_bounds(r):
    """Largest differences of (out, lse) from the fp64 results r that the arithmetic allows.

    Scores: products of bf16 queries and E4M3 keys (8 and 4 bits) are exact; 128 sums, the scale, log2(e) and the difference from
    the largest: 140 steps of at most 2^-23 of sum |q K| (2^-24 where a sum is rounded, twice that where it is cut).
    exp2 itself: 2^-22.  exp(x) is off by the score's difference, for weight and for sum, hence 2 delta.  Weights are rounded
    to bf16 for the products, 2^-8 (half a step, relative); n products and joined parts are summed in fp32, as is the
    sum itself.  The result is rounded once to bf16.  The largest weight of a row is kept between 2^-8 and 1.
    Weights and products below 2^-126 are not normal fp32 numbers and may count as 0: each key then lacks at most 2^-126 (|V| + 1) of
    a sum that is divided by at least 2^-8."""
    keys = np.maximum(r["keys"], 0)
    delta = 140 * 2.0**-23 * r["smax"] + 2.0**-22
    fp32 = 2.0**-23 * (keys + 64)
    lse = delta + fp32 + 2.0**-22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0))
    rel = (2.0**-8 + 2 * delta + 2 * fp32)[..., None]
    out = 2.0**-8 * np.abs(r["out"]) + rel * r["absum"] * (1 + 2.0**-8)
    out = out + 2.0**-118 * (1 + keys * (r["vmax"] + 1))[..., None]
    return out, lse


def turns(g, positions, rotary):
    """Cosines and sines fp32 [positions, rotary / 2, 2]."""
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(rotary // 2) * 2 / rotary)
    return np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
