"""Attention over the 4-bit cache at the ends of what numbers hold: the largest and smallest keys and values that
nm_kv4_append stores, scores of any size below 2^125, scales of any size.  Calls of few rows (row tiles) and the kernel
that takes prompts."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

from tests.kv4_util import attention_bounds, batch, bf16, filled_cache  # noqa: E402
from tests.test_gpu_kv4 import held_to, run_attention  # noqa: E402
from tests.test_gpu_kv4_prompts import extra  # noqa: E402

HUGE = 6 * 2.0**125
WAYS = [1, 5, 80]  # rows: the last one goes to the kernel for prompts, with rows behind the last sequence


def queries(x, rows):
    """Rows x [rows, Hq, D], and for prompts as many zeros behind them as make the call a large one."""
    Hq, D = x.shape[1:]
    return np.concatenate([x, np.zeros((extra(Hq) if rows > 64 else 0, Hq, D))])


def scale_bytes(cache, H, ps, D, values):
    x = cache.reshape(len(cache), H, -1)
    at = ps * D + (ps * D // 32 if values else 0)
    return x[:, :, at : at + ps * D // 32]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("n", [81, 700, 5000])
@pytest.mark.parametrize("equal", [False, True])
def test_values_near_the_largest_number(D, rows, n, equal):
    """Values of one sign up to 6 * 2^125: their weighted mean is a number whatever their count.  With queries of 0
    the weights are all alike."""
    say("largest values", D, rows, n, equal)
    g = np.random.default_rng(n + rows)
    H, Hq, ps = 1, 4, 64
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D, 118, 126)
    cache.reshape(N, H, -1)[:, :, ps * D // 2 : ps * D] &= 0x77
    scale_bytes(cache, H, ps, D, True)[:] = g.integers(250, 253, size=(N, H, ps * D // 32), dtype=np.uint8)
    q = queries(np.zeros((rows, Hq, D)) if equal else bf16(g.standard_normal((rows, Hq, D))), rows)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, f"D{D} rows {rows} n {n}")


@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("n", [81, 3000])
def test_values_near_the_smallest_number(rows, n):
    """Values of 2^-112 to 6 * 2^-111 among thousands of others, multiplied as 2^-12 of what they are: weights times values
    are not normal numbers.  An fp32 sum of what is below 2^-126 is kept in steps of 2^-149: n products are off by half a
    step each, n * 2^-150, times 2^12 and over weights that sum to at least 2^-8 that is n * 2^-130."""
    say("smallest values", rows, n)
    g = np.random.default_rng(n)
    H, Hq, D, ps = 1, 4, 128, 64
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D, 118, 126)
    scale_bytes(cache, H, ps, D, True)[:] = 16
    q = queries(bf16(g.standard_normal((rows, Hq, D))), rows)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows)
    held_to(out, lse, r, "smallest values")
    ro, ra = r["out"][:rows], r["absum"][:rows]
    delta = 2.0**-20 * r["srow"] + 140 * 2.0**-24 * r["smax"] + 2.0**-22
    rel = (2.0**-8 + 2 * delta + 2.0**-23 * (n + 64))[:rows, :, None]
    assert (np.abs(out[:rows] - ro) <= 2.0**-8 * np.abs(ro) + 1.01 * rel * ra + n * 2.0**-129).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("n", [200, 3000])
def test_keys_that_hold_the_largest_number(D, rows, n):
    """Two keys with a channel of 6 * 2^125 (an infinity, as nm_kv4_append keeps it).  Where the query's channel has
    their sign, the two take all the weight, half each; where it has the other, they take none."""
    say("largest keys", D, rows, n)
    g = np.random.default_rng(n + D)
    H, Hq, ps, ch, two = 1, 4, 64, 37, [3, 60]
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    k, v = (bf16(g.standard_normal((n, H, D))) for _ in range(2))
    k[two] = 0.0
    k[two, 0, ch] = HUGE
    every = np.array([0, n], np.int32)
    cache = np.zeros((N, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    kv4.append(cache, k, v, table, kv_len, every, ps)
    others = np.zeros_like(cache)  # the sequence without the two
    fewer = kv_len - 2
    kv4.append(others, np.delete(k, two, 0), np.delete(v, two, 0), table, fewer, every - [0, 2], ps)
    q = bf16(g.standard_normal((rows, Hq, D)))
    q[:, :, ch] = 1.5 * np.array([1, -1, 1, -1])
    q = queries(q, rows)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows)
    out, lse = out[:rows], lse[:rows]
    r = {a: b[:rows] for a, b in kv4.attention(q, others, table, fewer, q_start, ps, H, D**-0.5, 0).items()}
    bo, bl = attention_bounds(r)
    neg = [1, 3]
    assert (np.abs(out - r["out"])[:, neg] <= bo[:, neg]).all() and (np.abs(lse - r["lse"])[:, neg] <= bl[:, neg]).all()
    _, vs = kv4.rows_of(cache, table, kv_len, every, ps, H, D, n)
    mean, top = vs[two, 0].mean(0), D**-0.5 * 1.5 * HUGE
    # equal scores: equal weights, a power of two each; half the sum of two E2M1 numbers is rounded once
    assert (np.abs(out[:, [0, 2]] - mean) <= 2.0**-8 * np.abs(mean)).all()
    assert (np.abs(lse[:, [0, 2]] / top - 1) <= 2.0**-21).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("up", [10, 20, 31, 60, 110])
@pytest.mark.parametrize("order", ["any", "rising", "falling"])
def test_large_scores(D, rows, up, order):
    """Scores that are whole multiples of 2^(up - 1), exact in fp32 and up to 2^13 times that: keys of the
    largest one share the weight, all others have at most exp(-2^9) < 2^-738 of it, which is 0 in fp32.  lse: that score; c, two products and a sum round, and so does
    the factor back to natural logarithms (6 steps of 2^-24)."""
    say("large scores", D, rows, up, order)
    g = np.random.default_rng(up + rows)
    H, Hq, ps, n = 1, 4, 64, 700
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    k, v = kv4.E2M1[g.integers(0, 8, size=(n, H, D))] * g.choice([-1, 1], size=(n, H, D)), bf16(g.standard_normal((n, H, D)))
    k[:, 0, ::32] = 6.0  # the scale is 1
    q = g.integers(-3, 4, size=(rows, Hq, D)).astype(np.float64)
    if order != "any":  # by the scores of the first row and head
        by = np.argsort(k[:, 0] @ q[0, 0], kind="stable")
        k = k[by if order == "rising" else by[::-1]]
    q *= 2.0**up
    cache = np.zeros((N, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    kv4.append(cache, k, v, table, kv_len, np.array([0, n], np.int32), ps)
    q = queries(q, rows)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows, scale=1.0)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, 1.0, 0)
    out, lse, ro, ra, rl = out[:rows], lse[:rows], r["out"][:rows], r["absum"][:rows], r["lse"][:rows]
    assert np.isfinite(out).all()
    assert (np.abs(out - ro) <= 2.0**-8 * np.abs(ro) + 2.0**-8 * ra + 2.0**-700).all()
    assert (np.abs(lse - rl) <= 2.0**-21 * np.abs(rl) + 2.0**-20 * 16).all()


@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("scale,up_q,up_k", [(2.0**-100, 55, 45), (2.0**-125, 70, 55), (1e-40, 68, 64), (2.0**-149, 100, 49),
                                             (-(2.0**-60), 100, -40), (2.0**60, -30, -30), (2.0**100, -60, -40),
                                             (0.0, 100, 100), (0.0, 0, 0), (1e-30, 0, 0)])
def test_scales_of_any_size(rows, scale, up_q, up_k):
    """Products of queries and keys that pass the range of fp32 by themselves, and scores of ordinary size."""
    say("scale", rows, scale)
    g = np.random.default_rng(rows)
    H, Hq, D, ps, n = 1, 4, 128, 64, 300
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D, 126 + up_k, 128 + up_k)
    scale_bytes(cache, H, ps, D, True)[:] = g.integers(120, 128, size=(N, H, ps * D // 32), dtype=np.uint8)
    q = queries(bf16(np.ldexp(g.standard_normal((rows, Hq, D)), up_q)), rows)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, float(np.float32(scale)), 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows, scale=scale), r, f"scale {scale}")


@pytest.mark.parametrize("rows", WAYS)
@pytest.mark.parametrize("scale", [0.0, 2.0**-140, -(2.0**-100), 2.0**60])
def test_a_query_that_is_not_finite_at_any_scale(rows, scale):
    """NaN in its own row and head, also where the scale leaves nothing of the others."""
    say("not finite", rows, scale)
    g = np.random.default_rng(rows)
    H, Hq, D, ps, n = 1, 4, 64, 64, 300
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D)
    q = queries(bf16(g.standard_normal((rows, Hq, D))), rows)
    q[0, 1, 5], q[rows - 1, 2, 40], q[rows // 2, 0, 63] = np.inf, np.nan, -np.inf
    spoilt = ~np.isfinite(q[:rows]).all(-1)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows, scale=scale)
    out, lse = out[:rows], lse[:rows]
    assert np.isnan(out[spoilt]).all() and np.isnan(lse[spoilt]).all()
    assert np.isfinite(out[~spoilt]).all() and np.isfinite(lse[~spoilt]).all()
