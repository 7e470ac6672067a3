"""The choice of blocks of the 8-bit cache and attention over chosen blocks, on the GPU against oracle/kv8.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import filled_cache, poison, sections

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.test_gpu_kv8 import attention_case, dev, held_to, run_attention  # noqa: E402


def run_select(q, cache, table, kv_len, q_start, H, ps, top, first, last):
    out = torch.full((len(q), H, top), -2, dtype=torch.int32, device="cuda")
    nm.nm_kv8_select(dev_bf16(bits(q)), dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, top, first=first, last=last, out=out)
    return out.cpu().numpy()


def select_case(seed, rows, lens, Hq, H, D, ps, top, first, last, change=None, extra=0):
    g = np.random.default_rng(seed)
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]) + extra, Hq, D)))
    if change:
        change(g, cache, table, q)
    want = kv8.select(q, cache, table, kv_len, q_start, ps, H, top, first, last)
    got = run_select(q, cache, table, kv_len, q_start, H, ps, top, first, last)
    off = np.argwhere((got != want).any(-1))
    assert not len(off), f"{len(off)} rows, the first {off[0]}: {got[tuple(off[0])]}, not {want[tuple(off[0])]}"
    return got


@pytest.mark.parametrize("top,first,last", [(1, 0, 0), (1, 0, 1), (4, 1, 1), (5, 0, 2), (8, 2, 0), (100, 3, 4)])
@pytest.mark.parametrize("Hq,H,D,ps", [(4, 2, 128, 64), (3, 3, 64, 128), (20, 1, 128, 512)])
def test_choice(Hq, H, D, ps, top, first, last):
    say("choice", Hq, H, D, ps, top, first, last)
    lens = [1, 63, 64, 65, 300, 1000, 2500, 0]
    select_case(top * D, [1] * len(lens), lens, Hq, H, D, ps, top, first, last, extra=2)
    select_case(top * D, [5, 9, 0, 2], [2, 700, 10, 130], Hq, H, D, ps, top, first, last)


def test_long_rows_and_many_rows():
    say("long")
    select_case(1, [1, 1], [40000, 70001], 8, 2, 64, 512, 40, 1, 2)
    select_case(2, [1], [300000], 2, 1, 64, 512, 300, 1, 2)  # a table of more than 4096 blocks
    select_case(3, [400, 300], [900, 1800], 4, 1, 64, 256, 6, 1, 1)  # more rows than workgroups of sixteen waves are for


def test_sixteen_rows_a_workgroup_at_the_largest_table():
    """A table of 1024 blocks, as many as such rows' scores have room for."""
    say("1024 blocks")
    for D in (64, 128):
        select_case(4, [21], [65000], 2, 1, D, 512, 30, 1, 1)
        select_case(5, [9, 7, 3], [40000, 500, 64], 2, 1, D, 512, 300, 2, 2)


def test_scores_that_are_alike():
    """Blocks with the same bytes, in groups larger and smaller than what one wave ranks: the lowest of them."""
    say("alike")

    def copies(count):
        def change(g, cache, table, q):
            v, b, s = sections(cache, 64, 2, 64)
            pages = table[0, table[0] >= 0]
            for i, p in enumerate(pages):
                b[p], s[p] = b[pages[i % count]], s[pages[i % count]]
        return change

    for count in (1, 2, 3, 7, 50):
        for top in (1, 9, 40, 150):
            select_case(count + top, [1], [13000], 4, 2, 64, 64, top, 0, 1, change=copies(count))


def test_scores_that_differ_in_the_last_bits():
    """Two runs of bounds whose scores are 2^-40 of each other apart: fp32 sums could not tell them."""
    say("close")

    def change(g, cache, table, q):
        v, b, s = sections(cache, 64, 1, 64)
        pages = table[0, table[0] >= 0]
        b[:], s[:] = 0, 127
        q[:] = 0
        q[:, :, 0], q[:, :, 1] = 2.0**20, 2.0**-20
        b[pages, 0, 0, :, 0] = kv8.encode(np.array(448.0))
        b[pages, 0, 0, :, 1] = kv8.encode(g.integers(-8, 9, size=len(pages)) / 8.0)[:, None]
    got = select_case(3, [1], [6000], 2, 1, 64, 64, 20, 0, 0, change=change)
    assert len(set(got[0, 0])) == 20


def test_all_signs_and_zeros():
    say("signs")

    def change(g, cache, table, q):
        v, b, s = sections(cache, 64, 2, 128)
        s[..., 0] = g.integers(63, 183, size=s[..., 0].shape)
        b[:, :, :, :, ::2] &= 128  # zeros of both signs
        q[:, 0] = 0.0
    select_case(4, [1, 3], [3000, 2000], 4, 2, 128, 64, 12, 0, 0, change=change)


def test_queries_that_are_not_finite_take_the_lowest():
    say("not finite")

    def change(g, cache, table, q):
        q[0, 0, 3], q[1, 3, 100], q[2, 1, 0] = np.inf, np.nan, -np.inf
    got = select_case(5, [4], [3000], 4, 2, 128, 64, 6, 1, 2, change=change)
    assert (got[0, 0] == [0, 1, 2, 3, 45, 46]).all() and (got[1, 1] == got[0, 0]).all()


def test_blocks_without_a_page_are_not_taken():
    say("no page")

    def change(g, cache, table, q):
        table[0, [0, 5, 9]] = -1, len(cache), 2**31 - 1
    got = select_case(6, [2], [1000], 2, 1, 64, 64, 14, 2, 1, change=change)
    assert not np.isin([0, 5, 9], got).any() and (got[1, 0] == -1).sum() == 14 - 13


# ---- attention over chosen blocks ----

def drawn(top, high):
    return lambda g, T, H: g.integers(-1, high, size=(T, H, top)).astype(np.int32)


@pytest.mark.parametrize("top", [1, 3, 8, 9, 70, 200])
@pytest.mark.parametrize("Hq,H,D,ps", [(8, 2, 128, 64), (3, 3, 64, 128), (40, 2, 64, 256)])
def test_named_blocks(Hq, H, D, ps, top):
    """Any order, named twice (counted twice), behind the row's own block, none."""
    say("named", Hq, H, D, ps, top)
    attention_case(top + D, [1, 1, 1, 1], [1, 130, 700, 2000], Hq, H, D, ps, pick=drawn(top, 40))
    attention_case(top + D, [3, 1, 5, 0], [3, 64, 500, 9], Hq, H, D, ps, pick=drawn(top, 9), extra=1)


@pytest.mark.parametrize("window", [1, 64, 100, 333])
def test_named_blocks_and_a_window(window):
    say("named, window", window)
    attention_case(window, [1, 4], [500, 400], 8, 2, 128, 64, window=window, pick=drawn(12, 8))


def test_names_far_out_of_range():
    say("far names")

    def pick(g, T, H):
        s = np.full((T, H, 6), -1, dtype=np.int32)
        s[:, :, 1], s[:, :, 2], s[:, :, 3], s[:, :, 4] = 2**31 - 1, -(2**31), 2**26, 1
        return s
    attention_case(1, [1, 3, 1], [200, 140, 3], 4, 2, 128, 64, pick=pick)


def test_many_rows_with_named_blocks():
    say("many rows, named")
    attention_case(7, [150, 120], [700, 120], 4, 2, 64, 64, pick=drawn(5, 11))


def test_all_blocks_named_are_all_keys():
    say("all named")
    g = np.random.default_rng(3)
    H, D, ps, rows, lens = 2, 128, 64, [1, 4], [1000, 700]
    q, cache, table, kv_len, q_start, out, lse = attention_case(3, rows, lens, 8, H, D, ps)
    sel = run_select(q, cache, table, kv_len, q_start, H, ps, 20, 1, 1)
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, 4, selected=sel), r, "all named")


@pytest.mark.parametrize("seqs", [1, 3, 40])
def test_choice_and_attention_together(seqs):
    """As a decode step uses them; the chosen blocks hold more of the weight than any others."""
    say("together", seqs)
    g = np.random.default_rng(seqs)
    H, D, ps, top = 2, 128, 64, 12
    lens = [3000] + [int(n) for n in g.integers(1, 3000, seqs - 1)]
    table, kv_len, q_start, N = batch(g, [1] * seqs, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((seqs, 8, D)))
    sel = run_select(q, cache, table, kv_len, q_start, H, ps, top, 1, 2)
    assert (sel == kv8.select(q, cache, table, kv_len, q_start, ps, H, top, 1, 2)).all()
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0, sel)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, 1, selected=sel), r, f"{seqs} sequences")


@pytest.mark.parametrize("rows,lens", [([1, 1], [900, 40000]), ([21], [30000]), ([1], [200000]), ([600], [140000])])
def test_pages_that_were_never_written(rows, lens):
    """Any bytes as bounds and scales, NaN among them: blocks that the row has, each once, none without a page."""
    say("never written", rows, lens)
    g = np.random.default_rng(77)
    ps, H, D, Hq = 512, 1, 64, 2
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = g.integers(0, 256, size=(N, kv8.page_bytes(ps, H, D)), dtype=np.uint8)
    b, s = sections(cache, ps, H, D)[1:]
    b[::3] = 127
    s[1::4] = 255
    bad = g.random(table.shape) < 0.2
    table[bad] = np.where(g.random(table.shape) < 0.5, -1, N)[bad]
    q = bf16(g.standard_normal((int(q_start[-1]), Hq, D)))
    for top in (2, 7, 90):
        got = run_select(q, cache, table, kv_len, q_start, H, ps, top, 1, 1)
        for i, n in enumerate(rows):
            for t in range(q_start[i], q_start[i + 1]):
                own = (kv_len[i] - q_start[i + 1] + t) // 64
                x = got[t, 0]
                x = x[x != -1]
                assert (got[t, 0, : len(x)] == x).all() and (np.diff(x) > 0).all()
                assert (x >= 0).all() and (x <= own).all()
                pages = table[i, x * 64 // ps]
                assert ((pages >= 0) & (pages < N)).all()


@pytest.mark.parametrize("kind", ["plain", "alike", "not finite", "pages", "loud"])
@pytest.mark.parametrize("rows,lens,Hq,H,D,ps,top,first,last", [
    ([129], [5000], 32, 16, 128, 64, 9, 1, 1), ([260], [64000], 8, 8, 64, 512, 40, 0, 2), ([130, 3], [700, 9000], 16, 16, 128, 512, 100, 2, 3),
    ([40, 17, 0, 31, 9], [40, 900, 64, 31, 300], 32, 32, 64, 128, 3, 0, 0)])
def test_sixteen_rows_a_workgroup(rows, lens, Hq, H, D, ps, top, first, last, kind):
    """More than 2048 choices, of sequences of 16 rows and more on average."""
    say("sixteen rows", rows, lens, Hq, H, D, ps, top, kind)
    assert sum(rows) * H > 2048 and sum(rows) >= 16 * len(rows)

    def change(g, cache, table, q):
        _, b, s = sections(cache, ps, H, D)
        if kind == "alike":
            b[:], s[:] = b[:1, :, :1], 120
        if kind == "not finite":
            q[3, 0, 1], q[7, -1, 5], q[20] = np.inf, np.nan, 0
        if kind == "pages":
            bad = g.random(table.shape) < 0.3
            table[bad] = np.where(g.random(table.shape) < 0.5, -1, len(cache))[bad]
        if kind == "loud":
            s[g.random(s.shape) < 0.2] = 182  # among quiet ones: first scores decide about few blocks
    select_case(len(rows) * D, rows, lens, Hq, H, D, ps, top, first, last, change=change, extra=1)


def test_sixteen_rows_a_workgroup_behind_a_wide_table():
    """A table of 1024 blocks, the most that such rows' scores have room for, at the larger dimension."""
    say("sixteen rows, wide")
    g = np.random.default_rng(9)
    ps, Hq, H, D, rows, lens = 512, 16, 8, 128, [300], [20000]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    wide = np.full((1, 1024 * 64 // ps), -1, dtype=np.int32)
    wide[:, : table.shape[1]] = table
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((rows[0], Hq, D)))
    want = kv8.select(q, cache, wide, kv_len, q_start, ps, H, 20, 1, 1)
    assert (run_select(q, cache, wide, kv_len, q_start, H, ps, 20, 1, 1) == want).all()
