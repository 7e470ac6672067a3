"""The 8-bit cache where tables are wide or the cache is large: each form of the choice behind more blocks than one wave holds, and pages behind
4 GiB.  Against oracle/kv8.py."""
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
from tests.test_gpu_kv8 import dev, held_to, run_attention  # noqa: E402
from tests.test_gpu_kv8_select import run_select  # noqa: E402


def changed(kind, g, cache, table, q, ps, H, D):
    _, b, s = sections(cache, ps, H, D)
    if kind == "alike":
        b[:], s[:] = b[:1, :, :1], 120
    if kind == "alike by fifty":
        pages = table[0, table[0] >= 0]
        for i, p in enumerate(pages):
            b[p], s[p] = b[pages[i % 50]], s[pages[i % 50]]
    if kind == "not finite":
        q[0, 0, 1], q[-1, -1, 5] = np.inf, np.nan
    if kind == "pages":
        bad = g.random(table.shape) < 0.3
        table[bad] = np.where(g.random(table.shape) < 0.5, -1, len(cache))[bad]
    if kind == "loud":
        s[g.random(s.shape) < 0.2] = 182  # among quiet ones: first scores decide about few blocks


# short: single tokens of so many short sequences beside the long ones, which make the workgroups small; blocks: of the table
FORMS = [
    ("sixteen waves a row, 4096 blocks", [1, 2], [100000, 66000], 0, 1600),
    ("four waves a row, 4096 blocks", [1, 1], [100000, 67000], 520, 3000),
    ("four waves a row, 16384 blocks", [1, 1], [80000, 270000], 520, 5000),
    ("four waves a row, the widest table", [2], [90000], 520, 16384),
    ("two launches", [1, 3], [140000, 66000], 0, 2400),
    ("two launches, the widest table", [1], [270000], 3, 16384),
]


@pytest.mark.parametrize("kind", ["plain", "alike", "alike by fifty", "not finite", "pages", "loud"])
@pytest.mark.parametrize("name,rows,lens,short,blocks", FORMS)
def test_choice_among_more_blocks_than_one_wave_holds(name, rows, lens, short, blocks, kind):
    say("wide", name, kind)
    g = np.random.default_rng(blocks)
    ps, H, Hq, D = 512, 1, 2, 64
    rows, lens = rows + [1] * short, lens + [int(n) for n in g.integers(1, 400, short)]
    table, kv_len, q_start, N = batch(g, rows, lens, ps, extra_cols=0)
    assert table.shape[1] * ps // 64 <= blocks
    table = np.pad(table, ((0, 0), (0, blocks * 64 // ps - table.shape[1])), constant_values=-1)
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]) + 1, Hq, D)))
    changed(kind, g, cache, table, q, ps, H, D)
    for top, first, last in ((30, 1, 2), (700, 0, 1)):
        want = kv8.select(q, cache, table, kv_len, q_start, ps, H, top, first, last)
        got = run_select(q, cache, table, kv_len, q_start, H, ps, top, first, last)
        off = np.argwhere((got != want).any(-1))
        assert not len(off), f"{len(off)} rows, the first {off[0]}: {got[tuple(off[0])]}, not {want[tuple(off[0])]}"


@pytest.mark.parametrize("D", [64, 128])
def test_a_short_row_of_a_wide_table(D):
    """A table for a long context, a few tokens so far: the choice and attention are those of a narrow one."""
    say("short row, wide table", D)
    g = np.random.default_rng(D)
    ps, H, Hq, rows, lens = 128, 2, 8, [1, 3, 1], [500, 700, 1]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]), Hq, D)))
    want = kv8.select(q, cache, table, kv_len, q_start, ps, H, 4, 1, 1)
    r, rs = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5), kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0, want)
    for blocks in (40, 700, 3000, 16384):
        wide = np.pad(table, ((0, 0), (0, blocks * 64 // ps - table.shape[1])), constant_values=-1)
        assert (run_select(q, cache, wide, kv_len, q_start, H, ps, 4, 1, 1) == want).all()
        held_to(*run_attention(q, cache, wide, kv_len, q_start, H, ps, 3), r, f"{blocks} blocks")
        held_to(*run_attention(q, cache, wide, kv_len, q_start, H, ps, 3, selected=want), rs, f"{blocks} blocks, chosen")


def test_unpack_and_chosen_blocks_behind_four_gibibytes():
    say("large cache")
    g = np.random.default_rng(6)
    ps, H, Hq, D = 64, 2, 8, 128
    N = (1 << 32) // kv8.page_bytes(ps, H, D) + 40
    rows, lens = [2, 150, 1], [300, 200, 700]
    table, kv_len, q_start, n = batch(g, rows, lens, ps)
    high = np.where(table >= 0, table + N - n, -1).astype(np.int32)
    small = filled_cache(g, n, ps, H, D)
    cache = torch.zeros((N, small.shape[1]), dtype=torch.uint8, device="cuda")
    cache[N - n :] = dev(small)
    T = int(q_start[-1])
    args = dev(high), dev(kv_len), dev(q_start)
    ko, vo = (torch.full((T + 1, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv8_unpack(cache, *args, ps, ko, vo)
    for got, want in zip((ko, vo), kv8.rows_of(small, table, kv_len, q_start, ps, H, D, T)):
        got = bf16_as_f64(host_bf16(got))
        assert (got[:T] == want).all() and (got[T] == 5).all()
    q = bf16(g.standard_normal((T, Hq, D)))
    sel = kv8.select(q, small, table, kv_len, q_start, ps, H, 3, 1, 1)
    out, lse = nm.nm_kv8_attention(dev_bf16(bits(q)), cache, *args, H, ps, 150, selected=dev(sel))
    r = kv8.attention(q, small, table, kv_len, q_start, ps, H, D**-0.5, 0, sel)
    held_to(bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64), r, "large cache, chosen")
