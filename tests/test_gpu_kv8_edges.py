"""Attention over the 8-bit cache where a row tile or a prompt meets blocks that hold nothing for it: pages that were never written or are
not there, sequences without tokens, windows, lengths behind the table.  Against oracle/kv8.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import say
from tests.kv4_util import batch, bf16
from tests.kv8_util import filled_cache, poison, sections

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

from tests.test_gpu_kv8 import held_to, run_attention  # noqa: E402


def without_page_zero(g, rows, lens, ps, H, D, **kw):
    """A batch that does not own page 0, whose bytes are all 255: codes and scales that are no numbers."""
    table, kv_len, q_start, N = batch(g, rows, lens, ps, **kw)
    table[table >= 0] += 1
    cache = filled_cache(g, N + 1, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    cache[0] = 255
    return table, kv_len, q_start, cache


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("room", [64, 64 * 80])
def test_no_tokens_behind_a_page_that_was_never_written(rows, room, D):
    """A slot whose pages were handed out, with rows but no tokens yet: zeros, whatever the pages hold."""
    say("no tokens", rows, room, D)
    g = np.random.default_rng(rows)
    H, Hq, ps = 2, 8, 64
    table = np.full((3, room // ps), -1, dtype=np.int32)
    table[0, 0], table[1, 0], table[2, 0] = 0, 1, 0
    kv_len, q_start = np.array([0, 40, 0], dtype=np.int32), np.array([0, rows, 2 * rows, 3 * rows], dtype=np.int32)
    cache = filled_cache(g, 2, ps, H, D)
    cache[0] = 255
    q = bf16(g.standard_normal((3 * rows, Hq, D)))
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "no tokens")
    sel = np.zeros((3 * rows, H, 2), dtype=np.int32)
    sel[:, :, 1] = -1
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows, selected=sel), r, "no tokens, named")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [3, 12])
def test_named_blocks_before_the_window_hold_anything(top, D):
    """Their pages may be another sequence's by now, or were never written."""
    say("before the window", top, D)
    g = np.random.default_rng(top)
    H, Hq, ps, window = 2, 8, 64, 100
    table, kv_len, q_start, cache = without_page_zero(g, [1, 4, 1], [700, 500, 90], ps, H, D)
    table[0, :9], table[1, :6] = 0, 0  # the windows begin at 600 and 397
    q = bf16(g.standard_normal((6, Hq, D)))
    sel = np.sort(g.integers(0, 11, size=(6, H, top)).astype(np.int32), -1)
    sel[:, :, 0] = 0
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, window, sel)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, 4, window=window, selected=sel), r, "named")


def prompt_rows(g, rows, kv_len, table, cache, q_start, Hq, H, D, ps, window, drawn=5):
    """A call of rows enough for workgroups of 128 of them (64 rows times heads for each compute unit); checked at each sequence's
    ends, at its first and last place and at drawn rows."""
    T = int(q_start[-1]) + 1
    assert T * Hq > 64 * torch.cuda.get_device_properties(0).multi_processor_count
    q = bf16(g.standard_normal((T, Hq, D)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, max(rows), window=window)
    assert (out[-1] == 77).all() and (lse[-1] == 77).all()
    room = table.shape[1] * ps
    for s, n in enumerate(rows):
        first = int(kv_len[s]) - n
        at = {0, n // 2, n - 1, -first - 1, -first, room - first - 1, room - first, room - first + window, *map(int, g.integers(0, max(n, 1), drawn))}
        for i in sorted(i for i in at if 0 <= i < n):
            t = int(q_start[s]) + i
            one = np.array([first + i + 1], dtype=np.int32)
            r = kv8.attention(q[t : t + 1], cache, table[s : s + 1], one, np.array([0, 1]), ps, H, D**-0.5, window)
            held_to(out[t : t + 1], lse[t : t + 1], r, f"sequence {s} row {i}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("ps", [64, 256])
def test_pages_of_a_prompt_that_are_not_there(ps, window, D):
    say("prompt, bad pages", ps, window, D)
    g = np.random.default_rng(ps + window)
    rows, H, Hq = [700, 500, 1], 1, 32
    table, kv_len, q_start, cache = without_page_zero(g, rows, [1300, 900, 400], ps, H, D)
    table[0, 2], table[0, 3], table[1, 0], table[0, table.shape[1] - 2], table[2, 0] = -1, len(cache), 2**31 - 1, -5, -(2**31)
    prompt_rows(g, rows, kv_len, table, cache, q_start, Hq, H, D, ps, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 63, 64, 700])
@pytest.mark.parametrize("rows,lens,longer", [([1100], [1200], 300), ([1100, 5], [700, 3], 0), ([600, 500, 2], [1000, 900, 70], 600)])
def test_prompts_at_the_ends_of_table_and_sequence(rows, lens, longer, window, D):
    """Lengths behind the table's last column (`longer` tokens), more rows than places, windows shorter than a block."""
    say("prompt, ends", rows, lens, longer, window, D)
    g = np.random.default_rng(len(rows) + window)
    H, Hq, ps = 2, 64, 64
    table, kv_len, q_start, cache = without_page_zero(g, rows, lens, ps, H, D, extra_cols=0)
    kv_len = kv_len + np.array([longer] + [0] * (len(rows) - 1), dtype=np.int32)
    if longer:  # what poison left behind the old end is looked at now
        cache[1:] = filled_cache(g, len(cache) - 1, ps, H, D)
    prompt_rows(g, rows, kv_len, table, cache, q_start, Hq, H, D, ps, window, drawn=2)


def test_prompts_of_one_token_and_many():
    """Single tokens, drafts and prompts in one call, over pages of every size."""
    say("prompt, mixed")
    for ps in (64, 128, 256, 512):
        g = np.random.default_rng(ps)
        rows, lens = [1, 600, 4, 0, 33, 500], [2000, 600, 90, 5, 33, 1100]
        table, kv_len, q_start, cache = without_page_zero(g, rows, lens, ps, 4, 128)
        prompt_rows(g, rows, kv_len, table, cache, q_start, 20, 4, 128, ps, 0, drawn=3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [False, True])
def test_the_rounding_of_a_dominant_key_cancels_in_prompts(far, D):
    """Values are all 1, and so is their mean.  One key of each row has nearly all the weight: first place 0, from place 500 on that, with 2^q
    times the weight, 4 <= q < 8, from place 900 on that, with 2^2q times; the others 2^-9q.  The largest weight is as large in the divisor as it was
    multiplied; of the rest, at most 2^-4 of it, roundings are 2^-12 of the result, and fp32 sums 1300 x 2^-23: less than half a step
    of bf16 below 1, 2^-9.  far: scores behind 28672 q0 in fp32, for all keys of a row alike."""
    say("dominant key", far, D)
    g = np.random.default_rng(D)
    rows, lens, H, Hq, ps = [1100, 200], [1100, 900], 2, 32, 64
    table, kv_len, q_start, cache = without_page_zero(g, rows, lens, ps, H, D)
    v, _, s = sections(cache, ps, H, D)
    kat, vat = kv8.places(D)
    v[...], s[...] = 0, 127
    v[:, :, :, vat.reshape(-1)] = 0x38
    v[:, :, :, kat[:, 0]] = kv8.encode(np.array(-8.0))
    v[:, :, :, kat[:, 1]] = kv8.encode(np.array(448.0))
    for place, x in ((0, 1.0), (500, 2.0), (900, 4.0)):
        for row in table[:, place // ps]:
            if row >= 0:
                v[row, :, 0, kat[place % ps, 0]] = kv8.encode(np.array(x))
    q = np.zeros((int(q_start[-1]) + 1, Hq, D))
    q[..., 0] = bf16(g.uniform(4, 7.96, q.shape[:2]))
    if far:
        q[..., 1] = bf16(g.uniform(-64, 64, q.shape[:2]))
    assert len(q) * Hq > 64 * torch.cuda.get_device_properties(0).multi_processor_count
    out, _ = run_attention(q, cache, table, kv_len, q_start, H, ps, 1100, scale=float(np.float32(np.log(2))))
    assert (out[:-1] == 1).all()
