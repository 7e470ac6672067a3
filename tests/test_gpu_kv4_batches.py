"""Batches of the 4-bit cache that are far from the usual ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.kv4_util import attention_bounds, bf16, bits, filled_cache  # noqa: E402
from tests.test_gpu_kv4 import attention_case, dev  # noqa: E402


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,used", [(1000, [0, 999]), (1000, [0, 1, 63, 64, 65, 500, 998]), (130, [128, 129]), (4097, [7, 4000, 4096])])
def test_rows_of_sequences_far_apart(D, S, used):
    """A wave's rows belong to sequences with many without rows between them."""
    say("far apart", D, S, used)
    g = np.random.default_rng(S)
    H, ps = 2, 64
    n = np.zeros(S, dtype=np.int64)
    n[used] = g.integers(1, 4, size=len(used))
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    kv_len = (n + g.integers(0, 60, size=S)).astype(np.int32)
    table = np.full((S, 1), -1, np.int32)
    table[used, 0] = g.permutation(len(used) + 2)[: len(used)]
    T = int(q_start[-1])
    k, v = (bf16(g.standard_normal((T, H, D))) for _ in range(2))
    cache = g.integers(0, 250, size=(len(used) + 2, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    cd, args = dev(cache), (dev(table), dev(kv_len), dev(q_start), ps)
    nm.nm_kv4_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args)
    kv4.append(cache, k, v, table, kv_len, q_start, ps)
    assert (cd.cpu().numpy() == cache).all()
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv4_unpack(cd, *args, ko, vo)
    kr, vr = kv4.rows_of(cache, table, kv_len, q_start, ps, H, D, T)
    assert (bf16_as_f64(host_bf16(ko)) == kr).all() and (bf16_as_f64(host_bf16(vo)) == vr).all()


def test_two_rows_at_the_ends_of_a_million_slots():
    """The search for a row's sequence takes a few looks, not one for each of the slots between two rows of a
    wave: 10 ms are a thousand times what the call takes, and a tenth of a million reads one after the other."""
    say("a million slots")
    S, H, D, ps = 1 << 20, 2, 128, 64
    q_start = torch.ones(S + 1, dtype=torch.int32, device="cuda")
    q_start[0], q_start[-1] = 0, 2
    kv_len = torch.full((S,), 1, dtype=torch.int32, device="cuda")
    table = torch.zeros((S, 1), dtype=torch.int32, device="cuda")
    table[-1] = 1
    x = torch.randn((2, H, D), device="cuda").to(torch.bfloat16)
    cache = torch.zeros((2, kv4.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for again in range(2):
        torch.cuda.synchronize()
        t0.record()
        nm.nm_kv4_append(x, x, cache, table, kv_len, q_start, ps)
        nm.nm_kv4_unpack(cache, table, kv_len, q_start, ps, a, b)
        t1.record()
        torch.cuda.synchronize()
    want = kv4.dequantize(*kv4.quantize(bf16_as_f64(host_bf16(x))))
    assert (bf16_as_f64(host_bf16(a)) == want).all() and (bf16_as_f64(host_bf16(b)) == want).all()
    assert int(cache.any(1).sum()) == 2
    assert t0.elapsed_time(t1) < 10, f"{t0.elapsed_time(t1)} ms"


@pytest.mark.parametrize("hint", [1 << 40, 1 << 61, (1 << 63) - 1])
def test_a_hint_of_any_size(hint):
    say("hint", hint)
    attention_case(5, [3, 1], [70, 33], 8, 2, 128, 64, max_q=hint)


def test_no_sequences():
    say("no sequences")
    cache = torch.zeros((2, kv4.page_bytes(64, 1, 64)), dtype=torch.uint8, device="cuda")
    table, kv_len, q_start = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((0, 1), 0, 1))
    x = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    nm.nm_kv4_append(x, x, cache, table, kv_len, q_start, 64)
    nm.nm_kv4_unpack(cache, table, kv_len, q_start, 64, x, x)
    out, lse = nm.nm_kv4_attention(x, cache, table, kv_len, q_start, 1, 64, 1)
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1) and int(cache.sum()) == 0


@pytest.mark.parametrize("rows", [2, 64, 3000])
def test_the_same_place_twice_stays_within_that_place(rows):
    """Rows of many sequences that share a page, all for one token of it: what ends up there is finite, and nothing else changes."""
    say("same place", rows)
    H, D, ps = 3, 128, 64
    g = np.random.default_rng(rows)
    x = bf16(g.standard_normal((rows, H, D)) * np.exp(4 * g.standard_normal((rows, 1, 1))))
    table = torch.ones((rows, 1), dtype=torch.int32, device="cuda")
    kv_len = torch.full((rows,), 21, dtype=torch.int32, device="cuda")
    q_start = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    before = g.integers(0, 250, size=(3, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    cd, xd = dev(before), dev_bf16(bits(x))
    nm.nm_kv4_append(xd, xd, cd, table, kv_len, q_start, ps)
    after = cd.cpu().numpy()
    mine = np.zeros((H, before.shape[1] // H), dtype=bool)
    for values in (False, True):
        at, sc = kv4.places(ps, D, values)
        mine[:, at[20]] = mine[:, sc[20]] = True
    mine = mine.reshape(-1)
    assert (after[[0, 2]] == before[[0, 2]]).all() and (after[1, ~mine] == before[1, ~mine]).all()
    one = [table[:1], kv_len[:1], q_start[:2]]
    for y in nm.nm_kv4_unpack(cd, *one, ps, *(torch.empty_like(xd[:1]) for _ in range(2))):
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("window", [0, 30000])
def test_long_runs_of_row_tiles(window):
    """Over 60 blocks to a wave, so that it reads the page table again within its run; whole rows, pieces, and
    short sequences between them in one run.  Some rows against the plain definition."""
    say("long runs", window)
    g = np.random.default_rng(31)
    Hq, H, D, ps, N = 32, 4, 64, 64, 50
    rows, lens = [60, 1, 2, 0, 8, 40], [65536, 70, 6000, 9, 50001, 30011]
    tiles = [-(-r * Hq // H // 16) for r in rows]
    units = H * sum(t * -(-n // 64) for t, n in zip(tiles, lens))
    assert window or units > 62 * 8 * torch.cuda.get_device_properties(0).multi_processor_count  # 8 waves to a CU
    cols = 65536 // ps
    table = g.integers(0, N, size=(len(rows), cols)).astype(np.int32)  # a small pool, its pages many times in a row
    kv_len, q_start = np.array(lens, np.int32), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    cache = filled_cache(g, N, ps, H, D)
    T = int(q_start[-1])
    q = bf16(g.standard_normal((T, Hq, D)))
    out, lse = nm.nm_kv4_attention(dev_bf16(bits(q)), dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, 1, window=window)
    out, lse = bf16_as_f64(host_bf16(out)), lse.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for t in (0, 17, 59, 60, 61, 62, 63, 66, 70, 71, 90, T - 1):
        s = int(np.searchsorted(q_start, t, side="right")) - 1
        length = kv_len[s : s + 1] - (q_start[s + 1] - 1 - t)  # the sequence as that row sees it
        r = kv4.attention(q[t : t + 1], cache, table[s : s + 1], length, np.array([0, 1]), ps, H, D**-0.5, window)
        bo, bl = attention_bounds(r)
        assert (np.abs(out[t] - r["out"][0]) <= bo[0]).all() and (np.abs(lse[t] - r["lse"][0]) <= bl[0]).all(), t
