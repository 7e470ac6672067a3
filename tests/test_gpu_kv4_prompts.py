"""Prompts over the 4-bit cache, in the kernel that takes a sequence's rows by the hundred.  Calls with few rows go
another way, so these have rows behind the last sequence, which must stay as they are."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4
from tests.gpu_util import dev_bf16, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.kv4_util import attention_bounds, batch, bf16, bits, filled_cache  # noqa: E402
from tests.test_gpu_kv4 import attention_case, dev, held_to, run_attention  # noqa: E402


def extra(Hq):
    """Rows that make a call of Hq heads a large one on up to 320 CUs: half a row tile of 16 rows to each wave, 8 waves a CU."""
    return 320 * 8 * 16 // 2 // Hq


@pytest.mark.parametrize("rows,lens", [([64], [64]), ([65, 1], [65, 400]), ([127, 128, 129], [127, 128, 129]),
                                       ([200, 7, 1, 0, 90], [333, 7, 500, 64, 90]), ([260], [700])])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (2, 2, 64), (6, 2, 128), (8, 1, 64)])
def test_prompts(rows, lens, Hq, H, D):
    say("prompts", rows, lens, Hq, H, D)
    attention_case(sum(rows), rows, lens, Hq, H, D, 64, extra=extra(Hq))


@pytest.mark.parametrize("rows", [0, 1, 9])
def test_a_lone_sequence_of_fewer_rows_than_the_hint_says(rows):
    say("lone", rows)
    attention_case(rows, [rows], [rows + 500], 8, 2, 128, 64, max_q=300, extra=extra(8))


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (5, 1, 64)])
def test_prompts_beside_long_sequences_of_single_tokens(Hq, H, D):
    """Both kinds in one launch, rows of the latter cut between workgroups."""
    say("mixed", Hq, H, D)
    rows, lens = [1, 200, 3, 1, 90, 0, 1, 8], [20000, 300, 5000, 1, 4000, 70, 0, 9000]
    attention_case(Hq, rows, lens, Hq, H, D, 64, dirty=False, extra=extra(Hq))
    attention_case(Hq, rows, lens, Hq, H, D, 128, window=700, dirty=False, extra=extra(Hq))


@pytest.mark.parametrize("ps", [128, 256, 512])
def test_page_sizes(ps):
    say("page size", ps)
    attention_case(ps, [90, 1, 40], [ps + 60, 3 * ps - 5, 2 * ps + 7], 8, 2, 128, ps, extra=extra(8))


def test_many_pages():
    """More blocks than a wave holds the places of at a time, and sequences past the number of lanes."""
    say("many pages")
    attention_case(4, [40], [9000], 4, 1, 64, 64, extra=extra(4), dirty=False)
    g = np.random.default_rng(2)
    rows, lens = [int(r) for r in g.integers(0, 4, size=150)], [int(n) for n in g.integers(4, 20, size=150)]
    rows[70], lens[70], rows[149], lens[149] = 80, 300, 70, 70
    attention_case(5, rows, lens, 4, 2, 64, 64, extra=extra(4), dirty=False)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 1000])
def test_windows(window):
    say("window", window)
    attention_case(window, [150, 1, 150], [150, 300, 513], 8, 2, 128, 64, window=window, extra=extra(8))
    attention_case(window, [150], [257], 2, 2, 64, 128, window=window, extra=extra(2))


@pytest.mark.parametrize("rows,lens", [([130, 1, 0, 0, 1], [70, 1, 9, 0, 0]), ([70, 80], [0, 5])])
def test_rows_without_keys(rows, lens):
    say("empty rows", rows, lens)
    attention_case(9, rows, lens, 8, 2, 128, 64, extra=extra(8))
    attention_case(9, rows, lens, 8, 2, 64, 64, window=3, extra=extra(8))


@pytest.mark.parametrize("scale", [1e-3, 3.0, -0.5, 0.0])
def test_scales_and_large_scores(scale):
    """Scores of hundreds, growing along the keys at times: what weights are relative to moves often."""
    say("scale", scale)
    attention_case(7, [70, 120], [200, 900], 4, 2, 128, 64, scale=scale, extra=extra(4))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [0.02, 0.3, -0.3])
def test_scores_that_rise_from_key_to_key(D, step):
    """Every 32 tokens bring a new largest score (or none ever does): pending weights follow the reference."""
    say("rising", D, step)
    g = np.random.default_rng(1)
    H, Hq, ps, n, rows = 1, 4, 64, 700, 100
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    k, v = np.zeros((n, H, D)), bf16(g.standard_normal((n, H, D)))
    k[:, 0, 0] = bf16(1 + step * np.arange(n) if step > 0 else 1 + step * np.arange(n)[::-1])
    k[:, 0, 32:] = bf16(0.1 * g.standard_normal((n, D - 32)))
    cache = np.zeros((N, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    kv4.append(cache, k, v, table, kv_len, np.array([0, n], np.int32), ps)
    q = bf16(np.concatenate([g.standard_normal((rows, Hq, D)), np.zeros((extra(Hq), Hq, D))]))
    q[:rows, :, 0] = 6.0
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, 1.0, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows, scale=1.0), r, f"rising {D} {step}")


def test_bad_pages_and_a_length_behind_the_table():
    say("bad pages")
    g = np.random.default_rng(100)
    H, D, ps, rows = 2, 128, 64, 100
    table, kv_len, q_start, N = batch(g, [rows] * 4, [500, 300, 200, 128], ps)
    table[0, 2], table[0, 3], table[1, 0], table[2, :] = -1, N, 2**31 - 1, -5
    kv_len[0] = table.shape[1] * ps + 20
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((4 * rows + extra(8), 8, D)))
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "bad pages")


def test_scale_bytes_at_both_ends():
    say("scale ends")
    g = np.random.default_rng(3)
    H, D, ps, rows = 1, 128, 64, 80
    table, kv_len, q_start, N = batch(g, [rows], [200], ps)
    for lo, hi in ((16, 18), (246, 250), (16, 250)):
        cache = filled_cache(g, N, ps, H, D, 120, 130)
        x = cache.reshape(N, H, -1)
        vs = ps * D + ps * D // 32
        x[:, :, vs:] = g.integers(lo, hi, size=x[:, :, vs:].shape, dtype=np.uint8)
        q = bf16(g.standard_normal((rows + extra(4), 4, D)))
        r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
        held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, f"V scales {lo}..{hi}")


@pytest.mark.parametrize("D", [64, 128])
def test_one_key_gives_its_value_exactly(D):
    say("one key", D)
    g = np.random.default_rng(11)
    H, ps, n, rows = 2, 64, 200, 70
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((rows + extra(8), 8, D)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows, window=1)
    _, v = kv4.rows_of(cache, table, kv_len, q_start, ps, H, D, rows)
    assert (out[:rows] == np.repeat(v, 4, axis=1)).all() and (out[rows:] == 77).all()


def test_a_query_that_is_not_finite_spoils_its_own_row_alone():
    say("not finite")
    g = np.random.default_rng(6)
    H, Hq, D, ps, rows = 2, 8, 128, 64, 150
    table, kv_len, q_start, N = batch(g, [rows], [300], ps)
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((rows + extra(Hq), Hq, D)))
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    bo, bl = attention_bounds({k: x[:rows] for k, x in r.items()})
    bad = dev_bf16(bits(q))
    spoilt = np.zeros((rows, Hq), dtype=bool)
    for t, h, ch, x in ((0, 0, 0, float("nan")), (60, 5, D - 1, float("inf")), (rows - 1, 3, 33, float("-inf"))):
        bad[t, h, ch] = x
        spoilt[t, h] = True
    out, lse = nm.nm_kv4_attention(bad, dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, rows)
    out, lse = out[:rows].double().cpu().numpy(), lse[:rows].double().cpu().numpy()
    assert np.isnan(out[spoilt]).all() and np.isnan(lse[spoilt]).all()
    assert (np.abs(out - r["out"][:rows])[~spoilt] <= bo[~spoilt]).all()
    assert (np.abs(lse - r["lse"][:rows])[~spoilt] <= bl[~spoilt]).all()


@pytest.mark.parametrize("Hq,H,D", [(32, 8, 128), (9, 3, 64)])
def test_prompts_that_fill_the_machine(Hq, H, D):
    """Enough rows of their own; a few of them, spread over all tiles, against the plain definition."""
    say("large", Hq, H, D)
    g = np.random.default_rng(Hq)
    ps, rows, lens = 64, [700, 1, 60 * 32 // Hq * 10, 5], [900, 2000, 60 * 32 // Hq * 10 + 64, 5]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    T = sum(rows)
    assert T * Hq > 320 * 8 * 16 // 2
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((T, Hq, D)))
    out, lse = nm.nm_kv4_attention(dev_bf16(bits(q)), dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, max(rows))
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for t in sorted({0, 699, 700, T - 1, *(int(x) for x in g.integers(0, T, size=60))}):
        s = int(np.searchsorted(q_start, t, side="right")) - 1
        length = kv_len[s : s + 1] - (q_start[s + 1] - 1 - t)  # the sequence as that row sees it
        r = kv4.attention(q[t : t + 1], cache, table[s : s + 1], length, np.array([0, 1]), ps, H, D**-0.5, 0)
        bo, bl = attention_bounds(r)
        assert (np.abs(out[t] - r["out"][0]) <= bo[0]).all() and (np.abs(lse[t] - r["lse"][0]) <= bl[0]).all(), t


def test_a_captured_batch_of_prompts_and_single_tokens():
    """One graph; queries, lengths, rows and the page table change between its replays, each as the eager call."""
    say("captured")
    g = np.random.default_rng(3)
    Hq, H, D, ps = 8, 2, 128, 64
    T = 400 + extra(Hq)
    plans = [([200, 1, 1, 90], [300, 9000, 64, 90]), ([1, 300, 2, 0], [700, 300, 5000, 80]), ([1, 1, 1, 1], [8000, 1, 0, 129]),
             ([0, 0, 400, 0], [5, 5, 4000, 5])]
    cols = 9000 // ps + 2
    N = 160
    cache = dev(filled_cache(g, N, ps, H, D))
    q, table = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, cols), dtype=torch.int32, device="cuda")
    kv_len, q_start = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 5))
    out, lse = torch.zeros_like(q), torch.zeros((T, Hq), device="cuda")
    ws = torch.empty(nm.nm_kv4_attention_workspace_bytes(T, 4, Hq, H, D, 400, cols * ps), dtype=torch.uint8, device="cuda")
    run = lambda o, e, w: nm.nm_kv4_attention(q, cache, table, kv_len, q_start, H, ps, 400, out=o, lse=e, workspace=w)  # noqa: E731
    run(out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run(out, lse, ws)
    for i, (rows, lens) in enumerate(plans * 2):
        q.copy_(torch.randn(q.shape, device="cuda"))
        table.copy_(dev(g.integers(0, N, size=(4, cols)).astype(np.int32)))
        kv_len.copy_(dev(np.array(lens, np.int32)))
        q_start.copy_(dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)))
        eager = torch.full_like(q, 3.0), torch.full_like(lse, 3.0)
        run(*eager, None)
        out.fill_(3.0)
        lse.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1]), f"replay {i}"
        n = sum(rows)
        assert torch.isfinite(out).all() and (out[n:] == 3).all() and (lse[n:] == 3).all()
