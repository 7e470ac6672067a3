"""The 4-bit key/value cache on the GPU against the plain definitions (oracle/kv4.py): tokens in and out bit for
bit, attention within the bounds its arithmetic allows (tests/kv4_util.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import attention_bounds, batch, bf16, bits, filled_cache, poison

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_attention(q, cache, table, kv_len, q_start, H, ps, max_q, scale=None, window=0, view=None):
    """q fp64 [T, Hq, D] (bf16 values) -> out, lse as fp64; rows that are not written stay 77."""
    T, Hq, D = q.shape
    qd = dev_bf16(bits(q)) if view is None else view
    out = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 77.0, device="cuda")
    nm.nm_kv4_attention(qd, dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, max_q, scale=scale, window=window,
                        out=out, lse=lse)
    torch.cuda.synchronize()
    return bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64)


def held_to(out, lse, r, what):
    tail = np.isnan(r["lse"])
    assert (out[tail] == 77).all() and (lse[tail] == 77).all(), f"{what}: rows behind the last sequence were written"
    bo, bl = attention_bounds({k: v[~tail] for k, v in r.items()})
    ro, rl = r["out"][~tail], r["lse"][~tail]
    out, lse = out[~tail], lse[~tail]
    empty = np.isinf(rl)
    assert (lse[empty] == -np.inf).all() and (out[empty] == 0).all(), f"{what}: rows without keys"
    assert np.isfinite(out).all() and np.isfinite(lse[~empty]).all(), f"{what}: not finite"
    worst = (np.abs(out - ro) / bo).max(initial=0), (np.abs(lse[~empty] - rl[~empty]) / bl[~empty]).max(initial=0)
    assert worst[0] <= 1 and worst[1] <= 1, f"{what}: out {worst[0]:.3f}, lse {worst[1]:.3f} of the bound"


def attention_case(seed, rows, lens, Hq, H, D, ps, window=0, max_q=None, dirty=True, extra=0, **kw):
    g = np.random.default_rng(seed)
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    if dirty:
        poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]) + extra, Hq, D)) * np.exp(0.5 * g.standard_normal((Hq, D))))
    scale = kw.get("scale", D**-0.5)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, scale, window)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, max_q or max(rows + [1]), scale, window)
    held_to(out, lse, r, f"{rows} {lens} {Hq}/{H} D{D} ps{ps} w{window}")
    return q, cache, table, kv_len, q_start, out, lse


# ---- tokens in and out ----

@pytest.mark.parametrize("H,D,ps,rows,before", [
    (1, 64, 64, [1], [0]), (8, 128, 64, [1, 1, 1], [63, 64, 0]), (2, 128, 128, [5, 0, 130], [61, 7, 127]),
    (3, 64, 256, [70, 3], [250, 0]), (2, 128, 512, [513], [3]), (1, 128, 64, [1] * 70, list(range(70)))])
def test_append_and_unpack_bit_for_bit(H, D, ps, rows, before):
    say("append", H, D, ps, rows)
    g = np.random.default_rng(D + ps)
    lens = [a + b for a, b in zip(rows, before)]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = g.integers(0, 256, size=(N, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    T = int(q_start[-1])
    k, v = (bf16(g.standard_normal((T, H, D)) * np.exp(2 * g.standard_normal((T, H, D)))) for _ in range(2))
    k[0, 0, :32], v[0, 0, 1] = 0.0, 3.0e38
    k[-1, -1, -32:] = bf16(1e-39 * g.standard_normal(32))  # subnormal
    cd = dev(cache)
    args = (dev(table), dev(kv_len), dev(q_start), ps)
    nm.nm_kv4_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args)
    want = cache.copy()
    kv4.append(want, k, v, table, kv_len, q_start, ps)
    assert (cd.cpu().numpy() == want).all()
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv4_unpack(cd, *args, ko, vo)
    kr, vr = kv4.rows_of(want, table, kv_len, q_start, ps, H, D, T)
    assert (bf16_as_f64(host_bf16(ko)) == kr).all() and (bf16_as_f64(host_bf16(vo)) == vr).all()


def test_every_bf16_magnitude_and_neighbour_is_rounded_as_defined():
    """Each finite bf16 number beside a largest one of its own, twice and four times its size."""
    say("rounding")
    u = np.arange(0x7F80, dtype=np.uint32)
    x = (u << 16).view(np.float32).astype(np.float64)
    blocks = np.zeros((3, len(x), 32))
    for i, f in enumerate((1.0, 2.0, 4.5)):
        blocks[i, :, 0] = bf16(np.minimum(x * f, 3.38e38))
        blocks[i, :, 1], blocks[i, :, 2] = x, -x
    rows = blocks.reshape(-1, 2, 64)
    T = len(rows)
    table, kv_len, q_start, N = batch(np.random.default_rng(0), [T], [T], 512, spare=0)
    cd = torch.zeros((N, kv4.page_bytes(512, 2, 64)), dtype=torch.uint8, device="cuda")
    args = (dev(table), dev(kv_len), dev(q_start), 512)
    xd = dev_bf16(bits(rows))
    nm.nm_kv4_append(xd, xd, cd, *args)
    ko, vo = torch.empty_like(xd), torch.empty_like(xd)
    nm.nm_kv4_unpack(cd, *args, ko, vo)
    want = kv4.dequantize(*kv4.quantize(rows))
    assert (bf16_as_f64(host_bf16(ko)) == want).all() and (bf16_as_f64(host_bf16(vo)) == want).all()


def test_rows_without_a_place_and_behind_the_last_sequence():
    """Places below 0, behind the table and on bad pages are not written and read as zeros."""
    say("no place")
    H, D, ps = 2, 64, 64
    table = np.array([[0, 9], [-1, 1], [2, -7], [3, 3]], dtype=np.int32)
    kv_len = np.array([70, 70, 3, 200], dtype=np.int32)  # page 9 of 4; no page 0; 5 rows but 3 places; 128 places
    q_start = np.array([0, 10, 20, 25, 100], dtype=np.int32)
    g = np.random.default_rng(4)
    cache = g.integers(0, 250, size=(4, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    T = 103
    k, v = (bf16(g.standard_normal((T, H, D))) for _ in range(2))
    cd = dev(cache)
    args = (dev(table), dev(kv_len), dev(q_start), ps)
    nm.nm_kv4_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args)
    want = cache.copy()
    kv4.append(want, k, v, table, kv_len, q_start, ps)
    assert (cd.cpu().numpy() == want).all()
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv4_unpack(cd, *args, ko, vo)
    kr, vr = kv4.rows_of(want, table, kv_len, q_start, ps, H, D, T)
    for a, b in ((ko, kr), (vo, vr)):
        a = bf16_as_f64(host_bf16(a))
        assert (a[100:] == 5).all() and (a[:100] == b[:100]).all()


# ---- attention ----

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 4), (8, 2), (5, 1), (16, 2), (7, 1), (40, 2), (24, 1)])
def test_one_token_of_each_sequence(Hq, H, D):
    say("decode", Hq, H, D)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 777]
    attention_case(Hq * D, [1] * len(lens), lens, Hq, H, D, 64)


@pytest.mark.parametrize("ps", [64, 128, 256, 512])
def test_page_sizes(ps):
    say("page size", ps)
    attention_case(ps, [1, 1, 3, 1, 40], [ps - 1, ps, ps + 1, 3 * ps - 5, 2 * ps + 7], 8, 2, 128, ps)


@pytest.mark.parametrize("rows", [2, 3, 4, 5, 8, 9, 17, 33])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (3, 3, 64), (8, 1, 64)])
def test_several_tokens(rows, Hq, H, D):
    say("rows", rows, Hq, H, D)
    attention_case(rows * Hq, [rows, rows, rows, 1], [rows, 64, 200 + rows, 130], Hq, H, D, 64)


@pytest.mark.parametrize("rows,lens", [([64], [64]), ([65, 1], [65, 400]), ([127, 128, 129], [127, 128, 129]),
                                       ([200, 7, 1, 0, 90], [333, 7, 500, 64, 90]), ([260], [700])])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (2, 2, 64), (6, 2, 128)])
def test_prompts(rows, lens, Hq, H, D):
    say("prompts", rows, lens, Hq, H, D)
    attention_case(sum(rows), rows, lens, Hq, H, D, 64)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("rows", [1, 5, 150])
def test_windows(window, rows):
    say("window", window, rows)
    attention_case(window + rows, [rows, rows, rows], [rows, 300, 513], 8, 2, 128, 64, window=window)
    attention_case(window + rows, [rows], [257], 2, 2, 64, 128, window=window)


@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [0, 5, 0]), ([4, 6], [2, 0]), ([130, 1, 0, 0, 1], [70, 1, 9, 0, 0]),
                                       ([0, 0], [5, 0])])
def test_rows_without_keys(rows, lens):
    """Sequences of length 0, and with more rows than places."""
    say("empty rows", rows, lens)
    attention_case(9, rows, lens, 8, 2, 128, 64, extra=2)
    attention_case(9, rows, lens, 8, 2, 64, 64, window=3, extra=2)


@pytest.mark.parametrize("rows", [1, 100])
def test_bad_pages_are_left_out(rows):
    say("bad pages", rows)
    g = np.random.default_rng(rows)
    H, D, ps = 2, 128, 64
    table, kv_len, q_start, N = batch(g, [rows] * 3, [500, 300, 200], ps)
    table[0, 2], table[0, 3], table[1, 0], table[2, :] = -1, N, 2**31 - 1, -5
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((3 * rows, 8, D)))
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "bad pages")


@pytest.mark.parametrize("rows", [1, 90])
def test_a_length_behind_the_table_stops_at_its_end(rows):
    say("table end", rows)
    g = np.random.default_rng(rows)
    table, kv_len, q_start, N = batch(g, [rows], [128], 64, extra_cols=0)
    kv_len[0] = 150
    cache = filled_cache(g, N, 64, 1, 64)
    q = bf16(g.standard_normal((rows, 4, 64)))
    r = kv4.attention(q, cache, table, kv_len, q_start, 64, 1, 0.125, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, 1, 64, rows), r, "table end")


@pytest.mark.parametrize("rows,hint", [(1, 200), (150, 1), (9, 1), (2, 1 << 20)])
def test_a_wrong_hint_changes_nothing_but_time(rows, hint):
    say("hint", rows, hint)
    attention_case(rows, [rows, 1], [rows + 70, 33], 8, 2, 128, 64, max_q=hint)


@pytest.mark.parametrize("scale", [1e-3, 3.0, -0.5, 0.0])
def test_scales_and_large_scores(scale):
    """Scores of hundreds: all weight on single keys; equal scores: a plain mean."""
    say("scale", scale)
    attention_case(7, [1, 70], [400, 200], 4, 2, 128, 64, scale=scale)


@pytest.mark.parametrize("rows", [1, 80])
def test_scale_bytes_at_both_ends(rows):
    """Values and keys of any size the format stores: the smallest, the largest and both in one sequence."""
    say("scale ends", rows)
    g = np.random.default_rng(3)
    H, D, ps = 1, 128, 64
    table, kv_len, q_start, N = batch(g, [rows], [200], ps)
    for lo, hi in ((16, 18), (246, 250), (16, 250)):  # 6 * 2^122 the largest: weighted sums stay below the largest bf16
        cache = filled_cache(g, N, ps, H, D, 120, 130)
        x = cache.reshape(N, H, -1)
        vs = ps * D + ps * D // 32
        x[:, :, vs:] = g.integers(lo, hi, size=x[:, :, vs:].shape, dtype=np.uint8)
        q = bf16(g.standard_normal((rows, 4, D)))
        r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
        held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, f"V scales {lo}..{hi}")
    cache = filled_cache(g, N, ps, H, D, 120, 130)
    x = cache.reshape(N, H, -1)
    x[:, :, ps * D : ps * D + ps * D // 32] = 16
    q = bf16(g.standard_normal((rows, 4, D)) * 1e30)
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "K scales 16")


@pytest.mark.parametrize("rows", [1, 6, 70])
def test_one_key_gives_its_value_exactly(rows):
    """A window of one: the weight is 1, the value of the row's own key comes back bit for bit."""
    say("one key", rows)
    g = np.random.default_rng(11)
    H, D, ps, n = 2, 128, 64, 200
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((rows, 8, D)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows, window=1)
    _, v = kv4.rows_of(cache, table, kv_len, q_start, ps, H, D, rows)
    assert (out == np.repeat(v, 4, axis=1)).all()


@pytest.mark.parametrize("rows", [1, 66])
def test_strided_rows_of_a_joint_projection(rows):
    """q, k and v are views of one [T, (Hq + 2 H) * D + 8] array, out a view of a wider one; the table has a row stride."""
    say("strides", rows)
    g = np.random.default_rng(rows)
    Hq, H, D, ps = 8, 2, 128, 64
    table, kv_len, q_start, N = batch(g, [rows, rows], [rows + 100, rows], ps)
    T, width = 2 * rows, (Hq + 2 * H) * D + 8
    qkv = bf16(g.standard_normal((T, width)))
    x = dev_bf16(bits(qkv))
    part = lambda a, n: x[:, a * D : (a + n) * D].unflatten(1, (n, D))  # noqa: E731
    q, k, v = part(0, Hq), part(Hq, H), part(Hq + H, H)
    cache = filled_cache(g, N, ps, H, D)
    cd = dev(cache)
    wide = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = dev(table)
    td = wide[:, : table.shape[1]]
    nm.nm_kv4_append(k, v, cd, td, dev(kv_len), dev(q_start), ps)
    host = lambda a, n: qkv[:, a * D : (a + n) * D].reshape(T, n, D)  # noqa: E731
    kv4.append(cache, host(Hq, H), host(Hq + H, H), table, kv_len, q_start, ps)
    assert (cd.cpu().numpy() == cache).all()
    big = torch.full((T, Hq * D + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, : Hq * D].unflatten(1, (Hq, D))
    lse = torch.full((T, Hq + 3), 77.0, device="cuda")
    nm.nm_kv4_attention(q, cd, td, dev(kv_len), dev(q_start), H, ps, rows, out=out, lse=lse[:, :Hq])
    assert (big[:, Hq * D :] == 3).all() and (lse[:, Hq:] == 77).all()
    r = kv4.attention(host(0, Hq), cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(bf16_as_f64(host_bf16(out)), lse[:, :Hq].cpu().numpy().astype(np.float64), r, "strides")


@pytest.mark.parametrize("rows", [1, 70])
def test_pages_far_into_a_large_cache(rows):
    """A cache of over 4 GiB, its pages in use at both ends: offsets pass 32 bits."""
    say("large cache", rows)
    g = np.random.default_rng(2)
    H, D, ps = 8, 128, 512
    nbytes = kv4.page_bytes(ps, H, D)
    N = (5 << 30) // nbytes
    small = filled_cache(g, 4, ps, H, D)
    cd = torch.zeros((N, nbytes), dtype=torch.uint8, device="cuda")
    cd[-3:] = dev(small[1:])
    cd[0] = dev(small[0])
    local, kv_len = np.array([[3, 0, 1, 2]], np.int32), np.array([1900], np.int32)
    far = np.array([[N - 1, 0, N - 3, N - 2]], np.int32)
    q_start = np.array([0, rows], np.int32)
    k, v = (bf16(g.standard_normal((rows, H, D))) for _ in range(2))
    nm.nm_kv4_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, dev(far), dev(kv_len), dev(q_start), ps)
    kv4.append(small, k, v, local, kv_len, q_start, ps)
    assert (cd[-3:].cpu().numpy() == small[1:]).all() and (cd[0].cpu().numpy() == small[0]).all()
    q = bf16(g.standard_normal((rows, H, D)))
    out = torch.empty((rows, H, D), dtype=torch.bfloat16, device="cuda")
    out, lse = nm.nm_kv4_attention(dev_bf16(bits(q)), cd, dev(far), dev(kv_len), dev(q_start), H, ps, rows, out=out)
    r = kv4.attention(q, small, local, kv_len, q_start, ps, H, D**-0.5, 0)
    held_to(bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64), r, "large cache")


@pytest.mark.parametrize("S", [65, 200, 1030])
def test_many_sequences(S):
    """More sequences than a wave has lanes, some without rows, a long one among short ones."""
    say("many", S)
    g = np.random.default_rng(S)
    rows = [int(r) for r in g.integers(0, 3, size=S)]
    lens = [int(n) for n in g.integers(0, 20, size=S)]
    rows[S // 2], lens[S // 2] = 2, 3000
    rows[-1], lens[-1] = 5, 90
    attention_case(S, rows, lens, 2, 1, 64, 64, dirty=False)


def test_no_rows_at_all():
    say("no rows")
    cache = torch.zeros((2, kv4.page_bytes(64, 1, 64)), dtype=torch.uint8, device="cuda")
    table, kv_len, q_start = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((2, 1), 2, 3))
    x = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    nm.nm_kv4_append(x, x, cache, table, kv_len, q_start, 64)
    nm.nm_kv4_unpack(cache, table, kv_len, q_start, 64, x, x)
    out, lse = nm.nm_kv4_attention(x, cache, table, kv_len, q_start, 1, 64, 1)
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1) and int(cache.sum()) == 0


def test_the_same_call_gives_the_same_bits():
    say("determinism")
    g = np.random.default_rng(0)
    table, kv_len, q_start, N = batch(g, [1, 5, 100, 1], [9000, 4000, 300, 64], 64)
    cache = filled_cache(g, N, 64, 2, 128)
    q = bf16(g.standard_normal((107, 16, 128)))
    first = run_attention(q, cache, table, kv_len, q_start, 2, 64, 100)
    for _ in range(5):
        again = run_attention(q, cache, table, kv_len, q_start, 2, 64, 100)
        assert (first[0] == again[0]).all() and (first[1] == again[1]).all()


def test_long_contexts():
    """Work split over the length and joined: 40000 tokens of one sequence, alone and beside short ones."""
    say("long")
    attention_case(1, [1], [40000], 4, 1, 128, 64, dirty=False)
    attention_case(2, [1, 1, 2, 1], [30000, 1, 5000, 0], 4, 1, 64, 256, dirty=False)
    attention_case(3, [20, 1], [9000, 12000], 8, 2, 128, 64, dirty=False)


def test_two_streams_at_once():
    say("streams")
    cases = [attention_case(s, [1, 9], [3000, 500], 8, 2, 128, 64, dirty=False) for s in (5, 6)]
    on = [torch.cuda.Stream() for _ in cases]
    args = []
    for q, cache, table, kv_len, q_start, *_ in cases:
        args.append((dev_bf16(bits(q)), dev(cache), dev(table), dev(kv_len), dev(q_start)))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st, a in zip(on, args):
            with torch.cuda.stream(st):
                got.append(nm.nm_kv4_attention(*a, 2, 64, 9))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert (bf16_as_f64(host_bf16(out)) == cases[i % 2][-2]).all()
        assert (lse.cpu().numpy() == cases[i % 2][-1]).all()
