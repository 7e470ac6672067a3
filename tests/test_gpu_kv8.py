"""The 8-bit key/value cache on the GPU against the plain definitions (oracle/kv8.py): tokens in and out bit for
bit, attention within the bounds its arithmetic allows (tests/kv8_util.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import attention_bounds, filled_cache, poison, sections, turns

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same_bytes(got, want, ps, H, D, what):
    got = got.cpu().numpy()
    for name, a, b in zip(("values", "bounds", "scales"), sections(got, ps, H, D), sections(want, ps, H, D)):
        off = np.argwhere(a != b)
        assert not len(off), f"{what}: {len(off)} bytes of {name} differ, the first at {off[0]}: {a[tuple(off[0])]}, not {b[tuple(off[0])]}"


def grown(g, cache, H, D, ps, N, before, rows, table, turn, interleaved, loud=1.0):
    """`before` tokens into the oracle's and the GPU's cache, then `rows` more; -> the second call's arguments."""
    cd = dev(cache)
    want = cache.copy()
    for lens, n, size in ((before, before, 1.0), ([a + b for a, b in zip(before, rows)], rows, loud)):
        q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        kv_len = np.array(lens, dtype=np.int32)
        T = int(q_start[-1])
        if T == 0:
            continue
        k, v = (bf16(size * g.standard_normal((T, H, D)) * np.exp(g.standard_normal((T, H, D)))) for _ in range(2))
        args = dev(table), dev(kv_len), dev(q_start), ps
        nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args, rotation=None if turn is None else dev(turn), interleaved=interleaved)
        kv8.append(want, k, v, table, kv_len, q_start, ps, turn, interleaved)
    return cd, want, args, kv_len, q_start, T


@pytest.mark.parametrize("rotary,interleaved", [(None, False), (1.0, False), (1.0, True), (0.5, False), (0.25, True)])
@pytest.mark.parametrize("H,D,ps,rows,before,loud", [
    (1, 64, 64, [1], [0], 1.0), (8, 128, 64, [1, 1, 1], [63, 64, 0], 1.0), (2, 128, 128, [5, 0, 130], [61, 7, 127], 8.0),
    (3, 64, 256, [70, 3], [250, 0], 100.0), (2, 128, 512, [513], [3], 30.0), (1, 128, 64, [1] * 70, list(range(70)), 0.01),
    (2, 64, 64, [2, 9, 1], [30, 1, 62], 3000.0)])
def test_append_and_unpack_bit_for_bit(H, D, ps, rows, before, loud, rotary, interleaved):
    say("append", H, D, ps, rows, rotary, interleaved)
    g = np.random.default_rng(D + ps + len(rows))
    table, _, _, N = batch(g, rows, [a + b for a, b in zip(rows, before)], ps)
    cache = g.integers(0, 256, size=(N, kv8.page_bytes(ps, H, D)), dtype=np.uint8)  # what lies there before does not matter
    turn = None if rotary is None else turns(g, table.shape[1] * ps, int(D * rotary))
    cd, want, args, kv_len, q_start, T = grown(g, cache, H, D, ps, N, before, rows, table, turn, interleaved, loud)
    same_bytes(cd, want, ps, H, D, "append")
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv8_unpack(cd, *args, ko, vo)
    kr, vr = kv8.rows_of(want, table, kv_len, q_start, ps, H, D, T)
    assert (bf16_as_f64(host_bf16(ko)) == kr).all() and (bf16_as_f64(host_bf16(vo)) == vr).all()


def test_every_bf16_magnitude_is_rounded_as_defined():
    """Each finite bf16 number in a block with a largest one of its own, of its size, twice, 4.5 and 1000 times."""
    say("rounding")
    u = np.arange(0x7F80, dtype=np.uint32)
    x = (u << 16).view(np.float32).astype(np.float64)
    few = x.reshape(-1, 32)  # 32 neighbours and their negatives a block
    for f in (1.0, 2.0, 4.5, 1000.0):
        D = 64
        tokens = np.concatenate([few, -few], 1)[:, None, :]  # [blocks, 1, 64]
        T = len(tokens)
        table, kv_len, q_start, N = batch(np.random.default_rng(0), [1] * T, [1] * T, 64, spare=0)
        tokens[:, 0, 5] = bf16(np.minimum(np.abs(tokens[:, 0]).max(-1) * f, 3.38e38))
        cd = torch.zeros((N, kv8.page_bytes(64, 1, D)), dtype=torch.uint8, device="cuda")
        want = np.zeros(cd.shape, dtype=np.uint8)
        xd = dev_bf16(bits(tokens))
        nm.nm_kv8_append(xd, xd, cd, dev(table), dev(kv_len), dev(q_start), 64)
        kv8.append(want, tokens, tokens, table, kv_len, q_start, 64)
        same_bytes(cd, want, 64, 1, D, f"factor {f}")


def test_rotation_rounds_once():
    """Turns by angles so small that a rounding to fp32 in between would leave ties."""
    say("rounds once")
    g = np.random.default_rng(3)
    H, D, ps, T = 2, 128, 64, 64
    table, kv_len, q_start, N = batch(g, [T], [T], ps, extra_cols=0)
    turn = np.zeros((ps, D // 2, 2), dtype=np.float32)
    turn[..., 0], turn[..., 1] = 1.0, g.choice([1e-9, -1e-9, 1e-12, 0.0], size=turn.shape[:2])
    k = g.integers(17, 32, size=(T, H, D)) * 2.0 ** g.integers(-3, 3, size=(T, H, D)) * g.choice([1, -1], size=(T, H, D))  # 5 bits: halfway between codes
    cd = torch.zeros((N, kv8.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda")
    want = np.zeros(cd.shape, dtype=np.uint8)
    kd = dev_bf16(bits(k))
    nm.nm_kv8_append(kd, kd, cd, dev(table), dev(kv_len), dev(q_start), ps, rotation=dev(turn))
    kv8.append(want, k, k, table, kv_len, q_start, ps, turn)
    same_bytes(cd, want, ps, H, D, "rounds once")


@pytest.mark.parametrize("D,rotary,interleaved,heads", [(128, 128, False, 8), (128, 64, True, 5), (64, 16, False, 3), (64, 64, True, 24)])
@pytest.mark.parametrize("inplace", [False, True])
def test_queries_are_rotated(D, rotary, interleaved, heads, inplace):
    """Against fp64; off by a rounding of products and sum in fp32 and one to bf16."""
    say("queries", D, rotary, interleaved, heads)
    g = np.random.default_rng(heads)
    rows, lens, ps = [1, 7, 0, 130], [200, 60, 5, 131], 128
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    T = int(q_start[-1]) + 2
    H = 1
    turn = turns(g, table.shape[1] * ps, rotary)
    q, k = bf16(g.standard_normal((T, heads, D))), bf16(g.standard_normal((T, H, D)))
    qd, kd = dev_bf16(bits(q)), dev_bf16(bits(k))
    out = qd if inplace else torch.full_like(qd, 9.0)
    cd = torch.zeros((N, kv8.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda")
    got = nm.nm_kv8_append(kd, kd, cd, dev(table), dev(kv_len), dev(q_start), ps, rotation=dev(turn), interleaved=interleaved, q=qd, q_out=out)
    assert got is out
    got = bf16_as_f64(host_bf16(out))
    assert (got[-2:] == (q[-2:] if inplace else 9.0)).all()
    for s in range(len(rows)):
        for i in range(rows[s]):
            t, p = q_start[s] + i, lens[s] - rows[s] + i
            if p < 0:
                assert (got[t] == (q[t] if inplace else 9.0)).all()
                continue
            want, size = kv8.rotate(q[t], p, turn, interleaved), kv8.rotate(np.abs(q[t]), p, np.abs(turn) * [1, -1], interleaved)
            size = np.maximum(size, np.abs(kv8.rotate(np.abs(q[t]), p, np.abs(turn), interleaved)))
            assert (np.abs(got[t] - want) <= 2.0**-8 * np.abs(want) + 2.0**-22 * size).all(), (s, i)


def test_tokens_that_are_not_finite_stay_by_themselves():
    say("not finite")
    g = np.random.default_rng(8)
    H, D, ps, rows, lens = 2, 128, 64, [20, 1, 3], [80, 64, 3]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    T = int(q_start[-1])
    k, v = (bf16(g.standard_normal((T, H, D))) for _ in range(2))
    k[3, 0, 17], k[5, 1, 0], k[20, 0, :] = np.inf, np.nan, -np.inf
    v[7, 0, 99], v[7, 0, 3], v[21, 1, 64], v[22, 0, 0] = np.nan, np.inf, -np.inf, np.nan
    cd, want = dev(cache), cache.copy()
    args = dev(table), dev(kv_len), dev(q_start), ps
    nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args)
    kv8.append(want, k, v, table, kv_len, q_start, ps)
    same_bytes(cd, want, ps, H, D, "not finite")
    q = bf16(g.standard_normal((T, 4, D)))
    r = kv8.attention(q, want, table, kv_len, q_start, ps, H, D**-0.5)
    nan = np.isnan(r["lse"])
    assert nan[3:20, :2].all() and nan[5:20, 2:].all() and not nan[:3].any() and nan.sum() < nan.size
    out, lse = nm.nm_kv8_attention(dev_bf16(bits(q)), cd, *args[:3], H, ps, 20)
    out, lse = bf16_as_f64(host_bf16(out)), lse.cpu().numpy()
    assert (np.isnan(out).any(-1) == nan).all() and (np.isnan(lse) == nan).all()


def test_rows_without_a_place_and_behind_the_last_sequence():
    """Places below 0, behind the table and on bad pages are not written and read as zeros."""
    say("no place")
    H, D, ps = 2, 64, 64
    table = np.array([[0, 9], [-1, 1], [2, -7], [3, 3]], dtype=np.int32)
    kv_len = np.array([70, 70, 3, 200], dtype=np.int32)  # page 9 of 4; no page 0; 5 rows but 3 places; 128 places
    q_start = np.array([0, 10, 20, 25, 89], dtype=np.int32)  # the last: places 136 on, none of them in the table
    g = np.random.default_rng(4)
    cache = filled_cache(g, 4, ps, H, D)
    T = 92
    k, v = (bf16(g.standard_normal((T, H, D))) for _ in range(2))
    cd = dev(cache)
    args = (dev(table), dev(kv_len), dev(q_start), ps)
    nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, *args)
    want = cache.copy()
    kv8.append(want, k, v, table, kv_len, q_start, ps)
    same_bytes(cd, want, ps, H, D, "no place")
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nm.nm_kv8_unpack(cd, *args, ko, vo)
    kr, vr = kv8.rows_of(want, table, kv_len, q_start, ps, H, D, T)
    for a, b in ((ko, kr), (vo, vr)):
        a = bf16_as_f64(host_bf16(a))
        assert (a[89:] == 5).all() and (a[:89] == b[:89]).all()


def test_tokens_taken_back_and_written_again():
    """A draft that is loud, taken back, and quiet tokens in its place: scale and bounds keep what they had, values are the new ones."""
    say("taken back")
    g = np.random.default_rng(11)
    H, D, ps = 2, 128, 64
    table = np.array([[0, 1, 2]], dtype=np.int32)
    cd, want = torch.zeros((3, kv8.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda"), np.zeros((3, kv8.page_bytes(ps, H, D)), dtype=np.uint8)
    for n, length, size in ((50, 50, 1.0), (10, 60, 50.0), (3, 55, 0.1), (20, 75, 1.0), (1, 64, 0.01), (2, 66, 1000.0)):
        k, v = (bf16(size * g.standard_normal((n, H, D))) for _ in range(2))
        kv_len, q_start = np.array([length], dtype=np.int32), np.array([0, n], dtype=np.int32)
        nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cd, dev(table), dev(kv_len), dev(q_start), ps)
        kv8.append(want, k, v, table, kv_len, q_start, ps)
        same_bytes(cd, want, ps, H, D, f"{n} to {length}")


# ---- attention ----

def run_attention(q, cache, table, kv_len, q_start, H, ps, max_q, scale=None, window=0, selected=None, view=None):
    """q fp64 [T, Hq, D] (bf16 values) -> out, lse as fp64; rows that are not written stay 77."""
    T, Hq, D = q.shape
    qd = dev_bf16(bits(q)) if view is None else view
    out = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 77.0, device="cuda")
    nm.nm_kv8_attention(qd, dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, max_q, scale=scale, window=window,
                        selected=None if selected is None else dev(selected), out=out, lse=lse)
    torch.cuda.synchronize()
    return bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64)


def held_to(out, lse, r, what):
    tail = r["keys"] < 0
    assert (out[tail] == 77).all() and (lse[tail] == 77).all(), f"{what}: rows behind the last sequence were written"
    bo, bl = attention_bounds({k: v[~tail] for k, v in r.items()})
    ro, rl = r["out"][~tail], r["lse"][~tail]
    out, lse = out[~tail], lse[~tail]
    empty = np.isneginf(rl)
    assert (lse[empty] == -np.inf).all() and (out[empty] == 0).all(), f"{what}: rows without keys"
    assert np.isfinite(out).all() and np.isfinite(lse[~empty]).all(), f"{what}: not finite"
    worst = (np.abs(out - ro) / bo).max(initial=0), (np.abs(lse[~empty] - rl[~empty]) / bl[~empty]).max(initial=0)
    assert worst[0] <= 1 and worst[1] <= 1, f"{what}: out {worst[0]:.3f}, lse {worst[1]:.3f} of the bound"


def attention_case(seed, rows, lens, Hq, H, D, ps, window=0, max_q=None, extra=0, pick=None, **kw):
    g = np.random.default_rng(seed)
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]) + extra, Hq, D)) * np.exp(0.5 * g.standard_normal((Hq, D))))
    scale = kw.get("scale", D**-0.5)
    selected = None if pick is None else pick(g, len(q), H)
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, scale, window, selected)
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, max_q or max(rows + [1]), scale, window, selected)
    held_to(out, lse, r, f"{rows} {lens} {Hq}/{H} D{D} ps{ps} w{window}")
    return q, cache, table, kv_len, q_start, out, lse


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


def test_long_contexts_are_split_and_joined():
    say("split")
    attention_case(5, [1, 2, 1], [9000, 4097, 20000], 8, 2, 128, 256)
    attention_case(6, [1], [30001], 4, 1, 64, 512)


@pytest.mark.parametrize("rows,lens", [([64], [64]), ([65, 1], [65, 400]), ([127, 128, 129], [127, 128, 129]),
                                       ([200, 7, 1, 0, 90], [333, 7, 500, 64, 90]), ([260], [700])])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (2, 2, 64), (6, 2, 128)])
def test_prompts(rows, lens, Hq, H, D):
    say("prompts", rows, lens, Hq, H, D)
    attention_case(sum(rows), rows, lens, Hq, H, D, 64)


@pytest.mark.parametrize("rows,lens,Hq,H,D,window", [
    ([700, 690, 1, 0, 40], [1300, 690, 2000, 9, 1500], 64, 1, 128, 0), ([700, 690, 1, 0, 40], [1300, 690, 2000, 9, 1500], 64, 1, 64, 0),
    ([1100], [1229], 64, 2, 128, 0), ([1100], [5000], 64, 2, 64, 500), ([1100, 3], [1229, 5000], 64, 2, 128, 77)])
def test_prompts_of_many_rows(rows, lens, Hq, H, D, window):
    """Enough rows for workgroups of 128 of them; checked on a few rows of each sequence, at the ends and drawn ones."""
    say("many rows", rows, lens, Hq, H, D, window)
    g = np.random.default_rng(sum(rows))
    ps = 64
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    assert int(q_start[-1]) * Hq > 256 * 2 * 4 * 16 // 2
    cache = filled_cache(g, N, ps, H, D)
    poison(cache, table, kv_len, ps, H, D)
    q = bf16(g.standard_normal((int(q_start[-1]) + 1, Hq, D)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, max(rows), window=window)
    assert (out[-1] == 77).all() and (lse[-1] == 77).all()
    for s, n in enumerate(rows):
        for i in sorted({0, n // 2, n - 1, *map(int, g.integers(0, max(n, 1), 6))} if n else ()):
            t = int(q_start[s]) + i
            one = np.array([lens[s] - n + i + 1], dtype=np.int32)
            r = kv8.attention(q[t : t + 1], cache, table[s : s + 1], one, np.array([0, 1]), ps, H, D**-0.5, window)
            held_to(out[t : t + 1], lse[t : t + 1], r, f"sequence {s} row {i}")


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
    attention_case(9, rows, lens, 8, 2, 64, 64, extra=2, pick=lambda g, T, H: g.integers(-1, 3, size=(T, H, 3)).astype(np.int32))


@pytest.mark.parametrize("rows", [1, 100])
def test_bad_pages_are_left_out(rows):
    say("bad pages", rows)
    g = np.random.default_rng(rows)
    H, D, ps = 2, 128, 64
    table, kv_len, q_start, N = batch(g, [rows] * 3, [500, 300, 200], ps)
    table[0, 2], table[0, 3], table[1, 0], table[2, :] = -1, N, 2**31 - 1, -5
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((3 * rows, 8, D)))
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "bad pages")
    sel = np.tile(np.arange(8, dtype=np.int32), (3 * rows, H, 1))
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows, selected=sel), r, "bad pages, all blocks named")


@pytest.mark.parametrize("rows", [1, 90])
def test_a_length_behind_the_table_stops_at_its_end(rows):
    say("behind the table", rows)
    g = np.random.default_rng(rows)
    H, D, ps = 1, 64, 64
    table, kv_len, q_start, N = batch(g, [rows], [200], ps, extra_cols=0)
    cache = filled_cache(g, N, ps, H, D)
    kv_len = np.array([330], dtype=np.int32)
    q = bf16(g.standard_normal((rows, 4, D)))
    r = kv8.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5)
    held_to(*run_attention(q, cache, table, kv_len, q_start, H, ps, rows), r, "behind the table")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-6])
@pytest.mark.parametrize("rows", [1, 40, 1100])
def test_scales(scale, rows):
    say("scale", scale, rows)
    if rows < 1000:
        attention_case(rows, [rows, 1], [300, 64], 4, 2, 128, 64, scale=scale)
        return
    g = np.random.default_rng(1)
    table, kv_len, q_start, N = batch(g, [rows], [rows], 64)
    cache = filled_cache(g, N, 64, 2, 128)
    q = bf16(g.standard_normal((rows, 64, 128)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, 2, 64, rows, scale=scale)
    for t in (0, 500, rows - 1):
        r = kv8.attention(q[t : t + 1], cache, table, np.array([t + 1]), np.array([0, 1]), 64, 2, scale)
        held_to(out[t : t + 1], lse[t : t + 1], r, f"row {t}")


@pytest.mark.parametrize("rows", [1, 1100])
def test_scores_and_values_at_the_ends_of_the_range(rows):
    """The largest values that the cache stores, scores of hundreds of thousands, and queries that are not finite in their own row alone."""
    say("range", rows)
    g = np.random.default_rng(2)
    H, Hq, D, ps, n = 2, 64, 128, 64, max(rows, 700)
    table, kv_len, q_start, N = batch(g, [rows], [n], ps)
    cache = filled_cache(g, N, ps, H, D, 60, 62)
    sc = sections(cache, ps, H, D)[2]
    sc[..., 0], sc[..., 1] = 130, 182
    q = bf16(100 * g.standard_normal((rows, Hq, D)))
    q[0, 3, 5], q[0, 7, 0], q[0, 9, 127] = np.inf, np.nan, -np.inf
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows)
    for t in (0, rows // 2, rows - 1):
        r = kv8.attention(q[t : t + 1], cache, table, np.array([n - rows + t + 1]), np.array([0, 1]), ps, H, D**-0.5)
        bad = np.isin(np.arange(Hq), [3, 7, 9]) if t == 0 else np.zeros(Hq, dtype=bool)
        assert np.isnan(out[t, bad]).all() and np.isnan(lse[t, bad]).all()
        held_to(out[t : t + 1, ~bad], lse[t : t + 1, ~bad], {k: v[:, ~bad] for k, v in r.items()}, f"row {t}")


@pytest.mark.parametrize("D", [64, 128])
def test_a_key_that_is_no_number_in_a_prompt(D):
    """Rows before it, in the same tiles, are what they are without it."""
    say("NaN in a prompt", D)
    g = np.random.default_rng(D)
    H, Hq, ps, rows = 2, 64, 64, 1100
    table, kv_len, q_start, N = batch(g, [rows], [rows], ps)
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((rows, Hq, D)))
    out, lse = run_attention(q, cache, table, kv_len, q_start, H, ps, rows)
    at = 517
    v = sections(cache, ps, H, D)[0]
    v[table[0, at // 64], 0, 0, kv8.places(D)[0][at % 64, 7]] = 255
    out2, lse2 = run_attention(q, cache, table, kv_len, q_start, H, ps, rows)
    first = np.arange(Hq) < Hq // H
    assert np.isnan(out2[at:, first]).all() and np.isnan(lse2[at:, first]).all()
    for a, b in ((out, out2), (lse, lse2)):
        assert (a[:at] == b[:at]).all() and (a[:, ~first] == b[:, ~first]).all()


def test_strided_rows_of_one_projection():
    """q, k and v as slices of one [T, (Hq + 2 H) D] tensor; out and lse with strides of their own."""
    say("strides")
    g = np.random.default_rng(13)
    Hq, H, D, ps, rows, lens = 8, 2, 128, 64, [3, 1, 70], [3, 100, 130]
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    T = int(q_start[-1])
    x = bf16(g.standard_normal((T, Hq + 2 * H, D)))
    xd = dev_bf16(bits(x))
    cache = filled_cache(g, N, ps, H, D)
    cd, want = dev(cache), cache.copy()
    args = dev(table), dev(kv_len), dev(q_start)
    turn = turns(g, table.shape[1] * ps, D)
    q = xd[:, :Hq]
    nm.nm_kv8_append(xd[:, Hq : Hq + H], xd[:, Hq + H :], cd, *args, ps, rotation=dev(turn), q=q, q_out=q)
    kv8.append(want, x[:, Hq : Hq + H], x[:, Hq + H :], table, kv_len, q_start, ps, turn)
    same_bytes(cd, want, ps, H, D, "strides")
    big, wide = torch.zeros((T, 2, Hq, D + 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, 3 * Hq), device="cuda")
    out, lse = big[:, 1, :, :D], wide[:, Hq : 2 * Hq]
    nm.nm_kv8_attention(q, cd, *args, H, ps, 70, out=out, lse=lse)
    a, b = nm.nm_kv8_attention(q.contiguous(), cd, *args, H, ps, 70)
    assert torch.equal(out, a) and torch.equal(lse, b)
    assert (big[:, 0] == 0).all() and (big[..., D:] == 0).all() and (wide[:, :Hq] == 0).all() and (wide[:, 2 * Hq :] == 0).all()
    qr = bf16_as_f64(host_bf16(q.contiguous()))
    r = kv8.attention(qr, want, table, kv_len, q_start, ps, H, D**-0.5)
    held_to(bf16_as_f64(host_bf16(a)), b.cpu().numpy().astype(np.float64), r, "strides")
