"""The plain definitions of the 4-bit cache (oracle/kv4.py) against closed forms and small cases by hand."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import kv4
from tests.kv4_util import bf16, four_pieces


def test_every_place_of_a_block_is_used_once():
    for ps in (64, 128, 256, 512):
        for D in (64, 128):
            seen = np.zeros(kv4.page_bytes(ps, 1, D), dtype=int)
            for values in (False, True):
                at, sc = kv4.places(ps, D, values)
                np.add.at(seen, at[:, ::2].reshape(-1), 1)
                assert (at[:, ::2] == at[:, 1::2]).all()
                np.add.at(seen, sc.reshape(-1), 1)
            assert (seen == 1).all()


def test_multiples_of_a_scale_are_kept_exactly():
    g = np.random.default_rng(0)
    x = kv4.E2M1[g.integers(0, 8, size=(50, 32))] * g.choice([-1.0, 1.0], size=(50, 32))
    x[:, 0] = 6.0
    for e in (-100, -7, 0, 30, 120):
        y = x * 2.0**e
        assert (kv4.dequantize(*kv4.quantize(y)) == y).all()


def test_a_value_is_off_by_at_most_one_unit():
    g = np.random.default_rng(1)
    x = bf16(g.standard_normal((200, 64)) * np.exp(g.standard_normal((200, 64))))
    code, byte = kv4.quantize(x)
    unit = np.repeat(np.exp2(byte - 127.0), 32, -1)
    assert (np.abs(kv4.dequantize(code, byte) - x) <= unit).all()


def test_ties_ends_and_zero():
    x = np.zeros((1, 32))
    x[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 7, -7]
    code, byte = kv4.quantize(x)
    assert byte[0, 0] == 127
    assert list(kv4.dequantize(code, byte)[0, :12]) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, 6, -6]
    code, byte = kv4.quantize(np.zeros((1, 32)))
    assert byte[0, 0] == 16 and (code == 0).all()
    top = np.full((1, 32), bf16(3.3895e38))
    code, byte = kv4.quantize(top)
    assert byte[0, 0] == 252 and np.isfinite(kv4.dequantize(code, byte).astype(np.float32)).all()


@pytest.mark.parametrize("window", [0, 1, 3])
def test_equal_keys_average_the_values(window):
    H, D, ps, n = 1, 64, 64, 5
    cache = np.zeros((1, kv4.page_bytes(ps, H, D)), dtype=np.uint8)
    v = np.zeros((n, H, D))
    v[:, 0] = np.array([1.0, 2.0, 3.0, 4.0, 6.0])[:, None]
    table, kv_len, q_start = np.zeros((1, 1), np.int32), np.array([n], np.int32), np.array([0, n], np.int32)
    kv4.append(cache, np.zeros((n, H, D)), v, table, kv_len, q_start, ps)
    r = kv4.attention(np.ones((n, 1, D)), cache, table, kv_len, q_start, ps, 1, 0.5, window)
    for i in range(n):
        first = max(0, i - window + 1) if window else 0
        assert np.allclose(r["out"][i, 0], v[first : i + 1, 0].mean(0), atol=1e-14)
        assert np.isclose(r["lse"][i, 0], np.log(i + 1 - first))


def test_pages_by_hand():
    table = np.array([[0, 1, -1, -1], [0, 2, 5, -1], [-1, -1, -1, -1]], dtype=np.int32)
    kv_len, refs = np.array([100, 192, 0], np.int32), np.array([2, 1, 1, 0, 0, 1, 0, 0], np.int32)
    moves, missing = kv4.fork([0], [2], table, kv_len, refs, 64)  # page 0 shared, page 1 (36 tokens) copied to 3
    assert list(table[2]) == [0, 3, -1, -1] and kv_len[2] == 100 and missing == 0
    assert moves.tolist() == [[1, 3]] and list(refs) == [3, 1, 1, 1, 0, 1, 0, 0]
    moves, missing = kv4.resize([64, 193, 100], table, kv_len, refs, 64)  # page 1 back, and out again
    assert list(table[0]) == [0, -1, -1, -1] and list(table[1]) == [0, 2, 5, 1] and missing == 0
    assert list(refs) == [3, 1, 1, 1, 0, 1, 0, 0] and (moves == -1).all()
    moves, missing = kv4.resize([65, 0, 400], table, kv_len, refs, 64)  # 400 tokens do not fit in four columns
    assert list(kv_len) == [65, 0, 100] and list(table[0]) == [0, 1, -1, -1] and list(refs) == [2, 1, 0, 1, 0, 0, 0, 0]
    moves, used = kv4.compact(table, kv_len, refs, 64, 4)
    assert used == 3 and moves.tolist() == [[3, 2], [-1, -1], [-1, -1], [-1, -1]]
    assert list(table[2]) == [0, 2, -1, -1] and list(refs) == [2, 1, 1, 0, 0, 0, 0, 0]


def test_growth_in_a_shared_page_takes_a_page_of_its_own():
    table, kv_len = np.array([[3, -1], [3, -1]], np.int32), np.array([10, 10], np.int32)
    refs = np.array([0, 0, 0, 2], np.int32)
    moves, missing = kv4.resize([11, 10], table, kv_len, refs, 64)
    assert table.tolist() == [[0, -1], [3, -1]] and moves.tolist() == [[3, 0], [-1, -1]] and list(refs) == [1, 0, 0, 1]


def test_a_pool_that_runs_out_serves_the_first():
    table, kv_len, refs = np.full((3, 2), -1, np.int32), np.zeros(3, np.int32), np.zeros(2, np.int32)
    moves, missing = kv4.resize([64, 100, 5], table, kv_len, refs, 64)
    assert missing == 2 and list(kv_len) == [64, 0, 0] and list(refs) == [1, 0]


def test_four_pieces_hold_every_query_number():
    """Every bf16 number of a block whose largest magnitude is in [1, 2), down to where all of it is below the bound."""
    q = np.concatenate([np.arange(128, 256) / 128.0 * 2.0**-d for d in range(40)])
    assert np.abs(four_pieces(q)).max() <= 2.0**-20
    assert (four_pieces(q[: 128 * 9]) == 0).all()  # within 2^-8 of the largest nothing is lost
