"""The plain definitions of the 8-bit cache (oracle/kv8.py) against closed forms and small cases by hand."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.kv4_util import bf16


def test_every_place_of_a_block_is_used_once():
    for D in (64, 128):
        seen = np.zeros(128 * D, dtype=int)
        for at in kv8.places(D):
            np.add.at(seen, at.reshape(-1), 1)
        assert (seen == 1).all()
        for ps, H in ((64, 1), (128, 3), (512, 8)):
            parts = [[], [], []]
            for h in range(H):
                for b in range(ps // 64):
                    for part, at, n in zip(parts, kv8.offsets(ps, H, D, h, b), (128 * D, 2 * D, 4)):
                        part += range(at, at + n)
            at = np.concatenate(parts)
            assert len(set(at)) == len(at) == at.max() + 1 <= kv8.page_bytes(ps, H, D) < at.max() + 129


def test_codes_are_the_type_torch_has():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(kv8.decode(codes.numpy()), codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    g = np.random.default_rng(0)
    x = np.clip(bf16(g.standard_normal(20000) * np.exp(3 * g.standard_normal(20000))), -448, 448)
    assert (kv8.encode(x) == torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()).all()


def test_ties_ends_and_zero():
    # 17/16 lies halfway between 1 and 9/8, 19/16 between 9/8 and 10/8: to the even codes; half of the smallest number to 0
    x = np.array([1.0, 17 / 16, 19 / 16, 21 / 16, 448.0, 500.0, -464.0, 2.0**-9, 2.0**-10, 1.5 * 2.0**-9, 0.0, -0.0])
    assert list(kv8.decode(kv8.encode(x))) == [1.0, 1.0, 1.25, 1.25, 448.0, 448.0, -448.0, 2.0**-9, 0.0, 2.0**-8, 0.0, 0.0]
    assert kv8.encode(np.array([np.nan]))[0] == kv8.NAN
    for top, byte in ((448.0, 127), (449.0, 128), (224.0, 126), (224.5, 127), (1.75 * 2.0**-3, 116), (0.0, 63), (2.0**-100, 63), (3e38, 182)):
        assert kv8.scale_byte(top) == byte


def one_page(H, D, n, before=0):
    return (np.zeros((1, kv8.page_bytes(64, H, D)), dtype=np.uint8), np.zeros((1, 1), np.int32), np.array([before + n], np.int32),
            np.array([0, n], np.int32))


def test_a_block_that_grows_louder_keeps_its_tokens():
    """Scales are powers of two: the earlier tokens come through a larger one unchanged while they stay normal numbers."""
    g = np.random.default_rng(1)
    H, D = 2, 64
    cache, table, _, _ = one_page(H, D, 1)
    k = kv8.decode(kv8.encode(g.uniform(1, 400, size=(3, H, D)) * g.choice([-1, 1], size=(3, H, D))))
    k[:, :, 0] = 448.0
    for i, f in enumerate((1.0, 16.0, 64.0)):
        kv8.append(cache, k[i : i + 1] * f, k[i : i + 1] * f, table, np.array([i + 1]), np.array([0, 1]), 64)
    K, V, b = kv8.unpack_pages(cache, 64, H, D)
    want = k * np.array([1.0, 16.0, 64.0])[:, None, None]
    assert (K[0, :, :3].transpose(1, 0, 2) == want).all() and (V[0, :, :3].transpose(1, 0, 2) == want).all()
    assert (b[0, :, 0, 0] == want.max(0)).all() and (b[0, :, 0, 1] == want.min(0)).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    g = np.random.default_rng(2)
    D, P = 64, 16
    x, angle = g.standard_normal((3, D)), g.uniform(0, 6, size=(5, P))
    turn = np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
    y = kv8.rotate(x, 4, turn, interleaved)
    z = x[:, : 2 * P].reshape(3, P, 2) if interleaved else x[:, : 2 * P].reshape(3, 2, P).transpose(0, 2, 1)
    w = (z[..., 0] + 1j * z[..., 1]) * (turn[4, :, 0].astype(float) + 1j * turn[4, :, 1])
    u = y[:, : 2 * P].reshape(3, P, 2) if interleaved else y[:, : 2 * P].reshape(3, 2, P).transpose(0, 2, 1)
    assert np.allclose(u[..., 0], w.real, atol=1e-15) and np.allclose(u[..., 1], w.imag, atol=1e-15)
    assert (y[:, 2 * P :] == x[:, 2 * P :]).all()


def test_equal_keys_average_the_values():
    H, D, n = 1, 64, 5
    cache, table, kv_len, q_start = one_page(H, D, n)
    v = np.zeros((n, H, D))
    v[:, 0] = np.array([1.0, 2.0, 3.0, 4.0, 6.0])[:, None]
    kv8.append(cache, np.zeros((n, H, D)), v, table, kv_len, q_start, 64)
    r = kv8.attention(np.ones((n, 2, D)), cache, table, kv_len, q_start, 64, H, 0.1)
    assert np.allclose(r["out"][:, 0, 0], [1, 1.5, 2, 2.5, 3.2]) and np.allclose(r["lse"][:, 1], np.log(np.arange(1, 6)))
    r = kv8.attention(np.ones((n, 2, D)), cache, table, kv_len, q_start, 64, H, 0.1, selected=np.array([[[0, -1]]] * 4 + [[[1, -1]]]))
    assert np.allclose(r["out"][:, 0, 0], [1, 1.5, 2, 2.5, 0]) and r["lse"][4, 0] == -np.inf


def test_no_key_beats_the_bound_of_its_block():
    g = np.random.default_rng(4)
    H, D, n = 1, 64, 200
    cache = np.zeros((4, kv8.page_bytes(64, H, D)), dtype=np.uint8)
    table, kv_len, q_start = np.arange(4, dtype=np.int32)[None], np.array([n]), np.array([0, n])
    k = bf16(g.standard_normal((n, H, D)))
    kv8.append(cache, k, k, table, kv_len, q_start, 64)
    K, _, b = kv8.unpack_pages(cache, 64, H, D)
    q = bf16(g.standard_normal((n, 2, D)))
    bound = np.array([[np.maximum(q[-1, h] * b[p, 0, 0, 0], q[-1, h] * b[p, 0, 0, 1]).sum() for p in range(4)] for h in range(2)]).sum(0)
    score = (K[:, 0] @ q[-1].T).sum(-1)
    score[3, n - 192 :] = -np.inf  # no tokens there
    assert (score.max(1) <= bound).all()
    sel = kv8.select(q, cache, table, kv_len, q_start, 64, H, 2, 0, 0)
    assert sorted(np.argsort(-bound, kind="stable")[:2]) == list(sel[-1, 0])
    assert (sel[0, 0] == [0, -1]).all() and (kv8.select(q, cache, table, kv_len, q_start, 64, H, 2, 1, 1)[-1, 0] == [0, 3]).all()
