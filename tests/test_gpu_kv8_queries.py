"""Queries rotated on the way into the 8-bit cache: the nearest bf16 number to the rotation in 64 bits, as keys are rounded once too."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import turns

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.test_gpu_kv8 import dev  # noqa: E402


def nearest_bf16(x):
    """fp64 -> bf16, ties to even, as fp64 (normal numbers and 0)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def rotated(q, turn, interleaved, rows, lens, ps=128, H=2):
    g = np.random.default_rng(0)
    T, heads, D = q.shape
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    k = dev_bf16(bits(bf16(g.standard_normal((T, H, D)))))
    cache = torch.zeros((N, kv8.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda")
    got = nm.nm_kv8_append(k, k, cache, dev(table), dev(kv_len), dev(q_start), ps, rotation=dev(turn), interleaved=interleaved, q=dev_bf16(bits(q)))
    want = np.concatenate([np.stack([kv8.rotate(q[int(q_start[s]) + i], lens[s] - n + i, turn, interleaved) for i in range(n)]) for s, n in enumerate(rows) if n])
    return bf16_as_f64(host_bf16(got)), nearest_bf16(want)


@pytest.mark.parametrize("D,rotary,interleaved,heads", [(128, 128, False, 8), (128, 64, True, 6), (64, 16, False, 4), (64, 64, True, 24), (128, 128, True, 40)])
@pytest.mark.parametrize("rows,lens", [([1, 1, 1, 1, 1], [1, 64, 65, 700, 129]), ([300, 7], [300, 260])])
def test_queries_are_rounded_once(rows, lens, D, rotary, interleaved, heads):
    say("queries", rows, D, rotary, interleaved, heads)
    g = np.random.default_rng(heads)
    turn = turns(g, 128 * 7, rotary)
    got, want = rotated(bf16(g.standard_normal((sum(rows), heads, D)) * np.exp(3 * g.standard_normal((heads, D)))), turn, interleaved, rows, lens)
    assert (got == want).all()


@pytest.mark.parametrize("D,interleaved", [(64, False), (64, True), (128, False), (128, True)])
def test_queries_next_to_ties(D, interleaved):
    """Odd numbers of 8 bits, one and a half times each lies halfway between two bf16 numbers, and a second product far below fp32's last bit
    that says which is nearer."""
    say("queries, ties", D, interleaved)
    g = np.random.default_rng(D)
    rows = lens = [90]
    turn = np.empty((256, D // 2, 2), dtype=np.float32)
    turn[..., 0], turn[..., 1] = 1.5, g.choice([1e-9, -1e-9, 1e-12, 0.0], size=turn.shape[:2])
    q = (2 * g.integers(64, 85, size=(90, 4, D)) + 1) * 2.0 ** g.integers(-3, 3, size=(90, 1, 1)) * g.choice([1, -1], size=(90, 4, D))
    got, want = rotated(q.astype(np.float64), turn, interleaved, rows, lens)
    assert (got == want).all()
