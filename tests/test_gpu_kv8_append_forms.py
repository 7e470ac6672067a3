"""The 8-bit cache's append at every number of new tokens of a block, on the GPU against oracle/kv8.py, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import dev_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import turns

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.test_gpu_kv8 import dev, same_bytes  # noqa: E402


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_any_number_of_new_tokens(tokens, D, interleaved):
    """From every kind of place in a block, into the next one too; scales that stay and that grow; numbers that are none."""
    g = np.random.default_rng(tokens * D + interleaved)
    H, ps = 2, 128
    for before in sorted({0, 1, (64 - tokens) // 2, 64 - tokens, 63}):
        for loud in (0.1, 50.0):
            say("new tokens", tokens, D, interleaved, before, loud)
            rows = [before + 3, tokens]
            table, _, _, N = batch(g, rows, [before + 3, before + tokens], ps)
            turn = turns(g, table.shape[1] * ps, D // 2)
            want = g.integers(0, 256, size=(N, kv8.page_bytes(ps, H, D)), dtype=np.uint8)
            cache = dev(want)
            for n, lens, size in (([before + 3, before], [before + 3, before], 1.0), ([0, tokens], [before + 3, before + tokens], loud)):
                q_start, kv_len = np.concatenate([[0], np.cumsum(n)]).astype(np.int32), np.array(lens, dtype=np.int32)
                T = int(q_start[-1])
                k, v = (bf16(size * g.standard_normal((T, H, D)) * np.exp(g.standard_normal((T, H, D)))) for _ in range(2))
                k[T // 2, 0, 3], v[T - 1, 1, D - 1], v[T // 3, 0, 0] = np.inf, np.nan, -np.inf
                nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cache, dev(table), dev(kv_len), dev(q_start), ps, rotation=dev(turn),
                                 interleaved=interleaved)
                kv8.append(want, k, v, table, kv_len, q_start, ps, turn, interleaved)
            same_bytes(cache, want, ps, H, D, f"{before} and {tokens}")
