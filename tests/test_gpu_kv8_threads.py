"""The choice of blocks of the 8-bit cache by several host threads at once."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

from oracle import kv8
from tests.gpu_util import dev_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import filled_cache

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.test_gpu_kv8 import dev  # noqa: E402


@pytest.mark.parametrize("D", [64, 128])
def test_tables_of_several_widths_at_once(D):
    """Rows by sixteens: their scores' room in LDS goes by the table's width, and is asked of the runtime for the kernel, not for a call."""
    say("threads", D)
    g = np.random.default_rng(D)
    H, ps, rows, top = 8, 512, 300, 9
    table, kv_len, q_start, N = batch(g, [rows], [20000], ps)
    cache, q = filled_cache(g, N, ps, H, D), bf16(g.standard_normal((rows, H, D)))
    want = kv8.select(q[:4], cache, table, kv_len - rows + 4, np.array([0, 4], dtype=np.int32), ps, H, top, 1, 1)
    cd, qd = dev(cache), dev_bf16(bits(q))
    tables = [np.pad(table, ((0, 0), (0, cols - table.shape[1])), constant_values=-1) for cols in (1024 * 64 // ps, 60, 600 * 64 // ps)]
    args = [(qd, cd, dev(t), dev(kv_len), dev(q_start), H, ps, top) for t in tables]
    torch.cuda.synchronize()
    lost = []

    def work(a):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [nm.nm_kv8_select(*a) for _ in range(100)]
                torch.cuda.current_stream().synchronize()
            x = got[0].cpu().numpy()
            if not all(torch.equal(got[0], y) for y in got) or (x[:4] != want).any():
                lost.append("another choice")
        except Exception as e:  # a launch that is refused
            lost.append(e)
    threads = [threading.Thread(target=work, args=(a,)) for a in args * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not lost, lost[0]
