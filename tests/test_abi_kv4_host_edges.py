"""Arguments of the 4-bit cache at the ends of their ranges (no GPU needed)."""
from __future__ import annotations

import contextlib
import os

import pytest

from tests.test_abi_kv4_host import HIP, L, OK, SHAPE, call  # noqa: F401


@pytest.mark.parametrize("scale", [2.0**126, -(2.0**126), 3.0e38])
def test_a_scale_whose_scores_pass_fp32_is_refused(L, scale):  # noqa: F811
    assert call(L, "nm_kv4_attention", scale=scale) == SHAPE


def test_no_sequences_have_no_arrays(L):  # noqa: F811
    """An array of no elements may have no address: the table's and the lengths' of no sequences."""
    for name in ("nm_kv4_append", "nm_kv4_unpack", "nm_kv4_attention"):
        assert call(L, name, S=0, T=0, page_table=None, kv_len=None) == OK, name
        assert call(L, name, S=0, T=1, page_table=None, kv_len=None) == SHAPE, name


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="would be launched, with addresses that are none")
def test_any_hint_reaches_the_launch(L):  # noqa: F811
    """As many rows as the type holds: with no device to launch on, that is all that is wrong."""
    for hint in ((1 << 63) - 1, 1 << 61, 1 << 40):
        assert call(L, "nm_kv4_attention", max_q_len=hint) == HIP


def test_workspace_sizes_are_asked_on_the_device_of_the_call(monkeypatch):
    """Two devices of different size: what a call on the second needs is not what the current one would."""
    import bitmask_spmv_amd as nm

    at = [0]

    class Library:
        def nm_kv4_attention_workspace_bytes(self, *sizes):
            return 1000 + at[0]

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d
        yield
        at[0] = before

    monkeypatch.setattr(nm, "lib", Library())
    monkeypatch.setattr(nm, "_current_device", lambda: at[0])
    monkeypatch.setattr(nm.torch.cuda, "device", device)
    nm._attention_workspace.cache_clear()
    try:
        sizes = (5, 3, 8, 2, 128, 1, 4096)
        for d in (1, 0, 1):
            assert nm._attention_workspace(d, *sizes) == 1000 + d
            assert at == [0]
    finally:
        nm._attention_workspace.cache_clear()
