"""Arguments of the 4-bit cache at the ends of their ranges (no GPU needed)."""
from __future__ import annotations

import pytest

from tests.test_abi_kv4_host import L, SHAPE, call  # noqa: F401


@pytest.mark.parametrize("scale", [2.0**126, -(2.0**126), 3.0e38])
def test_a_scale_whose_scores_pass_fp32_is_refused(L, scale):  # noqa: F811
    assert call(L, "nm_kv4_attention", scale=scale) == SHAPE
