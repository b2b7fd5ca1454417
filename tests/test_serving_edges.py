"""The serving calls without a GPU, beyond test_serving.py: workspace sizes of long tails."""

from __future__ import annotations

import pytest

from random_rotation_kv_b200 import binding as B


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("batch,hq,hkv,prefix", [(1, 32, 8, 0), (64, 64, 8, 0), (4, 8, 8, 1000)])
def test_shared_attention_workspace_is_bounded_in_tail_cap(d, batch, hq, hkv, prefix):
    """A unit of work leaves at most one state per range, however long the tails may be."""
    ws = B.rrq_attention_shared_workspace_bytes
    most = 148 + -(-prefix // 64)  # ranges without a GPU, and a state per tile of the prefix
    rows = batch * hq
    for cap in (1 << 14, 1 << 17, 1 << 20):
        size = ws(batch, hq, hkv, d, prefix, cap)
        assert 0 < size <= most * rows * (4 * d + 8) + rows * (4 * d + 4) + 64 * (batch * hkv + 300) + 4096, (cap, size)
    assert ws(batch, hq, hkv, d, prefix, 1 << 21) == ws(batch, hq, hkv, d, prefix, 1 << 20)
