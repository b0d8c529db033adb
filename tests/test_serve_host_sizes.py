"""Sizes of the serving calls' workspaces (no GPU)."""
import ctypes

import pytest

from compressed_attention_cvq_b200 import _binding as b


def prefix_bytes(n, **kw):
    d = dict(batch=12, n_q_heads=8, n_kv_heads=2, R=2, t_cap=2100)
    d.update(kw)
    return b.lib.cvq_prefix_workspace_bytes(ctypes.byref(b.make_shape(**d)), n)


@pytest.mark.parametrize("kw,step,ctas", [(dict(R=1), 128, 2), (dict(R=2), 256, 4), (dict(R=5, group_dim=64), 256, 4)])
def test_only_long_splits_keep_sums(kw, step, ctas):
    """Two outputs a row and CTA, only where a split has more than 32 steps of the cluster."""
    kept = 12 * 8 * ctas * 2 * 128 * 4
    short, long = (prefix_bytes(1, t_cap=t, **kw) for t in (32 * step, 32 * step + 64))
    assert long - short == kept
    for n in (2, 7):
        assert prefix_bytes(n, t_cap=n * 32 * step, **kw) - short == 12 * 8 * ctas * (n - 1) * 130 * 4
        assert prefix_bytes(n, t_cap=n * 32 * step + 64, **kw) - prefix_bytes(n, t_cap=n * 32 * step, **kw) == n * kept


def test_the_counters_come_first():
    p = b.cvq_paged(3, 32, 8, 128, 16, 10, 4, b.CVQ_BF16, 500000.0, 0)
    assert b.lib.cvq_paged_workspace_bytes(ctypes.byref(p), 4) == 65536 + 3 * 32 * 4 * 130 * 4
