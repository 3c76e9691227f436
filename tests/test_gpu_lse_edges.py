"""The log-sum-exp output at its edges."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache
from tests.test_gpu_cache import check, dev, inputs  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,s,topk", [(512, 40, 130), (512, 1, 1200), (512, 3, 0), (256, 3, 70), (256, 1, 700)])
def test_a_sink_past_every_logit(dev, d, s, topk):  # noqa: F811
    """An infinite sink, and finite ones whose logarithm to base 2 is past f32: o = 0 and lse = the sink
    (unsplit, split and without columns, both kernel families).  A NaN logit under one is NaN."""
    q, kv, _, sink, idx = inputs(dev, "bf16", 1, s, 16, d, 1500, topk, 7)
    sink[3], sink[7], sink[9], sink[11] = torch.inf, 3e38, -3e38, -torch.inf
    lse = torch.empty(1, s, 16, device=dev)
    o = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, lse=lse)
    if topk:
        _, want, _, tol = _cache.attention(q, _cache.rows_f64(kv, None, d), sink, idx, d ** -0.5)
        check(lse, want, tol, "lse")
    else:
        assert (lse == sink).all()
    assert (o[:, :, [3, 7]] == 0).all() and (lse[:, :, 3] == torch.inf).all()
    if topk:
        idx[0, s - 1] = torch.arange(topk, device=dev, dtype=torch.int32)
        q[0, s - 1, 3, 5] = torch.nan
        sa.sparse_attn(q, kv, sink, idx, d ** -0.5, lse=lse)
        assert lse[0, s - 1, 3].isnan() and not lse[0, s - 1, 4:].isnan().any()
