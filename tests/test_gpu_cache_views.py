"""Operators on parts of larger buffers: a later sequence of a packed cache."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests.test_gpu_cache import dev, inputs  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128, 192, 256, 384, 448, 512])
def test_row_weights_of_a_later_sequence(dev, fmt, d):  # noqa: F811
    """A sequence of a cache with an odd number of rows, as a view: what a copy of it gives."""
    q, kv, sc, sink, idx = inputs(dev, fmt, 4, 3, 20, d, 91, 70, d)
    lse = torch.empty(4, 3, 20, device=dev)
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse)
    got = torch.zeros(4, 91, dtype=torch.int64, device=dev)
    want = torch.zeros_like(got)
    for i in range(4):
        view = [t[i:i + 1] for t in (q, kv, lse, idx, sc)]
        copy = [t.clone() for t in view]
        sa.row_weights(*view[:4], d ** -0.5, got[i:i + 1], kv_scale=view[4])
        sa.row_weights(*copy[:4], d ** -0.5, want[i:i + 1], kv_scale=copy[4])
    assert torch.equal(got, want) and (want != 0).any()
