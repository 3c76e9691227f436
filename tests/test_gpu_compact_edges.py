"""compact_rows at its edges."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b", [1, 2])
def test_from_a_cache_without_rows(dev, b):  # noqa: F811
    """Every entry of kept is out of range: whole rows of zeros."""
    kept = torch.tensor([[0, -1, 3, -1, -1]], dtype=torch.int32, device=dev).repeat(b, 1)
    src = [torch.empty(b, 0, 256, dtype=torch.uint8, device=dev), torch.empty(b, 0, dtype=torch.int64, device=dev),
           torch.empty(b, 0, 5, 7, device=dev)]
    out = [torch.full((b, 6) + t.shape[2:], 9, dtype=t.dtype, device=dev) for t in src]
    sa.compact_rows(src, kept, out=out)
    for o in out:
        assert (o[:, :5] == 0).all() and (o[:, 5] == 9).all()
