"""The selection over clusters of CTAs whose shares, and whose threads' shares, are uneven, many times over."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,rows,keep,kind", [(1, 70001, 30000, "ties"), (19, 65537, 32001, "spread"),
                                              (3, 131073, 999, "ties"), (38, 33003, 20000, "spread")])
def test_the_same_every_time(dev, b, rows, keep, kind):  # noqa: F811
    rng = np.random.default_rng(rows)
    acc = rng.integers(0, 7 if kind == "ties" else 1 << 45, (b, rows))
    want_k, want_r = (torch.from_numpy(a).to(dev) for a in _cache.select(acc, keep, 128, 77))
    acc = torch.from_numpy(acc).to(dev)
    for _ in range(100):
        kept, remap = sa.evict_select(acc, keep, keep_first=128, keep_last=77)
        assert torch.equal(kept, want_k) and torch.equal(remap, want_r)
