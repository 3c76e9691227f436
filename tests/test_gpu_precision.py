"""How far the softmax statistics and the weights are off on ordinary inputs, in the root mean square: bounds
that sums or statistics held in fewer than 32 bits would break, where the worst-case bounds of the other
tests would not see them."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache
from tests.test_gpu_cache import dev, inputs  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23  # of f32


def rms(x):
    return float(x.double().square().mean().sqrt())


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("b,s,h,d,rows,topk", [(1, 64, 64, 512, 2000, 640), (4, 1, 64, 512, 2000, 1152),
                                               (1, 40, 128, 512, 900, 130), (1, 40, 64, 256, 900, 320),
                                               (2, 30, 32, 64, 900, 320)])
def test_statistics_are_f32(dev, fmt, b, s, h, d, rows, topk):  # noqa: F811
    """Logits of unit size.  A logit's products are added up with a rounding or a cut of partial sums of about its
    own size: the products' are as often up as down (sqrt(d) steps together), those of the partial sums,
    16 products apart, may all go one way (d / 16).  An exponential takes its argument and its result in f32 (at
    most 4 steps of arguments up to |l| + |lse|, 8 of results), a denominator's additions sqrt(topk), a logarithm
    2 and its result one of |lse|.  (Probabilities rounded to bf16 before they are summed would be off by 2^-9 / sqrt(3) each,
    over an effective topk / e of them: 7e-5 at 640, five times the bound.)"""
    q, kv, sc, sink, idx = inputs(dev, fmt, b, s, h, d, rows, topk, 3 * d + s)
    scale = d ** -0.5
    lse = torch.empty(b, s, h, device=dev)
    sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc, lse=lse)
    kv64 = _cache.rows_f64(kv, sc, d)
    l, _, _, seen = _cache.logits(q, kv64, idx, scale)
    l = torch.where(seen, l, -torch.inf)
    want = torch.logsumexp(torch.cat([l, sink.double().expand(b, s, h)[..., None]], -1), -1)
    size = float(want.abs().mean()) + 1.0
    dot = d ** 0.5 + d / 16
    assert rms(lse - want) < STEP * (dot + 4 * size + 8 + topk ** 0.5 + 2 + size)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, idx, scale, acc, kv_scale=sc)
    w, _ = _cache.row_weights(q, kv64, lse, idx, scale)
    there = w > 0
    off = (acc.double() * sa.WEIGHT_UNIT - w)[there] / w[there]
    # (the sum over heads: sqrt(h); the rounding to multiples of 2^-32 is far below)
    assert rms(off) < STEP * (dot + 4 * size + 8 + h ** 0.5)
