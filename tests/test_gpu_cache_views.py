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


@pytest.mark.parametrize("n,d,width,at", [(300, 512, 272, 0), (37, 64, 37, 3), (5000, 96, 64, 8), (2, 32, 17, 0)])
def test_act_quant_fp4_into_packed_rows(dev, n, d, width, at):  # noqa: F811
    """Codes and scales of a row side by side in one buffer, and everything of a row in one."""
    g = torch.Generator(device=dev).manual_seed(n)
    x = torch.randn(n, d, device=dev, generator=g).to(torch.bfloat16)
    codes = torch.empty(n, d // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(n, d // 32, dtype=torch.uint8, device=dev)
    rt = torch.empty_like(x)
    sa.act_quant_fp4(x, codes=codes, scales=scales, out_rt=rt)
    c, s = slice(at, at + d // 2), slice(at + d // 2, at + d // 2 + d // 32)
    buf = torch.full((n, width), 0xAB, dtype=torch.uint8, device=dev)
    sa.act_quant_fp4(x, codes=buf[:, c], scales=buf[:, s])
    assert torch.equal(buf[:, c], codes) and torch.equal(buf[:, s], scales)
    assert (buf[:, :at] == 0xAB).all() and (buf[:, s.stop:] == 0xAB).all()
    # x, its round trip, codes and scales, 16 bytes between them
    wide = torch.full((n, 5 * d + 64), 0xAB, dtype=torch.uint8, device=dev)
    row = wide.view(torch.bfloat16)
    row[:, :d] = x
    c = slice(4 * d + 32, 4 * d + 32 + d // 2)
    s = slice(c.stop, c.stop + d // 32)
    sa.act_quant_fp4(row[:, :d], out_rt=row[:, d + 8:2 * d + 8], codes=wide[:, c], scales=wide[:, s])
    assert torch.equal(row[:, :d], x) and torch.equal(row[:, d + 8:2 * d + 8], rt)
    assert torch.equal(wide[:, c], codes) and torch.equal(wide[:, s], scales)
    for gap in (slice(2 * d, 2 * d + 16), slice(4 * d + 16, c.start), slice(s.stop, None)):
        assert (wide[:, gap] == 0xAB).all()
