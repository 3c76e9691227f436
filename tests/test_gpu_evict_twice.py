"""A cache of fixed size over a long generation: evicted in place twice, with rows appended in between."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache
from tests.test_gpu_cache import check, dev  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp4", "fp8", "bf16"])
def test_evicted_twice_with_rows_appended(dev, fmt):  # noqa: F811
    """Rows are told apart by when they were appended; the weights of each are added up in 64 bits.  The rows that
    an eviction frees are used again, with accumulators that start at 0, and an index table and a map of all rows
    ever appended follow both evictions."""
    b, h, d, cap, keep, more = 3, 64, 512, 500, 200, 250
    scale = d ** -0.5
    g = torch.Generator(device=dev).manual_seed(4)
    width = {"fp4": d // 2, "fp8": d, "bf16": d}[fmt]
    kv = torch.zeros(b, cap, width, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device=dev)
    sc = None if fmt == "bf16" else torch.zeros(b, cap, d // 32, dtype=torch.uint8, device=dev)
    acc = torch.zeros(b, cap, dtype=torch.int64, device=dev)
    sink = torch.randn(h, device=dev, generator=g)
    name = torch.full((b, cap), -1, dtype=torch.int32, device=dev)  # which row is where
    n_names = 0
    weight = torch.zeros(b, 2000, dtype=torch.float64, device=dev)  # by name
    room = torch.zeros_like(weight)
    where = torch.empty(b, 0, dtype=torch.int32, device=dev)  # a name's row, -1 once it is gone
    live = 0

    def append(n):
        nonlocal n_names, live, where
        x = torch.randn(b, n, d, device=dev, generator=g).to(torch.bfloat16)
        at = slice(live, live + n)
        if fmt == "bf16":
            kv[:, at] = x
        else:
            quant = sa.act_quant_fp4 if fmt == "fp4" else sa.act_quant_fp8
            for bi in range(b):
                quant(x[bi], codes=kv[bi, at], scales=sc[bi, at])
        name[:, at] = torch.arange(n_names, n_names + n, device=dev, dtype=torch.int32)
        new = torch.arange(live, live + n, device=dev, dtype=torch.int32).expand(b, n)
        where = torch.cat([where, new], 1)
        n_names, live = n_names + n, live + n

    def attend():
        q = torch.randn(b, 2, h, d, device=dev, generator=g).to(torch.bfloat16)
        idx = torch.rand(b, 2, live, device=dev, generator=g).argsort(-1)[..., :130].to(torch.int32)
        lse = torch.empty(b, 2, h, device=dev)
        o = sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc, lse=lse)
        sa.row_weights(q, kv, lse, idx, scale, acc, kv_scale=sc)
        kv64 = _cache.rows_f64(kv, sc, d)
        want, _, tol, _ = _cache.attention(q, kv64, sink, idx, scale)
        check(o, want, tol, "o")
        w, t = _cache.row_weights(q, kv64, lse, idx, scale)
        weight.scatter_add_(1, name[:, :live].long(), w[:, :live])
        room.scatter_add_(1, name[:, :live].long(), t[:, :live])
        return idx

    append(450)
    for _ in range(2):
        for _ in range(3):
            idx = attend()
        names = name.gather(1, idx.long().view(b, -1))
        have = torch.full((b,), live, dtype=torch.int32, device=dev)
        kept, remap = sa.evict_select(acc, keep, keep_first=8, keep_last=16, live=have)
        tensors = [t for t in (kv, sc, acc, name) if t is not None]
        sa.compact_rows(tensors, kept, out=tensors)
        acc[:, keep:] = 0  # these rows are used again
        where = sa.remap_idx(where, remap)
        idx = sa.remap_idx(idx, remap).view(b, -1)
        live = keep
        # the tables agree with where the rows went
        stays = idx >= 0
        assert stays.any() and not stays.all()
        assert torch.equal(name.gather(1, idx.clamp(min=0).long())[stays], names[stays])
        assert torch.equal(where.gather(1, name[:, :live].long()),
                           torch.arange(live, device=dev, dtype=torch.int32).expand(b, live))
        assert (where >= 0).sum() == b * live
        append(more)
    attend()
    # every row's weight is its own
    at = name[:, :live].long()
    check(acc[:, :live].double() * sa.WEIGHT_UNIT, weight.gather(1, at), room.gather(1, at), "weights")
