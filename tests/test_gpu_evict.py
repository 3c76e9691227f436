"""Row weights and eviction on the GPU against plain 64-bit implementations, and the run of the whole:
write, attend, weigh, evict, attend again."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache
from tests.test_gpu_cache import CASES, check, dev, far_inputs, inputs  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


def _close(acc, q, kv, sc, lse, idx, scale, before=0):
    want, tol = _cache.row_weights(q, _cache.rows_f64(kv, sc, q.shape[-1]), lse, idx, scale)
    check((acc - before).double() * sa.WEIGHT_UNIT, want, tol, "weights")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}s{c[1]}h{c[2]}d{c[3]}k{c[5]}")
def test_row_weights(dev, case, fmt):  # noqa: F811
    b, s, h, d, rows, topk, extra = case
    empty = (b * s - 1,) if b * s > 1 else ()
    q, kv, sc, sink, idx = inputs(dev, fmt, b, s, h, d, rows, topk, 13 * b + s, empty=empty, **extra)
    lse = torch.empty(b, s, h, device=dev)
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, idx, d ** -0.5, acc, kv_scale=sc, workspace=ws)
    assert sa.read_status(ws) == 0
    _close(acc, q, kv, sc, lse, idx, d ** -0.5)
    # added to what is there, the same every time
    again = torch.arange(b * rows, device=dev).view(b, rows) << 33
    start = again.clone()
    sa.row_weights(q, kv, lse, idx, d ** -0.5, again, kv_scale=sc)
    assert torch.equal(again - start, acc)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("h,d,topk", [(128, 512, 1), (100, 512, 64), (128, 448, 130), (65, 384, 2), (128, 320, 200),
                                      (128, 256, 64), (64, 512, 1), (33, 384, 130)])
def test_row_weights_many_short_queries(dev, h, d, topk, fmt):  # noqa: F811
    """Several queries a CTA, one or two tiles each: every stage and every part of q is used again and
    again.  The same every time."""
    b, s, rows = 17, 40, 128
    q, kv, sc, sink, idx = inputs(dev, fmt, b, s, h, d, rows, topk, h + d + topk, distinct=topk <= rows)
    lse = torch.empty(b, s, h, device=dev)
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, idx, d ** -0.5, acc, kv_scale=sc)
    _close(acc, q, kv, sc, lse, idx, d ** -0.5)
    for _ in range(20):
        again = torch.zeros_like(acc)
        sa.row_weights(q, kv, lse, idx, d ** -0.5, again, kv_scale=sc)
        assert torch.equal(again, acc)


def test_row_weights_negative_scale_and_special_lse(dev):  # noqa: F811
    q, kv, sc, sink, idx = inputs(dev, "fp4", 1, 6, 16, 512, 200, 150, 3)
    lse = torch.full((1, 6, 16), 4.0, device=dev)
    acc = torch.zeros(1, 200, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, idx, -0.04, acc, kv_scale=sc)
    _close(acc, q, kv, sc, lse, idx, -0.04)
    acc.zero_()
    sa.row_weights(q, kv, torch.full_like(lse, torch.inf), idx, 0.04, acc, kv_scale=sc)
    assert (acc == 0).all()
    # weights are held to [0, h]; what is not a number adds nothing
    sa.row_weights(q, kv, torch.full_like(lse, -torch.inf), idx, 0.04, acc, kv_scale=sc)
    listed = torch.zeros(200, dtype=torch.int64, device=dev).scatter_add_(
        0, idx[idx >= 0].long(), torch.ones_like(idx[idx >= 0], dtype=torch.int64))
    assert torch.equal(acc[0], listed * 16 << 32)
    acc.zero_()
    sa.row_weights(q, kv, torch.full_like(lse, torch.nan), idx, 0.04, acc, kv_scale=sc)
    assert (acc == 0).all()


def test_row_weights_other_rows_may_hold_anything(dev):  # noqa: F811
    # infinities and NaNs in rows and heads' queries of other tokens do not spill over
    q, kv, _, sink, idx = inputs(dev, "bf16", 2, 3, 60, 512, 300, 100, 4, neg=0.2)
    idx = torch.where(idx == 7, 8, idx)
    lse = torch.empty(2, 3, 60, device=dev)
    sa.sparse_attn(q, kv, sink, idx, 0.04, lse=lse)
    acc, acc2 = (torch.zeros(2, 300, dtype=torch.int64, device=dev) for _ in range(2))
    sa.row_weights(q, kv, lse, idx, 0.04, acc)
    kv2, q2 = kv.clone(), q.clone()
    kv2[:, 7] = torch.nan
    q2[1, 2] = torch.inf                       # the last token's queries
    sa.row_weights(q2, kv2, lse, idx, 0.04, acc2)
    assert torch.equal(acc[0], acc2[0])
    only = torch.ones(300, dtype=torch.bool, device=dev)
    only[idx[1, 2][idx[1, 2] >= 0].long()] = False
    assert torch.equal(acc[1][only], acc2[1][only])


def test_row_weights_bad_index(dev):  # noqa: F811
    q, kv, sc, sink, idx = inputs(dev, "fp8", 2, 2, 64, 512, 300, 140, 6)
    lse = torch.full((2, 2, 64), 5.0, device=dev)
    bad = idx.clone()
    bad[1, 0, 5], bad[0, 1, 137] = 300, -2
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    acc, acc2 = (torch.zeros(2, 300, dtype=torch.int64, device=dev) for _ in range(2))
    sa.row_weights(q, kv, lse, bad, 0.04, acc, kv_scale=sc, workspace=ws)
    assert sa.read_status(ws, clear=True) == 4
    sa.row_weights(q, kv, lse, torch.where((bad >= 300) | (bad < -1), -1, bad), 0.04, acc2, kv_scale=sc,
                   workspace=ws)
    assert sa.read_status(ws) == 0 and torch.equal(acc, acc2)


@pytest.mark.parametrize("fmt,d,rows", [("bf16", 512, (1 << 32) // 1024 + 3000), ("fp4", 512, (1 << 32) // 256 + 4000),
                                        ("fp8", 64, (1 << 32) // 64 // 2 + 1000)])
def test_row_weights_cache_past_32_bits(dev, fmt, d, rows):  # noqa: F811
    b = 2 if d == 64 else 1
    q, (kv, sc, near), (far, far_sc, idx), sink = far_inputs(dev, fmt, b, rows, 64, d, 300, 15)
    lse = torch.empty(b, 1, 64, device=dev)
    sa.sparse_attn(q, kv, sink, near, d ** -0.5, kv_scale=sc, lse=lse)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    sa.row_weights(q, far, lse, idx, d ** -0.5, acc, kv_scale=far_sc)
    want = torch.zeros(b, 300, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, near, d ** -0.5, want, kv_scale=sc)
    assert torch.equal(acc.gather(1, idx[:, 0].long()), want)
    assert int((acc != 0).sum()) == int((want != 0).sum())
    _close(want, q, kv, sc, lse, near, d ** -0.5)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_row_weights_nothing_listed_and_no_rows(dev, fmt):  # noqa: F811
    q, kv, sc, sink, idx = inputs(dev, fmt, 2, 3, 16, 512, 40, 70, 9, neg=1.1, distinct=False)
    lse = torch.zeros(2, 3, 16, device=dev)
    acc = torch.full((2, 40), 5, dtype=torch.int64, device=dev)
    sa.row_weights(q, kv, lse, idx, 0.1, acc, kv_scale=sc)
    assert (acc == 5).all()
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    none = acc[:, :0].contiguous()
    no_kv = kv[:, :0].contiguous()
    no_sc = None if sc is None else sc[:, :0].contiguous()
    sa.row_weights(q, no_kv, lse, idx, 0.1, none, kv_scale=no_sc, workspace=ws)
    assert sa.read_status(ws) == 0
    idx[1, 2, 69] = 0  # out of range: there is no row 0
    sa.row_weights(q, no_kv, lse, idx, 0.1, none, kv_scale=no_sc, workspace=ws)
    assert sa.read_status(ws) == 4


# --------------------------------------------------------------------------------------------
# eviction
# --------------------------------------------------------------------------------------------

SELECT = [
    # b, rows, keep, first, last, kind, live
    (1, 1, 1, 0, 0, "random", None), (1, 1, 0, 0, 0, "random", None), (2, 10, 4, 0, 0, "random", None),
    (3, 1000, 300, 128, 16, "random", None), (2, 1025, 1024, 5, 5, "random", None),
    (4, 777, 100, 0, 100, "random", None),                 # nothing to choose: all of them protected
    (4, 777, 100, 50, 50, "random", None), (2, 500, 500, 0, 0, "random", None),
    (3, 5000, 1234, 128, 64, "ties", None), (3, 5000, 1234, 128, 64, "zero", None),
    (2, 5000, 700, 0, 0, "same", None), (2, 3333, 700, 7, 9, "extreme", None),
    (5, 2000, 600, 128, 64, "random", [0, 1, 500, 1999, 2000]),
    (5, 2000, 600, 128, 64, "ties", [599, 600, 601, -3, 99999]),
    (4, 300, 200, 128, 64, "random", [100, 130, 190, 250]),  # fewer rows than are protected
    (2, 40000, 16384, 128, 256, "random", None), (1, 100003, 777, 1, 0, "random", None),
    (1, 300000, 150000, 128, 1000, "heavy", None), (200, 64, 16, 4, 4, "ties", None),
    (2, 1000003, 400000, 128, 1000, "heavy", None),        # more rows than the cluster's shared memory holds
    (2, 1000003, 400000, 128, 1000, "ties", [999999, 5000]),
    (3, 16384, 5000, 0, 0, "near", None), (3, 70000, 30000, 3, 3, "near", None),  # equal as f32, not as integers
    (90, 20000, 7000, 128, 0, "zero", None), (1, 20000, 0, 0, 0, "random", None), (1, 20000, 20000, 0, 0, "random", None),
    (2, 50000, 300, 200, 100, "random", None),             # a cluster with nothing to choose
]


def _acc(rng, b, rows, kind):
    if kind == "ties":
        return rng.integers(0, 5, (b, rows)) << 40
    if kind == "zero":
        return np.where(rng.random((b, rows)) < 0.9, 0, rng.integers(0, 1 << 40, (b, rows)))
    if kind == "same":
        return np.full((b, rows), 123456789)
    if kind == "extreme":
        a = rng.integers(-2**63, 2**63 - 1, (b, rows))
        a[:, ::7], a[:, 1::7], a[:, 2::7] = 2**63 - 1, -2**63, 0
        return a
    if kind == "near":  # within one f32 step of one another: 2^44 and a step of 2^21
        return (1 << 44) + rng.integers(0, 1 << 20, (b, rows)) // 7
    if kind == "heavy":
        return (rng.random((b, rows)) ** 8 * 2.0 ** 45).astype(np.int64)
    return rng.integers(0, 1 << 45, (b, rows))


@pytest.mark.parametrize("case", SELECT, ids=lambda c: f"b{c[0]}r{c[1]}k{c[2]}f{c[3]}l{c[4]}{c[5]}"
                         f"{'-live' if c[6] else ''}")
def test_evict_select(dev, case):  # noqa: F811
    b, rows, keep, first, last, kind, live = case
    acc = _acc(np.random.default_rng(rows + keep), b, rows, kind).astype(np.int64)
    want_k, want_r = _cache.select(acc, keep, first, last, live)
    lv = None if live is None else torch.tensor(live, dtype=torch.int32, device=dev)
    kept, remap = sa.evict_select(torch.from_numpy(acc).to(dev), keep, keep_first=first, keep_last=last,
                                  live=lv)
    assert (kept.cpu().numpy() == want_k).all()
    assert (remap.cpu().numpy() == want_r).all()


def _gathered(t, kept, n):
    out = torch.zeros((t.shape[0], n) + t.shape[2:], dtype=t.dtype)
    for bi in range(t.shape[0]):
        for j in range(n):
            if kept[bi, j] >= 0:
                out[bi, j] = t[bi, kept[bi, j]]
    return out


@pytest.mark.parametrize("b,rows,keep,live", [(1, 9, 4, None), (3, 700, 200, [700, 150, 200]),
                                              (2, 5000, 4999, None), (2, 3000, 3000, None)])
def test_compact_rows(dev, b, rows, keep, live):  # noqa: F811
    g = torch.Generator().manual_seed(rows)
    acc = torch.randint(0, 1 << 40, (b, rows), generator=g)
    lv = None if live is None else torch.tensor(live, dtype=torch.int32, device=dev)
    kept, _ = sa.evict_select(acc.to(dev), keep, keep_first=2, keep_last=1, live=lv)
    host = [torch.randint(0, 256, (b, rows, 256), generator=g, dtype=torch.uint8),
            torch.randint(0, 256, (b, rows, 16), generator=g, dtype=torch.uint8), acc,
            torch.randint(0, 256, (b, rows, 3), generator=g, dtype=torch.uint8),
            torch.randn(b, rows, 5, 7, generator=g),
            torch.randint(0, 256, (b, rows), generator=g, dtype=torch.uint8),
            torch.randn(b, rows, 33, generator=g).to(torch.bfloat16),
            torch.randn(b, rows, 24, generator=g)]
    want = [_gathered(t, kept.cpu(), keep) for t in host]
    got = sa.compact_rows([t.to(dev) for t in host], kept)
    for g_, w in zip(got, want):
        assert g_.dtype == w.dtype and torch.equal(g_.cpu(), w)
    # into the leading rows of larger tensors: what lies behind them is left alone
    big = [torch.full((b, keep + 3) + t.shape[2:], 9, dtype=t.dtype, device=dev) for t in host]
    sa.compact_rows([t.to(dev) for t in host], kept, out=big)
    for g_, w in zip(big, want):
        assert torch.equal(g_[:, :keep].cpu(), w) and (g_[:, keep:] == 9).all()
    # in place, some of them as views whose sequences are further apart
    own = [t.to(dev) for t in host]
    wide = torch.full((b, rows + 5, 256), 77, dtype=torch.uint8, device=dev)
    wide[:, :rows] = own[0]
    own[0] = wide[:, :rows]
    res = sa.compact_rows(own, kept, out=own)
    for r, t, w, h in zip(res, own, want, host):
        assert r is t and torch.equal(t[:, :keep].cpu(), w) and torch.equal(t[:, keep:].cpu(), h[:, keep:])
    assert (wide[:, rows:] == 77).all()
    # some in place and others not, in one call
    mix = [host[0].to(dev), host[2].to(dev)]
    fresh = torch.empty(b, keep, dtype=torch.int64, device=dev)
    sa.compact_rows(mix, kept, out=[mix[0], fresh])
    assert torch.equal(mix[0][:, :keep].cpu(), want[0]) and torch.equal(fresh.cpu(), want[2])


def test_compact_rows_long_in_place(dev):  # noqa: F811
    # many chunks, the worst of moves: every row by one, and every second row
    for rows, kept_rows in ((50001, np.arange(1, 50001)), (50001, np.arange(0, 50001, 2))):
        t = torch.arange(rows * 8, device=dev, dtype=torch.int32).view(1, rows, 8)
        kept = torch.from_numpy(kept_rows.astype(np.int32))[None].to(dev)
        want = t[:, kept[0].long()].clone()
        sa.compact_rows([t], kept, out=[t])
        assert torch.equal(t[:, :kept.shape[1]], want)


def test_compact_rows_entries_out_of_range(dev):  # noqa: F811
    t = torch.ones(1, 4, 8, device=dev)
    kept = torch.tensor([[1, 4, -5]], dtype=torch.int32, device=dev)
    out, = sa.compact_rows([t], kept)
    assert (out[0, 0] == 1).all() and (out[0, 1:] == 0).all()


def test_compact_rows_past_32_bits(dev):  # noqa: F811
    rows = (1 << 32) // 256 + 5000
    t = torch.empty(1, rows, 256, dtype=torch.uint8, device=dev)
    kept = torch.cat([torch.arange(0, 3000, 7), torch.arange(rows - 4000, rows, 3)]).to(dev)
    n = len(kept)
    marks = torch.randint(0, 256, (n, 256), device=dev, dtype=torch.uint8)
    t[0, kept] = marks
    kept = kept.to(torch.int32)[None].contiguous()
    out, = sa.compact_rows([t], kept)
    assert torch.equal(out[0], marks)
    sa.compact_rows([t], kept, out=[t])
    assert torch.equal(t[0, :n], marks)


def test_remap_idx(dev):  # noqa: F811
    rng = np.random.default_rng(2)
    remap = torch.from_numpy(rng.integers(-1, 50, (3, 90)).astype(np.int32)).to(dev)
    idx = torch.from_numpy(rng.integers(-1, 90, (3, 7, 41)).astype(np.int32)).to(dev)
    idx[0, 0, 0], idx[1, 1, 1] = 90, -7
    ok = (idx >= 0) & (idx < 90)
    want = torch.where(ok, remap.gather(1, idx.clamp(0, 89).long().view(3, -1)).view(idx.shape), -1)
    assert torch.equal(sa.remap_idx(idx, remap), want.to(torch.int32))
    sa.remap_idx(idx, remap, out=idx)
    assert torch.equal(idx, want.to(torch.int32))


# --------------------------------------------------------------------------------------------
# the whole run
# --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("in_place", [False, True])
def test_write_attend_weigh_evict(dev, in_place):  # noqa: F811
    """A 4-bit cache with a ring in front: three decode steps, their weights accumulated, the cache
    halved, and a step over what stays, which is the attention over the old cache with the evicted
    entries empty."""
    b, h, d, W, n, topk, keep = 3, 64, 512, 8, 600, 200, 304
    g = torch.Generator(device=dev).manual_seed(1)
    rows, scale = W + n, d ** -0.5
    codes = torch.zeros(b, rows, d // 2, dtype=torch.uint8, device=dev)
    scales = torch.zeros(b, rows, d // 32, dtype=torch.uint8, device=dev)
    x = torch.randn(b, rows, d, device=dev, generator=g).to(torch.bfloat16)
    for bi in range(b):
        sa.act_quant_fp4(x[bi], codes=codes[bi], scales=scales[bi])
    sink = torch.randn(h, device=dev, generator=g)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    ws = sa.new_workspace(b, 1, h, d, rows, W + topk, sa.SA_KV_FP4_E2M1)
    total = torch.zeros(b, rows, dtype=torch.float64, device=dev)
    room = torch.zeros(b, rows, dtype=torch.float64, device=dev)
    lse = torch.empty(b, 1, h, device=dev)
    idx = torch.empty(b, 1, W + topk, dtype=torch.int32, device=dev)
    for step in range(3):
        pos = 4 * n + step
        new = torch.randn(b, 1, d, device=dev, generator=g).to(torch.bfloat16)
        sa.window_write_fp4(new, pos, codes=codes[:, :W], scales=scales[:, :W])
        q = torch.randn(b, 1, h, d, device=dev, generator=g).to(torch.bfloat16)
        score = torch.randn(b, 1, (pos + 1) // 4, device=dev, generator=g)
        sa.window_idxs(pos, 1, W, out=idx[:, :, :W], nbatch=b)
        sa.indexer_topk(score, pos, 4, topk, W, out=idx[:, :, W:])
        o = sa.sparse_attn(q, codes, sink, idx, scale, kv_scale=scales, lse=lse, workspace=ws)
        sa.row_weights(q, codes, lse, idx, scale, acc, kv_scale=scales, workspace=ws)
        kv64 = _cache.rows_f64(codes, scales, d)
        want, want_lse, o_tol, lse_tol = _cache.attention(q, kv64, sink, idx, scale)
        check(o, want, o_tol, "o")
        check(lse, want_lse, lse_tol, "lse")
        w, t = _cache.row_weights(q, kv64, lse, idx, scale)
        total, room = total + w, room + t
    check(acc.double() * sa.WEIGHT_UNIT, total, room, "weights")
    kept, remap = sa.evict_select(acc, keep, keep_first=W, keep_last=16)
    want_k, want_r = _cache.select(acc.cpu().numpy(), keep, W, 16)
    assert (kept.cpu().numpy() == want_k).all() and (remap.cpu().numpy() == want_r).all()
    gone = torch.where((idx >= 0) & (remap.gather(1, idx.clamp(min=0).long().view(b, -1))
                                     .view(idx.shape) < 0), -1, idx)
    want, _, o_tol, _ = _cache.attention(q, kv64, sink, gone, scale)
    moved = sa.compact_rows([codes, scales, acc], kept, out=[codes, scales, acc] if in_place else None)
    c2, s2, a2 = (t[:, :keep].contiguous() for t in moved)
    idx2 = sa.remap_idx(idx, remap)
    o2 = sa.sparse_attn(q, c2, sink, idx2, scale, kv_scale=s2, lse=lse)
    check(o2, want, o_tol, "after the eviction")
    assert (a2[:, :W] >= 0).all() and idx2.max() < keep


def test_captured_and_replayed_on_a_side_stream(dev):  # noqa: F811
    """A decode step (ring write, attention with lse, weights) and an eviction captured in one graph on
    a stream of their own, replayed twice on other contents: what direct calls give."""
    b, h, d, W, rows, topk, keep = 2, 64, 512, 8, 300, 100, 100
    scale = d ** -0.5
    q, kv, sc, sink, idx = inputs(dev, "fp4", b, 1, h, d, rows, topk, 21)
    new = torch.randn(b, 1, d, device=dev).to(torch.bfloat16)
    acc = torch.zeros(b, rows, dtype=torch.int64, device=dev)
    lse, o = torch.empty(b, 1, h, device=dev), torch.empty_like(q)
    ws = sa.new_workspace(b, 1, h, d, rows, topk, sa.SA_KV_FP4_E2M1)

    def step():
        sa.window_write_fp4(new, 5, codes=kv[:, :W], scales=sc[:, :W])
        sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc, lse=lse, out=o, workspace=ws)
        sa.row_weights(q, kv, lse, idx, scale, acc, kv_scale=sc, workspace=ws)
        kept, remap = sa.evict_select(acc, keep, keep_first=W)
        return [kept, remap, sa.remap_idx(idx, remap)] + sa.compact_rows([kv, sc, acc], kept)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            res = step()
    torch.cuda.synchronize()
    for seed in (1, 2):
        q.copy_(torch.randn(q.shape, device=dev, generator=torch.Generator(device=dev).manual_seed(seed)))
        new.mul_(-1.5)
        acc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in [o, lse] + res]
        acc.zero_()
        want = [o, lse] + step()
        torch.cuda.synchronize()
        for g_, w in zip(got, want):
            assert torch.equal(g_, w)


@pytest.mark.parametrize("call", ["sparse_attn", "evict_select", "compact_rows", "remap_idx"])
def test_outputs_of_a_call_on_another_stream(dev, call):  # noqa: F811
    """A call on a stream of its own does not write into memory that the current stream still reads."""
    n = 300000
    acc = torch.arange(n, device=dev)[None]
    kept = torch.arange(n, device=dev, dtype=torch.int32)[None]
    q, kv, sc, sink, idx = inputs(dev, "fp4", 1, 10, 64, 512, 700, 64, 3)
    run = {"sparse_attn": lambda st: [sa.sparse_attn(q, kv, sink, idx, 0.05, kv_scale=sc, stream=st)],
           "evict_select": lambda st: sa.evict_select(acc, n, stream=st),
           "compact_rows": lambda st: sa.compact_rows([kept], kept, stream=st),
           "remap_idx": lambda st: [sa.remap_idx(kept, kept, stream=st)]}[call]
    want = [t.clone() for t in run(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nbytes = want[0].numel() * want[0].element_size()
    old, copy = (torch.full((nbytes,), 7, dtype=torch.uint8, device=dev) for _ in range(2))
    copy.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    copy.copy_(old)
    del old
    got = run(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert (copy == 7).all()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_no_columns_captured(dev):  # noqa: F811
    """The call without columns (a memset and the sinks) in a graph."""
    q, kv, sc, sink, idx = inputs(dev, "fp4", 2, 3, 16, 512, 40, 0, 9)
    lse, o = torch.empty(2, 3, 16, device=dev), torch.empty_like(q)
    ws = sa.new_workspace(2, 3, 16, 512, 40, 0, sa.SA_KV_FP4_E2M1)
    graph = torch.cuda.CUDAGraph()
    sa.sparse_attn(q, kv, sink, idx, 0.1, kv_scale=sc, lse=lse, out=o, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sa.sparse_attn(q, kv, sink, idx, 0.1, kv_scale=sc, lse=lse, out=o, workspace=ws)
    lse.fill_(5)
    o.fill_(5)
    graph.replay()
    assert (o == 0).all() and (lse == sink).all()
