"""page_write and window_attn on the GPU, against their formulas in 64 bits."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from sparse_latent_attention_gb300._lib import SA_ERR_INDEX, SA_STATUS_BYTES
from tests import _cache, _paged
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)
from tests.test_gpu_norm import _far_rows

pytestmark = pytest.mark.gpu

EPS = 1e-6
MIX = ([1, 4, 0, 37, 1], [0, 90, 5, 0, 700])  # sequences' new tokens and what their caches held


def _rows(dev, n, d, seed, pad=0):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(n, d + pad, device=dev, generator=g) * torch.exp(torch.randn(n, 1, device=dev, generator=g))
    return x.to(torch.bfloat16)[:, :d]


def _pools(dev, bt, d, fmt, seed, pad=0):  # noqa: F811
    """pages, codes, scales with arbitrary contents (pad: rows that lie apart)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    shape = (bt.n_pages, bt.page)
    pages = torch.randn(*shape, d + pad, device=dev, generator=g).to(torch.bfloat16)[..., :d]
    if not fmt:
        return pages, None, None
    both = torch.randint(0, 256, (*shape, (d if fmt == "fp8" else d // 2) + d // 32 + pad), device=dev, generator=g,
                         dtype=torch.uint8)
    w = d if fmt == "fp8" else d // 2
    codes, scales = both[..., :w], both[..., w:w + d // 32]   # side by side in a row
    return (pages, codes, scales) if pad else (pages, codes.contiguous(), scales.contiguous())


def _want(bt, x, weight, rot):
    y = x[:bt.live].double() if weight is None else _paged.norm(x[:bt.live], weight, EPS)
    return y if rot is None else _paged.turned(y, rot, bt.positions().to(y.device))


def _check_rows(bt, y, pages, codes, scales, quant, before, rel):
    rows = bt.rows().to(y.device)
    for t, old in zip((pages, codes, scales), before):  # every other row is as it was
        if t is not None:
            other = torch.ones(bt.n_pages * bt.page, dtype=torch.bool, device=y.device)
            other[rows] = False
            assert torch.equal(t.flatten(0, 1)[other].view(torch.uint8), old.flatten(0, 1)[other].view(torch.uint8))
    # y's parts may cancel in a rotation: its error is relative to the pair's length
    if codes is not None:
        c, s = codes.flatten(0, 1)[rows], scales.flatten(0, 1)[rows]
        v = c.view(torch.float8_e4m3fn).double() if quant == "fp8" else _paged.fp4_values(c)
        _paged.check_codes(v, s, y, quant, rel)
        if pages is not None:
            rt = v * _paged.pow2(s.long() - 127).repeat_interleave(32, -1)
            assert torch.equal(pages.flatten(0, 1)[rows].double(), rt)
    elif quant is None:
        got = pages.flatten(0, 1)[rows].double()
        assert ((got - y).abs() <= (2.0 ** -8 + rel) * y.abs() + 2.0 ** -135).all()
    return rows


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,page,norm,rope,pad", [
    (512, 64, True, 64, 0), (512, 1, False, 0, 0), (512, 100, True, 512, 0), (64, 16, True, 2, 0), (32, 3, False, 32, 0),
    (448, 64, True, 64, 32), (1024, 48, True, 128, 0), (544, 64, True, 6, 0), (512, 64, True, 64, 1), (96, 5, True, 10, 3),
])
def test_page_write(dev, fmt, d, page, norm, rope, pad):  # noqa: F811
    bt = _paged.Batch(*MIX, page, d + page, spare=3)
    x = _rows(dev, bt.n, d, d, pad)
    w = 1 + 0.3 * torch.randn(d, device=dev) if norm else None
    rot = _paged.rotations(800, rope).to(dev) if rope else None
    quant = None if fmt == "bf16" else fmt
    pages, codes, scales = _pools(dev, bt, d, quant, 3, pad)
    before = [None if t is None else t.clone() for t in (pages, codes, scales)]
    ws = sa.new_window_workspace(bt.n, bt.b, 1, 64, 1, 0, page)
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, codes=codes, scales=scales, weight=w, eps=EPS,
                  rope=rot, workspace=ws)
    # (a rotation keeps what f32 loses: the error stays relative to the turned value but for a full cancellation)
    rows = _check_rows(bt, _want(bt, x, w, rot), pages, codes, scales, quant, before, _paged.NORM_REL)
    assert sa.read_status(ws) == 0
    # codes alone, and the round trip alone, are the same rows
    if quant:
        c2, s2 = before[1].clone(), before[2].clone()
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, codes=c2, scales=s2, weight=w, eps=EPS, rope=rot)
        assert torch.equal(c2, codes) and torch.equal(s2, scales)
        p2 = before[0].clone()
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=p2, quant=quant, weight=w, eps=EPS, rope=rot)
        assert torch.equal(p2.flatten(0, 1)[rows], pages.flatten(0, 1)[rows])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_page_write_quantises_as_act_quant(dev, fmt):  # noqa: F811
    """Without norm and rotation the codes are those of the library's quantisers, bit for bit."""
    bt = _paged.Batch([300], [13], 64, 1)
    x = _rows(dev, 300, 512, 2)
    _, codes, scales = _pools(dev, bt, 512, fmt, 3)
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, codes=codes, scales=scales)
    c = torch.empty(300, codes.shape[2], dtype=torch.uint8, device=dev)
    s = torch.empty(300, 16, dtype=torch.uint8, device=dev)
    (sa.act_quant_fp8 if fmt == "fp8" else sa.act_quant_fp4)(x, codes=c, scales=s)
    rows = bt.rows().to(dev)
    assert torch.equal(codes.flatten(0, 1)[rows], c) and torch.equal(scales.flatten(0, 1)[rows], s)


@pytest.mark.parametrize("b", [1, 31, 32, 33, 1000, 1100])
@pytest.mark.parametrize("each", [1, 17])
def test_page_write_many_sequences(dev, b, each):  # noqa: F811
    """A token's sequence among many, some without tokens, with few tokens a warp and with several."""
    new = [each if i % 5 != 3 or b == 1 else 0 for i in range(b)]
    bt = _paged.Batch(new, [(7 * i) % 50 for i in range(b)], 16, b)
    x = _rows(dev, bt.n, 64, b)
    pages, _, _ = _pools(dev, bt, 64, None, 4)
    before = pages.clone()
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages)
    _check_rows(bt, x.double(), pages, None, None, None, (before, None, None), 0.0)


def test_page_write_bad_pages(dev):  # noqa: F811
    """Positions without a page, past the table, below zero or past the rotations are not written."""
    bt = _paged.Batch([8, 8, 8, 8], [0, 60, 0, 90], 16, 5)
    x = _rows(dev, bt.n, 128, 6)
    pages, _, _ = _pools(dev, bt, 128, None, 7)
    before, rot = pages.clone(), _paged.rotations(95, 64).to(dev)
    bt.table[0, 0] = bt.n_pages            # no such page
    bt.table[1, 4] = -1                    # positions 64 .. 67
    bt.kv_len[2] = 3                       # its first five tokens have no position
    ws = sa.new_window_workspace(bt.n, 4, 1, 64, 1, 0, 16)
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, rope=rot, workspace=ws)
    assert sa.read_status(ws, clear=True) == SA_ERR_INDEX
    written = (pages != before).flatten(0, 1).any(-1).nonzero().flatten().tolist()
    want = [bt.row(1, p) for p in range(60, 64)] + [bt.row(2, p) for p in range(3)] + [bt.row(3, p) for p in range(90, 95)]
    assert sorted(written) == sorted(want)
    bt.kv_len[2], bt.kv_len[0] = 1 << 30, 8   # far past the table
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, workspace=ws)
    assert sa.read_status(ws, clear=True) == SA_ERR_INDEX
    # negative positions alone are no error
    few = _paged.Batch([4], [0], 16, 5)
    few.kv_len[0] = 2
    sa.page_write(x[:4], few.table, few.q_start, few.kv_len, pages=pages[:few.n_pages], workspace=ws)
    assert sa.read_status(ws) == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "bf16"])
def test_page_write_rounds_once(dev, fmt):  # noqa: F811
    """Millions of normed and turned values, to within 2^-36 of a border on its own side: of as many rounded to f32 on
    the way some would not be."""
    eps = float(torch.tensor(EPS))
    bt = _paged.Batch([8192], [0], 64, 8)
    x = _rows(dev, bt.n, 512, 9)
    w = 1 + 0.3 * torch.randn(512, device=dev, generator=torch.Generator(device=dev).manual_seed(10))
    rot = _paged.rotations(bt.n, 64).to(dev)
    y = _paged.turned(_paged.norm(x, w, eps), rot, bt.positions().to(dev))
    pages, codes, scales = _pools(dev, bt, 512, None if fmt == "bf16" else fmt, 11)
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, codes=codes, scales=scales, weight=w, eps=EPS, rope=rot)
    rows = bt.rows().to(dev)
    if fmt == "bf16":
        got = pages.flatten(0, 1)[rows].double()
        # half a step of the larger neighbour's
        step = _paged.pow2(torch.frexp(torch.maximum(got.abs(), y.abs())).exponent.long() - 9)
        assert ((got - y).abs() <= step + 2.0 ** -36 * y.abs()).all()
    else:
        c = codes.flatten(0, 1)[rows]
        v = c.view(torch.float8_e4m3fn).double() if fmt == "fp8" else _paged.fp4_values(c)
        # (a pair that cancels in the rotation keeps its error, which is relative to its length)
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[:, -64:] = (y[:, -64:].unflatten(1, (32, 2)).square().sum(-1, keepdim=True).sqrt().expand(-1, -1, 2).flatten(1)
                         < 256 * y[:, -64:].abs())
        _paged.check_codes(torch.where(keep, v, 0.0), scales.flatten(0, 1)[rows], torch.where(keep, y, 0.0), fmt, 2.0 ** -36)


def test_page_write_nan_and_inf(dev):  # noqa: F811
    bt = _paged.Batch([3], [0], 16, 5)
    x = _rows(dev, 3, 64, 6)
    x[0, 3], x[1, 40] = float("nan"), float("inf")
    for fmt in ("fp8", "fp4"):
        _, codes, scales = _pools(dev, bt, 64, fmt, 3)
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, codes=codes, scales=scales)
        c, s = codes.flatten(0, 1)[bt.rows().to(dev)], scales.flatten(0, 1)[bt.rows().to(dev)]
        v = c.view(torch.float8_e4m3fn).double() if fmt == "fp8" else _paged.fp4_values(c)
        y = x.double()
        assert v[0, 3].isnan() if fmt == "fp8" else v[0, 3] == 0
        assert v[1, 40] == (448 if fmt == "fp8" else 6) and int(s[1, 1]) < 255
        v[0, 3] = y[0, 3] = 0.0
        _paged.check_codes(v[[0, 2]], s[[0, 2]], y[[0, 2]], fmt, 0.0)
        _paged.check_codes(v[1:2, :32], s[1:2, :1], y[1:2, :32], fmt, 0.0)


# ---------------------------------------------------------------------------------------------
# window_attn
# ---------------------------------------------------------------------------------------------

def _attn_inputs(dev, bt, h, d, fmt, window, first, seed, peak=1.0):  # noqa: F811
    """q, sink, and a pool whose rows that no token sees hold NaN and infinities."""
    g = torch.Generator(device=dev).manual_seed(seed)
    q = (peak * torch.randn(bt.n, h, d, device=dev, generator=g)).to(torch.bfloat16)
    sink = torch.randn(h, device=dev, generator=g)
    rows = torch.randn(bt.n_pages * bt.page, d, device=dev, generator=g).to(torch.bfloat16)
    seen = torch.zeros(bt.n_pages * bt.page, dtype=torch.bool, device=dev)
    idx = bt.visible(window, first).to(dev)
    seen[idx[idx >= 0].long()] = True
    if fmt == "bf16":
        odd = torch.arange(len(rows), device=dev)[:, None] + torch.arange(d, device=dev)
        trash = torch.where(odd % 3 == 0, float("nan"), torch.where(odd % 3 == 1, float("inf"), -float("inf")))
        rows = torch.where(seen[:, None], rows, trash.to(torch.bfloat16))
        return q, sink, rows.view(bt.n_pages, bt.page, d), None
    codes = torch.empty(len(rows), d if fmt == "fp8" else d // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(len(rows), d // 32, dtype=torch.uint8, device=dev)
    (sa.act_quant_fp8 if fmt == "fp8" else sa.act_quant_fp4)(rows, codes=codes, scales=scales)
    codes[~seen], scales[~seen] = 0x7F, 255   # (e4m3's NaN; the largest scale)
    return q, sink, codes.view(bt.n_pages, bt.page, -1), scales.view(bt.n_pages, bt.page, -1)


def _attend(bt, q, pool, kv_scale, sink, scale, window, first, rot=None, with_lse=True):
    lse = torch.full(q.shape[:2], 77.0, device=q.device) if with_lse else None
    out = torch.full_like(q, 55.0)
    ws = sa.new_window_workspace(bt.n, bt.b, q.shape[1], q.shape[2], window, first, bt.page,
                                 sa.SA_KV_BF16 if kv_scale is None else
                                 sa.SA_KV_FP8_E4M3 if pool.shape[2] == q.shape[2] else sa.SA_KV_FP4_E2M1)
    ws[SA_STATUS_BYTES:].fill_(0xFF)   # (NaN wherever it is read unwritten)
    got = sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, scale, window, first=first,
                         kv_scale=kv_scale, out=out, lse=lse, rope=rot, workspace=ws)
    assert got is out
    assert sa.read_status(ws) == 0
    assert (out[bt.live:] == 55.0).all() and (lse is None or (lse[bt.live:] == 77.0).all())
    return out[:bt.live], None if lse is None else lse[:bt.live]


def _check_attn(bt, q, pool, kv_scale, sink, window, first, rot=None, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    o, lse = _attend(bt, q, pool, kv_scale, sink, scale, window, first, rot)
    want, lse_w, tol, lse_tol = _paged.attention(bt, q, pool, kv_scale, sink, scale, window, first, rot)
    off = ~((o.double() - want).abs() <= tol)
    assert not off.any(), f"{int(off.sum())} of {off.numel()} off, first {off.nonzero()[0].tolist()}: " \
                          f"{o[off][:4].tolist()} {want[off][:4].tolist()}"
    assert ((lse.double() - lse_w).abs() <= lse_tol)[lse_w.isfinite()].all()
    assert torch.equal(lse[lse_w.isinf()].double(), lse_w[lse_w.isinf()])
    alone, _ = _attend(bt, q, pool, kv_scale, sink, scale, window, first, rot, with_lse=False)
    assert torch.equal(alone, o)
    return o


ATTN = [  # new, held, page, h, d, window, first, spare
    ([1], [0], 64, 64, 512, 128, 4, 0),                    # a cache of one row
    ([1], [5000], 64, 64, 512, 128, 4, 0),                 # one token, its rows split over the GPU
    ([1] * 20, [37 * i for i in range(20)], 64, 64, 512, 100, 16, 3),
    ([1] * 5, [3000, 0, 64, 63, 9000], 32, 128, 512, 1024, 64, 0),
    ([130, 0, 1, 64], [0, 9, 700, 33], 64, 64, 512, 128, 4, 5),
    ([300], [0], 64, 64, 512, 128, 0, 0),
    ([70, 3], [1000, 100], 64, 128, 512, 300, 40, 0),
    ([257], [123], 32, 16, 512, 64, 7, 1),                 # eight tokens a tile
    ([200, 90], [0, 77], 64, 1, 512, 33, 2, 0),            # 128 tokens a tile
    ([33], [500], 64, 40, 512, 200, 0, 0),                 # a tile's edge inside a token
    ([50], [64], 64, 100, 512, 1, 0, 0),                   # itself alone
    ([9], [20], 64, 64, 512, 1, 12, 0),
    ([40], [300], 64, 64, 512, 4000, 500, 0),              # everything before it
    ([20], [300], 16, 64, 512, 128, 4, 0),                 # pages that end inside a tile
    ([20], [300], 100, 64, 512, 128, 4, 0),
    ([20], [300], 1, 64, 512, 128, 4, 0),
    ([30, 1], [0, 400], 64, 64, 64, 128, 4, 2),            # other head dims
    ([30, 1], [0, 400], 48, 40, 192, 100, 9, 0),
    ([5, 1], [0, 4000], 64, 128, 448, 2000, 0, 0),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", ATTN, ids=[str(i) for i in range(len(ATTN))])
def test_window_attn(dev, case, fmt):  # noqa: F811
    new, held, page, h, d, window, first, spare = case
    bt = _paged.Batch(new, held, page, 11, spare)
    q, sink, pool, sc = _attn_inputs(dev, bt, h, d, fmt, window, first, 12, peak=2.0)
    _check_attn(bt, q, pool, sc, sink, window, first)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("rope", [2, 64, 512])
@pytest.mark.parametrize("new,held", [([40, 0, 70], [0, 3, 600]), ([1, 1], [5000, 10])])
def test_window_attn_turned_back(dev, fmt, rope, new, held):  # noqa: F811
    bt = _paged.Batch(new, held, 64, 13, 2)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 14)
    _check_attn(bt, q, pool, sc, sink, 128, 4, rot=_paged.rotations(5001, rope).to(dev))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_sinks_and_scales(dev, fmt):  # noqa: F811
    bt = _paged.Batch([20, 1], [0, 300], 64, 15)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 64, 4, 16)
    sink[0], sink[1], sink[2], sink[3] = -float("inf"), 80.0, -80.0, float("inf")
    for scale in (512 ** -0.5, -0.1, 0.0):
        o = _check_attn(bt, q, pool, sc, sink, 64, 4, scale=scale)
        assert (o[:, 3] == 0).all()


def test_window_attn_peaks(dev):  # noqa: F811
    """Logits that rise along the row, and far apart: the running maximum moves again and again."""
    bt = _paged.Batch([64], [900], 64, 17)
    q, sink, pool, _ = _attn_inputs(dev, bt, 64, 512, "bf16", 800, 32, 18, peak=8.0)
    at = torch.tensor([bt.row(0, p) for p in range(964)], device=dev)
    pool.view(-1, 512)[at] *= torch.linspace(0.1, 3.0, 964, device=dev)[:, None].to(torch.bfloat16)
    _check_attn(bt, q, pool, None, sink, 800, 32)


def test_window_attn_bad_pages(dev):  # noqa: F811
    """A position without a page is not attended to, and noted; entries that no token meets are not looked at;
    a token without a position attends to nothing."""
    for fmt in ("bf16", "fp8"):
        bt = _paged.Batch([3, 4], [500, 0], 64, 19)
        q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 20)
        want, _ = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
        bt.table[0, 1:5] = 1 << 30                       # positions 64 .. 319: out of everybody's sight
        got, _ = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
        assert torch.equal(got, want)
        hold = bt.table[0, 6].item()
        bt.table[0, 6] = bt.n_pages                      # positions 384 .. 447
        ws = sa.new_window_workspace(7, 2, 64, 512, 128, 4, 64, sa.SA_KV_FP8_E4M3 if sc is not None else 0)
        got = sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 128, first=4, kv_scale=sc,
                             workspace=ws)
        assert sa.read_status(ws, clear=True) == SA_ERR_INDEX
        bt.table_cpu[0, 6] = hold
        idx = bt.visible(128, 4).to(dev)
        lost = (idx // 64) == hold
        idx = torch.where(lost, -1, idx).to(torch.int32)
        kv = _cache.rows_f64(torch.nan_to_num(pool.view(1, -1, 512).float(), 0, 0, 0).to(torch.bfloat16) if sc is None
                             else pool.view(1, -1, 512), None if sc is None else sc.view(1, -1, 16).clamp(max=140), 512)
        kv = torch.nan_to_num(kv)
        o, _, tol, _ = _cache.attention(q[None], kv, sink, idx[None], 0.05)
        assert ((got.double() - o[0]).abs() <= tol[0]).all()
        bt.table[0, 6] = hold
        bt.kv_len[1] = 2                                  # tokens 0 and 1 of the second have no position
        got, lse = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
        assert (got[3:5] == 0).all() and torch.allclose(lse[3:5], sink.expand(2, -1)) and torch.equal(got[:3], want[:3])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_graph(dev, fmt):  # noqa: F811
    """A captured step replayed with other lengths, pages and contents: the write, then the attention."""
    bt = _paged.Batch([1, 1, 2], [100, 400, 40], 64, 21)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 22)
    x = _rows(dev, 4, 512, 23)
    ws = sa.new_window_workspace(4, 3, 64, 512, 128, 4, 64, sa.SA_KV_FP8_E4M3 if sc is not None else 0)
    put = dict(pages=pool) if sc is None else dict(codes=pool, scales=sc)

    def step():
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, workspace=ws, **put)
        return sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 128, first=4, kv_scale=sc,
                              workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    for k in range(3):
        nxt = _paged.Batch([1, 1, 2], [100 + 30 * k, 300 - k, 64 * k], 64, 30 + k)
        m = min(nxt.max_pages, bt.max_pages)
        bt.table.fill_(-1)
        bt.table[:, :m] = nxt.table[:, :m] % pool.shape[0]
        bt.table_cpu, bt.held = bt.table.cpu(), nxt.held
        # (distinct pages: the pool is smaller than the new batch may ask for)
        free = iter(torch.randperm(pool.shape[0], generator=torch.Generator().manual_seed(k)).tolist())
        for i in range(3):
            for j in range(-(-(nxt.held[i] + bt.new[i]) // 64)):
                bt.table_cpu[i, j] = next(free)
        bt.table.copy_(bt.table_cpu)
        bt.kv_len.copy_(nxt.kv_len)
        q2, _, pool2, sc2 = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 40 + k)
        for a, b in ((q, q2), (pool, pool2), (sc, sc2)):
            if a is not None:
                a.copy_(b)
        x.copy_(_rows(dev, 4, 512, 50 + k))
        graph.replay()
        assert sa.read_status(ws) == 0
        want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 128, 4)
        assert ((o.double() - want).abs() <= tol).all()


def test_a_decode_loop(dev):  # noqa: F811
    """Norm, write and attention as a program uses them: a prompt in pieces, then tokens one by one, against the
    whole sequence at once; the window's pages behind it are given back on the way."""
    d, h, window, first, page, total = 512, 64, 100, 4, 32, 230
    g = torch.Generator(device=dev).manual_seed(60)
    raw = torch.randn(total, d, device=dev, generator=g).to(torch.bfloat16)
    q = torch.randn(total, h, d, device=dev, generator=g).to(torch.bfloat16)
    w, sink = 1 + 0.1 * torch.randn(d, device=dev, generator=g), torch.randn(h, device=dev, generator=g)
    rot = _paged.rotations(total, 64).to(dev)
    one = _paged.Batch([total], [0], page, 61)
    pool = torch.zeros(one.n_pages, page, d, dtype=torch.bfloat16, device=dev)
    x = sa.add_rms_norm(raw, w)
    sa.page_write(x, one.table, one.q_start, one.kv_len, pages=pool, rope=rot, quant="fp8")
    whole = sa.window_attn(q, pool, sink, one.table, one.q_start, one.kv_len, d ** -0.5, window, first=first, rope=rot)
    fresh, outs, at = torch.zeros_like(pool), [], 0
    for n in [90, 33, 64] + [1] * 43:
        bt = _paged.Batch([n], [at], page, 61, extra_pages=one.n_pages)
        table = one.table.clone()
        behind = max(0, at - window) // page      # pages that nobody sees any more, but the first
        table[0, 1:behind] = -1
        xs = sa.add_rms_norm(raw[at:at + n], w)
        sa.page_write(xs, table, bt.q_start, bt.kv_len, pages=fresh, rope=rot, quant="fp8")
        ws = sa.new_window_workspace(n, 1, h, d, window, first, page)
        outs.append(sa.window_attn(q[at:at + n], fresh, sink, table, bt.q_start, bt.kv_len, d ** -0.5, window,
                                   first=first, rope=rot, workspace=ws))
        assert sa.read_status(ws) == 0
        at += n
    want, _, tol, _ = _paged.attention(one, q, pool, None, sink, d ** -0.5, window, first, rot)
    assert torch.equal(fresh.flatten(0, 1)[one.rows().to(dev)], pool.flatten(0, 1)[one.rows().to(dev)])
    for got in (whole, torch.cat(outs)):
        assert ((got.double() - want).abs() <= tol).all()


def test_streams_and_workspaces(dev):  # noqa: F811
    """Two calls at once on streams of their own, each with its own workspace, and outputs made on the stream."""
    bts = [_paged.Batch([1] * 9, [200 * i for i in range(9)], 64, 70 + k) for k in range(2)]
    ins = [_attn_inputs(dev, bt, 64, 512, "fp8" if k else "bf16", 256, 8, 72 + k) for k, bt in enumerate(bts)]
    streams = [torch.cuda.Stream() for _ in bts]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got = [sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 256, first=8, kv_scale=sc, stream=st)
               for bt, (q, sink, pool, sc), st in zip(bts, ins, streams)]
    torch.cuda.synchronize()
    for bt, (q, sink, pool, sc), o in zip(bts, ins, got):
        want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 256, 8)
        assert ((o.double() - want).abs() <= tol).all()


def test_nothing_to_do(dev):  # noqa: F811
    z = dict(dtype=torch.int32, device=dev)
    q = torch.empty(0, 64, 512, dtype=torch.bfloat16, device=dev)
    pool, sink = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device=dev), torch.zeros(64, device=dev)
    assert sa.window_attn(q, pool, sink, torch.zeros(1, 2, **z), torch.zeros(2, **z), torch.zeros(1, **z), 1.0, 8).shape == q.shape
    sa.page_write(q[:, 0], torch.zeros(1, 2, **z), torch.zeros(2, **z), torch.zeros(1, **z), pages=pool)
    # no sequence: everything is left as it was
    out = torch.full((3, 64, 512), 5.0, dtype=torch.bfloat16, device=dev)
    sa.window_attn(torch.zeros_like(out), pool, sink, torch.zeros(0, 2, **z), torch.zeros(1, **z), torch.zeros(0, **z),
                   1.0, 8, out=out)
    assert (out == 5.0).all()


# ---------------------------------------------------------------------------------------------
# calls that the cases above do not make
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("b,h", [(33, 64), (1100, 16), (400, 128)])
def test_window_attn_many_sequences(dev, b, h, fmt):  # noqa: F811
    """A task's sequence among many, a run of them without tokens, some with more than a tile."""
    new = [0 if i % 5 == 3 or 60 <= i < 200 else 9 if i % 50 == 7 else 1 for i in range(b)]
    bt = _paged.Batch(new, [(37 * i) % 150 for i in range(b)], 32, b, spare=2)
    q, sink, pool, sc = _attn_inputs(dev, bt, h, 512, fmt, 40, 3, b + 1)
    _check_attn(bt, q, pool, sc, sink, 40, 3)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("new,held", [([1], [0]), ([1, 1, 2], [0, 40, 200]), ([1], [700])])
@pytest.mark.parametrize("rope", [0, 64])
def test_window_attn_parts_without_positions(dev, new, held, rope, fmt):  # noqa: F811
    """A window far longer than the caches: most of the parts that a token's positions are cut into have none."""
    bt = _paged.Batch(new, held, 64, 80)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 1 << 16, 100, 81, peak=2.0)
    _check_attn(bt, q, pool, sc, sink, 1 << 16, 100, rot=_paged.rotations(800, rope).to(dev) if rope else None)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_tokens_without_positions(dev, fmt):  # noqa: F811
    """Hundreds of sequences one behind the other whose caches are shorter than their new tokens, a few that are not."""
    b = 900
    bt = _paged.Batch([1] * b, [50] * b, 64, 82)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 30, 2, 83)
    want, lse_w = _attend(bt, q, pool, sc, sink, 0.05, 30, 2)
    want, lse_w = want.clone(), lse_w.clone()
    none = torch.ones(b, dtype=torch.bool, device=dev)
    none[[0, 300, 301, 777, 899]] = False
    bt.kv_len[none] = 0
    bt.kv_len[5] = -(1 << 31)
    got, lse = _attend(bt, q, pool, sc, sink, 0.05, 30, 2)
    assert torch.equal(got[~none], want[~none]) and torch.equal(lse[~none], lse_w[~none])
    assert (got[none] == 0).all() and torch.allclose(lse[none], sink.expand(int(none.sum()), -1))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [90, 1])
@pytest.mark.parametrize("page", [64, 16])
def test_window_attn_far_past_the_table(dev, new, page, fmt):  # noqa: F811
    """The largest length there is: noted, nothing read past the table, and the other sequences are right."""
    bt = _paged.Batch([new, 3], [400, 70], page, 84)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 85)
    want, _ = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
    ws = sa.new_window_workspace(bt.n, 2, 64, 512, 128, 4, page, sa.SA_KV_FP8_E4M3 if sc is not None else 0)
    for length in (2 ** 31 - 1, (bt.max_pages + 5) * page):
        bt.kv_len[0] = length
        got = sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 128, first=4, kv_scale=sc, workspace=ws)
        assert sa.read_status(ws, clear=True) == SA_ERR_INDEX
        assert torch.equal(got[new:], want[new:])
        # what is left of it are the first rows, which are in the table
        kv = _cache.rows_f64(pool.view(-1, pool.shape[2])[[bt.row(0, p) for p in range(4)]][None] if sc is None else
                             pool.view(-1, 512)[[bt.row(0, p) for p in range(4)]][None],
                             None if sc is None else sc.view(-1, 16)[[bt.row(0, p) for p in range(4)]][None], 512)
        idx = torch.arange(4, dtype=torch.int32, device=dev).expand(1, new, 4).contiguous()
        if length == 2 ** 31 - 1:
            o, _, tol, _ = _cache.attention(q[None, :new], kv, sink, idx, 0.05)
            assert ((got[:new].double() - o[0]).abs() <= tol[0]).all()


@pytest.mark.parametrize("page", [64, 16])
def test_window_attn_without_a_table(dev, page):  # noqa: F811
    """A table of no pages: every position is past it, nothing is attended to, and that is noted."""
    q = torch.randn(3, 64, 512, device=dev).to(torch.bfloat16)
    pool, sink = torch.full((2, page, 512), float("nan"), dtype=torch.bfloat16, device=dev), torch.randn(64, device=dev)
    i = dict(dtype=torch.int32, device=dev)
    ws, lse = sa.new_window_workspace(3, 2, 64, 512, 128, 4, page), torch.zeros(3, 64, device=dev)
    o = sa.window_attn(q, pool, sink, torch.zeros(2, 0, **i), torch.tensor([0, 1, 3], **i), torch.tensor([9, 70], **i), 0.05,
                       128, first=4, lse=lse, workspace=ws)
    assert sa.read_status(ws) == SA_ERR_INDEX and (o == 0).all() and torch.allclose(lse, sink.expand(3, -1))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,page,window,first", [(512, 16, 5000, 10), (512, 1, 90, 600), (256, 64, 5000, 10), (64, 64, 60, 600),
                                                 (64, 5, 1, 100), (448, 32, 1 << 20, 0)])
def test_window_attn_longer_than_the_table(dev, d, page, window, first, fmt):  # noqa: F811
    """A table of fewer positions than a token may see, in the kernels that gather by row: all of them are looked at, and
    a position past them is still an error."""
    bt = _paged.Batch([40, 0, 1], [100, 9, 300], page, 102, 2)
    rot = _paged.rotations(400, 64).to(dev) if d == 512 else None
    q, sink, pool, sc = _attn_inputs(dev, bt, 40, d, fmt, window, first, 103, peak=2.0)
    _check_attn(bt, q, pool, sc, sink, window, first, rot=rot)
    bt.kv_len[2] = bt.max_pages * page + 1
    ws = sa.new_window_workspace(bt.n, bt.b, 40, d, window, first, page,
                                 {"bf16": sa.SA_KV_BF16, "fp8": sa.SA_KV_FP8_E4M3, "fp4": sa.SA_KV_FP4_E2M1}[fmt])
    sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, window, first=first, kv_scale=sc, workspace=ws)
    assert sa.read_status(ws) == SA_ERR_INDEX


def test_window_attn_rotation_past_its_table(dev):  # noqa: F811
    """A position that the rotations do not hold counts as their last one, and is noted."""
    bt = _paged.Batch([4], [96], 64, 86)
    q, sink, pool, _ = _attn_inputs(dev, bt, 64, 512, "bf16", 64, 0, 87)
    rot = _paged.rotations(100, 64).to(dev)
    call = lambda r, **kw: sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 64, rope=r, **kw)
    ws = sa.new_window_workspace(4, 1, 64, 512, 64, 0, 64)
    got = call(rot[:98].contiguous(), workspace=ws)
    assert sa.read_status(ws, clear=True) == SA_ERR_INDEX
    held = rot.clone()
    held[98:] = rot[97]
    assert torch.equal(got, call(held, workspace=ws)) and sa.read_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [64, 16])
def test_window_attn_nan_rows(dev, fmt, page):  # noqa: F811
    """A row that is NaN: NaN for the tokens that see it, nothing to the others of the same tile."""
    bt = _paged.Batch([120], [30], page, 88)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 16, 3, 89)
    want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 16, 3)
    for p in (60, 77, 130, 149):
        flat = pool.view(-1, 512)
        if sc is None:
            flat[bt.row(0, p)] = float("nan")
        else:
            flat[bt.row(0, p)] = 0x7F
    got, lse = _attend(bt, q, pool, sc, sink, 0.05, 16, 3)
    at = bt.positions()
    sees = torch.zeros(bt.n, dtype=torch.bool)
    for p in (60, 77, 130, 149):
        sees |= (at >= p) & (at < p + 16)
    sees = sees.to(dev)
    assert got[sees].isnan().all() and lse[sees].isnan().all()
    assert ((got[~sees].double() - want[~sees]).abs() <= tol[~sees]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_window_attn_takes_a_strided_table(dev, fmt):  # noqa: F811
    """The page table as columns of a wider one; another table is the same rows elsewhere."""
    bt = _paged.Batch([5, 1, 70], [100, 300, 0], 64, 90)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 128, 4, 91)
    want, _ = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
    wide = torch.full((bt.b, bt.max_pages + 9), 1 << 30, dtype=torch.int32, device=dev)
    wide[:, 4:4 + bt.max_pages] = bt.table
    plain, bt.table = bt.table, wide[:, 4:4 + bt.max_pages]
    got, _ = _attend(bt, q, pool, sc, sink, 0.05, 128, 4)
    assert torch.equal(got, want)
    x = _rows(dev, bt.n, 512, 92)
    a, b = torch.zeros_like(pool), torch.zeros_like(pool)
    if fmt == "bf16":
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=a)
        sa.page_write(x, plain, bt.q_start, bt.kv_len, pages=b)
    else:
        sa.page_write(x, bt.table, bt.q_start, bt.kv_len, codes=a, scales=torch.zeros_like(sc))
        sa.page_write(x, plain, bt.q_start, bt.kv_len, codes=b, scales=torch.zeros_like(sc))
    assert torch.equal(a, b) and (a != 0).any()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_page_write_scales_behind_a_pages_codes(dev, fmt):  # noqa: F811
    """Pages that hold their codes and behind them their scales, in one buffer."""
    bt = _paged.Batch([40, 1], [0, 100], 64, 93)
    d, w = 512, 512 if fmt == "fp8" else 256
    x = _rows(dev, bt.n, d, 94)
    both = torch.full((bt.n_pages, 64 * (w + 16)), 0x55, dtype=torch.uint8, device=dev)
    codes, scales = both[:, :64 * w].unflatten(1, (64, w)), both[:, 64 * w:].unflatten(1, (64, 16))
    before = (None, codes.clone(), scales.clone())
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, codes=codes, scales=scales)
    _check_rows(bt, x.double(), None, codes, scales, fmt, before, 0.0)


def test_graphs_that_share_a_workspace(dev):  # noqa: F811
    """Two captured calls whose parts go through one workspace, replayed in turn on a stream."""
    ins = []
    ws = None
    for k, (window, fmt) in enumerate([(2000, "bf16"), (3000, "fp8")]):
        bt = _paged.Batch([1, 2], [1500 + 300 * k, 2500], 64, 95 + k)
        ins.append((bt, window, *_attn_inputs(dev, bt, 64, 512, fmt, window, 8, 97 + k)))
    size = max(sa.window_workspace_size(3, 2, 64, 512, w, 8, 64, f) for w, f in ((2000, 0), (3000, sa.SA_KV_FP8_E4M3)))
    assert size > SA_STATUS_BYTES + 256  # (parts there are)
    ws = torch.zeros(size, dtype=torch.uint8, device=dev)
    graphs, outs = [], []
    for bt, window, q, sink, pool, sc in ins:
        out = torch.empty_like(q)
        call = lambda: sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, window, first=8,
                                      kv_scale=sc, workspace=ws, out=out)
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append(out)
    for _ in range(10):
        for g, out in zip(graphs, outs):
            out.fill_(9.0)
            g.replay()
    assert sa.read_status(ws) == 0
    for (bt, window, q, sink, pool, sc), out in zip(ins, outs):
        want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, window, 8)
        assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_past_32_bits(dev, fmt):  # noqa: F811
    """q and o of more than 2^31 elements and a pool of more than 2^32 bytes, the last sequence at the end of all three."""
    tail, long, h = _paged.Batch([40], [60], 64, 99), 33100, 128
    q, sink, small, sc_small = _attn_inputs(dev, tail, h, 512, fmt, 32, 5, 100)
    n_pages = 72000 if fmt == "bf16" else 140000
    assert long * h * 512 > 1 << 31 and n_pages * 64 * small.shape[2] * small.element_size() > 1 << 32
    pool = torch.zeros(n_pages, *small.shape[1:], dtype=small.dtype, device=dev)
    sc = None if sc_small is None else torch.zeros(n_pages, *sc_small.shape[1:], dtype=torch.uint8, device=dev)
    pool[-tail.n_pages:] = small
    if sc is not None:
        sc[-tail.n_pages:] = sc_small
    table = torch.full((2, -(-long // 64)), -1, dtype=torch.int32, device=dev)
    table[0] = torch.arange(table.shape[1], device=dev)
    table[1, :tail.max_pages] = torch.where(tail.table >= 0, tail.table + n_pages - tail.n_pages, -1)
    qs = torch.zeros(long + 40, h, 512, dtype=torch.bfloat16, device=dev)
    qs[long:] = q
    out = torch.full_like(qs, 3.0)
    q_start = torch.tensor([0, long, long + 40], dtype=torch.int32, device=dev)
    kv_len = torch.tensor([long, 100], dtype=torch.int32, device=dev)
    sa.window_attn(qs, pool, sink, table, q_start, kv_len, 0.05, 32, first=5, kv_scale=sc, out=out)
    want, _, tol, _ = _paged.attention(tail, q, small, sc_small, sink, 0.05, 32, 5)
    assert ((out[long:].double() - want).abs() <= tol).all()
    assert (out[:long:997] == 0).all() and (out[long - 1] == 0).all()   # (zero rows)
    # and the write
    x = _rows(dev, 40, 512, 101)
    x_all = torch.zeros(long + 40, 512, dtype=torch.bfloat16, device=dev)
    x_all[long:] = x
    before = [None if t is None else t[-tail.n_pages:].clone() for t in (pool, sc)]
    if fmt == "bf16":
        sa.page_write(x_all, table, q_start, kv_len, pages=pool)
        _check_rows(tail, x.double(), pool[-tail.n_pages:], None, None, None, (before[0], None, None), 0.0)
    else:
        sa.page_write(x_all, table, q_start, kv_len, codes=pool, scales=sc)
        _check_rows(tail, x.double(), None, pool[-tail.n_pages:], sc[-tail.n_pages:], "fp8", (None, *before), 0.0)


NOT_FINITE = (float("nan"), float("inf"), -float("inf"), 3.3e38)  # (the last: finite, but for its logits)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("h", [1, 16, 40, 64, 128])
@pytest.mark.parametrize("page,d", [(64, 512), (16, 512), (64, 256)])
@pytest.mark.parametrize("value", NOT_FINITE)
def test_window_attn_q_that_is_not_finite(dev, value, page, d, h, fmt):  # noqa: F811
    """A row of q that is not finite changes its own o and no other: not that of its token's other heads, of tokens in
    the same tile, of the sequence before, nor of the last one where it belongs to no sequence."""
    bt = _paged.Batch([40, 3, 9, 21], [70, 200, 0, 31], page, 104, spare=12)
    q, sink, pool, sc = _attn_inputs(dev, bt, h, d, fmt, 16, 3, 105)
    want, lse_w = _attend(bt, q, pool, sc, sink, 0.05, 16, 3)
    want, lse_w = want.clone(), lse_w.clone()
    bad = torch.zeros(bt.n, h, dtype=torch.bool, device=dev)
    bad[7, h // 2] = bad[20, 0] = bad[20, h - 1] = True     # inside a sequence
    bad[43, 0] = bad[52, h // 3] = True                     # the first token of the next one
    bad[bt.live:] = True                                    # behind the last
    odd = q.clone()
    odd[..., 200] = torch.where(bad, value, q[..., 200].float()).to(torch.bfloat16)
    odd[bt.live:] = value
    got, lse = _attend(bt, odd, pool, sc, sink, 0.05, 16, 3)
    ok = ~bad[:bt.live]
    assert torch.equal(got[ok], want[ok]) and torch.equal(lse[ok], lse_w[ok])
    if value != value:
        assert got[~ok].isnan().all() and lse[~ok].isnan().all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_q_and_rows_that_are_not_finite(dev, fmt):  # noqa: F811
    """Both at once: tokens that see a NaN row are NaN, a NaN row of q is, and the rest are as without either."""
    bt = _paged.Batch([90, 5], [30, 0], 64, 106, spare=7)
    q, sink, pool, sc = _attn_inputs(dev, bt, 64, 512, fmt, 16, 3, 107)
    want, _ = _attend(bt, q, pool, sc, sink, 0.05, 16, 3)
    want = want.clone()
    pool.view(-1, pool.shape[2])[bt.row(0, 60)] = float("nan") if sc is None else 0x7F
    q[[33, 80, 91], 11], q[bt.live:] = float("nan"), float("nan")
    got, _ = _attend(bt, q, pool, sc, sink, 0.05, 16, 3)
    at = bt.positions().to(dev)
    nan = torch.zeros(bt.live, 64, dtype=torch.bool, device=dev)
    nan[:90][(at[:90] >= 60) & (at[:90] < 76)] = True
    nan[[33, 80, 91], 11] = True
    assert got[nan].isnan().all() and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("h", [16, 64, 128])
@pytest.mark.parametrize("held", [(10, 0, 40, 130), (200, 31, 5, 0, 100, 9), (600, 20, 20, 20, 20, 700)])
def test_window_attn_tasks_of_few_blocks(dev, held, h, fmt):  # noqa: F811
    """Tasks of one block between others of two and more, many for each pair of SMs: the roles run ahead of one another
    by as many tasks as they may."""
    rng = torch.Generator().manual_seed(108)
    at = torch.randint(0, len(held), (900,), generator=rng).tolist()
    bt = _paged.Batch([1] * len(at), [held[i] for i in at], 32, 109)
    q, sink, pool, sc = _attn_inputs(dev, bt, h, 512, fmt, 100, 3, 110)
    first = _check_attn(bt, q, pool, sc, sink, 100, 3).clone()
    for _ in range(10):
        assert torch.equal(_attend(bt, q, pool, sc, sink, 512 ** -0.5, 100, 3)[0], first)


@pytest.mark.parametrize("eps", [0.0, 1e-44, EPS])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,pad", [(64, 0), (512, 0), (1024, 0), (512, 1)])
def test_page_write_squares_outside_f32(dev, d, pad, fmt, eps):  # noqa: F811
    """Rows whose squares are below or beyond what f32 holds, and an eps that is none, or less than they are."""
    eps = float(torch.tensor(eps))
    bt = _paged.Batch([12], [5], 16, 111)
    x = torch.zeros(12, d + pad, dtype=torch.bfloat16, device=dev)[:, :d].copy_(_far_rows(dev, d))
    w, rot = torch.linspace(0.5, 1.5, d, device=dev), _paged.rotations(17, 64).to(dev)
    pages, codes, scales = _pools(dev, bt, d, None if fmt == "bf16" else fmt, 112)
    before = [None if t is None else t.clone() for t in (pages, codes, scales)]
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, codes=codes, scales=scales, weight=w, eps=eps)
    y = _paged.norm(x, w, eps)
    _check_rows(bt, y, pages, codes, scales, None if fmt == "bf16" else fmt, before, _paged.NORM_REL)
    # (turned: a pair that cancels keeps an error relative to its length)
    sa.page_write(x, bt.table, bt.q_start, bt.kv_len, pages=pages, weight=w, eps=eps, rope=rot)
    turned = _paged.turned(y, rot, bt.positions().to(dev))
    size = y.clone()
    size[:, -64:] = y[:, -64:].unflatten(1, (32, 2)).norm(dim=-1, keepdim=True).expand(-1, -1, 2).flatten(1)
    got = pages.flatten(0, 1)[bt.rows().to(dev)].double()
    # (and below bf16's normal numbers a rounding is off by up to 2^-134)
    assert ((got - turned).abs() <= 2.0 ** -8 * turned.abs() + _paged.NORM_REL * size.abs() + 2.0 ** -134).all()


@pytest.mark.parametrize("d,page", [(512, 64), (512, 16), (128, 64)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_window_attn_one_workspace_for_all_batches(dev, fmt, d, page):  # noqa: F811
    """A workspace made for the largest batch serves the smaller ones, whose positions are cut into parts."""
    kind = sa.SA_KV_BF16 if fmt == "bf16" else sa.SA_KV_FP8_E4M3
    ws = sa.new_window_workspace(150, 150, 64, d, 2000, 8, page, kind)
    for n in (150, 1, 40, 2, 9, 150):
        bt = _paged.Batch([1] * n, [(977 * i + 2500) % 4000 for i in range(n)], page, 113 + n)
        q, sink, pool, sc = _attn_inputs(dev, bt, 64, d, fmt, 2000, 8, 114)
        o = sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 2000, first=8, kv_scale=sc, workspace=ws)
        want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 2000, 8)
        assert sa.read_status(ws) == 0 and ((o.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("d,page", [(512, 64), (512, 16), (64, 64)])
def test_window_attn_of_everything(dev, d, page, fmt):  # noqa: F811
    """The largest window, its workspace made for the call: as large as the table's positions need."""
    bt = _paged.Batch([300, 1], [0, 500], page, 115, 2)
    q, sink, pool, sc = _attn_inputs(dev, bt, 16, d, fmt, 1000, 0, 116)
    o = sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, (1 << 30) - 9, first=8, kv_scale=sc)
    want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 1000, 0)
    assert ((o[:bt.live].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("h,held", [(1, (0, 10, 31)), (8, (0, 20, 200)), (1, (31, 32, 33, 64, 100))])
def test_window_attn_many_small_tasks(dev, held, h, fmt):  # noqa: F811
    """Two thousand sequences of no, one or two tokens and few rows, again and again: the same result every time."""
    g = torch.Generator().manual_seed(117)
    new, at = torch.randint(0, 3, (2000,), generator=g).tolist(), torch.randint(0, len(held), (2000,), generator=g).tolist()
    bt = _paged.Batch(new, [held[i] for i in at], 64, 118)
    q, sink, pool, sc = _attn_inputs(dev, bt, h, 512, fmt, 40, 3, 119)
    ws = sa.new_window_workspace(bt.n, bt.b, h, 512, 40, 3, 64, {"bf16": sa.SA_KV_BF16, "fp8": sa.SA_KV_FP8_E4M3,
                                                                  "fp4": sa.SA_KV_FP4_E2M1}[fmt])
    call = lambda: sa.window_attn(q, pool, sink, bt.table, bt.q_start, bt.kv_len, 0.05, 40, first=3, kv_scale=sc, workspace=ws)
    want, _, tol, _ = _paged.attention(bt, q, pool, sc, sink, 0.05, 40, 3)
    first = call()
    assert ((first.double() - want).abs() <= tol).all()
    same = torch.ones((), dtype=torch.bool, device=dev)
    for _ in range(200):
        same &= (call() == first).all()
    assert same and sa.read_status(ws) == 0
