"""add_rms_norm on the GPU, against the formula in 64 bits."""

from __future__ import annotations

import math

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _paged
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _inputs(dev, n, d, kind, seed, pad=0, big=1.0):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(seed)
    x = (big * torch.randn(n, d + pad, device=dev, generator=g)).to(torch.bfloat16)[:, :d]
    w = 1 + 0.3 * torch.randn(d, device=dev, generator=g)
    r = None
    if kind != "none":
        r = 3 * torch.randn(n, d + pad, device=dev, generator=g)
        r = (r if kind == "f32" else r.to(torch.bfloat16))[:, :d]
    return x, w, r


def _check(x, w, r0, r1, out, codes, scales, eps=EPS):
    """Everything a call returned, from the residual as it was (r0)."""
    h = x.double()
    if r0 is not None:
        # the sum of two bf16, or of a bf16 and an f32, rounded once
        s = h + r0.double()
        step = 2.0 ** -8 if r0.dtype == torch.bfloat16 else 2.0 ** -24
        assert ((r1.double() - s).abs() <= step * s.abs() + 2.0 ** -140).all()
        h = r1.double()
    y = _paged.norm(h, w, eps)
    if out is not None:
        assert ((out.double() - y).abs() <= (2.0 ** -8 + _paged.NORM_REL) * y.abs() + 2.0 ** -135).all()
    if codes is not None:
        _paged.check_codes(codes.view(torch.float8_e4m3fn).double(), scales, y, "fp8", _paged.NORM_REL)


@pytest.mark.parametrize("kind", ["none", "bf16", "f32"])
@pytest.mark.parametrize("n,d,pad", [
    (1, 32, 0), (5, 512, 0), (3, 544, 8), (7, 1024, 0), (2, 1056, 0), (64, 4096, 0), (200, 4096, 16), (1, 8192, 0),
    (160, 8192, 0), (3, 8224, 0), (2, 16384, 0), (2, 16416, 0), (1, 32768, 0),   # each chunk count, full and ragged
    (4, 512, 1), (3, 8192, 3), (2, 32768, 1),                                    # rows at odd places
    (1, 1, 0), (9, 33, 0), (2, 1000, 0), (3, 5001, 2), (1, 32767, 0),            # odd lengths (bf16 only)
])
def test_norm(dev, kind, n, d, pad):  # noqa: F811
    x, w, r = _inputs(dev, n, d, kind, 17 * d + n, pad)
    for quant in (False, True) if d % 32 == 0 else (False,):
        res = None if r is None else r.clone() if pad == 0 else torch.empty_strided(
            r.shape, r.stride(), dtype=r.dtype, device=dev).copy_(r)
        codes = torch.full((n, d), 0x55, dtype=torch.uint8, device=dev) if quant else None
        scales = torch.full((n, d // 32), 0x55, dtype=torch.uint8, device=dev) if quant else None
        out = sa.add_rms_norm(x, w, residual=res, eps=EPS, codes=codes, scales=scales)
        assert (out is None) == quant
        _check(x, w, r, res, out, codes, scales)


@pytest.mark.parametrize("kind,d", [("bf16", 4096), ("f32", 4096), ("none", 512), ("f32", 1024)])
def test_rounds_once(dev, kind, d):  # noqa: F811
    """Millions of codes, to within 2^-36 of a border on their own side: of as many rounded to f32 on the way some
    would not be."""
    n, eps = (1 << 22) // d, float(torch.tensor(EPS))
    x, w, r = _inputs(dev, n, d, kind, d)
    codes = torch.empty(n, d, dtype=torch.uint8, device=dev)
    scales = torch.empty(n, d // 32, dtype=torch.uint8, device=dev)
    out = torch.empty(n, d, dtype=torch.bfloat16, device=dev)
    sa.add_rms_norm(x, w, residual=r, eps=EPS, out=out, codes=codes, scales=scales)
    y = _paged.norm((x if r is None else r).double(), w, eps)
    _paged.check_codes(codes.view(torch.float8_e4m3fn).double(), scales, y, "fp8", 2.0 ** -36)
    got = out.double()
    step = _paged.pow2(torch.frexp(torch.maximum(got.abs(), y.abs())).exponent.long() - 9)   # half a step
    assert ((got - y).abs() <= step + 2.0 ** -36 * y.abs()).all()


def test_both_outputs_and_in_place(dev):  # noqa: F811
    x, w, r = _inputs(dev, 37, 1536, "bf16", 5)
    want, res = sa.add_rms_norm(x, w, residual=r.clone()), r.clone()
    xx, codes = x.clone(), torch.empty(37, 1536, dtype=torch.uint8, device=dev)
    scales = torch.empty(37, 48, dtype=torch.uint8, device=dev)
    got = sa.add_rms_norm(xx, w, residual=res, out=xx, codes=codes, scales=scales)
    assert got is xx and torch.equal(xx, want)
    _check(x, w, r, res, xx, codes, scales)
    alone = torch.empty_like(codes), torch.empty_like(scales)
    sa.add_rms_norm(x, w, residual=r.clone(), codes=alone[0], scales=alone[1])
    assert torch.equal(alone[0], codes) and torch.equal(alone[1], scales)


def test_wide_and_any_alignment_agree(dev):  # noqa: F811
    """A row at an odd place takes another kernel: its y is the same up to the sum's own rounding."""
    x, w, _ = _inputs(dev, 50, 4096, "none", 6)
    odd = torch.empty(50, 4097, dtype=torch.bfloat16, device=dev)[:, 1:]
    odd.copy_(x)
    a, b = sa.add_rms_norm(x, w).double(), sa.add_rms_norm(odd, w).double()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs()).all() and (a != b).double().mean() < 1e-3


def test_extremes(dev):  # noqa: F811
    n, d = 6, 256
    x = torch.zeros(n, d, device=dev)
    w = torch.ones(d, device=dev)
    x[1] = 1e-30
    x[2] = 1e18                                     # (its squares' sum is the largest that f32 holds, about)
    x[3, 5] = 1.0
    x[4] = 1e-3
    x[5] = torch.arange(d, device=dev) - 100.0
    x = x.to(torch.bfloat16)
    codes, scales = torch.empty(n, d, dtype=torch.uint8, device=dev), torch.empty(n, 8, dtype=torch.uint8, device=dev)
    _check(x, w, None, None, sa.add_rms_norm(x, w), None, None)
    sa.add_rms_norm(x, w, codes=codes, scales=scales)
    _check(x, w, None, None, None, codes, scales)
    assert (sa.add_rms_norm(x[:1], w) == 0).all()
    # a NaN or an infinity in a row is that row's alone
    bad = x.clone()
    bad[1, 7], bad[4, 9] = float("nan"), float("inf")
    got, want = sa.add_rms_norm(bad, w), sa.add_rms_norm(x, w)
    assert got[1].isnan().all() and torch.equal(got[[0, 2, 3, 5]], want[[0, 2, 3, 5]])
    assert got[4, 9].isnan() and (got[4, :9] == 0).all()
    # a weight beyond 8 bits' largest value saturates with its block's scale; zero weights give zeros
    w2 = w.clone()
    w2[:32], w2[32:64] = float("inf"), 0.0
    sa.add_rms_norm(x[5:], w2, codes=codes[5:], scales=scales[5:])
    v = codes[5].view(torch.float8_e4m3fn).float()
    assert (v[:32].abs() == 448).all() and (v[32:64] == 0).all() and (scales[5] < 255).all()


@pytest.mark.parametrize("d", [64, 512, 4096])
def test_squares_at_the_edges_of_f32(dev, d):  # noqa: F811
    """One element whose square is all but the largest that f32 holds, rows of few or of many magnitudes, and squares
    below the smallest normal."""
    x = torch.zeros(5, d, device=dev)
    x[0, 3] = 1.7e19
    x[1, 3], x[1, 40] = 1e19, -1.2e19
    x[2] = 2.0 ** torch.linspace(-30, 62 - 0.5 * math.log2(d), d, device=dev)
    x[3] = 2.0 ** torch.linspace(-60, 0, d, device=dev).flip(0)
    x[4] = 3e-23                                     # (eps is all of the mean)
    x = x.to(torch.bfloat16)
    w = torch.linspace(0.5, 1.5, d, device=dev)
    _check(x, w, None, None, sa.add_rms_norm(x, w), None, None)
    _check(x[:4], w, None, None, sa.add_rms_norm(x[:4], w, eps=0.0), None, None, eps=0.0)


def test_rows_of_nothing(dev):  # noqa: F811
    w = torch.ones(64, device=dev)
    assert sa.add_rms_norm(torch.empty(0, 64, dtype=torch.bfloat16, device=dev), w).shape == (0, 64)


def test_graph_and_stream(dev):  # noqa: F811
    """Captured once and replayed on new contents; on a stream of its own, out comes from that stream."""
    x, w, r = _inputs(dev, 33, 2048, "f32", 8)
    res = r.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = sa.add_rms_norm(x, w, residual=res, stream=side)
    side.synchronize()
    _check(x, w, r, res, out, None, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sa.add_rms_norm(x, w, residual=res)
    for seed in (9, 10):
        x2, _, r2 = _inputs(dev, 33, 2048, "f32", seed)
        x.copy_(x2)
        res.copy_(r2)
        graph.replay()
        _check(x, w, r2, res, out, None, None)


def _far_rows(dev, d):  # noqa: F811
    """f32 rows whose squares, or the sum of them, are below or beyond what f32 holds."""
    g = torch.Generator(device=dev).manual_seed(d)
    z = torch.randn(12, d, device=dev, generator=g)
    for i, m in enumerate((1e-12, 1e-18, 1e-21, 3e-23, 1e-30, 1e-37, 2e-38, 1e20, 1e25, 6e37)):
        z[i] *= m
    z[9].clamp_(-3e38, 3e38)
    z[10] *= torch.where(torch.arange(d, device=dev) % 3 == 0, 1e22, 1.0)   # large ones, and others beside them
    z[11] = 0.0
    z[11, d // 2] = 4e-39                                                   # one element, below the smallest normal
    return z


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, EPS])
@pytest.mark.parametrize("kind", ["none", "bf16", "f32"])
@pytest.mark.parametrize("d,pad", [(64, 0), (512, 0), (1024, 0), (4096, 0), (8192, 0), (32768, 0), (512, 1), (33, 0)])
def test_squares_outside_f32(dev, d, pad, kind, eps):  # noqa: F811
    """Rows of any magnitude, with an eps that is none, or less than they are: y is the formula's."""
    z = _far_rows(dev, d)
    eps = float(torch.tensor(eps))
    w = torch.linspace(0.5, 1.5, d, device=dev)
    wide = torch.zeros(12, d + pad, dtype=torch.bfloat16, device=dev)[:, :d]
    r = None
    if kind == "none":
        wide.copy_(z)
    else:
        r = z.to(torch.bfloat16) if kind == "bf16" else z
    res = None if r is None else r.clone()
    out = sa.add_rms_norm(wide, w, residual=res, eps=eps)
    _check(wide, w, r, res, None, None, None)
    y = _paged.norm(wide if r is None else res, w, eps)
    # (bf16's smallest number is 2^-133: below the normal ones a rounding is off by up to 2^-134)
    assert ((out.double() - y).abs() <= (2.0 ** -8 + _paged.NORM_REL) * y.abs() + 2.0 ** -134).all()
    if d % 32 == 0:
        codes = torch.empty(12, d, dtype=torch.uint8, device=dev)
        scales = torch.empty(12, d // 32, dtype=torch.uint8, device=dev)
        res = None if r is None else r.clone()
        sa.add_rms_norm(wide, w, residual=res, eps=eps, codes=codes, scales=scales)
        _check(wide, w, r, res, None, codes, scales, eps=eps)


@pytest.mark.parametrize("d", [512, 4096, 96])
def test_rows_between_one_another(dev, d):  # noqa: F811
    """Codes and scales side by side in a row; x, the residual and out as columns of one buffer: no byte is another's."""
    x, w, r = _inputs(dev, 9, d, "bf16", d)
    both = torch.full((9, d + d // 32), 0x55, dtype=torch.uint8, device=dev)
    codes, scales = both[:, :d], both[:, d:]
    wide = torch.cat([x, r, torch.full_like(x, 5.0), torch.full((9, 8), 7.0, dtype=x.dtype, device=dev)], 1)
    sa.add_rms_norm(wide[:, :d], w, residual=wide[:, d:2 * d], out=wide[:, 2 * d:3 * d], codes=codes, scales=scales)
    assert torch.equal(wide[:, :d], x) and (wide[:, 3 * d:] == 7.0).all()
    _check(x, w, r, wide[:, d:2 * d], wide[:, 2 * d:3 * d], codes, scales)
    with pytest.raises(sa.SparseAttnError):   # (a column further: the residual's last)
        sa.add_rms_norm(wide[:, :d], w, residual=wide[:, d:2 * d], out=wide[:, 2 * d - 1:3 * d - 1])
    with pytest.raises(sa.SparseAttnError):
        sa.add_rms_norm(x, w, codes=codes, scales=both[:, d - 1:d - 1 + d // 32])
    with pytest.raises(sa.SparseAttnError):   # (rows of another distance)
        sa.add_rms_norm(wide[:, :d], w, out=wide.view(-1)[d:].as_strided((9, d), (wide.stride(0) - 8, 1)))
