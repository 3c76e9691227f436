"""The 4-bit cache on the GPU: quantiser, ring write, sparse_attn over it, and the log-sum-exp output,
against plain 64-bit implementations."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import sparse_latent_attention_gb300 as sa
from sparse_latent_attention_gb300 import _lib, build, workloads
from tests import _cache, _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    sa.load()
    return torch.device("cuda:0")


# --------------------------------------------------------------------------------------------
# quantiser and ring write: bit-exact
# --------------------------------------------------------------------------------------------

def _rows(rng, n, d, special=True):
    x = rng.standard_normal((n, d)).astype(np.float32)
    x *= np.exp(rng.uniform(-60, 60, (n, d // 32))).repeat(32, axis=1).astype(np.float32)
    bits = workloads.to_bf16_bits(x)
    if special and n >= 8:
        bits[0] = 0                                     # zeros, and zeros with a sign
        bits[1] = 0x8000
        bits[2, :32] = workloads.to_bf16_bits(np.float32([6.0] + [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0,
                                                                  -0.25, -5.0] * 3 + [0.0] * 4))
        bits[3, :32] = 0x40C1                           # just above 6: the next scale
        bits[4, :32] = workloads.to_bf16_bits(np.float32([1e-6, -2e-5] * 16))  # below the floor
        bits[5, :4] = [0x7F80, 0xFF80, 0x7FC0, 0xFFC1]  # infinities and NaNs
        bits[6, :32] = 0x7F7F                           # the largest finite value
        bits[7, :32] = [0x7FC0, 0xFFFF] * 16            # nothing but NaNs
    return bits


@pytest.mark.parametrize("n,d,stride,offset", [
    (1, 32, 32, 0), (9, 64, 64, 0), (300, 512, 512, 0), (97, 512, 520, 8), (40, 96, 96, 0),
    (33, 512, 513, 0), (33, 512, 512, 1), (1000, 1024, 1024, 0)])
def test_act_quant_fp4_bit_exact(dev, n, d, stride, offset):
    bits = _rows(np.random.default_rng(n + d), n, d)
    want_c, want_s, want_v = _cache.quantise(bits)
    buf = torch.zeros(n * stride + offset + 8, dtype=torch.bfloat16, device=dev)
    x = buf[offset:offset + n * stride].view(n, stride)[:, :d]
    x.copy_(_gpu.u16_to_bf16_tensor(bits, dev))
    rt = torch.full((n + 1, d), 7.0, dtype=torch.bfloat16, device=dev)
    codes = torch.full((n + 1, d // 2), 0xAB, dtype=torch.uint8, device=dev)
    scales = torch.full((n + 1, d // 32), 0x55, dtype=torch.uint8, device=dev)
    sa.act_quant_fp4(x, out_rt=rt[:n], codes=codes[:n], scales=scales[:n])
    assert (scales[:n].cpu().numpy() == want_s).all()
    assert (codes[:n].cpu().numpy() == want_c).all()
    assert np.array_equal(rt[:n].double().cpu().numpy(), want_v)
    assert np.array_equal(np.signbit(rt[:n].double().cpu().numpy()), np.signbit(want_v))
    # the row behind the last is left alone
    assert (rt[n] == 7.0).all() and (codes[n] == 0xAB).all() and (scales[n] == 0x55).all()
    # one output at a time, strided codes, and in place
    wide = torch.full((n, d // 2 + 3), 0xAB, dtype=torch.uint8, device=dev)
    sa.act_quant_fp4(x, codes=wide[:, 1:1 + d // 2])
    assert (wide[:, 1:1 + d // 2].cpu().numpy() == want_c).all()
    assert (wide[:, 0] == 0xAB).all() and (wide[:, 1 + d // 2:] == 0xAB).all()
    sa.act_quant_fp4(x, out_rt=x)
    assert np.array_equal(x.double().cpu().numpy(), want_v)


def test_act_quant_fp4_every_bf16_value(dev):
    allv = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    mag = ((allv & 0x7FFF).astype(np.uint32) << 16).view(np.float32)
    for amax in (6.0, 4.0, 1e-3, 3e30):
        keep = allv[mag <= amax]
        blk = np.zeros((len(keep) + 30) // 31 * 31, np.uint16)
        blk[:len(keep)] = keep
        blk = blk.reshape(-1, 31)
        top = np.full((len(blk), 1), workloads.to_bf16_bits(np.float32([amax]))[0], np.uint16)
        rows = np.concatenate([blk, top], axis=1)
        want_c, want_s, want_v = _cache.quantise(rows)
        x = _gpu.u16_to_bf16_tensor(rows, dev)
        codes = torch.empty((len(rows), 16), dtype=torch.uint8, device=dev)
        scales = torch.empty((len(rows), 1), dtype=torch.uint8, device=dev)
        rt = torch.empty_like(x)
        sa.act_quant_fp4(x, out_rt=rt, codes=codes, scales=scales)
        assert (codes.cpu().numpy() == want_c).all(), amax
        assert (scales.cpu().numpy() == want_s).all(), amax
        assert np.array_equal(rt.double().cpu().numpy(), want_v), amax


@pytest.mark.parametrize("nb,seqlen,start,window,rows,d", [
    (1, 12, 0, 8, 8, 512), (2, 12, 5, 8, 20, 64), (3, 1, 13, 8, 30, 512), (3, 1, 32768, 128, 300, 512),
    (1, 300, 0, 128, 128, 96), (2, 5, 0, 8, 8, 512), (1, 1, 2**40 + 3, 7, 9, 32)])
def test_window_write_fp4_bit_exact(dev, nb, seqlen, start, window, rows, d):
    bits = _rows(np.random.default_rng(nb + seqlen), nb * seqlen, d)
    codes, scales, values = (a.reshape(nb, seqlen, -1) for a in _cache.quantise(bits))
    want_c = np.full((nb, rows, d // 2), 0xAB, np.uint8)
    want_s = np.full((nb, rows, d // 32), 0x55, np.uint8)
    want_v = np.full((nb, rows, d), 7.0)
    for t in range(seqlen):
        slot = (start + t) % window
        want_c[:, slot], want_s[:, slot], want_v[:, slot] = codes[:, t], scales[:, t], values[:, t]
    c = torch.full((nb, rows, d // 2), 0xAB, dtype=torch.uint8, device=dev)
    s = torch.full((nb, rows, d // 32), 0x55, dtype=torch.uint8, device=dev)
    rt = torch.full((nb, rows, d), 7.0, dtype=torch.bfloat16, device=dev)
    x = _gpu.u16_to_bf16_tensor(bits, dev).view(nb, seqlen, d)
    sa.window_write_fp4(x, start, codes=c[:, :window], scales=s[:, :window], ring_rt=rt[:, :window])
    assert (c.cpu().numpy() == want_c).all()
    assert (s.cpu().numpy() == want_s).all()
    assert np.array_equal(rt.double().cpu().numpy(), want_v)


# --------------------------------------------------------------------------------------------
# sparse_attn over a 4-bit cache, and lse
# --------------------------------------------------------------------------------------------

def inputs(dev, fmt, b, s, h, d, rows, topk, seed, neg=0.1, empty=(), distinct=True, q_scale=1.0,
           sink_scale=1.0):
    """q, kv, kv_scale, sink, idx of a call; kv in format fmt of N(0, 1) rows."""
    g = torch.Generator(device=dev).manual_seed(seed)
    q = (torch.randn(b, s, h, d, device=dev, generator=g) * q_scale).to(torch.bfloat16)
    sink = torch.randn(h, device=dev, generator=g) * sink_scale
    kv = torch.randn(b, rows, d, device=dev, generator=g).to(torch.bfloat16)
    if distinct and topk <= rows:
        idx = torch.rand(b, s, rows, device=dev, generator=g).argsort(-1)[..., :topk]
    else:
        idx = torch.randint(0, max(rows, 1), (b, s, topk), device=dev, generator=g)
    drop = torch.rand(b, s, topk, device=dev, generator=g) < neg
    idx = torch.where(drop, -1, idx).to(torch.int32).contiguous()
    for t in empty:
        idx.view(-1, topk)[t] = -1
    if fmt == "bf16":
        return q, kv, None, sink, idx
    codes = torch.empty(b, rows, d if fmt == "fp8" else d // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(b, rows, d // 32, dtype=torch.uint8, device=dev)
    quant = sa.act_quant_fp8 if fmt == "fp8" else sa.act_quant_fp4
    quant(kv.view(-1, d), codes=codes.view(b * rows, -1), scales=scales.view(b * rows, -1))
    return q, codes, scales, sink, idx


def check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    # (equal infinities are equal)
    bad &= ~(torch.isinf(want) & (got.double() == want))
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), got.double()[bad][:4], want[bad][:4], tol[bad][:4])


CASES = [
    # b, s, h, d, rows, topk, extra
    (1, 1, 64, 512, 700, 640, {}),                       # one token, split idx columns
    (3, 1, 64, 512, 5000, 1152, {}),                     # decode: pieces merged
    (2, 1, 128, 512, 3001, 2176, {}),                    # two head blocks
    (2, 37, 64, 512, 300, 200, {}),                      # ragged tail
    (1, 9, 100, 512, 700, 650, {}),                      # partial head block
    (1, 12, 8, 512, 200, 130, {}),
    (1, 5, 1, 512, 3, 1, {}),                            # one head, one entry
    (1, 13, 64, 512, 64, 64, dict(distinct=False)),      # repeated rows
    (2, 30, 64, 512, 90, 200, dict(distinct=False)),
    (1, 300, 64, 512, 640, 128, dict(neg=0.0)),          # more tokens than SMs
    (2, 9, 64, 512, 400, 130, dict(neg=0.97)),           # nearly everything masked
    (2, 7, 64, 512, 400, 130, dict(q_scale=8.0)),        # large logits
    (1, 8, 64, 512, 100, 100, dict(sink_scale=60.0)),    # sinks far from the logits
    (1, 20, 4, 64, 48, 16, {}),                          # the other head dims
    (2, 11, 100, 192, 90, 70, {}),
    (1, 13, 64, 256, 640, 513, {}),
    (3, 1, 16, 128, 900, 700, {}),
    (1, 3, 64, 448, 90, 65, {}),
    (2, 5, 70, 320, 200, 140, {}),
    (1, 4, 128, 384, 300, 257, {}),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}s{c[1]}h{c[2]}d{c[3]}k{c[5]}")
def test_sparse_attn_fp4(dev, case):
    b, s, h, d, rows, topk, extra = case
    empty = (b * s - 1,) if b * s > 1 else ()
    q, kv, sc, sink, idx = inputs(dev, "fp4", b, s, h, d, rows, topk, 31 * b + s + topk, empty=empty, **extra)
    lse = torch.full((b, s, h), 99.0, device=dev)
    ws = sa.new_workspace(b, s, h, d, rows, topk, sa.SA_KV_FP4_E2M1)
    o = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse, workspace=ws)
    assert sa.read_status(ws) == 0
    want, want_lse, o_tol, lse_tol = _cache.attention(q, _cache.rows_f64(kv, sc, d), sink, idx, d ** -0.5)
    check(o, want, o_tol, "o")
    check(lse, want_lse, lse_tol, "lse")
    for t in empty:
        assert (o.view(-1, h, d)[t] == 0).all()
        assert (lse.view(-1, h)[t] == sink).all()
    # the same bits as the round trip's bf16 rows, and as the call without lse
    rt = _cache.rows_f64(kv, sc, d).to(torch.bfloat16)
    lse16 = torch.empty_like(lse)
    o16 = sa.sparse_attn(q, rt, sink, idx, d ** -0.5, lse=lse16)
    assert torch.equal(o.view(torch.int16), o16.view(torch.int16))
    assert torch.equal(lse, lse16)
    plain = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc)
    assert torch.equal(o.view(torch.int16), plain.view(torch.int16))


@pytest.mark.parametrize("family", ["tcgen05", "mma"])
def test_fp4_families(dev, family):
    q, kv, sc, sink, idx = inputs(dev, "fp4", 2, 5, 64, 512, 500, 300, 5)
    o = sa.sparse_attn(q, kv, sink, idx, 512 ** -0.5, kv_scale=sc, family=family)
    want, _, tol, _ = _cache.attention(q, _cache.rows_f64(kv, sc, 512), sink, idx, 512 ** -0.5)
    check(o, want, tol, family)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("b,s,h,d,rows,topk", [(2, 1, 64, 512, 900, 640), (1, 33, 64, 512, 300, 130),
                                               (2, 3, 20, 128, 100, 70), (1, 2, 16, 64, 600, 520)])
def test_lse(dev, fmt, b, s, h, d, rows, topk):
    q, kv, sc, sink, idx = inputs(dev, fmt, b, s, h, d, rows, topk, 77 + s, empty=(1,))
    sink[0], sink[1], sink[2] = -torch.inf, 300.0, -300.0  # no sink; a sink that is the whole denominator
    lse = torch.empty(b, s, h, device=dev)
    o = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse)
    plain = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc)
    assert torch.equal(o.view(torch.int16), plain.view(torch.int16))
    _, want, _, tol = _cache.attention(q, _cache.rows_f64(kv, sc, d), sink, idx, d ** -0.5)
    check(lse, want, tol, fmt)


def test_fp4_with_rope_and_lse(dev):
    b, s, h, d = 2, 9, 64, 512
    q, kv, sc, sink, idx = inputs(dev, "fp4", b, s, h, d, 300, 200, 8)
    rot = torch.from_numpy(workloads.rope_table(40, 64, seed=3)).to(dev)
    lse, lse0 = torch.empty(b, s, h, device=dev), torch.empty(b, s, h, device=dev)
    o = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse, rope=(rot, 11))
    o2 = sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, rope=(rot, 11))
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, kv_scale=sc, lse=lse0)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse0)
    want, _, tol, _ = _cache.attention(q, _cache.rows_f64(kv, sc, d), sink, idx, d ** -0.5)
    c, sn = (rot[11:11 + s, :, i].double()[None, :, None, :] for i in (0, 1))
    a, bb = want[..., 448::2].clone(), want[..., 449::2].clone()
    ta, tb = tol[..., 448::2].clone(), tol[..., 449::2].clone()
    want[..., 448::2], want[..., 449::2] = a * c + bb * sn, bb * c - a * sn
    tol[..., 448::2] = tol[..., 449::2] = ta + tb   # |cos|, |sin| <= 1, and the rounding of the result
    check(o, want, tol, "rotated")


@pytest.mark.parametrize("d,s,topk", [(512, 40, 130), (512, 1, 1200), (256, 3, 70)])
def test_lse_of_logits_that_are_not_numbers(dev, d, s, topk):
    """A NaN in a head's q makes that head's lse NaN; the other heads' stay."""
    q, kv, sc, sink, idx = inputs(dev, "bf16", 1, s, 16, d, 1500, topk, 7)
    idx[0, s - 1] = torch.arange(topk, device=dev, dtype=torch.int32)
    want, got = (torch.empty((1, s, 16), dtype=torch.float32, device=dev) for _ in range(2))
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, lse=want)
    q[0, s - 1, 5, 3] = float("nan")
    sa.sparse_attn(q, kv, sink, idx, d ** -0.5, lse=got)
    assert got[0, s - 1, 5].isnan()
    got[0, s - 1, 5] = want[0, s - 1, 5]
    assert torch.equal(got, want)


def test_no_columns_and_no_tokens(dev):
    for d in (512, 128):
        q, kv, sc, sink, idx = inputs(dev, "fp4", 2, 3, 16, d, 40, 0, 9)
        lse = torch.empty(2, 3, 16, device=dev)
        o = sa.sparse_attn(q, kv, sink, idx, 0.1, kv_scale=sc, lse=lse)
        assert (o == 0).all() and (lse == sink).all()
        q0, lse0 = q[:0], lse[:0]
        o = sa.sparse_attn(q0, kv[:0], sink, idx[:0], 0.1, kv_scale=sc[:0], lse=lse0)
        assert o.shape == q0.shape


def test_fp4_rows_are_finite_whatever_their_bytes(dev):
    # every code with every scale byte: a row decodes to finite values, so a tile's unlisted rows
    # cannot disturb the others
    d, h = 512, 64
    g = torch.Generator(device=dev).manual_seed(4)
    kv = torch.randint(0, 256, (1, 256, d // 2), device=dev, generator=g, dtype=torch.uint8)
    sc = torch.arange(256, device=dev, dtype=torch.uint8)[:, None].expand(256, d // 32)[None].contiguous()
    q = torch.zeros(1, 4, h, d, dtype=torch.bfloat16, device=dev)
    sink = torch.full((h,), -torch.inf, device=dev)
    # q = 0: every listed row weighs the same, o is the rows' mean
    idx = torch.tensor([[252, 253, 254, 255], [100, 110, 120, 130], [0, 1, 2, 3], [255, -1, -1, -1]],
                       dtype=torch.int32, device=dev)[None].contiguous()
    kv[0, 252:] &= 0x33                                  # magnitudes to 1.5: sums of four stay finite
    for family in ("tcgen05", "mma"):
        o = sa.sparse_attn(q, kv, sink, idx, 0.1, kv_scale=sc, family=family)
        want, _, tol, _ = _cache.attention(q, _cache.rows_f64(kv, sc, d), sink, idx, 0.1)
        assert torch.isfinite(o.float()).all()
        # (sums of subnormals: a unit of the smallest bf16)
        check(o, want, tol + 2.0 ** -132, family)


def test_fp4_bad_index_sets_status(dev):
    q, kv, sc, sink, idx = inputs(dev, "fp4", 2, 1, 64, 512, 300, 200, 10)
    bad = idx.clone()
    bad[1, 0, 5], bad[0, 0, 7] = 300, -2
    ws = sa.new_workspace(2, 1, 64, 512, 300, 200, sa.SA_KV_FP4_E2M1)
    o = sa.sparse_attn(q, kv, sink, bad, 0.05, kv_scale=sc, workspace=ws)
    assert sa.read_status(ws, clear=True) == 4
    good = torch.where((bad >= 300) | (bad < -1), -1, bad)
    o2 = sa.sparse_attn(q, kv, sink, good, 0.05, kv_scale=sc, workspace=ws)
    assert sa.read_status(ws) == 0 and torch.equal(o, o2)


# --------------------------------------------------------------------------------------------
# calls at the edges
# --------------------------------------------------------------------------------------------

def test_quant_rows_gigabytes_apart(dev):
    """Row offsets past 32 bits: a stride of 1 GB (32-bit products), and one past 2^31 elements."""
    rng = np.random.default_rng(3)
    for n, stride in ((6, (1 << 29) + 8), (3, (1 << 31) + 8)):
        bits = _rows(rng, n, 64, special=False)
        want_c, want_s, want_v = _cache.quantise(bits)
        buf = torch.empty((n - 1) * stride + 64, dtype=torch.bfloat16, device=dev)
        x = buf.as_strided((n, 64), (stride, 1))
        x.copy_(_gpu.u16_to_bf16_tensor(bits, dev))
        codes = torch.empty(n, 32, dtype=torch.uint8, device=dev)
        scales = torch.empty(n, 2, dtype=torch.uint8, device=dev)
        sa.act_quant_fp4(x, codes=codes, scales=scales, out_rt=x)
        assert (codes.cpu().numpy() == want_c).all() and (scales.cpu().numpy() == want_s).all()
        assert np.array_equal(x.double().cpu().numpy(), want_v)
        del buf, x


def far_inputs(dev, fmt, b, rows, h, d, topk, seed):
    """inputs() over a long cache: only the rows that idx names are filled (the others hold whatever the
    memory holds), among them the first and the last."""
    q, kv, sc, sink, _ = inputs(dev, fmt, b, 1, h, d, topk, topk, seed, neg=0.0)
    g = torch.Generator(device=dev).manual_seed(seed)
    at = torch.stack([torch.randperm(rows - 2, device=dev, generator=g)[:topk] + 1 for _ in range(b)])
    at[:, 0], at[:, -1] = 0, rows - 1
    bi = torch.arange(b, device=dev)[:, None]
    far = torch.empty((b, rows, kv.shape[2]), dtype=kv.dtype, device=dev)
    far[bi, at] = kv
    far_sc = None
    if sc is not None:
        far_sc = torch.empty((b, rows, sc.shape[2]), dtype=sc.dtype, device=dev)
        far_sc[bi, at] = sc
    near = torch.arange(topk, device=dev, dtype=torch.int32).expand(b, 1, topk).contiguous()
    return q, (kv, sc, near), (far, far_sc, at.to(torch.int32)[:, None].contiguous()), sink


@pytest.mark.parametrize("d", [512, 256])
def test_fp4_cache_past_32_bits(dev, d):
    rows = (1 << 32) // (d // 2) // 2 + 4000   # two sequences: codes past 4 GB
    q, (kv, sc, near), (far, far_sc, idx), sink = far_inputs(dev, "fp4", 2, rows, 64, d, 200, 12)
    lse = torch.empty(2, 1, 64, device=dev)
    o = sa.sparse_attn(q, far, sink, idx, d ** -0.5, kv_scale=far_sc, lse=lse)
    want, want_lse, tol, lse_tol = _cache.attention(q, _cache.rows_f64(kv, sc, d), sink, near, d ** -0.5)
    check(o, want, tol, "o")
    check(lse, want_lse, lse_tol, "lse")


def test_fp4_nothing_listed_and_no_rows(dev):
    for d in (512, 64):
        q, kv, sc, sink, idx = inputs(dev, "fp4", 2, 3, 16, d, 40, 70, 9, neg=1.1, distinct=False)
        lse = torch.empty(2, 3, 16, device=dev)
        assert (idx == -1).all()
        o = sa.sparse_attn(q, kv, sink, idx, 0.1, kv_scale=sc, lse=lse)
        assert (o == 0).all() and (lse == sink).all()
        o = sa.sparse_attn(q, kv[:, :0].contiguous(), sink, idx, 0.1, kv_scale=sc[:, :0].contiguous(), lse=lse)
        assert (o == 0).all() and (lse == sink).all()


def test_fp4_through_the_static_scratch(dev):
    q, kv, sc, sink, idx = inputs(dev, "fp4", 3, 1, 64, 512, 900, 640, 14)
    want = sa.sparse_attn(q, kv, sink, idx, 0.05, kv_scale=sc)
    o = torch.empty_like(q)
    P = ctypes.c_void_p
    st = _lib.load().sa_sparse_attn_static_scratch(
        P(q.data_ptr()), P(kv.data_ptr()), P(sc.data_ptr()), 2, P(sink.data_ptr()), P(idx.data_ptr()),
        ctypes.c_float(0.05), ctypes.c_int64(3), ctypes.c_int64(1), 64, 512, ctypes.c_int64(900), 640,
        P(o.data_ptr()), None, P(torch.cuda.current_stream().cuda_stream))
    assert st == 0 and torch.equal(o, want)


def test_two_graphs_share_a_workspace(dev):
    """Two captured decode steps that use one workspace, replayed in turn on one stream."""
    scale = 512 ** -0.5
    sets = [inputs(dev, "fp4", 2, 1, 64, 512, 700, 640, seed) for seed in (1, 2)]
    ws = sa.new_workspace(2, 1, 64, 512, 700, 640, sa.SA_KV_FP4_E2M1)
    want = [sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc).clone() for q, kv, sc, sink, idx in sets]
    outs = [torch.empty_like(s[0]) for s in sets]
    graphs = []
    for (q, kv, sc, sink, idx), o in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_two_streams_at_once(dev):
    """Calls with workspaces of their own on two streams at the same time."""
    scale = 512 ** -0.5
    sets = [inputs(dev, fmt, 4, 1, 64, 512, 2000, 1152, 5) for fmt in ("fp4", "fp8")]
    want = [sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc) for q, kv, sc, sink, idx in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, ((q, kv, sc, sink, idx), st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append(sa.sparse_attn(q, kv, sink, idx, scale, kv_scale=sc))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)
