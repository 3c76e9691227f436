"""The C ABI of the 4-bit cache and of eviction without a GPU: every declared symbol is there, and bad
arguments are refused before anything touches CUDA."""

from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from sparse_latent_attention_gb300 import _lib, build

INVALID, UNSUPPORTED, WORKSPACE, OK = (_lib.SA_ERR_INVALID_ARG, _lib.SA_ERR_UNSUPPORTED,
                                       _lib.SA_ERR_WORKSPACE, _lib.SA_OK)


def at(n, off=0):
    """An address that is never read: every call below fails its checks or has nothing to do."""
    return ctypes.c_void_p((n << 40) + off)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols("cache")
    assert set(names) == {"sa_act_quant_fp4", "sa_window_write_fp4", "sa_sparse_attn_lse", "sa_row_weights",
                          "sa_evict_select", "sa_compact_rows", "sa_remap_idx"}
    for n in names:
        assert hasattr(lib, n), n


def test_fp4_is_a_kv_format(lib):
    f = lib.sa_sparse_attn_workspace_size
    for d in (64, 512):
        assert f(64, 1, 64, d, 8320, 1152, 2) == f(64, 1, 64, d, 8320, 1152, 1)
    call = [at(1), at(2), None, 2, at(3), at(4), 0.1, 1, 2, 4, 64, 8, 4, at(5), None, 0, None]
    assert lib.sa_sparse_attn(*call) == INVALID           # no scales
    call[2] = at(6)
    assert lib.sa_sparse_attn(*call) == WORKSPACE         # nothing else is wrong
    call[10], call[2] = 512, at(6, 8)
    assert lib.sa_sparse_attn(*call) == INVALID           # scales not 16-byte aligned
    call[2], call[13] = at(6), at(2, 8 * 256 - 16)
    assert lib.sa_sparse_attn(*call) == INVALID           # o in the codes' last row
    call[13] = at(2, 8 * 256)
    assert lib.sa_sparse_attn(*call) == WORKSPACE         # o right behind them


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(d=33), INVALID), (dict(d=0), INVALID), (dict(n=-1), INVALID),
    (dict(n=1, x=None), INVALID), (dict(n=1, xs=63), INVALID), (dict(n=1, rt=None, codes=None, scales=None), INVALID),
    (dict(n=1, rts=63), INVALID), (dict(n=1, cs=31), INVALID), (dict(n=1, ss=1), INVALID),
    (dict(n=1, x=at(1, 1)), INVALID), (dict(n=1, rt=at(2, 1)), INVALID),
    (dict(n=2, rt=at(1, 64)), INVALID),                   # a shifted overlap
    (dict(n=2, rt=at(1), rts=128), INVALID),              # in place with another stride
    (dict(n=2, codes=at(1, 100)), INVALID), (dict(n=2, scales=at(1, 100)), INVALID),
    (dict(n=2, codes=at(2, 100)), INVALID), (dict(n=2, scales=at(3, 10)), INVALID),
])
def test_act_quant_fp4_refuses(lib, change, code):
    a = dict(x=at(1), n=0, d=64, xs=64, rt=at(2), rts=64, codes=at(3), cs=32, scales=at(4), ss=2)
    a.update(change)
    assert lib.sa_act_quant_fp4(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(nb=0), OK), (dict(sl=0), OK), (dict(d=40), INVALID), (dict(window=0), INVALID),
    (dict(start=-1), INVALID), (dict(rt=None, codes=None, scales=None), INVALID), (dict(x=None), INVALID),
    (dict(xs=60), INVALID), (dict(rts=60), INVALID), (dict(cs=31), INVALID), (dict(ss=1), INVALID),
    (dict(rtb=8 * 64 - 1), INVALID), (dict(cb=8 * 32 - 1), INVALID), (dict(sb=8 * 2 - 1), INVALID),
    (dict(rt=at(1)), INVALID), (dict(codes=at(1, 8)), INVALID), (dict(scales=at(1, 8)), INVALID),
])
def test_window_write_fp4_refuses(lib, change, code):
    a = dict(x=at(1), nb=2, sl=3, d=64, xs=64, start=5, window=8, rt=at(2), rts=64, rtb=8 * 64, codes=at(3),
             cs=32, cb=8 * 32, scales=at(4), ss=2, sb=16)
    a.update(change)
    assert lib.sa_window_write_fp4(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    ({}, WORKSPACE), (dict(lse=None), INVALID), (dict(lse=at(6, 2)), INVALID), (dict(lse=at(5, 64)), INVALID),
    (dict(lse=at(1)), INVALID), (dict(lse=at(2)), INVALID), (dict(lse=at(3)), INVALID), (dict(lse=at(4)), INVALID),
    (dict(fmt=3), INVALID), (dict(fmt=2), INVALID), (dict(b=0, lse=None), OK),
    (dict(rot=at(7)), WORKSPACE), (dict(rot=at(7), rope_dim=63), INVALID), (dict(rot=at(7), start=15), INVALID),
    (dict(rot=at(7), d=256), UNSUPPORTED), (dict(rope_dim=63), WORKSPACE), (dict(rot=at(6)), INVALID),
    (dict(ws=at(8), ws_bytes=1 << 20, lse=at(8, 128)), INVALID),
])
def test_sparse_attn_lse_refuses(lib, change, code):
    a = dict(q=at(1), kv=at(2), kv_scale=None, fmt=0, sink=at(3), idx=at(4), scale=0.1, b=1, s=2, h=64, d=512,
             rows=8, topk=4, o=at(5), lse=at(6), ws=None, ws_bytes=0, rot=None, npos=16, rope_dim=64, start=3)
    a.update(change)
    assert lib.sa_sparse_attn_lse(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    ({}, WORKSPACE), (dict(b=0, q=None), OK), (dict(topk=0, idx=None), OK), (dict(fmt=3), INVALID),
    (dict(fmt=1), INVALID), (dict(kv_scale=at(9)), INVALID), (dict(fmt=2, kv_scale=at(9, 4)), INVALID),
    (dict(fmt=2, kv_scale=at(9)), WORKSPACE), (dict(h=0), INVALID), (dict(h=129), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(topk=-1), INVALID), (dict(q=None), INVALID), (dict(kv=None), INVALID),
    (dict(lse=None), INVALID), (dict(idx=None), INVALID), (dict(acc=None), INVALID),
    (dict(acc=at(6, 4)), INVALID), (dict(q=at(1, 8)), INVALID), (dict(kv=at(2, 8)), INVALID),
    (dict(acc=at(1, 64)), INVALID), (dict(acc=at(2, 64)), INVALID), (dict(acc=at(3)), INVALID),
    (dict(acc=at(4)), INVALID), (dict(rows=0, kv=None, acc=None), WORKSPACE),
    (dict(ws=at(8), ws_bytes=255), WORKSPACE), (dict(ws=at(8, 64), ws_bytes=256), INVALID),
    (dict(ws=at(6), ws_bytes=256), INVALID), (dict(topk=2**31 - 1), UNSUPPORTED),
    (dict(topk=2**31 - 129), WORKSPACE),
])
def test_row_weights_refuses(lib, change, code):
    a = dict(q=at(1), kv=at(2), kv_scale=None, fmt=0, lse=at(3), idx=at(4), scale=0.1, b=1, s=2, h=64, d=512,
             rows=8, topk=4, acc=at(6), ws=None, ws_bytes=0)
    a.update(change)
    assert lib.sa_row_weights(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(b=0), OK), (dict(rows=0, keep=0, first=0, last=0), OK), (dict(keep=101), INVALID),
    (dict(keep=-1), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=40, last=11), INVALID), (dict(first=51, last=0), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows=(1 << 31) - 65535), UNSUPPORTED), (dict(rows=(1 << 31) - 65536, acc=None), INVALID),
    (dict(first=2**63 - 1, last=2**63 - 1), INVALID), (dict(acc=None), INVALID), (dict(kept=None), INVALID),
    (dict(remap=None), INVALID), (dict(acc=at(1, 4)), INVALID), (dict(kept=at(3, 2)), INVALID),
    (dict(live=at(2, 2)), INVALID), (dict(kept=at(1, 8)), INVALID), (dict(remap=at(1, 8)), INVALID),
    (dict(kept=at(4, 8)), INVALID), (dict(kept=at(2)), INVALID), (dict(remap=at(2)), INVALID),
])
def test_evict_select_refuses(lib, change, code):
    a = dict(acc=at(1), live=at(2), b=2, rows=100, keep=50, first=8, last=8, kept=at(3), remap=at(4))
    a.update(change)
    assert lib.sa_evict_select(*a.values(), None) == code


def _compact(lib, src, dst, row, sb, db, b=2, rows=10, keep=5, kept=at(9)):
    n = len(src)
    P, I = ctypes.c_void_p * max(n, 1), ctypes.c_int64 * max(n, 1)
    return lib.sa_compact_rows(n, P(*src), P(*dst), I(*row), I(*sb), I(*db), b, rows, keep, kept, None)


def test_compact_rows_refuses(lib):
    A, B, C = (n << 40 for n in (1, 2, 3))
    ok = ([A], [B], [16], [160], [80])
    assert _compact(lib, *ok, b=0) == OK and _compact(lib, *ok, keep=0) == OK
    assert _compact(lib, [], [], [], [], []) == OK
    assert _compact(lib, [A] * 9, [B] * 9, [16] * 9, [160] * 9, [80] * 9) == INVALID
    assert _compact(lib, *ok, b=-1) == INVALID and _compact(lib, *ok, rows=-1) == INVALID
    assert _compact(lib, *ok, kept=None) == INVALID and _compact(lib, *ok, kept=at(9, 2)) == INVALID
    assert _compact(lib, *ok, rows=1 << 31) == UNSUPPORTED
    for k, v in ((0, [None]), (1, [None]), (2, [0]), (3, [159]), (4, [79])):
        bad = list(ok)
        bad[k] = v
        assert _compact(lib, *bad) == INVALID, k
    assert _compact(lib, [A], [A], [16], [160], [80]) == INVALID            # in place, other distances
    assert _compact(lib, [A], [A], [16], [160], [160], keep=11) == INVALID  # in place, more rows than there are
    assert _compact(lib, [A], [A + 16], [16], [160], [160]) == INVALID      # a shifted overlap
    assert _compact(lib, [A, C], [B, A], [16, 16], [160] * 2, [80] * 2) == INVALID   # into another's source
    assert _compact(lib, [A, C], [B, B + 64], [16, 16], [160] * 2, [80] * 2) == INVALID
    assert _compact(lib, [A], [(9 << 40) - 64], [16], [160], [80]) == INVALID        # into kept


def test_remap_idx_refuses(lib):
    f = lib.sa_remap_idx
    assert f(at(1), 0, 5, at(2), 9, at(3), None) == OK and f(None, 2, 0, at(2), 9, None, None) == OK
    assert f(at(1), -1, 5, at(2), 9, at(3), None) == INVALID
    assert f(None, 2, 5, at(2), 9, at(3), None) == INVALID
    assert f(at(1), 2, 5, None, 9, at(3), None) == INVALID
    assert f(at(1), 2, 5, at(2), 9, at(3, 2), None) == INVALID
    assert f(at(1), 2, 5, at(2), 9, at(1, 8), None) == INVALID       # a shifted overlap
    assert f(at(1), 2, 5, at(2), 9, at(2, 8), None) == INVALID       # over the map


def _host(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: sa.act_quant_fp4(_host(2, 64, dtype=torch.bfloat16), out_rt=_host(2, 64, dtype=torch.bfloat16)),
    lambda: sa.window_write_fp4(_host(1, 2, 64, dtype=torch.bfloat16), 0,
                                ring_rt=_host(1, 2, 64, dtype=torch.bfloat16)),
    lambda: sa.row_weights(_host(1, 2, 4, 64, dtype=torch.bfloat16), _host(1, 8, 64, dtype=torch.bfloat16),
                           _host(1, 2, 4), _host(1, 2, 4, dtype=torch.int32), 0.1,
                           _host(1, 8, dtype=torch.int64)),
    lambda: sa.evict_select(_host(1, 8, dtype=torch.int64), 4),
    lambda: sa.compact_rows([_host(1, 8)], _host(1, 4, dtype=torch.int32)),
    lambda: sa.remap_idx(_host(1, 8, dtype=torch.int32), _host(1, 8, dtype=torch.int32)),
])
def test_host_tensors_are_refused(call):
    with pytest.raises((TypeError, ValueError)):
        call()
