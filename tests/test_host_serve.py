"""The paged cache, its window attention and the residual norm without a GPU: exported symbols, workspace sizes,
and every refusal before anything is enqueued."""

from __future__ import annotations

import ctypes
import os
import random
import re

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from sparse_latent_attention_gb300 import _lib, build

OK, INVALID, UNSUPPORTED, WORKSPACE = (_lib.SA_OK, _lib.SA_ERR_INVALID_ARG, _lib.SA_ERR_UNSUPPORTED,
                                       _lib.SA_ERR_WORKSPACE)


def at(n, off=0):
    """A made-up device address (never dereferenced), far from those of other n."""
    return ctypes.c_void_p((n << 40) + off)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_exports_every_declared_symbol(lib):
    names = _lib.declared_symbols("serve")
    assert set(names) == {"sa_add_rms_norm", "sa_page_write", "sa_window_attn", "sa_window_attn_workspace_size"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("change,code", [
    (dict(n=0, x=None), OK), (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(kind=3), INVALID), (dict(kind=0), INVALID), (dict(res=None), INVALID),
    (dict(out=None, codes=None, scales=None), INVALID), (dict(scales=None), INVALID), (dict(codes=None), INVALID),
    (dict(d=63), INVALID), (dict(d=32800, xs=32800, rs=32800, os=32800, cs=32800, ss=1025), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=at(1, 1)), INVALID), (dict(xs=63), INVALID), (dict(w=None), INVALID),
    (dict(w=at(2, 2)), INVALID), (dict(res=at(3, 1)), INVALID), (dict(kind=2, res=at(3, 2)), INVALID),
    (dict(rs=63), INVALID), (dict(os=63), INVALID), (dict(out=at(4, 1)), INVALID), (dict(cs=63), INVALID),
    (dict(ss=1), INVALID), (dict(out=at(1), os=72), INVALID), (dict(out=at(1, 128)), INVALID),
    (dict(out=at(3)), INVALID), (dict(res=at(1, 2)), INVALID), (dict(codes=at(1, 383)), INVALID),
    (dict(codes=at(4, 10)), INVALID), (dict(scales=at(5, 191)), INVALID), (dict(scales=at(3, 383)), INVALID),
    (dict(out=at(2, 254)), INVALID), (dict(kind=2, scales=at(3, 767)), INVALID),
])
def test_add_rms_norm_refuses(lib, change, code):
    a = dict(x=at(1), n=3, d=64, xs=64, w=at(2), eps=1e-6, res=at(3), kind=1, rs=64, out=at(4), os=64, codes=at(5),
             cs=64, scales=at(6), ss=2)
    a.update(change)
    assert lib.sa_add_rms_norm(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(n=0, x=None), OK), (dict(b=0, q_start=None), OK), (dict(n=-1), INVALID), (dict(d=40), INVALID),
    (dict(d=0), INVALID), (dict(d=1056, xs=1056, pgs=1056, pgp=1 << 20, cs=1056, ss=40), UNSUPPORTED),
    (dict(n=1 << 31), UNSUPPORTED), (dict(n_pages=1 << 38), UNSUPPORTED),
    (dict(n_pages=1 << 31, page=1), UNSUPPORTED), (dict(n_pages=1 << 62), UNSUPPORTED), (dict(max_pages=1 << 31), UNSUPPORTED),
    (dict(b=1 << 31), UNSUPPORTED), (dict(xs=1 << 62), INVALID), (dict(ts=1 << 62), INVALID), (dict(pgp=1 << 60), INVALID),
    (dict(pgs=1 << 60), INVALID), (dict(cp=1 << 60), INVALID), (dict(ss=1 << 62), INVALID),
    (dict(b=-1), INVALID),
    (dict(n_pages=-1), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID), (dict(max_pages=-1), INVALID), (dict(quant=3), INVALID),
    (dict(quant=0), INVALID), (dict(codes=None, scales=None, pages=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=None), INVALID), (dict(x=at(1, 1)), INVALID), (dict(xs=63), INVALID), (dict(q_start=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(table=None), INVALID), (dict(table=at(2, 2)), INVALID),
    (dict(ts=3), INVALID), (dict(pages=at(5, 1)), INVALID), (dict(pgs=63), INVALID), (dict(pgp=511), INVALID),
    (dict(cs=63), INVALID), (dict(cp=511), INVALID), (dict(ss=1), INVALID), (dict(sp=15), INVALID),
    (dict(w=at(8, 2)), INVALID), (dict(w=at(8), eps=-1.0), INVALID), (dict(rot=at(9, 4)), INVALID),
    (dict(rot=at(9), rope=63), INVALID), (dict(rot=at(9), rope=66), INVALID), (dict(rot=at(9), rope=0), INVALID),
    (dict(rot=at(9), npos=-1), INVALID), (dict(status=at(10, 2)), INVALID),
    (dict(pages=at(1, 64)), INVALID), (dict(codes=at(1, 64)), INVALID), (dict(scales=at(1, 64)), INVALID),
    (dict(codes=at(5, 64)), INVALID), (dict(scales=at(6, 64)), INVALID), (dict(codes=at(2, 4)), INVALID),
    (dict(codes=at(3, 4)), INVALID), (dict(codes=at(4, 4)), INVALID), (dict(w=at(5, 64)), INVALID),
    (dict(rot=at(5, 64)), INVALID), (dict(status=at(6, 64)), INVALID),
])
def test_page_write_refuses(lib, change, code):
    a = dict(x=at(1), n=3, d=64, xs=64, table=at(2), max_pages=4, ts=4, q_start=at(3), kv_len=at(4), b=2, n_pages=10,
             page=8, quant=1, pages=at(5), pgs=64, pgp=512, codes=at(6), cs=64, cp=512, scales=at(7), ss=2, sp=16, w=None,
             eps=1e-6, rot=None, npos=100, rope=64, status=None)
    a.update(change)
    assert lib.sa_page_write(*a.values(), None) == code


def test_page_write_takes_rows_between_one_another(lib):
    """Codes and scales side by side in a row or in a page are no overlap; a byte further they are one.  (The calls
    stop at a misaligned status word, which is looked at first, or at the overlap: neither is enqueued.)"""
    a = dict(x=at(1), n=3, d=64, xs=64, table=at(2), max_pages=4, ts=4, q_start=at(3), kv_len=at(4), b=2, n_pages=10,
             page=8, quant=1, pages=None, pgs=0, pgp=0, codes=at(6), cs=66, cp=528, scales=at(6, 63), ss=66, sp=528,
             w=None, eps=1e-6, rot=None, npos=0, rope=0, status=None)
    assert lib.sa_page_write(*a.values(), None) == INVALID           # the row's last code
    a.update(cs=64, scales=at(6, 511), ss=2)
    assert lib.sa_page_write(*a.values(), None) == INVALID           # the page's last code
    a.update(scales=at(6, 513))
    assert lib.sa_page_write(*a.values(), None) == INVALID           # the next page's first


@pytest.mark.parametrize("change,code", [
    ({}, WORKSPACE), (dict(n=0, q=None), OK), (dict(b=0), OK), (dict(fmt=3), INVALID), (dict(fmt=1), INVALID),
    (dict(scale_ptr=at(9)), INVALID), (dict(fmt=1, scale_ptr=at(9, 4)), INVALID), (dict(fmt=1, scale_ptr=at(9)), WORKSPACE),
    (dict(n=-1), INVALID), (dict(h=0), INVALID), (dict(h=129), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(d=576), UNSUPPORTED), (dict(window=0), INVALID), (dict(window=1 << 30), INVALID), (dict(first=-1), INVALID),
    (dict(first=(1 << 30) - 128), INVALID), (dict(window=1 << 24, max_pages=1 << 18, ts=1 << 18), WORKSPACE),
    (dict(window=1 << 24, max_pages=(1 << 18) + 1, ts=1 << 19), UNSUPPORTED), (dict(window=1 << 29), WORKSPACE),
    (dict(window=(1 << 24) - 4, max_pages=1 << 20, ts=1 << 20), WORKSPACE),
    (dict(page=0), INVALID), (dict(n_pages=-1), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_pages=1 << 25), UNSUPPORTED), (dict(n=1 << 25), UNSUPPORTED),
    (dict(n=1 << 58), UNSUPPORTED), (dict(b=1 << 31), UNSUPPORTED), (dict(max_pages=1 << 31), UNSUPPORTED),
    (dict(n_pages=1 << 62), UNSUPPORTED), (dict(ts=1 << 62), INVALID), (dict(rot=at(10), npos=1 << 60), INVALID),
    (dict(max_pages=-1), INVALID),
    (dict(ts=3), INVALID), (dict(q=None), INVALID), (dict(q=at(1, 8)), INVALID), (dict(kv=None), INVALID),
    (dict(kv=at(2, 8)), INVALID), (dict(sink=None), INVALID), (dict(sink=at(3, 2)), INVALID), (dict(o=None), INVALID),
    (dict(o=at(7, 8)), INVALID), (dict(o=at(7, 16)), INVALID), (dict(o=at(7, 32)), WORKSPACE),
    (dict(o=at(7, 16), page=48), WORKSPACE), (dict(o=at(7, 16), d=256), WORKSPACE), (dict(o=at(7, 8), d=256), INVALID),
    (dict(table=None), INVALID), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID),
    (dict(q_start=at(5, 2)), INVALID), (dict(lse=at(8, 2)), INVALID), (dict(rot=at(10)), WORKSPACE),
    (dict(rot=at(10, 4)), INVALID), (dict(rot=at(10), rope=63), INVALID), (dict(rot=at(10), npos=0), INVALID),
    (dict(rot=at(10), d=256), UNSUPPORTED), (dict(o=at(1)), INVALID), (dict(o=at(2, 64)), INVALID), (dict(o=at(4)), INVALID),
    (dict(o=at(5)), INVALID), (dict(o=at(6)), INVALID), (dict(o=at(3)), INVALID), (dict(lse=at(7, 64)), INVALID),
    (dict(lse=at(1, 64)), INVALID), (dict(lse=at(2, 64)), INVALID), (dict(rot=at(10), lse=at(10)), INVALID),
    (dict(ws=at(11), ws_bytes=255), WORKSPACE), (dict(ws=at(11, 64), ws_bytes=1 << 30), INVALID),
    (dict(ws=at(7), ws_bytes=1 << 30), INVALID), (dict(ws=at(2), ws_bytes=1 << 30), INVALID),
    (dict(lse=at(11, 128), ws=at(11), ws_bytes=1 << 30), INVALID),
])
def test_window_attn_refuses(lib, change, code):
    a = dict(q=at(1), kv=at(2), scale_ptr=None, fmt=0, sink=at(3), table=at(4), max_pages=4, ts=4, q_start=at(5),
             kv_len=at(6), scale=0.1, n=3, b=2, h=64, d=512, n_pages=10, page=64, window=128, first=4, o=at(7), lse=at(8),
             rot=None, npos=100, rope=64, ws=None, ws_bytes=0)
    a.update(change)
    assert lib.sa_window_attn(*a.values(), None) == code


def test_window_attn_workspace_size(lib):
    f = lib.sa_window_attn_workspace_size
    for fmt in (0, 1, 2):
        assert f(0, 0, 64, 512, 128, 4, 64, fmt) >= _lib.SA_STATUS_BYTES
        assert f(8192, 3, 64, 512, 128, 4, 64, fmt) >= _lib.SA_STATUS_BYTES
    for bad in ((-1, 1, 64, 512, 128, 4, 64, 0), (1, 1, 0, 512, 128, 4, 64, 0), (1, 1, 64, 500, 128, 4, 64, 0),
                (1, 1, 64, 512, 0, 4, 64, 0), (1, 1, 64, 512, 128, -1, 64, 0), (1, 1, 64, 512, 128, 4, 0, 0),
                (1, 1, 64, 512, 128, 4, 64, 3), (1 << 25, 1, 64, 512, 128, 4, 64, 0),
                (1 << 58, 1, 64, 512, 128, 4, 64, 0)):
        assert f(*bad) == 0
    with pytest.raises(sa.SparseAttnError):
        sa.window_workspace_size(1, 1, 64, 500, 128, 4, 64)


def test_workspace_size_without_tokens(lib):
    """A batch of no tokens, or of no sequences, over a long table: the status word and no more."""
    for b, s in ((0, 4), (4, 0), (0, 0)):
        for d, fmt in ((512, 0), (512, 1), (512, 2), (128, 0)):
            assert lib.sa_sparse_attn_workspace_size(b, s, 64, d, 4096, 2048, fmt) == _lib.SA_STATUS_BYTES


def test_host_tensors_are_refused():
    """Tensors that are not on a GPU, or of another type, are refused before the library is called."""
    i = dict(dtype=torch.int32)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(TypeError):
        sa.add_rms_norm(x, w)
    with pytest.raises(TypeError):
        sa.page_write(x, torch.zeros(1, 1, **i), torch.zeros(2, **i), torch.zeros(1, **i), pages=torch.zeros(1, 8, 64))
    with pytest.raises(TypeError):
        sa.window_attn(x[:, None], torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1), torch.zeros(1, 1, **i),
                       torch.zeros(2, **i), torch.zeros(1, **i), 1.0, 8)
    with pytest.raises(TypeError):
        sa.add_rms_norm(None, w)


from tests.test_host_calls import DEV, bf16, calls, i32, on_device, u8  # noqa: E402, F401 (calls: a fixture)


def _batch():
    return on_device(2, 3, dtype=i32), on_device(3, dtype=i32), on_device(2, dtype=i32)


SERVE = {
    "sa_add_rms_norm": lambda **kw: sa.add_rms_norm(on_device(4, 64, dtype=bf16), on_device(64),
                                                    **{"out": on_device(4, 64, dtype=bf16), **kw}),
    "sa_page_write": lambda **kw: sa.page_write(on_device(4, 64, dtype=bf16), *_batch(),
                                                **{"pages": on_device(5, 8, 64, dtype=bf16), **kw}),
    "sa_window_attn": lambda **kw: sa.window_attn(
        on_device(4, 2, 64, dtype=bf16), on_device(5, 8, 64, dtype=bf16), on_device(2), *_batch(), 0.1, 8,
        **{"out": on_device(4, 2, 64, dtype=bf16), "workspace": on_device(1024, dtype=u8), **kw}),
}


@pytest.mark.parametrize("name", SERVE)
def test_calls_run_on_their_tensors_device(calls, monkeypatch, name):  # noqa: F811
    """With another device current: that of the tensors is current for the call, on its own stream or the given one."""
    monkeypatch.setattr(sa, "_current_device", lambda: 0)
    SERVE[name]()
    stream = type("Stream", (), {"cuda_stream": 77})()
    SERVE[name](stream=stream)
    assert calls["calls"] == [(name, DEV, 1000 + DEV), (name, DEV, 77)]


@pytest.mark.parametrize("name,kw", [
    ("sa_add_rms_norm", dict(out=torch.zeros(4, 64, dtype=torch.bfloat16))),
    ("sa_add_rms_norm", dict(residual=torch.zeros(4, 64))),
    ("sa_add_rms_norm", dict(codes=torch.zeros(4, 64, dtype=torch.uint8), scales=torch.zeros(4, 2, dtype=torch.uint8))),
    ("sa_page_write", dict(pages=torch.zeros(5, 8, 64, dtype=torch.bfloat16))),
    ("sa_page_write", dict(weight=torch.zeros(64))), ("sa_page_write", dict(rope=torch.zeros(9, 4, 2))),
    ("sa_page_write", dict(workspace=torch.zeros(256, dtype=torch.uint8))),
    ("sa_window_attn", dict(out=torch.zeros(4, 2, 64, dtype=torch.bfloat16))),
    ("sa_window_attn", dict(lse=torch.zeros(4, 2))), ("sa_window_attn", dict(rope=torch.zeros(9, 4, 2))),
    ("sa_window_attn", dict(workspace=torch.zeros(256, dtype=torch.uint8))),
])
def test_tensors_elsewhere_are_refused(calls, monkeypatch, name, kw):  # noqa: F811
    """A host tensor among those of a device: its address never reaches the library."""
    monkeypatch.setattr(sa, "_current_device", lambda: DEV)
    with pytest.raises((TypeError, ValueError)):
        SERVE[name](**kw)
    assert not calls["calls"]


def test_the_widening_warps_stages():
    """window_attn over codes: a warp that widens waits by a phase's parity for a stage of the ring of four, which is
    safe only where it knows that the stage's use before the last has ended: where it had that use itself, and waited for
    its turn then.  So whatever blocks the tasks have, a stage's uses are all of one set of warps.  (Which stages of a task
    a set has is the source's expression.)"""
    with open(os.path.join(build.CSRC, "sa_window_tc.cu")) as f:
        source = f.read()
    start = re.search(r"const int n0 = ([^;]+);\s*int put = n0;.*?for \(int n = n0; n < stages; n \+= 2\)", source, re.S)
    assert start
    start = compile(start[1].replace("(int)", ""), "n0", "eval")
    rng = random.Random(1)
    for _ in range(50):
        seq, owner = 0, {}
        for _ in range(100):
            stages = rng.choice([0, 1, 1, 2, 3, 4, 5, 9])
            for turn in (0, 1):
                for n in range(eval(start, {"turn": turn, "seq": seq}), stages, 2):
                    assert owner.setdefault((seq + n) % 4, turn) == turn, (seq, n)
            seq += stages


def _interleavings(program, tiles, count):
    """Whether two warps that run `program` for each of some tiles always read the other's value of the same tile: every
    order of their steps is tried.  A step: ("write",), ("read",), ("arrive", barrier) or ("wait", barrier, flip), a wait
    for the phase with the parity of the tile's number, flipped or not; a barrier's phase has `count` arrivals."""
    bars = sorted({s[1] for s in program if len(s) > 1})
    seen, todo = set(), [((0, 0), (-1, -1), (0,) * len(bars))]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, slot, arrived = state
        moved = False
        for me in (0, 1):
            if at[me] == tiles * len(program):
                continue
            tile, step = divmod(at[me], len(program))
            step, slots, counts = program[step], list(slot), list(arrived)
            if step[0] == "write":
                slots[me] = tile
            elif step[0] == "read":
                if slot[1 - me] != tile:
                    return False
            elif step[0] == "arrive":
                counts[bars.index(step[1])] += 1
            elif (arrived[bars.index(step[1])] // count) % 2 == (tile + step[2]) % 2:
                continue                              # (the phase at hand has the parity that is waited for)
            moved = True
            todo.append((tuple(a + (i == me) for i, a in enumerate(at)), tuple(slots), tuple(counts)))
        assert moved or at == (tiles * len(program),) * 2, f"both warps wait: {at}"
    return True


def test_the_maxima_that_two_warps_trade():
    """window_attn's softmax: a row's two halves, in two warps, trade their maxima through shared memory tile by tile.
    The steps are those of the source, in its order; neither warp may overwrite a maximum that the other has yet to
    read, however far it is ahead."""
    with open(os.path.join(build.CSRC, "sa_window_tc.cu")) as f:
        source = f.read()
    part = source[source.index("- softmax\n"):source.index("- epilogue\n")]
    step = re.compile(r"M\.mx\[b\]\[(me|me \^ 64)\]( = )?"
                      r"|(arrive|wait\w*)\(M\.(\w+)\[grp\]\[w & 1\], (lane|g >> 1|\(g >> 1\) \^ 1u)[,)]")
    program = []
    for m in step.finditer(part):
        if m[1]:
            assert (m[1] == "me") == bool(m[2])
            program.append(("write",) if m[2] else ("read",))
        else:
            program.append(("arrive", m[4]) if m[3] == "arrive" else ("wait", m[4], int("^" in m[5])))
    for bar in {s[1] for s in program if len(s) > 1}:
        assert re.findall(rf"mbar_init\(smem_addr\(&M\.{bar}\[b\]\[\d\]\), (\d+)\)", source) == ["2", "2"], bar
    assert program.count(("write",)) == program.count(("read",)) == 1
    assert _interleavings(program, 5, 2)
    # (without the wait for the reader, one warp's next maximum may come first)
    assert not _interleavings([("write",), ("arrive", "a"), ("wait", "a", 0), ("read",)], 5, 2)


@pytest.mark.parametrize("fmt,d,page", [(0, 512, 64), (1, 512, 64), (2, 512, 32), (0, 512, 16), (1, 512, 1), (0, 256, 64),
                                        (2, 64, 64)])
@pytest.mark.parametrize("h", [1, 16, 64, 100, 128])
def test_window_attn_workspace_of_the_largest_batch(lib, fmt, d, page, h):
    """A workspace of the size for n tokens, b sequences, window and first is taken by every call of no more.  (The calls
    stop at its misaligned address, which is looked at after its size.)"""
    a = dict(q=at(1), kv=at(2), scale_ptr=at(9) if fmt else None, fmt=fmt, sink=at(3), table=at(4), max_pages=400, ts=400,
             q_start=at(5), kv_len=at(6), scale=0.1, n=3, b=2, h=h, d=d, n_pages=1000, page=page, window=128, first=4, o=at(7),
             lse=None, rot=None, npos=0, rope=0, ws=at(11, 64), ws_bytes=0)
    for n, b, window, first in ((200, 200, 1024, 64), (400, 3, 333, 0), (7, 7, 4096, 128), (1, 1, 5000, 9)):
        size = lib.sa_window_attn_workspace_size(n, b, h, d, window, first, page, fmt)
        for m in {k for k in (1, 2, 3, n // 9, n // 5, n // 3, n // 2, n - 1, n) if 0 < k <= n}:
            for seqs in {1, min(2, b), min(m, b)}:
                for w, f in ((window, first), (window // 2 + 1, first), (window // 7 + 1, first // 2), (1, 0), (64, 0)):
                    assert lib.sa_window_attn_workspace_size(m, seqs, h, d, w, f, page, fmt) <= size
                    for pages in (400, 9, 1):
                        a.update(n=m, b=seqs, window=w, first=f, max_pages=pages, ts=pages, ws_bytes=size)
                        assert lib.sa_window_attn(*a.values(), None) == INVALID, (n, m, seqs, w, f, pages)
    a.update(ws_bytes=size, ws=None)
    assert lib.sa_window_attn(*a.values(), None) == WORKSPACE


@pytest.mark.parametrize("fmt,d,page", [(0, 512, 64), (1, 512, 16), (0, 256, 64), (2, 64, 5)])
@pytest.mark.parametrize("n,pages", [(3, 4), (4096, 8), (1, 400), (65536, 1), (7, 0)])
def test_window_attn_workspace_of_the_tables_positions(lib, fmt, d, page, n, pages):
    """A window beyond the page table's positions asks for no more than one of as many."""
    a = dict(q=at(1), kv=at(2), scale_ptr=at(9) if fmt else None, fmt=fmt, sink=at(3), table=at(4), max_pages=pages, ts=pages,
             q_start=at(5), kv_len=at(6), scale=0.1, n=n, b=1, h=16, d=d, n_pages=1000, page=page, window=1, first=0, o=at(7),
             lse=None, rot=None, npos=0, rope=0, ws=at(11, 64), ws_bytes=0)
    held = max(pages * page, 1)
    a.update(ws_bytes=lib.sa_window_attn_workspace_size(n, 1, 16, d, held, 0, page, fmt))
    for window, first in ((held, 5), (2 * held + 77, 0), (1 << 20, 1 << 20), ((1 << 30) - 9, 8), (1, 1 << 29)):
        a.update(window=window, first=first)
        assert lib.sa_window_attn(*a.values(), None) == INVALID, (window, first)   # (the workspace's address)
    assert a["ws_bytes"] < 256 + (24 << 20) + n * (4 * held + 4) + 1024


@pytest.mark.parametrize("change", [
    dict(scales=at(5, 63)), dict(scales=at(5, 65)),                     # the last code; the next row's first
    dict(out=at(1, 126)), dict(out=at(1, 134)), dict(res=at(1, 126)),   # x's last column; the next row's first
    dict(n=4, ss=67),                                                   # rows of another distance
    dict(cs=64, ss=64),                                                 # a row that leaves no room
])
def test_add_rms_norm_refuses_rows_that_share_a_byte(lib, change):
    a = dict(x=at(1), n=3, d=64, xs=130, w=at(2), eps=1e-6, res=at(3), kind=1, rs=130, out=at(4), os=130, codes=at(5),
             cs=66, scales=at(5, 64), ss=66)
    a.update(change)
    assert lib.sa_add_rms_norm(*a.values(), None) == INVALID
