"""sparse_attn for GB300: DeepSeek V4.1's index-gathered latent attention with an attention sink.

The public calls take torch CUDA tensors and pass their device pointers to the C-ABI library
(libsa.so, include/sparse_attn.h) on the current stream.  PyTorch provides device memory and
streams only; all the arithmetic runs in the library's sm_103a kernels.

    o = sparse_attn(q, kv, sink, idx, softmax_scale)            # bf16 kv
    o = sparse_attn(q, codes, sink, idx, scale, kv_scale=e8m0)  # fp8 e4m3 kv + e8m0 scales
    window_idxs(start_pos, seqlen, window, out=idx[..., :window])
    act_quant_fp8(x, out_rt=x)                                  # in-place block-32 round trip

A cache held in 4 bits (e2m1 codes, two to a byte, and e8m0 scales), and its eviction by weight:

    act_quant_fp4(x, codes=codes, scales=scales)                # or window_write_fp4
    o = sparse_attn(q, codes, sink, idx, scale, kv_scale=scales, lse=lse)
    row_weights(q, codes, lse, idx, scale, acc, kv_scale=scales)    # acc += each row's weight
    kept, remap = evict_select(acc, n_keep, keep_first=window)
    codes, scales, acc = compact_rows([codes, scales, acc], kept)
    idx = remap_idx(idx, remap)

A cache in pages that sequences of different lengths share, attended to by position, and the norm before it:

    h = add_rms_norm(x, weight, residual=stream)                # stream += x, its norm (or 8-bit codes of it)
    page_write(rows, page_table, q_start, kv_len, pages=pages, weight=w, rope=rot)
    o = window_attn(q, pages, sink, page_table, q_start, kv_len, scale, window, first=4)
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import (SA_KV_BF16, SA_KV_FP4_E2M1, SA_KV_FP8_E4M3, SA_SCORE_BF16, SA_SCORE_F32,
                   SA_STATUS_BYTES, SparseAttnError, load, status_string)

__all__ = ["sparse_attn", "window_idxs", "act_quant_fp8", "window_write", "indexer_topk",
           "candidate_blocks", "hc_split_sinkhorn",
           "act_quant_fp4", "window_write_fp4", "row_weights", "evict_select", "compact_rows",
           "remap_idx", "WEIGHT_UNIT",
           "add_rms_norm", "page_write", "window_attn", "window_workspace_size", "new_window_workspace",
           "workspace_size", "new_workspace", "read_status", "SparseAttnError", "SA_KV_BF16",
           "SA_KV_FP8_E4M3", "SA_KV_FP4_E2M1", "SA_SCORE_F32", "SA_SCORE_BF16", "load"]

# row_weights' accumulators are int64 multiples of this: acc * WEIGHT_UNIT are the weights in f32
WEIGHT_UNIT = 2.0 ** -32


# What a call costs on the host is mostly attribute reads and argument objects, so pointers and streams go
# to ctypes as integers (its argument types are declared) and a tensor's properties are read once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (a PyTorch without CUDA has none)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _status(dev, name, stream, *args) -> int:
    """A library call's sa_status, on the device (its index) that the tensors are on: with that device
    current, on ``stream`` or the device's current stream."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _status(dev, name, stream, *args)
    return getattr(load(), name)(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)


def _call(name, dev, stream, *args):
    """The same, an error raised."""
    st = _status(dev, name, stream, *args)
    if st:
        _lib.check(st, name)


def _new(stream, make):
    """make()'s tensor, for a call that runs on ``stream``: from that stream's memory when one is given,
    where it is filled and where a block that other work still reads is not handed out, and kept while the
    current stream, on which the caller will use it, has work queued."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _need(t, name, dtype, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _on(t, name, like):
    """t (or None) is on like's device."""
    if t is not None and t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")


def workspace_size(b, s, h, d, rows, topk, kv_format=SA_KV_BF16) -> int:
    n = int(load().sa_sparse_attn_workspace_size(b, s, h, d, rows, topk, kv_format))
    if n == 0:
        raise SparseAttnError(_lib.SA_ERR_UNSUPPORTED, "sa_sparse_attn_workspace_size")
    return n


def new_workspace(b, s, h, d, rows, topk, kv_format=SA_KV_BF16, device="cuda") -> torch.Tensor:
    """A zeroed uint8 workspace of the size the library asks for (status word cleared)."""
    return torch.zeros(workspace_size(b, s, h, d, rows, topk, kv_format), dtype=torch.uint8,
                       device=device)


FAMILIES = {"auto": _lib.SA_FAMILY_AUTO, "tcgen05": _lib.SA_FAMILY_TCGEN05,
            "mma": _lib.SA_FAMILY_MMA_SYNC}


def _kv_format(kv, kv_scale, b, d, dev):
    """The kv format of a cache: bf16 [b, rows, d] without scales; with them, uint8 [b, rows, d] is
    e4m3 and uint8 [b, rows, d / 2] is e2m1."""
    _need(kv, "kv", torch.bfloat16 if kv_scale is None else torch.uint8, dev)
    shape = tuple(kv.shape)
    if len(shape) != 3 or shape[0] != b:
        fmt = None
    elif kv_scale is None:
        fmt = SA_KV_BF16 if shape[2] == d else None
    else:
        fmt = SA_KV_FP8_E4M3 if shape[2] == d else SA_KV_FP4_E2M1 if 2 * shape[2] == d else None
    if fmt is None:
        raise ValueError(f"kv shape {shape} does not match {b} sequences of head_dim {d}")
    if kv_scale is not None:
        _need(kv_scale, "kv_scale", torch.uint8, dev)
        if kv_scale.shape != (b, shape[1], d // 32):
            raise ValueError(f"kv_scale shape {tuple(kv_scale.shape)} != {(b, shape[1], d // 32)}")
    return fmt


def sparse_attn(q, kv, sink, idx, softmax_scale, *, kv_scale=None, out=None, workspace=None,
                rope=None, family=None, lse=None, stream=None) -> torch.Tensor:
    """o[b, s, h, d] (bf16) = sparse_attn(q, kv, sink, idx, softmax_scale).

    q [b, s, h, d] bf16; kv [b, rows, d] bf16, or uint8 e4m3 codes [b, rows, d] or uint8 e2m1
    codes [b, rows, d / 2] (two to a byte, see act_quant_fp4) with kv_scale [b, rows, d/32]
    uint8 e8m0; sink [h] f32; idx [b, s, topk] int32 (-1 = empty).
    lse: an f32 tensor [b, s, h] that receives the log of each softmax's denominator (the sink's
    term included), e.g. for row_weights.
    rope=(rot, start_pos): also rotate o's last rot.shape[1] * 2 dims back by the inverse rotary
    embedding of positions start_pos + si, rot [positions, rope_dim / 2, 2] f32 (cos, sin).
    family: None (= "auto"), "tcgen05" or "mma" -- the kernel family that computes the call."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    b, s, h, d = q.shape
    fmt = _kv_format(kv, kv_scale, b, d, dev)
    rows = kv.shape[1]
    _need(sink, "sink", torch.float32, dev)
    if tuple(sink.shape) != (h,):
        raise ValueError(f"sink shape {tuple(sink.shape)} != ({h},)")
    _need(idx, "idx", torch.int32, dev)
    if idx.dim() != 3 or idx.shape[0] != b or idx.shape[1] != s:
        raise ValueError(f"idx shape {tuple(idx.shape)} does not match q {tuple(q.shape)}")
    topk = idx.shape[2]
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q))
    else:
        _need(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _new(stream, lambda: new_workspace(b, s, h, d, rows, topk, fmt, device=dev))
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    if family is not None and family not in FAMILIES:
        raise ValueError(f"family must be one of {sorted(FAMILIES)}")
    if rope is not None:
        if family not in (None, "auto", "tcgen05"):
            raise ValueError("the fused rotation runs in the tcgen05 family only")
        rot, start_pos = rope
        _need(rot, "rot", torch.float32, dev)
        if rot.dim() != 3 or rot.shape[2] != 2:
            raise ValueError(f"rot shape {tuple(rot.shape)} is not [positions, rope_dim / 2, 2]")
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
        if tuple(lse.shape) != (b, s, h):
            raise ValueError(f"lse shape {tuple(lse.shape)} != {(b, s, h)}")
        if family not in (None, "auto"):
            raise ValueError("lse comes from the family that the call is routed to")
        if rope is not None and rot.numel() == 0 and q.numel():  # (its address would say: no rotation)
            raise ValueError("rot is empty")
        turn = (_ptr(rot), rot.shape[0], 2 * rot.shape[1], int(start_pos)) if rope else (None, 0, 0, 0)
        _call("sa_sparse_attn_lse", dev.index, stream, _ptr(q), _ptr(kv), _ptr(kv_scale), fmt, _ptr(sink),
              _ptr(idx), float(softmax_scale), b, s, h, d, rows, topk, _ptr(out), _ptr(lse),
              _ptr(workspace), workspace.numel(), *turn)
        return out
    call = (_ptr(q), _ptr(kv), _ptr(kv_scale), fmt, _ptr(sink), _ptr(idx), float(softmax_scale), b, s, h, d,
            rows, topk, _ptr(out), _ptr(workspace), workspace.numel())
    if rope is not None:
        _call("sa_sparse_attn_rope", dev.index, stream, *call, _ptr(rot), rot.shape[0], 2 * rot.shape[1],
              int(start_pos))
    elif family is not None:
        _call("sa_sparse_attn_family", dev.index, stream, *call, FAMILIES[family])
    else:
        _call("sa_sparse_attn", dev.index, stream, *call)
    return out


def _score_format(score, name="score"):
    if not isinstance(score, torch.Tensor) or not score.is_cuda or score.dim() != 3:
        raise TypeError(f"{name} must be a 3-D CUDA tensor")
    if not score.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if score.dtype == torch.float32:
        return SA_SCORE_F32
    if score.dtype == torch.bfloat16:
        return SA_SCORE_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {score.dtype}")


def hc_split_sinkhorn(mixes, hc_scale, hc_base, hc=4, sinkhorn_iters=20, eps=1e-6, *,
                      stream=None):
    """hc_split_sinkhorn: mixes [..., (2 + hc) * hc] f32, hc_scale [3], hc_base [(2 + hc) * hc]
    -> (pre [..., hc], post [..., hc], comb [..., hc, hc]), all f32."""
    for t, name in ((mixes, "mixes"), (hc_scale, "hc_scale"), (hc_base, "hc_base")):
        _need(t, name, torch.float32, mixes.device)
    mix = (2 + hc) * hc
    if mixes.shape[-1] != mix or tuple(hc_scale.shape) != (3,) or tuple(hc_base.shape) != (mix,):
        raise ValueError(f"shapes do not fit hc = {hc}: mixes [..., {mix}], hc_scale [3], "
                         f"hc_base [{mix}]")
    lead = tuple(mixes.shape[:-1])
    n = mixes.numel() // mix
    pre, post, comb = (_new(stream, lambda: torch.empty(lead + tail, dtype=torch.float32,
                                                        device=mixes.device))
                       for tail in ((hc,), (hc,), (hc, hc)))
    _call("sa_hc_split_sinkhorn", mixes.get_device(), stream, _ptr(mixes), n, hc, _ptr(hc_scale),
          _ptr(hc_base), int(sinkhorn_iters), float(eps), _ptr(pre), _ptr(post), _ptr(comb))
    return pre, post, comb


def candidate_blocks(logits, start_pos, ratio, topk_blocks, block_size, *, out=None,
                     stream=None) -> torch.Tensor:
    """select_candidate_blocks: logits [b, s, n_comp] (f32 or bf16) -> bool mask [b, s, n_comp],
    True inside the topk_blocks best blocks of block_size positions (the block of the query's
    newest visible position always kept, -inf blocks never)."""
    fmt = _score_format(logits, "logits")
    b, s, n = logits.shape
    if out is None:
        out = _new(stream, lambda: torch.empty((b, s, n), dtype=torch.bool, device=logits.device))
    elif out.dtype != torch.bool or tuple(out.shape) != (b, s, n) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bool tensor of shape {(b, s, n)}")
    _on(out, "out", logits)
    _call("sa_candidate_blocks", logits.get_device(), stream, _ptr(logits), fmt, b, s, n, int(start_pos),
          int(ratio), int(topk_blocks), int(block_size), _ptr(out))
    return out


def indexer_topk(score, start_pos, ratio, index_topk, offset, *, candidates=None, out=None,
                 stream=None):
    """The indexer's selection: score [b, s, n_comp] (f32 or bf16, n_comp = (start_pos + s) //
    ratio) -> idx [b, s, k] int32, k = min(index_topk, n_comp): the top-k positions in position
    order, + offset, -1 for a position the query does not see.  ``candidates`` (bool [b, s,
    n_comp], e.g. from candidate_blocks) masks the scores outside it first.  ``out`` may be a
    column slice of a wider idx tensor (its row and batch strides are used)."""
    fmt = _score_format(score)
    b, s, n = score.shape
    if candidates is not None and (candidates.dtype != torch.bool or tuple(candidates.shape) !=
                                   (b, s, n) or not candidates.is_contiguous()):
        raise ValueError(f"candidates must be a contiguous bool tensor of shape {(b, s, n)}")
    _on(candidates, "candidates", score)
    k = min(int(index_topk), n)
    if out is None:
        out = _new(stream, lambda: torch.empty((b, s, k), dtype=torch.int32, device=score.device))
    if out.dtype != torch.int32 or not out.is_cuda or tuple(out.shape) != (b, s, k) or (
            k > 0 and out.stride(2) != 1):
        raise ValueError(f"out must be a CUDA int32 tensor of shape {(b, s, k)} with unit column "
                         "stride")
    _on(out, "out", score)
    ld = out.stride(1) if s > 1 else max(k, out.stride(1))
    bstride = out.stride(0) if b > 1 else s * ld
    _call("sa_indexer_topk", score.get_device(), stream, _ptr(score), fmt, _ptr(candidates), b, s, n,
          int(start_pos), int(ratio), int(index_topk), int(offset), _ptr(out), ld, bstride)
    return out


def window_idxs(start_pos, seqlen, window, *, out=None, nbatch=1, stream=None, device="cuda"):
    """Window index table [nbatch, seqlen, window] (int32), written into ``out`` when given
    (``out`` may be a column slice of a wider idx tensor: its row and batch strides are used)."""
    if out is None:
        out = _new(stream, lambda: torch.empty((nbatch, seqlen, window), dtype=torch.int32, device=device))
    if out.dtype != torch.int32 or not out.is_cuda:
        raise TypeError("out must be a CUDA int32 tensor")
    if out.dim() == 2:
        out3 = out.unsqueeze(0)
    else:
        out3 = out
    if tuple(out3.shape) != (nbatch, seqlen, window) or out3.stride(2) != 1:
        raise ValueError(f"out shape {tuple(out.shape)} / strides do not fit ({nbatch}, {seqlen}, "
                         f"{window}) with unit column stride")
    ld = out3.stride(1) if seqlen > 1 else max(window, out3.stride(1))
    bstride = out3.stride(0) if nbatch > 1 else seqlen * ld
    _call("sa_window_idxs", out.get_device(), stream, start_pos, seqlen, window, _ptr(out3), ld, nbatch,
          bstride)
    return out


def act_quant_fp8(x, *, out_rt=None, codes=None, scales=None, stream=None):
    """Block-32 e4m3 quantisation of the rows of a 2-D bf16 tensor (last dim contiguous).

    Writes the bf16 round trip into ``out_rt`` (may be ``x`` itself), the e4m3 codes into
    ``codes`` and the e8m0 block scales into ``scales`` (each a 2-D tensor with unit column
    stride; rows may be strided, e.g. one ring slot per sequence of a cache)."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype != torch.bfloat16 or not x.is_cuda:
        raise ValueError("x must be a 2-D CUDA bf16 tensor with unit column stride")
    n, d = x.shape

    def rows_of(t, name, dtype, width):
        if t is None:
            return None, 0
        if t.dim() != 2 or t.dtype != dtype or t.stride(1) != 1 or tuple(t.shape) != (n, width):
            raise ValueError(f"{name} must be a 2-D {dtype} tensor of shape ({n}, {width}) with "
                             "unit column stride")
        _on(t, name, x)
        return t, t.stride(0)

    rt, rts = rows_of(out_rt, "out_rt", torch.bfloat16, d)
    cd, cds = rows_of(codes, "codes", torch.uint8, d)
    sc, scs = rows_of(scales, "scales", torch.uint8, d // 32)
    _call("sa_act_quant_fp8", x.get_device(), stream, _ptr(x), n, d, x.stride(0), _ptr(rt), rts, _ptr(cd),
          cds, _ptr(sc), scs)


def window_write(x, start_pos, *, ring_rt=None, codes=None, scales=None, stream=None):
    """The ring write with act_quant fused (sa_window_write): row t of x[bi] (the new token at
    position start_pos + t of sequence bi) goes to ring slot (start_pos + t) % window.

    x is a 3-D CUDA bf16 tensor [nbatch, seqlen, d] (last dim contiguous, rows of a sequence
    equally spaced, sequences seqlen rows apart).  The rings are 3-D tensors [nbatch, window, d]
    (bf16 round trip ``ring_rt``, e4m3 ``codes``) or [nbatch, window, d / 32] (e8m0 ``scales``)
    with unit column stride; they may be strided views of a larger cache, e.g. its first window
    rows."""
    if x.dim() != 3 or x.stride(2) != 1 or x.dtype != torch.bfloat16 or not x.is_cuda:
        raise ValueError("x must be a 3-D CUDA bf16 tensor with unit column stride")
    nb, sl, d = x.shape
    if nb > 1 and x.stride(0) != sl * x.stride(1):
        raise ValueError("the sequences of x must be seqlen rows apart")
    window = None

    def ring_of(t, name, dtype, width):
        nonlocal window
        if t is None:
            return None, 0, 0
        if (t.dim() != 3 or t.dtype != dtype or t.stride(2) != 1 or t.shape[0] != nb
                or t.shape[2] != width):
            raise ValueError(f"{name} must be a 3-D {dtype} tensor of shape ({nb}, window, {width})"
                             " with unit column stride")
        if window is None:
            window = t.shape[1]
        elif t.shape[1] != window:
            raise ValueError("the rings must have the same window")
        _on(t, name, x)
        return t, t.stride(1), t.stride(0)

    rt, rts, rtb = ring_of(ring_rt, "ring_rt", torch.bfloat16, d)
    cd, cds, cdb = ring_of(codes, "codes", torch.uint8, d)
    sc, scs, scb = ring_of(scales, "scales", torch.uint8, d // 32)
    if window is None:
        raise ValueError("give at least one of ring_rt, codes, scales")
    _call("sa_window_write", x.get_device(), stream, _ptr(x), nb, sl, d, x.stride(1) if sl > 1 else d,
          int(start_pos), window, _ptr(rt), rts, rtb, _ptr(cd), cds, cdb, _ptr(sc), scs, scb)


def act_quant_fp4(x, *, out_rt=None, codes=None, scales=None, stream=None):
    """Block-32 e2m1 quantisation of the rows of a 2-D bf16 tensor (last dim contiguous).

    s = the smallest power of two with max|x| <= 6 s in the block (max|x| at least 1e-4, s at most
    2^125), each code the e2m1 value nearest to x / s (ties to even, saturating; NaN counts as 0).
    Writes the bf16 round trip into ``out_rt`` (may be ``x`` itself), the codes, two to a byte
    (element 2k in the low four bits), into ``codes`` [n, d / 2] and the e8m0 block scales into
    ``scales`` [n, d / 32] (each a 2-D tensor with unit column stride; rows may be strided)."""
    shape, stride = x.shape, x.stride()
    if (len(shape) != 2 or x.dtype != torch.bfloat16 or not x.is_cuda
            or (shape[1] > 1 and stride[1] != 1)):
        raise ValueError("x must be a 2-D CUDA bf16 tensor with unit column stride")
    n, d = shape
    dev = x.get_device()

    def rows_of(t, name, dtype, width):
        if t is None:
            return None, 0
        stride = t.stride()
        if t.dtype != dtype or t.shape != (n, width) or (width > 1 and stride[1] != 1):
            raise ValueError(f"{name} must be a 2-D {dtype} tensor of shape ({n}, {width}) with "
                             "unit column stride")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected {x.device}")
        return t.data_ptr(), stride[0] if n > 1 else max(width, stride[0])

    _call("sa_act_quant_fp4", dev, stream, x.data_ptr(), n, d,
          stride[0] if n > 1 else max(d, stride[0]), *rows_of(out_rt, "out_rt", torch.bfloat16, d),
          *rows_of(codes, "codes", torch.uint8, d // 2),
          *rows_of(scales, "scales", torch.uint8, d // 32))


def window_write_fp4(x, start_pos, *, ring_rt=None, codes=None, scales=None, stream=None):
    """The ring write into a 4-bit cache: window_write with rows quantised as act_quant_fp4 does.

    x is a 3-D CUDA bf16 tensor [nbatch, seqlen, d] (last dim contiguous, rows of a sequence
    equally spaced, sequences seqlen rows apart); row t of x[bi] goes to ring slot
    (start_pos + t) % window.  The rings are 3-D tensors ``codes`` [nbatch, window, d / 2],
    ``scales`` [nbatch, window, d / 32] and ``ring_rt`` [nbatch, window, d] (bf16 round trip)
    with unit column stride; they may be strided views of a larger cache."""
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or stride[2] != 1 or x.dtype != torch.bfloat16 or not x.is_cuda:
        raise ValueError("x must be a 3-D CUDA bf16 tensor with unit column stride")
    nb, sl, d = shape
    xs = stride[1] if sl > 1 else stride[0] if nb > 1 else d
    if nb > 1 and stride[0] != sl * xs:
        raise ValueError("the sequences of x must be seqlen rows apart")
    dev = x.get_device()
    given = [t for t in (ring_rt, codes, scales) if t is not None]
    if not given or given[0].dim() != 3:
        raise ValueError("give at least one of ring_rt, codes, scales, as 3-D tensors")
    window = given[0].shape[1]

    def ring_of(t, name, dtype, width):
        if t is None:
            return None, 0, 0
        stride = t.stride()
        if t.dtype != dtype or t.shape != (nb, window, width) or (width > 1 and stride[2] != 1):
            raise ValueError(f"{name} must be a {dtype} tensor of shape ({nb}, {window}, {width}) with "
                             "unit column stride")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected {x.device}")
        return t.data_ptr(), stride[1] if window > 1 else max(width, stride[1]), stride[0]

    _call("sa_window_write_fp4", dev, stream, x.data_ptr(), nb, sl, d, xs, int(start_pos), window,
          *ring_of(ring_rt, "ring_rt", torch.bfloat16, d),
          *ring_of(codes, "codes", torch.uint8, d // 2),
          *ring_of(scales, "scales", torch.uint8, d // 32))


def row_weights(q, kv, lse, idx, softmax_scale, acc, *, kv_scale=None, workspace=None,
                stream=None) -> torch.Tensor:
    """Adds to acc the attention weight each cache row received:

        acc[bi, idx[bi, si, c]] += sum over heads of e^(softmax_scale q.kv - lse)   (in units of 2^-32)

    for every query and every entry that is not -1.  q, kv, kv_scale, idx and softmax_scale are
    sparse_attn's; lse [b, s, h] f32 is what sparse_attn(..., lse=) wrote; acc [b, rows] int64 is
    fixed point (acc * WEIGHT_UNIT are the weights), so the sums are the same in any order.
    Returns acc."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    if q.dim() != 4:
        raise ValueError(f"q shape {tuple(q.shape)} is not [b, s, h, d]")
    b, s, h, d = q.shape
    fmt = _kv_format(kv, kv_scale, b, d, dev)
    rows = kv.shape[1]
    _need(lse, "lse", torch.float32, dev)
    if lse.shape != (b, s, h):
        raise ValueError(f"lse shape {tuple(lse.shape)} != {(b, s, h)}")
    _need(idx, "idx", torch.int32, dev)
    shape = idx.shape
    if len(shape) != 3 or shape[0] != b or shape[1] != s:
        raise ValueError(f"idx shape {tuple(idx.shape)} does not match q {tuple(q.shape)}")
    _need(acc, "acc", torch.int64, dev)
    if acc.shape != (b, rows):
        raise ValueError(f"acc shape {tuple(acc.shape)} != {(b, rows)}")
    if workspace is None:
        workspace = _new(stream, lambda: torch.zeros(SA_STATUS_BYTES, dtype=torch.uint8, device=dev))
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    _call("sa_row_weights", dev.index, stream, _ptr(q), _ptr(kv), _ptr(kv_scale), fmt, _ptr(lse), _ptr(idx),
          float(softmax_scale), b, s, h, d, rows, shape[2], _ptr(acc), _ptr(workspace),
          workspace.numel())
    return acc


def evict_select(acc, n_keep, *, keep_first=0, keep_last=0, live=None, stream=None):
    """Which rows of each sequence's cache stay: (kept [b, n_keep], remap [b, rows]) int32.

    acc [b, rows] int64 (row_weights'); live [b] int32: the sequences' rows in use (None: all).
    Of a sequence's L rows in use min(n_keep, L) stay: its first keep_first and last keep_last, and
    of the others those with the largest acc (equal ones lowest row first).  kept lists them in
    ascending order, then -1; remap holds each row's place in kept, -1 for a row that goes."""
    _need(acc, "acc", torch.int64)
    if acc.dim() != 2:
        raise ValueError(f"acc shape {tuple(acc.shape)} is not [b, rows]")
    b, rows = acc.shape
    if live is not None:
        _need(live, "live", torch.int32, acc.device)
        if tuple(live.shape) != (b,):
            raise ValueError(f"live shape {tuple(live.shape)} != ({b},)")
    n_keep = int(n_keep)
    if not 0 <= n_keep <= rows:
        raise ValueError(f"n_keep {n_keep} is not within [0, {rows}]")
    dev = acc.device
    kept = _new(stream, lambda: torch.empty((b, n_keep), dtype=torch.int32, device=dev))
    remap = _new(stream, lambda: torch.empty((b, rows), dtype=torch.int32, device=dev))
    _call("sa_evict_select", acc.get_device(), stream, _ptr(acc), _ptr(live), b, rows, n_keep,
          int(keep_first), int(keep_last), _ptr(kept), _ptr(remap))
    return kept, remap


def compact_rows(tensors, kept, *, out=None, stream=None):
    """Gathers the kept rows of a list of tensors [b, rows, ...] (any dtype; e.g. a cache's codes,
    its scales and its accumulators): row j of each result is row kept[bi, j], zeros where that is
    -1.

    ``out``: None (new tensors [b, n_keep, ...]), or a list of tensors [b, n_keep or more, ...]
    whose first n_keep rows are written; a tensor may be its own out (in place; kept then has to
    ascend, as evict_select's does).  What lies behind them stays: before rows are appended there
    again, their accumulators have to be zeroed (acc[:, n_keep:] = 0), or a new row starts with the
    weight of the one that was there.  Rows of a sequence are contiguous; sequences may be apart (a
    cache's leading rows).  Returns the list of results."""
    tensors = list(tensors)
    _need(kept, "kept", torch.int32)
    if kept.dim() != 2:
        raise ValueError(f"kept shape {tuple(kept.shape)} is not [b, n_keep]")
    (b, n_keep), dev = kept.shape, kept.get_device()
    n = len(tensors)
    if not 0 < n <= _lib.SA_COMPACT_MAX_TENSORS:
        raise ValueError(f"give 1 to {_lib.SA_COMPACT_MAX_TENSORS} tensors")
    outs = [None] * n if out is None else list(out)
    if len(outs) != n:
        raise ValueError("out must list one tensor for each of tensors")
    rows = None
    src, dst, row_bytes, src_b, dst_b = [], [], [], [], []

    def of(t, what, shape, stride, size):
        """The bytes of a row of t, whose rows are contiguous."""
        if t.is_contiguous() and shape[1] and b:
            return size * (t.numel() // (b * shape[1]))
        elements, apart = 1, False
        for extent, step in zip(reversed(shape[2:]), reversed(stride[2:])):
            apart |= extent > 1 and step != elements
            elements *= extent
        apart |= shape[1] > 1 and stride[1] != elements
        if apart and t.numel():
            raise ValueError(f"{what} must have contiguous rows")
        return size * elements

    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or t.get_device() != dev:
            raise TypeError(f"tensors[{i}] must be a tensor on {kept.device}")
        shape, stride = t.shape, t.stride()
        if rows is None and len(shape) > 1:
            rows = shape[1]
        if len(shape) < 2 or shape[0] != b or shape[1] != rows:
            raise ValueError(f"tensors[{i}] must be [{b}, {rows}, ...]")
        size = t.element_size()
        row_bytes.append(of(t, "a tensor", shape, stride, size))
        o = outs[i]
        if o is None:
            o = outs[i] = _new(stream, lambda: torch.empty((b, n_keep, *shape[2:]), dtype=t.dtype,
                                                           device=t.device))
        elif (o.get_device() != dev or o.dtype != t.dtype or o.dim() != len(shape) or o.shape[0] != b
              or o.shape[1] < n_keep or o.shape[2:] != shape[2:]):
            raise ValueError(f"out[{i}] must be a {t.dtype} tensor [{b}, {n_keep} or more, ...] like "
                             f"tensors[{i}]")
        else:
            of(o, "an out", o.shape, o.stride(), size)
        src.append(t.data_ptr())
        dst.append(o.data_ptr())
        src_b.append(stride[0] * size)
        dst_b.append(o.stride(0) * size)
    # one array of 64-bit words holds the five lists
    words = (ctypes.c_int64 * (5 * n))(*src, *dst, *row_bytes, *src_b, *dst_b)
    at = ctypes.addressof(words)
    _call("sa_compact_rows", dev, stream, n, at, at + 8 * n, at + 16 * n, at + 24 * n, at + 32 * n, b,
          rows, n_keep, kept.data_ptr())
    return outs


def remap_idx(idx, remap, *, out=None, stream=None) -> torch.Tensor:
    """A table of row numbers after an eviction: out[bi, ...] = remap[bi, idx[bi, ...]], -1 where
    idx is -1.  idx int32 [b, ...], remap int32 [b, rows]; out may be idx itself.  (An earlier
    eviction's remap is such a table too: remap_idx(earlier, remap) is the two in one.)"""
    _need(idx, "idx", torch.int32)
    _need(remap, "remap", torch.int32, idx.device)
    if remap.dim() != 2 or idx.dim() < 1 or idx.shape[0] != remap.shape[0]:
        raise ValueError(f"remap shape {tuple(remap.shape)} does not match idx {tuple(idx.shape)}")
    if out is None:
        out = _new(stream, lambda: torch.empty_like(idx))
    else:
        _need(out, "out", torch.int32, idx.device)
        if out.shape != idx.shape:
            raise ValueError("out must have idx's shape")
    b, rows = remap.shape
    _call("sa_remap_idx", idx.get_device(), stream, _ptr(idx), b, idx.numel() // b if b else 0, _ptr(remap),
          rows, _ptr(out))
    return out


def read_status(workspace, clear=False, stream=None) -> int:
    """The workspace status word as an sa_status (synchronises the stream)."""
    if not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    return _status(workspace.get_device(), "sa_read_status", stream, _ptr(workspace), int(bool(clear)))


# The calls below are made once a layer and token: their checks are one look at what is usual, and the precise ones, which
# name what is wrong, only where that look finds something else.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_functions = {}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(name, dev, stream, *args):
    """_call for the functions that a step makes many calls of: the library's function looked up once."""
    if stream is not None or dev != _current_device():
        return _call(name, dev, stream, *args)
    f = _functions.get(name)
    if f is None:
        f = _functions.setdefault(name, getattr(load(), name))
    st = f(*args, _raw_stream(dev))
    if st:
        _lib.check(st, name)


def _check_rows(t, name, dtypes, shape, dev):
    """Raises what is wrong with a tensor of strided rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA {' or '.join(map(str, dtypes))} tensor")
    if tuple(t.shape) != shape or (t.numel() and shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have shape {shape} and unit column stride, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def add_rms_norm(x, weight, *, residual=None, eps=1e-6, out=None, codes=None, scales=None, stream=None):
    """residual += x (in place), and the root-mean-square norm of the sum (of x without a residual):
    y = h * rsqrt(mean(h^2) + eps) * weight, h as the residual holds it.

    x [n, d] bf16; weight [d] f32; residual [n, d] bf16 or f32.  y goes to ``out`` [n, d] bf16, which may be
    ``x`` itself and is made (and returned) when neither it nor ``codes`` is given, and, quantised as
    act_quant_fp8 quantises, to ``codes`` [n, d] and ``scales`` [n, d / 32] uint8.  All but the weight with
    unit column stride; rows may be strided.  Returns out (None when only codes were asked for)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype is not _BF16:
        raise TypeError("x must be a CUDA bf16 tensor")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    n, d = shape
    xs, xc = x.stride()
    if xc != 1 and d > 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    dev = x.get_device()
    many = n > 1

    def rows_of(t, name, dtypes, width):
        """(address, distance of its rows) of a tensor of rows."""
        if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == (n, width) and t.get_device() == dev
                and (t.stride(1) == 1 or width < 2)):
            _check_rows(t, name, dtypes, (n, width), dev)
        return t.data_ptr(), t.stride(0) if many else width

    if not (isinstance(weight, torch.Tensor) and weight.dtype is _F32 and weight.shape == (d,)
            and weight.get_device() == dev and weight.is_contiguous()):
        _need(weight, "weight", _F32, x.device)
        raise ValueError(f"weight shape {tuple(weight.shape)} != ({d},)")
    kind, res, rs = _lib.SA_RESIDUAL_NONE, None, 0
    if residual is not None:
        res, rs = rows_of(residual, "residual", (_BF16, _F32), d)
        kind = _lib.SA_RESIDUAL_F32 if residual.dtype is _F32 else _lib.SA_RESIDUAL_BF16
    if (codes is None) != (scales is None):
        raise ValueError("give codes and scales together")
    cd = sc = po = None
    cs = ss = os_ = 0
    if codes is not None:
        if d % 32:
            raise ValueError(f"blocks of 32 need a row of a multiple of 32, got {d}")
        cd, cs = rows_of(codes, "codes", (_U8,), d)
        sc, ss = rows_of(scales, "scales", (_U8,), d // 32)
    if out is not None:
        po, os_ = rows_of(out, "out", (_BF16,), d)
    elif codes is None:
        if stream is None and x.is_contiguous():
            out = torch.empty_like(x)
        else:
            out = _new(stream, lambda: torch.empty(shape, dtype=_BF16, device=x.device))
        po, os_ = out.data_ptr(), d
    if n and d:
        _launch("sa_add_rms_norm", dev, stream, x.data_ptr(), n, d, xs if many else d, weight.data_ptr(),
                eps, res, kind, rs, po, os_, cd, cs, sc, ss)
    return out


def _batch(page_table, q_start, kv_len, dev):
    """The packed batch's tables: (b, max_pages, distance of the table's rows)."""
    try:
        b, max_pages = page_table.shape
        if (page_table.dtype is _I32 and q_start.dtype is _I32 and kv_len.dtype is _I32
                and page_table.get_device() == q_start.get_device() == kv_len.get_device() == dev
                and kv_len.shape == (b,) and q_start.shape == (b + 1,) and kv_len.is_contiguous()
                and q_start.is_contiguous() and (page_table.is_contiguous() or page_table.stride(1) == 1)):
            return b, max_pages, page_table.stride(0) if b > 1 else max_pages
    except (AttributeError, ValueError):
        pass
    for t, name, dim in ((page_table, "page_table", 2), (q_start, "q_start", 1), (kv_len, "kv_len", 1)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != _I32:
            raise TypeError(f"{name} must be a CUDA int32 tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
        if t.dim() != dim or (t.numel() > 1 and t.stride(-1) != 1):
            raise ValueError(f"{name} must have {dim} dimension{'s' if dim > 1 else ''} and unit column stride")
    raise ValueError(f"page_table {tuple(page_table.shape)} and q_start {tuple(q_start.shape)} do not fit "
                     f"the {kv_len.shape[0]} sequences of kv_len")


_QUANT = {None: SA_KV_BF16, "fp8": SA_KV_FP8_E4M3, "fp4": SA_KV_FP4_E2M1}
_NO_POOL = (None, 0, 0)


def page_write(x, page_table, q_start, kv_len, *, pages=None, codes=None, scales=None, quant=None, weight=None,
               eps=1e-6, rope=None, workspace=None, stream=None):
    """New latent rows into their pages (sa_page_write): normed (with ``weight`` [d] f32), their last dims
    turned by their position's rotation (``rope`` [positions, rope_dim / 2, 2] f32: cos, sin), and held in bf16,
    8 or 4 bits.

    x [n, d] bf16: the packed batch's new tokens; q_start [b + 1], kv_len [b] and page_table [b, max_pages]
    int32: sequence i owns tokens q_start[i] .. q_start[i + 1] - 1, the last of them at position kv_len[i] - 1,
    and position p lies in page page_table[i][p // page].  Tokens from q_start[b] on are left out.
    codes [n_pages, page, d] (e4m3) or [n_pages, page, d / 2] (e2m1) with scales [n_pages, page, d / 32], uint8,
    receive the quantised rows.  pages [n_pages, page, d] bf16 receives the rows, as they are quantised where
    codes are given or ``quant`` ("fp8", "fp4") says so, else rounded to bf16.  All with unit column stride; pages
    and rows may be strided.
    workspace: one of new_workspace or new_window_workspace, whose status word notes a position without a page
    (or past the rotations); such a row is not written."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype is not _BF16:
        raise TypeError("x must be a CUDA bf16 tensor")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    n, d = x.shape
    dev = x.get_device()
    b, max_pages, table_stride = _batch(page_table, q_start, kv_len, dev)
    n_pages = page = None

    def pool_of(t, name, dtype, width):
        """(address, distance of rows, of pages) of a pool of rows of ``width``."""
        nonlocal n_pages, page
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
            raise TypeError(f"{name} must be a {dtype} tensor")
        shape, (ps, rs, cs) = t.shape, t.stride() if t.dim() == 3 else (0, 0, 0)
        if page is None and cs:
            n_pages, page, _ = shape
        if shape != (n_pages, page, width) or cs != 1:
            raise ValueError(f"{name} shape {tuple(shape)} does not fit rows of {width}"
                             f"{'' if page is None else f' in {n_pages} pages of {page}'} with unit column stride")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected {x.device}")
        return t.data_ptr(), rs if page > 1 else width, ps

    fmt = _QUANT.get(quant)
    if fmt is None:
        raise ValueError("quant must be None, 'fp8' or 'fp4'")
    if (codes is None) != (scales is None):
        raise ValueError("give codes and scales together")
    pg = cd = sc = _NO_POOL
    if codes is not None:
        width = codes.shape[-1] if isinstance(codes, torch.Tensor) and codes.dim() else 0
        held = SA_KV_FP4_E2M1 if 2 * width == d else SA_KV_FP8_E4M3
        cd = pool_of(codes, "codes", _U8, width if held == SA_KV_FP4_E2M1 else d)
        sc = pool_of(scales, "scales", _U8, d // 32)
        if quant is not None and held != fmt:
            raise ValueError(f"quant {quant} does not fit codes of shape {tuple(codes.shape)}")
        fmt = held
    if pages is not None:
        pg = pool_of(pages, "pages", _BF16, d)
    if page is None:
        raise ValueError("give pages, or codes and scales")
    w = turn = None
    npos = rope_dim = 0
    if weight is not None:
        if not (isinstance(weight, torch.Tensor) and weight.dtype is _F32 and weight.shape == (d,)
                and weight.get_device() == dev and weight.is_contiguous()):
            _need(weight, "weight", _F32, x.device)
            raise ValueError(f"weight shape {tuple(weight.shape)} != ({d},)")
        w = weight.data_ptr()
    if rope is not None:
        turn, npos, rope_dim = _rotation(rope, dev, x)
    status = None
    if workspace is not None:
        _need(workspace, "workspace", _U8, x.device)
        if workspace.numel() < SA_STATUS_BYTES:
            raise ValueError("workspace is too small")
        status = workspace.data_ptr()
    _launch("sa_page_write", dev, stream, x.data_ptr(), n, d, x.stride(0) if n > 1 else d, page_table.data_ptr(),
            max_pages, table_stride, q_start.data_ptr(), kv_len.data_ptr(), b, n_pages, page, fmt, *pg, *cd, *sc,
            w, eps, turn, npos, rope_dim, status)


def _rotation(rope, dev, like):
    """A table of rotations by position: (address, positions, rope_dim)."""
    if not (isinstance(rope, torch.Tensor) and rope.dtype is _F32 and rope.get_device() == dev and rope.is_contiguous()):
        _need(rope, "rope", _F32, like.device)
    shape = rope.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError(f"rope shape {tuple(shape)} is not [positions, rope_dim / 2, 2]")
    if not shape[0] or not shape[1]:  # (its address would say: no rotation)
        raise ValueError("rope is empty")
    return rope.data_ptr(), shape[0], 2 * shape[1]


def window_workspace_size(n, b, h, d, window, first, page, kv_format=SA_KV_BF16) -> int:
    """Bytes of workspace that window_attn needs for any batch of at most n tokens of b sequences.  (A window may
    be given as the positions that the page table holds, with first 0, where it reaches beyond them.)"""
    size = int(load().sa_window_attn_workspace_size(n, b, h, d, window, first, page, kv_format))
    if size == 0:
        raise SparseAttnError(_lib.SA_ERR_UNSUPPORTED, "sa_window_attn_workspace_size")
    return size


def new_window_workspace(n, b, h, d, window, first, page, kv_format=SA_KV_BF16, device="cuda") -> torch.Tensor:
    """A workspace of that size, its status word cleared."""
    ws = torch.empty(window_workspace_size(n, b, h, d, window, first, page, kv_format), dtype=torch.uint8,
                     device=device)
    ws[:SA_STATUS_BYTES].zero_()
    return ws


def window_attn(q, pages, sink, page_table, q_start, kv_len, softmax_scale, window, *, first=0, kv_scale=None,
                out=None, lse=None, rope=None, workspace=None, stream=None) -> torch.Tensor:
    """o[n, h, d] (bf16): each token of a packed batch attends to the last ``window`` positions of its sequence,
    its own among them, and to the sequence's ``first`` first ones, over a cache held in pages (sa_window_attn).

    q [n, h, d] bf16; pages [n_pages, page, d] bf16, or uint8 codes [n_pages, page, d] (e4m3) or
    [n_pages, page, d / 2] (e2m1) with kv_scale [n_pages, page, d / 32] uint8; sink [h] f32; page_table, q_start
    and kv_len as in page_write, the cache with the tokens' own rows in it.  Rows of ``out`` and ``lse`` from
    q_start[b] on are left as they were.
    lse: an f32 tensor [n, h] that receives the log of each softmax's denominator (the sink's term included).
    rope [positions, rope_dim / 2, 2] f32: also turn o's last dims back by each token's position (d = 512)."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dtype is _BF16 and q.is_contiguous()):
        _need(q, "q", _BF16)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q shape {tuple(shape)} is not [n, h, d]")
    n, h, d = shape
    dev = q.get_device()
    if not isinstance(pages, torch.Tensor) or pages.dim() != 3:
        raise ValueError("pages must be a tensor [n_pages, page, .]")
    n_pages, page, _ = pages.shape
    fmt = SA_KV_BF16
    if not (kv_scale is None and pages.dtype is _BF16 and pages.get_device() == dev and pages.shape[2] == d
            and pages.is_contiguous()):
        fmt = _kv_format(pages, kv_scale, n_pages, d, q.device)
    b, max_pages, table_stride = _batch(page_table, q_start, kv_len, dev)
    if not (isinstance(sink, torch.Tensor) and sink.dtype is _F32 and sink.shape == (h,) and sink.get_device() == dev
            and sink.is_contiguous()):
        _need(sink, "sink", _F32, q.device)
        raise ValueError(f"sink shape {tuple(sink.shape)} != ({h},)")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(stream, lambda: torch.empty_like(q))
    elif not (isinstance(out, torch.Tensor) and out.dtype is _BF16 and out.shape == shape and out.get_device() == dev
              and out.is_contiguous()):
        _need(out, "out", _BF16, q.device)
        raise ValueError("out must have q's shape")
    lp = None
    if lse is not None:
        if not (isinstance(lse, torch.Tensor) and lse.dtype is _F32 and lse.shape == (n, h) and lse.get_device() == dev
                and lse.is_contiguous()):
            _need(lse, "lse", _F32, q.device)
            raise ValueError(f"lse shape {tuple(lse.shape)} != {(n, h)}")
        lp = lse.data_ptr()
    turn, npos, rope_dim = _NO_POOL if rope is None else _rotation(rope, dev, q)
    if workspace is None:
        held = max(max_pages * page, 1)  # (positions beyond them need no room)
        seen = min(window, held)
        workspace = _new(stream, lambda: new_window_workspace(n, b, h, d, seen, min(first, held - seen), page, fmt, q.device))
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is _U8 and workspace.get_device() == dev
              and workspace.is_contiguous()):
        _need(workspace, "workspace", _U8, q.device)
    _launch("sa_window_attn", dev, stream, q.data_ptr(), pages.data_ptr(), None if kv_scale is None else kv_scale.data_ptr(),
            fmt, sink.data_ptr(), page_table.data_ptr(), max_pages, table_stride, q_start.data_ptr(), kv_len.data_ptr(),
            softmax_scale, n, b, h, d, n_pages, page, window, first, out.data_ptr(), lp, turn, npos, rope_dim,
            workspace.data_ptr(), workspace.numel())
    return out
