"""Plain 64-bit implementations of the 4-bit cache, its attention, the row weights and the eviction,
written from their definitions, for the tests."""

from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(bits: np.ndarray):
    """bf16 bits [n, d] -> codes [n, d / 2], scales [n, d / 32] (uint8), values [n, d] f64."""
    x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    n, d = x.shape
    x = np.where(np.isnan(x), 0.0, x).reshape(n, d // 32, 32)
    amax = np.maximum(np.abs(x).max(-1), np.float64(np.float32(1e-4)))
    e = np.full(amax.shape, -140)
    while (todo := (amax > 6.0 * np.exp2(e)) & (e < 125)).any():
        e = e + todo
    s = np.exp2(e.astype(np.float64))[..., None]
    a = np.minimum(np.abs(x) / s, 6.0)
    far = np.abs(a[..., None] - LEVELS)
    near = far.argmin(-1)                       # the lower of two equally near levels ...
    tie = (near < 7) & (np.take_along_axis(far, np.minimum(near + 1, 7)[..., None], -1)[..., 0]
                        == np.take_along_axis(far, near[..., None], -1)[..., 0])
    near = near + (tie & (near % 2 == 1))       # ... unless it is the odd one
    sign = np.signbit(x) & ~np.isnan((bits.astype(np.uint32) << 16).view(np.float32)
                                     .reshape(n, d // 32, 32))
    code = (near + 8 * sign).astype(np.uint8).reshape(n, d // 2, 2)
    values = (np.where(sign, -1.0, 1.0) * LEVELS[near] * s).reshape(n, d)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).astype(np.uint8), values


def rows_f64(kv: torch.Tensor, kv_scale, d: int) -> torch.Tensor:
    """A cache [b, rows, .] of any format as f64 [b, rows, d]."""
    if kv_scale is None:
        return kv.double()
    if kv.shape[-1] == d:
        v = kv.view(torch.float8_e4m3fn).double()
        e = kv_scale.double() - 127
    else:
        lut = torch.tensor(np.concatenate([LEVELS, -LEVELS]), device=kv.device)
        v = torch.stack([lut[(kv & 15).int()], lut[(kv >> 4).int()]], -1).flatten(-2)
        e = kv_scale.double().clamp(max=252) - 127
    two = torch.from_numpy(np.exp2(np.arange(-127, 129).astype(np.float64))).to(kv.device)
    return v * two[(e + 127).long()].repeat_interleave(32, -1)


def logits(q, kv64, idx, scale):
    """(l [b, s, h, topk], size of the terms summed for each, the rows, which entries name a row)."""
    b, s, topk = idx.shape
    bi = torch.arange(b, device=idx.device)[:, None, None]
    k = kv64[bi, idx.clamp(min=0).long()]                        # [b, s, topk, d]
    l = scale * torch.einsum("bshd,bstd->bsht", q.double(), k)
    size = abs(scale) * torch.einsum("bshd,bstd->bsht", q.double().abs(), k.abs())
    return l, size, k, (idx >= 0)[:, :, None, :]


def logit_error(size, d):
    """A bound on the error of an f32 dot product of d terms whose magnitudes add up to ``size``,
    each addition rounded or cut to f32 (2^-23)."""
    return d * 2.0 ** -23 * size


def attention(q, kv64, sink, idx, scale):
    """o, lse, and bounds on what a kernel that sums in f32 and takes p and o in bf16 may be off."""
    d = q.shape[-1]
    l, size, k, seen = logits(q, kv64, idx, scale)
    l = torch.where(seen, l, -torch.inf)
    sk = sink.double().expand(l.shape[:-1])
    lse = torch.logsumexp(torch.cat([l, sk[..., None]], -1), -1)
    p = torch.where(seen, (l - lse[..., None]).exp(), 0.0)
    o = torch.einsum("bsht,bstd->bshd", p, k)
    mass = torch.einsum("bsht,bstd->bshd", p, k.abs())
    # a logit's error moves p (and the denominator) by as much relatively; exponentials, their
    # arguments (|l| and |lse| in f32) and the sums add a few f32 roundings a term
    dl = torch.where(seen, logit_error(size, d), 0.0).amax(-1)
    arg = torch.where(seen, l.abs(), 0.0).amax(-1) + lse.abs().nan_to_num(posinf=0.0)
    rel = 2 * dl + (8 * arg + l.shape[-1] + 32) * 2.0 ** -23
    # a sink far above the logits: o = (sum of e_j v_j) / den with e_j <= 2^8 (relative to a running
    # maximum that may lag by that much) and den beyond 2^126, whose reciprocal is below f32's normal
    # numbers and may be flushed to zero: off by at most 2^-126, so o by 2^-126 2^8 (sum of |v_j|)
    lost = torch.where(seen[..., None], k.abs()[:, :, None], 0.0).sum(3) * 2.0 ** -118
    # p to bf16 and o to bf16: half a step (2^-8) each
    o_tol = (2.0 ** -8 + rel[..., None]) * mass + 2.0 ** -8 * o.abs() + lost
    return o, lse, o_tol, rel + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def row_weights(q, kv64, lse, idx, scale):
    """Weights [b, rows] and a bound on the error of f32 exponentials and sums over heads, rounded
    to multiples of 2^-32."""
    d = q.shape[-1]
    b, rows = kv64.shape[:2]
    l, size, _, seen = logits(q, kv64, idx, scale)
    p = torch.where(seen, (l - lse.double()[..., None]).exp(), 0.0)
    rel = logit_error(size, d) + (8 * (l.abs() + lse.double().abs()[..., None]) + 32) * 2.0 ** -23
    tol = torch.where(seen, p * (rel + q.shape[2] * 2.0 ** -24), 0.0).sum(2) + 2.0 ** -33
    at = idx.clamp(min=0).long().view(b, -1)
    z = torch.zeros(b, rows, dtype=torch.float64, device=idx.device)
    return z.scatter_add(1, at, p.sum(2).view(b, -1)), z.scatter_add(1, at, tol.view(b, -1))


def select(acc: np.ndarray, n_keep, first, last, live=None):
    """kept [b, n_keep] and remap [b, rows], by sorting each sequence's rows."""
    b, rows = acc.shape
    kept = np.full((b, n_keep), -1, np.int32)
    remap = np.full((b, rows), -1, np.int32)
    for bi in range(b):
        n = rows if live is None else int(min(max(live[bi], 0), rows))
        lo = min(first, n)
        hi = max(lo, n - last)
        forced = np.r_[0:lo, hi:n]
        # ~acc falls where acc rises (and has no overflow); a stable sort leaves the lower of equal rows first
        rest = lo + np.argsort(~acc[bi, lo:hi], kind="stable")
        stay = np.sort(np.r_[forced, rest[:min(n_keep, n) - len(forced)]])
        kept[bi, :len(stay)] = stay
        remap[bi, stay] = np.arange(len(stay))
    return kept, remap
