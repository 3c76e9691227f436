"""Plain 64-bit implementations of the paged cache's write, the window attention over it and the residual
norm, written from their definitions, for the tests; and packed batches to run them on."""

from __future__ import annotations

import torch

from tests import _cache

NORM_REL = 2.0 ** -19  # of y in f32: a thread adds up to 32 squares (32 roundings of 2^-24, half of it in the
#                        root), the rest of the sum, the factor and the products round a few times more


class Batch:
    """b sequences with ``new`` tokens each, the last at position held + new - 1, in pages given out in a
    random order; `spare` more tokens behind the last sequence."""

    def __init__(self, new, held, page, seed, spare=0, dev="cuda", extra_pages=2):
        self.new, self.held, self.page = new, held, page
        self.b, self.live = len(new), sum(new)
        self.n = self.live + spare
        total = [a + c for a, c in zip(new, held)]
        per = [-(-t // page) for t in total]
        self.max_pages = max(per + [1]) + 1
        self.n_pages = sum(per) + extra_pages
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(self.n_pages, generator=g)
        table = torch.full((self.b, self.max_pages), -7, dtype=torch.int32)
        at = 0
        for i, k in enumerate(per):
            table[i, :k] = order[at:at + k]
            at += k
        self.table_cpu = table
        self.table = table.to(dev)
        self.q_start = torch.tensor([0] + new).cumsum(0).int().to(dev)
        self.kv_len = torch.tensor(total, dtype=torch.int32, device=dev)

    def tokens(self):
        """(token, sequence, position) of each live token."""
        t = 0
        for i in range(self.b):
            for j in range(self.new[i]):
                yield t, i, self.held[i] + j
                t += 1

    def row(self, i, p):
        return int(self.table_cpu[i, p // self.page]) * self.page + p % self.page

    def rows(self):
        """The pool row of each live token."""
        return torch.tensor([self.row(i, p) for _, i, p in self.tokens()], dtype=torch.long)

    def positions(self):
        return torch.tensor([p for _, _, p in self.tokens()], dtype=torch.long)

    def visible(self, window, first):
        """Index table [live, .]: the pool rows that each token sees, -1 behind them."""
        lists = []
        for _, i, p in self.tokens():
            lo = max(0, p - window + 1)
            lists.append([self.row(i, j) for j in list(range(min(first, lo))) + list(range(lo, p + 1))])
        width = max([len(v) for v in lists] + [1])
        return torch.tensor([v + [-1] * (width - len(v)) for v in lists], dtype=torch.int32).view(-1, width)


def norm(h, weight, eps):
    h = h.double()
    return h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def rotations(positions, rope, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(positions, rope // 2, generator=g, dtype=torch.float64) * 6.283
    return torch.stack([a.cos(), a.sin()], -1).float()


def turned(y, rot, positions, back=False):
    """The last dims of y [n, ., d] (f64) turned by each row's position."""
    w = rot.double()[positions]
    while w.dim() < y.dim() + 1:
        w = w.unsqueeze(1)
    r = 2 * rot.shape[1]
    a, b, c, s = y[..., -r::2], y[..., -r + 1::2], w[..., 0], w[..., 1] * (-1 if back else 1)
    z = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y[..., :-r], z], -1)


def pow2(e):
    """2^e as f64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def half_step(a, fmt):
    """Half the distance between the format's neighbours around |a| (f64)."""
    e = torch.frexp(a.abs()).exponent.long() - 1
    return pow2(e.clamp(min=-6, max=8) - 4) if fmt == "fp8" else pow2(e.clamp(min=0, max=2) - 2)


def check_codes(values, scale_bytes, y, fmt, rel):
    """values [n, d] (f64, the codes as numbers) and scale bytes [n, d / 32] are a quantisation of y [n, d], known
    to a relative error of rel."""
    top = {"fp8": 448.0, "fp4": 6.0}[fmt]
    s = pow2(scale_bytes.long() - 127)
    amax = y.abs().unflatten(-1, (-1, 32)).amax(-1).clamp(min=float(torch.tensor(1e-4)))
    assert (amax * (1 - rel) <= top * s).all(), "a scale is too small"
    assert (amax * (1 + rel) > top * s / 2).all(), "a scale is too large"
    a = y / s.repeat_interleave(32, -1)
    # (half a step of the larger neighbour's, where the value lies at a power of two)
    tol = torch.maximum(half_step(a, fmt), half_step(values, fmt)) + rel * a.abs()
    bad = ~((values - a).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} codes off, first {bad.nonzero()[0].tolist()}"


def fp4_values(codes):
    lut = torch.tensor(list(_cache.LEVELS) + [-v for v in _cache.LEVELS], device=codes.device, dtype=torch.float64)
    return torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)


def attention(bt, q, pool, kv_scale, sink, scale, window, first, rot=None):
    """o, lse of the live tokens, and bounds on a kernel's errors (see _cache.attention)."""
    d = q.shape[-1]
    idx = bt.visible(window, first).to(q.device)
    used = idx[idx >= 0].unique().long()
    flat = pool.flatten(0, 1)[used]                # (only rows that a token sees: the others hold anything)
    sc = None if kv_scale is None else kv_scale.flatten(0, 1)[used][None]
    kv = _cache.rows_f64(flat[None], sc, d)
    at = torch.full((pool.shape[0] * pool.shape[1] + 1,), -1, device=q.device, dtype=torch.long)
    at[used] = torch.arange(len(used), device=q.device)
    idx = at[idx.long()]
    o, lse, tol, lse_tol = _cache.attention(q[None, :bt.live], kv, sink, idx[None], scale)
    o, lse, tol, lse_tol = o[0], lse[0], tol[0], lse_tol[0]
    if rot is not None:
        # the rotation is of the f32 result: o's own rounding (2^-8 |o|) is of the turned value, and the rest of
        # the error of both parts of a pair (the weights' rounding among it) may come into each
        r = 2 * rot.shape[1]
        rest = tol - 2.0 ** -8 * o.abs()
        o = turned(o, rot.to(o.device), bt.positions().to(o.device), back=True)
        both = rest[..., -r:].unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(*rest.shape[:-1], r // 2, 2).flatten(-2)
        tol = torch.cat([rest[..., :-r], both * (1 + 2.0 ** -20)], -1) + 2.0 ** -8 * o.abs()
        tol[..., -r:] += 2.0 ** -22 * both + 2.0 ** -22 * o[..., -r:].abs() + 2.0 ** -22
    return o, lse, tol, lse_tol
