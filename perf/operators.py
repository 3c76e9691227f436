"""The 4-bit cache and its eviction: the cases these operators are measured on, and their plain forms.

quant    rows quantised to 4 bits: blocks of 32 along d, e2m1 codes (two to a byte, the even element in
         the low four bits) and one e8m0 scale a block:  s = 2^ceil(log2(max(|x|) / 6)) (max(|x|) at least
         1e-4), code = e2m1 of x / s to the nearest, ties to even
ring     the same for new tokens, written to their slots (position mod window) of a cache
attn     sparse_attn over a cache held in 4 bits, with the log-sum-exp of every query
weights  the attention weight each cache row received: over all queries and heads, the sum of
         e^(scale q.k - lse), for bf16, e4m3 and e2m1 caches
evict    the rows of a cache with the most weight kept: the selection, the cache (codes, scales and
         weights) gathered into a smaller one, and the index table renumbered
"""

import math

import torch

own = False  # set by whoever runs the file: False computes the plain forms, True calls the library

BLOCK = 32
UNIT = 2.0 ** -32  # the weights are held as int64 multiples of this


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's new row of each of 64 sequences into its 128-slot ring
        dict(name="ring_decode", op="ring", b=64, s=1, d=512, start=32768, window=128, rows=8320),
        # a prefill's 8192 tokens and 2048 compressed rows
        dict(name="quant_prefill", op="quant", n=10240, d=512, stride=512),
        # a cache of 64 sequences converted at once
        dict(name="quant_cache", op="quant", n=532480, d=512, stride=512),
        # one sequence's next token: latency
        dict(name="attn_single", op="attn", b=1, s=1, h=64, d=512, rows=8320, topk=640, window=128,
             neg=0.0, peak=1.0),
        # a decode batch (64 heads, 1152 rows a query)
        dict(name="attn_decode", op="attn", b=64, s=1, h=64, d=512, rows=8320, topk=1152, window=128,
             neg=0.0, peak=1.0),
        # the long decode (128 heads, 2176 rows a query, 5 % of them empty)
        dict(name="attn_long", op="attn", b=256, s=1, h=128, d=512, rows=32896, topk=2176, window=128,
             neg=0.05, peak=1.0),
        # an odd prefill over a 4-bit cache, the first queries seeing few rows
        dict(name="attn_prefill", op="attn", b=1, s=2047, h=64, d=512, rows=2558, topk=639, window=128,
             neg=0.0, peak=2.0),
        # the weights of one step of one sequence over a bf16 cache: latency
        dict(name="weights_single", op="weights", fmt="bf16", b=1, s=1, h=64, d=512, rows=8320,
             topk=640, window=128, neg=0.0, peak=2.0),
        # the weights of a prefill's queries over its own bf16 rows
        dict(name="weights_prefill", op="weights", fmt="bf16", b=1, s=4096, h=64, d=512, rows=5120,
             topk=640, window=128, neg=0.0, peak=2.0),
        # the weights of a long decode step over the 4-bit cache
        dict(name="weights_long", op="weights", fmt="fp4", b=256, s=1, h=128, d=512, rows=32896,
             topk=2176, window=128, neg=0.05, peak=1.0),
        # one sequence's cache halved, ring and newest rows kept
        dict(name="evict_single", op="evict", b=1, rows=8320, keep=4224, d=512, first=128, last=64,
             ragged=False, topk=1152),
        # a batch of ragged long sequences cut to 16384 rows
        dict(name="evict_batch", op="evict", b=64, rows=32896, keep=16384, d=512, first=128, last=256,
             ragged=True, topk=2176),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "ring", "attn", "attn", "weights", "weights", "evict"])
    if op == "quant":
        d = 32 * rng.choice([2, 3, 4, 6, 8, 16, 16, 16])
        return dict(op=op, n=_log(rng, 1, 400000), d=d, stride=d + rng.choice([0, 0, 8, 64, 1]))
    if op == "ring":
        window, s = rng.choice([8, 100, 128]), rng.choice([1, 1, 37, 512])
        return dict(op=op, b=_log(rng, 1, 256), s=s, d=64 * rng.choice([1, 4, 8, 8]),
                    start=0 if s > 1 else rng.randrange(1, 200000), window=window,
                    rows=window + rng.randrange(0, 4000))
    if op == "evict":
        rows = _log(rng, 200, 40000)
        keep = max(2, int(rows * rng.uniform(0.1, 0.95)))
        first = min(128, keep // 3)
        last = rng.randrange(0, keep // 3 + 1)
        return dict(op=op, b=_log(rng, 1, 48), rows=rows, keep=keep, d=rng.choice([64, 256, 512, 512]),
                    first=first, last=last, ragged=rng.random() < 0.5, topk=rng.choice([16, 200, 1152]))
    d = rng.choice([64, 128, 192, 256, 448, 512, 512, 512, 512, 512])
    h = rng.choice([1, 4, 16, 40, 64, 64, 100, 128])
    window = rng.choice([8, 128])
    if rng.random() < 0.5:  # decode
        b, s = _log(rng, 1, 200), 1
        topk = window + _log(rng, 1, 2048)
        rows = topk + _log(rng, 1, 8000)
        neg = rng.choice([0.0, 0.05, 0.9])
    else:                   # prefill: each query its window and what it sees of s / 4 compressed rows
        b, s = rng.choice([1, 1, 2]), _log(rng, 2, 1500)
        topk = window + min(512, max(1, s // 4))
        rows = s + max(1, s // 4)
        neg = 0.0
    c = dict(op=op, b=b, s=s, h=h, d=d, rows=rows, topk=topk, window=window, neg=neg,
             peak=rng.choice([1.0, 2.0]))
    if op == "weights":
        c["fmt"] = rng.choice(["bf16", "fp8", "fp4"])
    return c


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _index_table(c, g):
    """idx [b, s, topk]: the window's columns, then distinct rows behind the window in ascending
    order, with empty entries (-1): before a prefill's first token, where a query sees fewer rows than
    columns, and, at a decode step, scattered ones."""
    b, s, rows, topk, w = (c[k] for k in ("b", "s", "rows", "topk", "window"))
    j = torch.arange(w, device="cuda")
    if s == 1:
        win = ((rows + j) % w).expand(b, 1, w)  # the whole ring, oldest first
        pick = torch.rand(b, 1, rows - w, device="cuda", generator=g)
        tail = pick.topk(topk - w, dim=-1).indices.sort(-1).values + w
        idx = torch.cat([win, tail], -1)
        drop = torch.rand(idx.shape, device="cuda", generator=g) < c["neg"]
        return torch.where(drop, -1, idx).to(torch.int32)
    i = torch.arange(s, device="cuda")[:, None]
    win = (i - w + 1 + j).clamp(min=-1).expand(b, s, w)
    n = rows - s
    pick = torch.rand(b, s, n, device="cuda", generator=g)
    pick = torch.where(torch.arange(n, device="cuda") < (i + 1) // 4, pick, -1.0)
    best = pick.topk(topk - w, dim=-1)
    tail = torch.where(best.values >= 0, best.indices, n).sort(-1).values
    tail = torch.where(tail < n, tail + s, -1)
    return torch.cat([win, tail], -1).to(torch.int32)


def _cache(c, g, fmt):
    """A cache [b, rows, .] of N(0, 1) rows, as its format holds them (rows drawn from a pool)."""
    b, rows, d = c["b"], c["rows"], c["d"]
    pool = torch.randn(4096, d, device="cuda", generator=g).to(torch.bfloat16)
    at = torch.randint(0, 4096, (b, rows), device="cuda", generator=g)
    if fmt == "bf16":
        return pool[at], None
    if fmt == "fp4":
        codes, scales, _ = _quantised(pool)
        return codes[at], scales[at]
    x = pool.float().view(4096, d // BLOCK, BLOCK)
    e = _ceil_log2(x.abs().amax(-1).clamp(min=1e-4) / 448.0)
    codes = (x / _pow2(e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(4096, d)
    return codes[at], (e + 127).to(torch.uint8)[at]


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "quant":
        x = torch.randn(c["n"], c["stride"], device="cuda", generator=g)
        st["x"] = x.mul_(torch.exp(torch.randn(c["n"], 1, device="cuda", generator=g))) \
            .to(torch.bfloat16)[:, :c["d"]]
        st["rt"] = torch.empty(c["n"], c["d"], dtype=torch.bfloat16, device="cuda")
        st["codes"] = torch.empty(c["n"], c["d"] // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(c["n"], c["d"] // BLOCK, dtype=torch.uint8, device="cuda")
    elif c["op"] == "ring":
        st["x"] = torch.randn(c["b"], c["s"], c["d"], device="cuda", generator=g).to(torch.bfloat16)
        st["codes"], st["scales"] = _cache(c, g, "fp4")
    elif c["op"] == "evict":
        b, rows, d = c["b"], c["rows"], c["d"]
        # most rows hardly seen, a few seen by almost every query, a third never
        w = torch.rand(b, rows, device="cuda", generator=g)
        w = torch.where(w < 0.3, 0.0, (w - 0.3) ** 6 * 1000)
        st["acc"] = (w.double() / UNIT).to(torch.int64)
        st["codes"] = torch.randint(0, 256, (b, rows, d // 2), device="cuda", generator=g,
                                    dtype=torch.uint8)
        st["scales"] = torch.randint(118, 130, (b, rows, d // BLOCK), device="cuda", generator=g,
                                     dtype=torch.uint8)
        st["live"] = torch.randint(c["keep"] // 2, rows + 1, (b,), device="cuda", generator=g,
                                   dtype=torch.int32) if c["ragged"] else None
        idx = torch.randint(0, rows, (b, 1, c["topk"]), device="cuda", generator=g)
        empty = torch.rand(b, 1, c["topk"], device="cuda", generator=g) < 0.05
        st["idx"] = torch.where(empty, -1, idx).to(torch.int32)
    else:
        b, s, h, d = (c[k] for k in ("b", "s", "h", "d"))
        st["q"] = (torch.randn(b, s, h, d, device="cuda", generator=g) * c["peak"]).to(torch.bfloat16)
        st["sink"] = torch.randn(h, device="cuda", generator=g)
        st["scale"] = float(d) ** -0.5
        st["idx"] = _index_table(c, g)
        st["kv"], st["kv_scale"] = _cache(c, g, c.get("fmt", "fp4"))
        if c["op"] == "weights":  # what the attention of these queries returned
            st["lse"] = _attn(st)[1]
    return st


# --------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------

def _ceil_log2(v):
    """ceil(log2 v) of positive f32 values, exactly."""
    m, e = torch.frexp(v)
    return torch.where(m == 0.5, e - 1, e).float()


def _pow2(e):
    """2^e of whole e >= -126 as f32, exactly (exp2 is not)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantised(x):
    """codes, scales and values of the rows of x."""
    n, d = x.shape
    v = x.float().reshape(n, d // BLOCK, BLOCK)
    e = _ceil_log2(v.abs().amax(-1).clamp(min=1e-4) / 6.0).clamp(max=125)
    s = _pow2(e)[..., None]
    a = v.abs() / s
    # the three-bit magnitude: how many midpoints lie below, a midpoint itself going to the even code
    up = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    values = torch.copysign(level[up.long()] * s, v).reshape(n, d).to(torch.bfloat16)
    code = (up + 8 * torch.signbit(v)).to(torch.uint8).reshape(n, d // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8), values


def _rows_f32(kv, kv_scale, d):
    """Cache rows [..., .] as f32 [..., d]."""
    if kv_scale is None:
        return kv.float()
    if kv.shape[-1] == d:
        v = kv.view(torch.float8_e4m3fn).float()
    else:
        level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=kv.device)
        level = torch.cat([level, -level])
        v = torch.stack([level[(kv & 15).int()], level[(kv >> 4).int()]], -1)
    s = _pow2(kv_scale.to(torch.int32) - 127)[..., None]
    return (v.reshape(*kv_scale.shape, BLOCK) * s).reshape(*kv.shape[:-1], d)


def _gathered(st):
    """The rows that idx names, f32 [b, s, topk, d], and which entries name one."""
    idx, d = st["idx"], st["q"].shape[-1]
    b, s, topk = idx.shape
    at = (torch.arange(b, device="cuda")[:, None], idx.clamp(min=0).long().view(b, -1))
    kv = st["kv"][at]
    sc = None if st["kv_scale"] is None else st["kv_scale"][at]
    return _rows_f32(kv, sc, d).view(b, s, topk, d), (idx >= 0)[:, :, None, :]


def _attn(st):
    k, seen = _gathered(st)
    logit = (st["q"].float() @ k.transpose(-1, -2)) * st["scale"]
    logit = torch.where(seen, logit, -math.inf)
    sink = st["sink"].expand(logit.shape[:-1])
    m = torch.maximum(logit.amax(-1), sink)
    p = torch.exp(logit - m[..., None])
    den = p.sum(-1) + torch.exp(sink - m)
    return ((p @ k) / den[..., None]).to(torch.bfloat16), m + torch.log(den)


def _weights(st):
    k, seen = _gathered(st)
    logit = (st["q"].float() @ k.transpose(-1, -2)) * st["scale"]
    p = torch.where(seen, torch.exp(logit - st["lse"][..., None]), 0.0).sum(2)
    b, rows = st["kv"].shape[:2]
    acc = torch.zeros(b, rows, dtype=torch.float64, device="cuda")
    return acc.scatter_add_(1, st["idx"].clamp(min=0).long().view(b, -1), p.double().view(b, -1)).float()


def _evict(st):
    c, acc, codes = st["case"], st["acc"], st["codes"]
    b, rows = acc.shape
    row = torch.arange(rows, device="cuda").expand(b, rows)
    live = torch.full((b, 1), rows, device="cuda") if st["live"] is None else st["live"].long()[:, None]
    forced = (row < c["first"]) | (row >= live - c["last"])
    key = torch.where(row >= live, -1, torch.where(forced, 1 << 62, acc))
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    best = torch.where(best < live, best, rows).sort(1).values
    kept = torch.where(best < rows, best, -1)
    there = kept[..., None] >= 0
    at = (torch.arange(b, device="cuda")[:, None], kept.clamp(min=0))
    slot = torch.arange(c["keep"], device="cuda").expand(b, -1)
    remap = torch.full((b, rows + 1), -1, device="cuda").scatter_(1, best, slot)[:, :rows]
    idx = torch.where(st["idx"] < 0, -1, remap.gather(1, st["idx"].clamp(min=0).long().view(b, -1))
                      .view(st["idx"].shape))
    return {"kept": kept.to(torch.int32), "remap": remap.to(torch.int32), "idx": idx.to(torch.int32),
            "codes": torch.where(there, codes[at], 0), "scales": torch.where(there, st["scales"][at], 0),
            "acc": torch.where(kept >= 0, acc[at], 0)}


def _ring(st):
    c = st["case"]
    x, w = st["x"], c["window"]
    t = torch.arange(max(0, c["s"] - w), c["s"], device="cuda")
    codes, scales, _ = _quantised(x[:, t].reshape(-1, c["d"]))
    slot = (c["start"] + t) % w
    st["codes"][:, slot] = codes.view(c["b"], len(t), -1)
    st["scales"][:, slot] = scales.view(c["b"], len(t), -1)
    return {"codes": st["codes"][:, :w], "scales": st["scales"][:, :w]}


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "quant":
        codes, scales, values = _quantised(state["x"])
        return {"codes": codes, "scales": scales, "values": values}
    if c["op"] == "ring":
        return _ring(state)
    if c["op"] == "attn":
        o, lse = _attn(state)
        return {"o": o, "lse": lse}
    if c["op"] == "weights":
        return {"weights": _weights(state)}
    return _evict(state)


def _workspace(sa, c, st):
    """The workspace such a program keeps from step to step."""
    if "ws" not in st:
        fmt = {"bf16": sa.SA_KV_BF16, "fp8": sa.SA_KV_FP8_E4M3, "fp4": sa.SA_KV_FP4_E2M1}
        st["ws"] = sa.new_workspace(c["b"], c["s"], c["h"], c["d"], c["rows"], c["topk"],
                                    fmt[c.get("fmt", "fp4")])
    return st["ws"]


def _run_own(c, st):
    import sparse_latent_attention_gb300 as sa
    if c["op"] == "quant":
        sa.act_quant_fp4(st["x"], out_rt=st["rt"], codes=st["codes"], scales=st["scales"])
        return {"codes": st["codes"], "scales": st["scales"], "values": st["rt"]}
    if c["op"] == "ring":
        codes, scales = st["codes"][:, :c["window"]], st["scales"][:, :c["window"]]
        sa.window_write_fp4(st["x"], c["start"], codes=codes, scales=scales)
        return {"codes": codes, "scales": scales}
    if c["op"] == "attn":
        lse = torch.empty(st["q"].shape[:3], dtype=torch.float32, device="cuda")
        o = sa.sparse_attn(st["q"], st["kv"], st["sink"], st["idx"], st["scale"],
                           kv_scale=st["kv_scale"], lse=lse, workspace=_workspace(sa, c, st))
        return {"o": o, "lse": lse}
    if c["op"] == "weights":
        acc = torch.zeros(c["b"], c["rows"], dtype=torch.int64, device="cuda")
        sa.row_weights(st["q"], st["kv"], st["lse"], st["idx"], st["scale"], acc,
                       kv_scale=st["kv_scale"], workspace=_workspace(sa, c, st))
        return {"weights": acc * sa.WEIGHT_UNIT}
    kept, remap = sa.evict_select(st["acc"], c["keep"], keep_first=c["first"], keep_last=c["last"],
                                  live=st["live"])
    codes, scales, acc = sa.compact_rows([st["codes"], st["scales"], st["acc"]], kept)
    return {"kept": kept, "remap": remap, "idx": sa.remap_idx(st["idx"], remap),
            "codes": codes, "scales": scales, "acc": acc}


# --------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------

def _row_bytes(c):
    fmt, d = c.get("fmt", "fp4"), c["d"]
    return 2 * d if fmt == "bf16" else d + d // 32 if fmt == "fp8" else d // 2 + d // 32


def work(case):
    c = case
    if c["op"] == "quant":
        return {"bytes": c["n"] * (2 * c["d"] + 2 * c["d"] + c["d"] // 2 + c["d"] // 32), "flops": 0}
    if c["op"] == "ring":
        n = c["b"] * min(c["s"], c["window"])
        return {"bytes": n * (2 * c["d"] + c["d"] // 2 + c["d"] // 32), "flops": 0}
    if c["op"] == "evict":
        b, rows, keep = c["b"], c["rows"], c["keep"]
        row = c["d"] // 2 + c["d"] // 32 + 8
        return {"bytes": b * (rows * (8 + 4) + keep * (4 + 2 * row) + 2 * 4 * c["topk"]), "flops": 0}
    b, s, h, d, topk = (c[k] for k in ("b", "s", "h", "d", "topk"))
    # each row that some query lists is read once: at a prefill all of them, at a decode step topk
    seen = b * (c["rows"] if s > 1 else topk)
    n = b * s * h
    pairs = n * topk
    if c["op"] == "attn":
        return {"bytes": seen * _row_bytes(c) + n * (4 * d + 4) + 4 * b * s * topk + 4 * h,
                "flops": 4 * pairs * d}
    return {"bytes": seen * _row_bytes(c) + n * (2 * d + 4) + 4 * b * s * topk + 4 * b * c["rows"],
            "flops": 2 * pairs * d}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------

def _two_to(e):
    """2^e as f64, exactly."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _decoded(byte, scale, fmt):
    """Stored rows as f64, from the formats' definitions."""
    if fmt == "bf16":
        return byte.double()
    if fmt == "fp4":
        byte = torch.stack([byte % 16, byte // 16], -1).flatten(-2)
        exp_bits, man_bits, bias = 2, 1, 1
    else:
        exp_bits, man_bits, bias = 4, 3, 7
    b = byte.to(torch.int32)
    man = (b % 2 ** man_bits).double() / 2 ** man_bits
    exp = (b // 2 ** man_bits % 2 ** exp_bits).double()
    neg = b // 2 ** (man_bits + exp_bits) == 1
    mag = torch.where(exp == 0, man * 2.0 ** (1 - bias), (1 + man) * 2.0 ** (exp - bias))
    s = _two_to(scale.long() - 127).repeat_interleave(BLOCK, -1)
    return torch.where(neg, -mag, mag) * s


def exact(case, seed):
    c = case
    if c["op"] in ("evict", "ring"):
        return None
    st = prepare(case, seed)
    if c["op"] == "quant":
        x = st["x"].double().unflatten(-1, (-1, BLOCK))
        top = x.abs().amax(-1, keepdim=True).clamp(min=1e-4)
        # the smallest power of two that keeps the largest value within 6, and the nearest value of
        # the format's grid: steps of a half up to 2, of 1 up to 4, of 2 up to 6
        p = _two_to(torch.ceil(torch.log2(top / 6)))
        p = torch.where(top > 6 * p, 2 * p, torch.where(top <= 3 * p, p / 2, p))
        a = (x / p).abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        return {"codes": None, "scales": None,
                "values": (torch.sign(x) * torch.round(a / step) * step * p).flatten(-2)}
    b, s, topk = st["idx"].shape
    rows = st["idx"].long().flatten(1)
    seq = torch.arange(b, device="cuda").repeat_interleave(s * topk)
    flat = seq * c["rows"] + rows.clamp(min=0).flatten()
    sc = st["kv_scale"]
    k = _decoded(st["kv"].flatten(0, 1)[flat], None if sc is None else sc.flatten(0, 1)[flat],
                 c.get("fmt", "fp4")).view(b * s, topk, c["d"])
    q = st["q"].double().view(b * s, c["h"], c["d"])
    e = torch.einsum("nhd,ntd->nht", q, k).mul_(st["scale"])
    gone = (st["idx"] < 0).view(b * s, 1, topk)
    if c["op"] == "weights":
        w = e.sub_(st["lse"].double().view(b * s, c["h"], 1)).exp_().masked_fill_(gone, 0.0).sum(1)
        out = torch.zeros(b * c["rows"], dtype=torch.float64, device="cuda")
        return {"weights": out.index_add_(0, flat, w.flatten()).view(b, c["rows"])}
    lse = torch.logsumexp(torch.cat([e.masked_fill_(gone, -math.inf),
                                     st["sink"].double().view(1, -1, 1).expand(b * s, -1, 1)], -1), -1)
    o = torch.einsum("nht,ntd->nhd", (e - lse[..., None]).exp_(), k)
    return {"o": o.view(b, s, c["h"], c["d"]), "lse": lse.view(b, s, c["h"])}
