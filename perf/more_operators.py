"""The paged latent cache, its window attention and the norm before it: the cases these operators are measured
on, and their plain forms.

A batch of sequences is packed: sequence i owns tokens q_start[i] .. q_start[i + 1] - 1 of x and q, its cache
holds kv_len[i] rows with this step's, and its new token t is at position kv_len[i] - (its new tokens) + t.
Position p of sequence i lives in row p mod page of page page_table[i][p / page] of a pool that all share.

append   new latent rows into their pages: y = x rsqrt(mean(x^2) + eps) w, the last rope_dim dims turned by
         their position's rotation ((a, b) -> (a c - b s, a s + b c)), and held as bf16, as the bf16 round trip
         of a block-32 quantisation, or as its codes and scales:  s = 2^ceil(log2(max(|y|) / top)) (max(|y|) at
         least 1e-4), code = y / s to the nearest, ties to even (e4m3: top 448, e2m1: top 6)
norm     residual += x (held in the residual's type), y = residual rsqrt(mean(residual^2) + eps) w, as bf16 or
         as e4m3 codes with the scales of blocks of 32
attn     each new token p attends to positions p - window + 1 .. p and 0 .. first - 1 (rows serve as keys and
         values, the sink joins the denominator):
         o = sum_j e^(scale q.k_j) k_j / (e^sink + sum_j e^(scale q.k_j)), its rope dims turned back
"""

import math
import random

import torch

own = False  # set by whoever runs the file: False computes the plain forms, True calls the library

BLOCK = 32
EPS = 1e-6
THETA = 10000.0


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's new row of each of 64 sequences, into 8-bit pages: latency
        dict(name="append_decode", op="append", b=64, n=64, ctx=32768, page=64, d=512, fmt="fp8", norm=True,
             rope=64),
        # the rows of a ragged batch of prompts, into bf16 pages that hold the 8-bit round trip
        dict(name="append_prefill", op="append", b=5, n=10240, ctx=0, page=64, d=512, fmt="bf16_fp8",
             norm=True, rope=64),
        # many prompts at once, into 4-bit pages
        dict(name="append_bulk", op="append", b=33, n=65536, ctx=4096, page=128, d=512, fmt="fp4", norm=True,
             rope=64),
        # one token's residual and norm: latency
        dict(name="norm_single", op="norm", n=1, d=4096, fmt="bf16", residual="bf16", pad=0),
        # a decode batch of a wide stream, the norm's output in 8 bits
        dict(name="norm_decode", op="norm", n=256, d=8192, fmt="fp8", residual="bf16", pad=0),
        # a prompt's tokens, the stream kept in 32 bits
        dict(name="norm_prefill", op="norm", n=8191, d=4096, fmt="fp8", residual="f32", pad=0),
        # one sequence's next token: latency
        dict(name="attn_single", op="attn", b=1, n=1, ctx=5000, h=64, d=512, window=128, first=4, page=64,
             fmt="bf16", rope=64, lse=False),
        # a decode batch over 8-bit pages
        dict(name="attn_decode", op="attn", b=64, n=64, ctx=32768, h=64, d=512, window=1024, first=64,
             page=64, fmt="fp8", rope=64, lse=False),
        # a large decode batch of 128 heads, long windows
        dict(name="attn_long", op="attn", b=256, n=256, ctx=100000, h=128, d=512, window=4096, first=128,
             page=64, fmt="bf16", rope=0, lse=False),
        # a few drafted tokens of each sequence checked at once, few heads, 4-bit pages
        dict(name="attn_draft", op="attn", b=48, n=240, ctx=9000, h=16, d=512, window=512, first=16, page=32,
             fmt="fp4", rope=0, lse=True),
        # a prompt through a layer of the default window
        dict(name="attn_prefill", op="attn", b=1, n=4095, ctx=0, h=64, d=512, window=128, first=4, page=64,
             fmt="bf16", rope=64, lse=False),
        # pieces of three long prompts (some of them behind a cached part), a wide window
        dict(name="attn_chunk", op="attn", b=3, n=4096, ctx=6000, h=128, d=512, window=2048, first=64,
             page=64, fmt="bf16", rope=0, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "norm", "attn", "attn"])
    if op == "norm":
        d = rng.choice([_log(rng, 1, 512) * 32, _log(rng, 1, 512) * 32, _log(rng, 1, 16000)])
        fmt = rng.choice(["bf16", "fp8"]) if d % 32 == 0 else "bf16"
        return dict(op=op, n=min(_log(rng, 1, 16384), 2 ** 25 // d), d=d, fmt=fmt,
                    residual=rng.choice(["none", "bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 1, 8, 64]))
    if op == "append":
        d = 64 * rng.choice([1, 2, 3, 7, 8, 8, 8, 8])
        b = _log(rng, 1, 200)
        n = b if rng.random() < 0.4 else b + _log(rng, 1, 50000)
        return dict(op=op, b=b, n=n, ctx=rng.choice([0, 100, 5000, 60000]), page=rng.choice([1, 16, 48, 64, 256]),
                    d=d, fmt=rng.choice(["bf16", "bf16_fp8", "fp8", "fp8", "fp4"]), norm=rng.random() < 0.7,
                    rope=rng.choice([0, 2, 64, 64, 64]))
    d = rng.choice([64, 128, 192, 256, 448, 512, 512, 512, 512, 512, 512, 512])
    h = rng.choice([1, 8, 16, 40, 64, 64, 100, 128])
    window, first = _log(rng, 1, 4096), rng.choice([0, 0, 4, 37, 128])
    kind = rng.choice(["decode", "decode", "draft", "prefill", "prefill"])
    if kind == "prefill":
        b = rng.choice([1, 1, 2, 5])
        n = b + _log(rng, 1, 4096)
    else:
        b = _log(rng, 1, 256)
        n = b if kind == "decode" else b + _log(rng, 1, 4 * b)
    n = max(b, min(n, 2 ** 39 // (h * d * (window + first)), 2 ** 23 // (window + first)))
    return dict(op=op, b=b, n=n, ctx=rng.choice([0, 700, 20000]) if kind == "prefill" else _log(rng, 2, 100000),
                h=h, d=d, window=window, first=first, page=rng.choice([16, 32, 64, 64, 128, 100]),
                fmt=rng.choice(["bf16", "bf16", "fp8", "fp4"]),
                rope=64 if d == 512 and rng.random() < 0.5 else 0, lse=rng.random() < 0.5)


def _lens(c):
    """Each sequence's new tokens (they add up to n, one at least) and the rows its cache held before."""
    rng = random.Random(c["b"] * 1000003 + c["n"])
    cuts = sorted(rng.randrange(0, c["n"] - c["b"] + 1) for _ in range(c["b"] - 1))
    cuts = [0] + cuts + [c["n"] - c["b"]]
    new = [cuts[i + 1] - cuts[i] + 1 for i in range(c["b"])]
    held = [rng.randrange(c["ctx"] // 2, c["ctx"] + 1) for _ in range(c["b"])]
    return new, held


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rotations(positions, rope):
    """[positions, rope / 2, 2]: cos and sin of position x theta^(-2 k / rope), the angles in 64 bits."""
    k = torch.arange(rope // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * THETA ** (-2 * k / rope)
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _plan(c, g, reach):
    """The batch on the device: q_start, kv_len, page_table (pages in random order; those that no position
    of `reach`, a list of ranges for each sequence, falls in are -1) and the number of pages."""
    new, held = _lens(c)
    page = c["page"]
    total = [a + b for a, b in zip(new, held)]
    table = torch.full((c["b"], -(-max(total) // page)), -1, dtype=torch.int64)
    used = []
    for i in range(c["b"]):
        need = sorted({j for lo, hi in reach(new[i], held[i]) if hi > lo for j in range(lo // page, (hi - 1) // page + 1)})
        used += [(i, j) for j in need]
    at = torch.tensor(used)
    order = torch.randperm(len(used), device="cuda", generator=g).cpu()
    table[at[:, 0], at[:, 1]] = order
    start = torch.tensor([0] + new).cumsum(0)
    return dict(q_start=start.int().cuda(), kv_len=torch.tensor(total).int().cuda(), table=table.int().cuda(),
                n_pages=len(used), last=max(total))


def _pool(c, g, n_pages):
    """A pool of pages [n_pages, page, .] of N(0, 1) rows, as its format holds them (drawn from fewer)."""
    d, page = c["d"], c["page"]
    some = torch.randn(4096, d, device="cuda", generator=g)
    at = torch.randint(0, 4096, (n_pages, page), device="cuda", generator=g)
    if c["fmt"] == "bf16":
        return some.to(torch.bfloat16)[at], None
    top = 448.0 if c["fmt"] == "fp8" else 6.0
    v, e = _scaled(some, top)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8) if c["fmt"] == "fp8" else _packed(_fp4_codes(v))
    return codes[at], (e + 127).to(torch.uint8)[at]


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "norm":
        width = c["d"] + c["pad"]
        x = torch.randn(c["n"], width, device="cuda", generator=g) * torch.exp(
            torch.randn(c["n"], 1, device="cuda", generator=g))
        st["x"] = x.to(torch.bfloat16)[:, :c["d"]]
        st["weight"] = 1 + 0.2 * torch.randn(c["d"], device="cuda", generator=g)
        if c["residual"] != "none":
            r = 4 * torch.randn(c["n"], c["d"], device="cuda", generator=g)
            st["residual"] = r if c["residual"] == "f32" else r.to(torch.bfloat16)
        if c["fmt"] == "fp8":
            st["codes"] = torch.empty(c["n"], c["d"], dtype=torch.uint8, device="cuda")
            st["scales"] = torch.empty(c["n"], c["d"] // BLOCK, dtype=torch.uint8, device="cuda")
        return st
    if c["op"] == "append":
        st.update(_plan(c, g, lambda new, held: [(held, held + new)]))
        n, d, page = c["n"], c["d"], c["page"]
        x = torch.randn(n, d, device="cuda", generator=g)
        st["x"] = (x * torch.exp(0.5 * torch.randn(n, 1, device="cuda", generator=g))).to(torch.bfloat16)
        st["weight"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=g) if c["norm"] else None
        st["rot"] = _rotations(st["last"], c["rope"]) if c["rope"] else None
        st["pages"] = torch.randn(st["n_pages"], page, d, device="cuda", generator=g).to(torch.bfloat16)
        if c["fmt"] in ("fp8", "fp4"):
            st["codes"] = torch.randint(0, 127, (st["n_pages"], page, d if c["fmt"] == "fp8" else d // 2),
                                        device="cuda", generator=g, dtype=torch.uint8)
            st["scales"] = torch.randint(118, 130, (st["n_pages"], page, d // BLOCK), device="cuda",
                                         generator=g, dtype=torch.uint8)
        return st
    w, f = c["window"], c["first"]
    st.update(_plan(c, g, lambda new, held: [(0, min(f, held + new)), (max(0, held - w + 1), held + new)]))
    st["q"] = torch.randn(c["n"], c["h"], c["d"], device="cuda", generator=g).mul_(1.5).to(torch.bfloat16)
    st["sink"] = torch.randn(c["h"], device="cuda", generator=g)
    st["scale"] = float(c["d"]) ** -0.5
    st["pages"], st["kv_scale"] = _pool(c, g, st["n_pages"])
    st["rot"] = _rotations(st["last"], c["rope"]) if c["rope"] else None
    return st


# --------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------

def _ceil_log2(v):
    """ceil(log2 v) of positive f32 values, exactly."""
    m, e = torch.frexp(v)
    return torch.where(m == 0.5, e - 1, e)


def _pow2(e):
    """2^e of whole e >= -126 as f32, exactly (exp2 is not)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scaled(y, top):
    """Rows y (f32) over their blocks' scales, and the scales' exponents."""
    v = y.reshape(*y.shape[:-1], -1, BLOCK)
    # (a power of two below v / top times a number in [1, 2): the quotient's rounding cannot cross it)
    e = _ceil_log2(v.abs().amax(-1).clamp(min=1e-4) / top)
    return (v / _pow2(e)[..., None]).reshape(y.shape), e


def _fp4_codes(a):
    """The e2m1 codes of a (ties to even)."""
    m = a.abs()
    up = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    return (up + 8 * torch.signbit(a)).to(torch.uint8)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _fp4_values(code):
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    return torch.cat([level, -level])[code.int()]


def _times_scale(v, e):
    return (v.reshape(*e.shape, BLOCK) * _pow2(e)[..., None]).reshape(v.shape)


def _where(st):
    """Each token's sequence and position."""
    start = st["q_start"].long()
    token = torch.arange(st["case"]["n"], device="cuda")
    seq = torch.searchsorted(start, token, right=True) - 1
    return seq, st["kv_len"].long()[seq] - (start[seq + 1] - token)


def _normed(x, weight):
    """x rsqrt(mean(x^2) + eps) w in f64: a value next to a border between two codes goes to its own side."""
    v = x.double()
    if weight is None:
        return v
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * weight.double()


def _append(st):
    c = st["case"]
    seq, pos = _where(st)
    y = _normed(st["x"], st["weight"])
    if st["rot"] is not None:
        turn = st["rot"][pos].double()
        a, b = y[:, -c["rope"]::2], y[:, -c["rope"] + 1::2]
        turned = torch.stack([a * turn[..., 0] - b * turn[..., 1], a * turn[..., 1] + b * turn[..., 0]], -1)
        y = torch.cat([y[:, :-c["rope"]], turned.flatten(-2)], -1)
    y = y.float()
    at = (st["table"].long()[seq, pos // c["page"]], pos % c["page"])
    if c["fmt"] == "bf16":
        st["pages"][at] = y.to(torch.bfloat16)
        return {"pages": st["pages"]}
    fp4 = c["fmt"] == "fp4"
    v, e = _scaled(y, 6.0 if fp4 else 448.0)
    code = _fp4_codes(v) if fp4 else v.to(torch.float8_e4m3fn)
    st["pages"][at] = _times_scale(_fp4_values(code) if fp4 else code.float(), e).to(torch.bfloat16)
    if c["fmt"] != "bf16_fp8":
        st["codes"][at] = _packed(code) if fp4 else code.view(torch.uint8)
        st["scales"][at] = (e + 127).to(torch.uint8)
    return _append_outputs(st)


def _append_outputs(st):
    """The pages as the values they stand for (with codes, their round trip lies beside them)."""
    if st["case"]["fmt"] == "fp8":
        return {"pages": st["pages"], "codes": st["codes"].view(torch.float8_e4m3fn)}
    return {"pages": st["pages"]}


def _norm(st):
    c, h = st["case"], st["x"]
    if "residual" in st:
        h = (h.float() + st["residual"].float()).to(st["residual"].dtype)
        st["residual"].copy_(h)
    h = h.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["weight"]
    if c["fmt"] == "bf16":
        return _norm_outputs(st, y.to(torch.bfloat16))
    v, e = _scaled(y, 448.0)
    st["codes"].copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    st["scales"].copy_((e + 127).to(torch.uint8))
    return _norm_outputs(st, None)


def _norm_outputs(st, out):
    """bf16 rows, or the codes and the scales as the numbers they stand for; the stream beside them."""
    got = {"out": out} if out is not None else {"codes": st["codes"].view(torch.float8_e4m3fn),
                                                "scales": st["scales"].view(torch.float8_e8m0fnu)}
    return dict(got, residual=st["residual"]) if "residual" in st else got


def _seen(st):
    """The rows that each token may see, first ones and window: positions [n, first + window], and which of
    the columns name one."""
    c = st["case"]
    seq, pos = _where(st)
    f, w = c["first"], c["window"]
    head = torch.arange(f, device="cuda").expand(c["n"], f)
    tail = pos[:, None] - w + 1 + torch.arange(w, device="cuda")
    at = torch.cat([head, tail], -1)
    ok = torch.cat([head <= pos[:, None], tail >= f], -1)
    at = at.clamp(min=0)
    at = torch.where(ok, at, pos[:, None])
    return seq, pos, (st["table"].long()[seq[:, None], at // c["page"]], at % c["page"]), ok


def _attn(st):
    c = st["case"]
    _, pos, at, ok = _seen(st)
    k = st["pages"][at]
    if c["fmt"] == "bf16":
        k = k.float()
    else:
        v = k.view(torch.float8_e4m3fn).float() if c["fmt"] == "fp8" else \
            _fp4_values(torch.stack([k & 15, k >> 4], -1).flatten(-2))
        k = _times_scale(v, st["kv_scale"][at].int() - 127)
    logit = (st["q"].float() @ k.transpose(-1, -2)) * st["scale"]
    logit = torch.where(ok[:, None, :], logit, -math.inf)
    m = torch.maximum(logit.amax(-1), st["sink"])
    p = torch.exp(logit - m[..., None])
    den = p.sum(-1) + torch.exp(st["sink"] - m)
    o = (p @ k) / den[..., None]
    if st["rot"] is not None:
        turn = st["rot"][pos][:, None]
        a, b = o[..., -c["rope"]::2], o[..., -c["rope"] + 1::2]
        back = torch.stack([a * turn[..., 0] + b * turn[..., 1], b * turn[..., 0] - a * turn[..., 1]], -1)
        o = torch.cat([o[..., :-c["rope"]], back.flatten(-2)], -1)
    o = o.to(torch.bfloat16)
    return {"o": o, "lse": m + torch.log(den)} if c["lse"] else {"o": o}


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "append":
        return _append(state)
    return _norm(state) if c["op"] == "norm" else _attn(state)


def _run_own(c, st):
    import sparse_latent_attention_gb300 as sa
    if c["op"] == "norm":
        out = sa.add_rms_norm(st["x"], st["weight"], residual=st.get("residual"), eps=EPS,
                              codes=st.get("codes"), scales=st.get("scales"))
        return _norm_outputs(st, out)
    if c["op"] == "append":
        sa.page_write(st["x"], st["table"], st["q_start"], st["kv_len"], pages=st["pages"],
                      codes=st.get("codes"), scales=st.get("scales"),
                      quant="fp8" if c["fmt"] == "bf16_fp8" else None, weight=st["weight"], eps=EPS,
                      rope=st["rot"])
        return _append_outputs(st)
    lse = torch.empty(c["n"], c["h"], dtype=torch.float32, device="cuda") if c["lse"] else None
    if "ws" not in st:  # the workspace such a program keeps from step to step
        st["ws"] = sa.new_window_workspace(c["n"], c["b"], c["h"], c["d"], c["window"], c["first"], c["page"],
                                           {"bf16": sa.SA_KV_BF16, "fp8": sa.SA_KV_FP8_E4M3,
                                            "fp4": sa.SA_KV_FP4_E2M1}[c["fmt"]])
    o = sa.window_attn(st["q"], st["pages"], st["sink"], st["table"], st["q_start"], st["kv_len"], st["scale"],
                       c["window"], first=c["first"], kv_scale=st["kv_scale"], rope=st["rot"], lse=lse,
                       workspace=st["ws"])
    return {"o": o, "lse": lse} if c["lse"] else {"o": o}


# --------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        r = {"none": 0, "bf16": 4, "f32": 8}[c["residual"]]
        y = c["d"] + c["d"] // BLOCK if c["fmt"] == "fp8" else 2 * c["d"]
        return {"bytes": c["n"] * ((2 + r) * c["d"] + y) + 4 * c["d"], "flops": 0}
    d = c["d"]
    row = {"bf16": 2 * d, "bf16_fp8": 2 * d, "fp8": d + d // 32, "fp4": d // 2 + d // 32}[c["fmt"]]
    if c["op"] == "append":
        kept = row + (2 * d if c["fmt"] in ("fp8", "fp4") else 0)
        return {"bytes": c["n"] * (2 * d + kept + 4 * c["rope"]), "flops": 0}
    # a sequence's rows: those that its first new token's window reaches to its last token, and the first
    # ones before them; a token's: min(window, position + 1) and the first ones in front of those
    w, f, rows, pairs = c["window"], c["first"], 0, 0
    for new, held in zip(*_lens(c)):
        lo = max(0, held - w + 1)
        rows += held + new - lo + min(f, lo)
        for p in (range(held, held + new) if held < w + f else ()):
            pairs += min(w, p + 1) + min(f, max(0, p - w + 1))
        pairs += 0 if held < w + f else new * (w + f)
    n = c["n"] * c["h"]
    return {"bytes": rows * row + n * (4 * d + (4 if c["lse"] else 0)) + 4 * c["n"] * c["rope"],
            "flops": 4 * c["h"] * pairs * d}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------

def _place(c):
    """(sequence, position) of each token, on the host, from the lengths."""
    new, held = _lens(c)
    return [i for i in range(c["b"]) for _ in range(new[i])], [held[i] + t for i in range(c["b"]) for t in range(new[i])]


def _two_to(e):
    """2^e as f64, exactly."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _block_exponent(y, top):
    """The smallest whole e with max |block| <= top 2^e."""
    m = y.abs().unflatten(-1, (-1, BLOCK)).amax(-1).clamp(min=1e-4)
    e = torch.ceil(torch.log2(m / top)).long()
    e = torch.where(m > top * _two_to(e), e + 1, e)
    return torch.where(m <= top * _two_to(e - 1), e - 1, e)


def _held(y, top):
    """The codes' values and scales, as f64, of rows y: each element over its block's scale, to the nearest value
    of the format's grid (top 448: steps of an eighth of the power of two below, 2^-9 at least, top 6: of a half
    of it, 0.5 at least)."""
    s = _two_to(_block_exponent(y, top))
    a = y.unflatten(-1, (-1, BLOCK)) / s[..., None]
    e = torch.frexp(a.abs()).exponent.long() - 1
    step = _two_to(e.clamp(min=-6) - 3) if top == 448.0 else _two_to(e.clamp(min=0) - 1)
    return torch.round(a / step) * step, s


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "norm":
        h = st["x"].double()
        if "residual" in st:
            h += st["residual"].double()
            stream = h.clone()
            if c["residual"] == "bf16":  # the norm is that of the stream as it is held
                h = h.float().to(torch.bfloat16).double()
            else:
                h = h.float().double()
        y = torch.einsum("nd,n,d->nd", h, (torch.einsum("nd,nd->n", h, h) / c["d"] + EPS) ** -0.5,
                         st["weight"].double())
        if c["fmt"] == "bf16":
            got = {"out": y}
        else:
            codes, s = _held(y, 448.0)
            got = {"codes": codes.flatten(-2), "scales": s}
        return dict(got, residual=stream) if "residual" in st else got
    seq, pos = (torch.tensor(v, device="cuda") for v in _place(c))
    table = st["table"].long()
    if c["op"] == "append":
        y = st["x"].double()
        if c["norm"]:
            y = torch.einsum("nd,n,d->nd", y, (torch.einsum("nd,nd->n", y, y) / c["d"] + EPS) ** -0.5,
                             st["weight"].double())
        if c["rope"]:
            z = torch.view_as_complex(y[:, c["d"] - c["rope"]:].reshape(c["n"], -1, 2).contiguous())
            z = z * torch.view_as_complex(st["rot"].double())[pos]
            y = torch.cat([y[:, :c["d"] - c["rope"]], torch.view_as_real(z).flatten(1)], 1)
        flat = table[seq, pos // c["page"]] * c["page"] + pos % c["page"]
        if c["fmt"] != "bf16":
            codes, s = _held(y, 6.0 if c["fmt"] == "fp4" else 448.0)
            y = (codes * s[..., None]).flatten(-2)
        pages = st["pages"].double().flatten(0, 1).index_copy(0, flat, y).view(st["pages"].shape)
        if c["fmt"] != "fp8":
            return {"pages": pages}
        held = st["codes"].view(torch.float8_e4m3fn).double().flatten(0, 1)
        return {"pages": pages, "codes": held.index_copy(0, flat, codes.flatten(-2)).view(st["codes"].shape)}
    # position by position over each sequence's rows, a piece of the tokens at a time
    out, lses, flat = [], [], st["pages"].flatten(0, 1)
    scales = None if st["kv_scale"] is None else st["kv_scale"].flatten(0, 1)
    piece = max(1, 2 ** 30 // (max(c["h"], c["d"]) * (c["window"] + c["first"])))
    for a in range(0, c["n"], piece):
        i, p = seq[a:a + piece], pos[a:a + piece, None]
        at = torch.arange(c["first"] + c["window"], device="cuda") + 0 * p
        at = torch.where(at >= c["first"], p - (at - c["first"]), at)
        gone = (at < 0) | (at > p)
        gone[:, c["first"]:] |= at[:, c["first"]:] < c["first"]
        at = torch.where(gone, p, at)
        row = table[i[:, None], at // c["page"]] * c["page"] + at % c["page"]
        k = _decoded(flat[row], None if scales is None else scales[row], c["fmt"])
        e = torch.einsum("nhd,ntd->nht", st["q"][a:a + piece].double(), k).mul_(st["scale"])
        e = e.masked_fill_(gone[:, None, :], -math.inf)
        z = torch.logsumexp(torch.cat([e, st["sink"].double()[None, :, None].expand(len(i), -1, 1)], -1), -1)
        o = torch.einsum("nht,ntd->nhd", (e - z[..., None]).exp_(), k)
        if c["rope"]:
            t = torch.view_as_complex(o[..., c["d"] - c["rope"]:].unflatten(-1, (-1, 2)).contiguous())
            t = t * torch.view_as_complex(st["rot"].double())[p[:, 0]].conj()[:, None]
            o = torch.cat([o[..., :c["d"] - c["rope"]], torch.view_as_real(t).flatten(-2)], -1)
        out.append(o)
        lses.append(z)
    return {"o": torch.cat(out), "lse": torch.cat(lses)} if c["lse"] else {"o": torch.cat(out)}


def _decoded(byte, scale, fmt):
    """Stored rows as f64, from the formats' definitions."""
    if fmt == "bf16":
        return byte.double()
    if fmt == "fp4":
        byte = torch.stack([byte % 16, byte // 16], -1).flatten(-2)
        exp_bits, man_bits, bias = 2, 1, 1
    else:
        exp_bits, man_bits, bias = 4, 3, 7
    every = torch.arange(256, device="cuda")
    man = (every % 2 ** man_bits).double() / 2 ** man_bits
    exp = (every // 2 ** man_bits % 2 ** exp_bits).double()
    mag = torch.where(exp == 0, man * 2.0 ** (1 - bias), (1 + man) * 2.0 ** (exp - bias))
    value = torch.where(every // 2 ** (man_bits + exp_bits) % 2 == 1, -mag, mag)
    return (value[byte.int()].unflatten(-1, (-1, BLOCK)) * _two_to(scale.long() - 127)[..., None]).flatten(-2)
