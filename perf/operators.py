"""Cases of the decode-step operators: rotary positions, the quantized paged
key-value cache (written and read back) and the attention of one new token
over it.

``own`` chooses between the plain form (elementary torch operations in
float32) and the library's calls; both take what ``prepare`` returns.
``exact`` states the same results in float64, apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # the positions of one decode step: a batch of 64 sequences, one token each
        dict(name="rotary decode", op="rotary", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128,
             layout="half", dtype="bf16", scaling="none", max_pos=32768, inverse=False),
        # a long prompt far out in a stretched context, half of each head rotated in adjacent pairs
        dict(name="rotary prompt", op="rotary", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=64,
             layout="interleaved", dtype="bf16", scaling="yarn", max_pos=1 << 20, inverse=False),
        # the gradient (the inverse rotation) of an odd number of f32 rows with heads of 80, 40 of them rotated
        dict(name="rotary inverse f32", op="rotary", tokens=2999, q_heads=16, kv_heads=16, head_dim=80, rotary_dim=40,
             layout="half", dtype="f32", scaling="linear", max_pos=131072, inverse=True),
        # the new tokens of one decode step of 256 sequences
        dict(name="cache step", op="cache", tokens=256, kv_heads=8, head_dim=128, page_size=16, fmt="fp8_token"),
        # a prompt of 16384 tokens
        dict(name="cache prompt", op="cache", tokens=16384, kv_heads=8, head_dim=128, page_size=64, fmt="mxfp8"),
        # an odd number of prompt tokens with wide heads at four bits
        dict(name="cache mxfp4", op="cache", tokens=5003, kv_heads=4, head_dim=256, page_size=32, fmt="mxfp4"),
        # the first answers to a short question: one sequence of a few hundred tokens
        dict(name="attention short", op="attention", batch=1, min_len=333, max_len=333, q_heads=32, kv_heads=8,
             head_dim=128, page_size=16, fmt="bf16", window=0),
        # one very long document: all parallelism has to come from its length
        dict(name="attention long", op="attention", batch=1, min_len=131072, max_len=131072, q_heads=32, kv_heads=8,
             head_dim=128, page_size=64, fmt="fp8_token", window=0),
        # a serving batch of sequences at very different lengths
        dict(name="attention ragged", op="attention", batch=64, min_len=1, max_len=8191, q_heads=64, kv_heads=8,
             head_dim=128, page_size=16, fmt="mxfp8", window=0),
        # many short chats with one key-value head per query head
        dict(name="attention many", op="attention", batch=256, min_len=0, max_len=515, q_heads=16, kv_heads=16,
             head_dim=64, page_size=16, fmt="bf16", window=0),
        # a layer that looks back a few thousand tokens only, wide heads at four bits
        dict(name="attention window", op="attention", batch=32, min_len=2000, max_len=16384, q_heads=16, kv_heads=4,
             head_dim=256, page_size=32, fmt="mxfp4", window=4096),
        # the largest: a full batch of long sequences, unquantized
        dict(name="attention large", op="attention", batch=48, min_len=8192, max_len=16384, q_heads=32, kv_heads=8,
             head_dim=128, page_size=32, fmt="bf16", window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "attention", "attention"])
    if op == "rotary":
        head_dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log_int(rng, 1, 16384), q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8]),
                    kv_heads=kv_heads, head_dim=head_dim,
                    rotary_dim=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), max_pos=_log_int(rng, 2048, 1 << 20),
                    inverse=rng.random() < 0.3)
    if op == "cache":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 5, 8]),
                    head_dim=rng.choice([64, 128, 256]), page_size=rng.choice([16, 32, 64, 128]),
                    fmt=rng.choice(["bf16", "fp8_token", "mxfp8", "mxfp4"]))
    batch = _log_int(rng, 1, 256)
    top = min(131072, 500000 // batch)
    max_len = _log_int(rng, 1, top)
    kv_heads = rng.choice([1, 2, 4, 8])
    return dict(op=op, batch=batch, min_len=rng.choice([0, max_len // 4, max_len]), max_len=max_len,
                q_heads=kv_heads * rng.choice([1, 2, 4, 6, 8, 16]), kv_heads=kv_heads,
                head_dim=rng.choice([64, 128, 128, 256]) if kv_heads <= 4 else rng.choice([64, 128]),
                page_size=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["bf16", "fp8_token", "mxfp8", "mxfp4"]),
                window=rng.choice([0, 0, 0, max(1, max_len // 3)]))


def _lengths(case):
    """The sequence lengths of an attention case: spread evenly from min_len
    to max_len, both among them where there are two."""
    lo, hi, b = case["min_len"], case["max_len"], case["batch"]
    return ([hi, lo] + [lo + int((hi - lo + 1) * ((i * GOLDEN) % 1.0)) for i in range(2, b)])[:b]


def _code_bytes(fmt, d):
    """Bytes of one row of d values and of its scales."""
    return {"bf16": 2 * d, "fp8_token": d, "mxfp8": d, "mxfp4": d // 2}[fmt], \
        {"bf16": 0, "fp8_token": 4, "mxfp8": d // 32, "mxfp4": d // 32}[fmt]


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * case["head_dim"] * size + 8 * case["tokens"] + 4 * case["rotary_dim"],
                "flops": 3 * n * case["rotary_dim"]}
    row = sum(_code_bytes(case["fmt"], case["head_dim"]))
    if case["op"] == "cache":
        n = 2 * case["tokens"] * case["kv_heads"]      # rows of K and V: written from bf16, read back to bf16
        return {"bytes": n * (4 * case["head_dim"] + 2 * row) + 16 * case["tokens"], "flops": 4 * n * case["head_dim"]}
    seen = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
    heads = case["batch"] * case["q_heads"]
    return {"bytes": 2 * seen * case["kv_heads"] * row + heads * (4 * case["head_dim"] + 4)
            + 4 * (seen // case["page_size"] + 2 * case["batch"]),
            "flops": 4 * seen * case["q_heads"] * case["head_dim"]}


# ---------------------------------------------------------------------------
# inputs

def _inv_freq(case):
    """float64 frequencies and the factor on cos and sin, as a program has
    them from its configuration."""
    r = case["rotary_dim"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":
        factor, length = 16.0, 65536.0
        dim = lambda turns: r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(0.0, math.floor(dim(32.0))), min(r - 1.0, math.ceil(dim(1.0)))
        keep = 1 - ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _page_unit(fmt, ps, d):
    """Bytes of one head of one page: K codes, V codes, K scales, V scales."""
    code, scale = _code_bytes(fmt, d)
    return ps * code, ps * scale, 2 * ps * (code + scale)


def _e2m1(x):
    a = x.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c | ((x < 0).to(torch.uint8) << 3)


def _quantize(x, fmt):
    """float32 rows [..., d] -> (code bytes [..., code bytes], scale bytes [..., scale bytes])."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8), x.new_empty(x.shape[:-1] + (0,), dtype=torch.uint8)
    if fmt == "fp8_token":
        top = x.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))   # a true f32 division
        return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s.contiguous().view(torch.uint8)
    emax = 8 if fmt == "mxfp8" else 2
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, (torch.frexp(top)[1] - 1 - emax + 127).clamp(0, 254), 127)
    y = (g * torch.exp2((127 - e).double()).float()).flatten(-2)
    scales = e.squeeze(-1).to(torch.uint8)
    if fmt == "mxfp8":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scales
    c = _e2m1(y)
    return c[..., 0::2] | (c[..., 1::2] << 4), scales


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(codes, scales, fmt):
    """Code and scale bytes of rows -> float32 rows [..., d]."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    if fmt == "fp8_token":
        return codes.contiguous().view(torch.float8_e4m3fn).float() * scales.contiguous().view(torch.float32)
    if fmt == "mxfp8":
        x = codes.contiguous().view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        x = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = torch.exp2(scales.double() - 127).float()
    return (x.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _rows_of(units, fmt, ps, d):
    """Page units [..., unit] -> K codes, K scales, V codes, V scales, each [..., ps, bytes]."""
    nc, ns, _ = _page_unit(fmt, ps, d)
    kc, vc, ks, vs = units.split([nc, nc, ns, ns], -1)
    kc, vc, ks = (t.unflatten(-1, (ps, -1)) if t.shape[-1] else t.unsqueeze(-2) for t in (kc, vc, ks))
    # the scale bytes of V's 32-blocks lie by block, then by token
    vs = vs.unflatten(-1, (ps, -1)) if fmt == "fp8_token" else \
        vs.unflatten(-1, (-1, ps)).transpose(-1, -2) if ns else vs.unsqueeze(-2)
    return kc, ks, vc, vs


def _to_units(kc, ks, vc, vs, fmt):
    if fmt in ("mxfp8", "mxfp4"):
        vs = vs.transpose(-1, -2)
    return torch.cat([t.flatten(-2) for t in (kc, vc, ks, vs)], -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    d = case["head_dim"]
    if case["op"] == "rotary":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        # q and k as they come out of one product with v beside them
        qkv = normal(t, hq + 2 * hk, d).to(dt)
        pos = torch.randint(0, case["max_pos"], (1,), generator=g, device=DEV) if t > 256 else None
        pos = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV) if pos is None else \
            (pos + torch.arange(t, device=DEV)) % case["max_pos"]
        f, factor = _inv_freq(case)
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], positions=pos, inv_freq=f.to(DEV), factor=factor)
    hk, ps, fmt = case["kv_heads"], case["page_size"], case["fmt"]
    unit = _page_unit(fmt, ps, d)[2]
    if case["op"] == "cache":
        t = case["tokens"]
        pages = -(-t // ps) + 3
        kv = normal(t, 2 * hk, d) * torch.exp2(normal(t, 2 * hk, 1))
        kv[:, :hk, ::32] *= 4.0                       # keys have channels that stand out
        kv = kv.to(torch.bfloat16)
        slots = torch.randperm(pages * ps, generator=g, device=DEV)[:t] if t <= 256 else \
            (torch.randperm(pages, generator=g, device=DEV)[:, None] * ps
             + torch.arange(ps, device=DEV)).flatten()[:t].contiguous()
        back = slots[torch.randperm(t, generator=g, device=DEV)]
        return dict(case=case, k=kv[:, :hk], v=kv[:, hk:], slots=slots, read_slots=back,
                    cache=torch.zeros(pages * hk * unit, dtype=torch.uint8, device=DEV), desc=_desc(case, pages))
    b = case["batch"]
    order = torch.randperm(b, generator=g, device=DEV)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)[order]
    per_seq = -(-case["max_len"] // ps)
    need = -(-lens.long() // ps)
    pages = int(need.sum()) + 3
    at = torch.cumsum(need, 0) - need
    col = torch.arange(per_seq, device=DEV)
    ids = torch.randperm(pages, generator=g, device=DEV)
    table = torch.where(col < need[:, None], ids[(at[:, None] + col).clamp(max=pages - 1)], -1).int()
    cache = torch.empty((pages, hk, unit), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (hk * ps * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k, v = normal(n, hk, ps, d), normal(n, hk, ps, d)
        k[..., ::32] *= 3.0                           # keys have channels that stand out
        cache[p:p + n] = _to_units(*_quantize(k.to(torch.bfloat16).float(), fmt),
                                   *_quantize(v.to(torch.bfloat16).float(), fmt), fmt)
    q = normal(b, case["q_heads"] + 2 * hk, d).to(torch.bfloat16)[:, :case["q_heads"]]
    return dict(case=case, q=q, cache=cache.view(-1), table=table, lens=lens, scale=d ** -0.5, desc=_desc(case, pages))


def _desc(case, pages):
    """What names the cache to both forms."""
    return dict(fmt=case["fmt"], pages=pages, page_size=case["page_size"], heads=case["kv_heads"], dim=case["head_dim"])


# ---------------------------------------------------------------------------
# one pass

def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case)
    return _PLAIN[case["op"]](state, case)


def _own_rotary(s, case):
    import quantized_gemm_packed_amd as hum
    return hum.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], layout=case["layout"], factor=s["factor"],
                      inverse=case["inverse"])


def _own_desc(s):
    import quantized_gemm_packed_amd as hum
    if "own_desc" not in s:                           # the handle a program keeps with its cache
        d = s["desc"]
        s["own_desc"] = hum.make_kv_desc(d["fmt"], d["pages"], d["page_size"], d["heads"], d["dim"])
    return s["own_desc"]


def _own_cache(s, case):
    import quantized_gemm_packed_amd as hum
    d = _own_desc(s)
    hum.kv_write(d, s["cache"], s["k"], s["v"], s["slots"])
    return hum.kv_read(d, s["cache"], s["read_slots"])


def _own_attention(s, case):
    import quantized_gemm_packed_amd as hum
    return hum.kv_attention(_own_desc(s), s["cache"], s["q"], s["table"], s["lens"], scale=s["scale"],
                            window=case["window"], return_lse=True)


def _plain_rotary(s, case):
    r = case["rotary_dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    c = (angle.cos() * s["factor"]).float()[:, None]
    n = (angle.sin() * s["factor"]).float()[:, None]
    if case["inverse"]:
        n = -n

    def turn(x):
        y = x.float()
        if case["layout"] == "half":
            x0, x1 = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat((x0 * c - x1 * n, x0 * n + x1 * c), -1)
        else:
            x0, x1 = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack((x0 * c - x1 * n, x0 * n + x1 * c), -1).flatten(-2)
        return torch.cat((z, y[..., r:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _plain_cache(s, case):
    fmt, ps, d, hk = case["fmt"], case["page_size"], case["head_dim"], case["kv_heads"]
    units = s["cache"].view(-1, hk, _page_unit(fmt, ps, d)[2])
    rows = _rows_of(units, fmt, ps, d)                # views of the cache: [pages, heads, ps, bytes]
    page, at = s["slots"] // ps, s["slots"] % ps
    for x, (codes, scales) in ((s["k"], rows[:2]), (s["v"], rows[2:])):
        c, sc = _quantize(x.float(), fmt)
        codes[page, :, at] = c
        if fmt != "bf16":
            scales[page, :, at] = sc
    page, at = s["read_slots"] // ps, s["read_slots"] % ps

    def back(codes, scales):
        return _values(codes[page, :, at], scales[page, :, at] if fmt != "bf16" else None, fmt).to(torch.bfloat16)

    return back(*rows[:2]), back(*rows[2:])


def _plain_attention(s, case):
    fmt, ps, d, hk, b = case["fmt"], case["page_size"], case["head_dim"], case["kv_heads"], case["batch"]
    lens, table = s["lens"].long()[:, None], s["table"]
    units = s["cache"].view(-1, hk, _page_unit(fmt, ps, d)[2])
    first = torch.zeros_like(lens)
    if case["window"]:                                # only the pages that the window reaches
        first = (lens - case["window"]).clamp(min=0) // ps
        n = min(table.shape[1], case["window"] // ps + 2)
        col = first + torch.arange(n, device=DEV)
        table = table.gather(1, col.clamp(max=table.shape[1] - 1))
        table = torch.where(col < s["table"].shape[1], table, -1)
    pos = first * ps + torch.arange(table.shape[1] * ps, device=DEV)
    seen = (pos < lens) & (pos >= lens - case["window"] if case["window"] else pos >= 0)
    seen &= (table >= 0).repeat_interleave(ps, 1)
    kc, ks, vc, vs = _rows_of(units[table.clamp(min=0).long()], fmt, ps, d)   # [b, pages, heads, ps, bytes]
    k = _values(kc, ks, fmt).transpose(1, 2).flatten(2, 3)                     # [b, heads, tokens, d]
    v = _values(vc, vs, fmt).transpose(1, 2).flatten(2, 3)
    q = s["q"].float().view(b, hk, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o.view(b, -1, d).to(torch.bfloat16), (top + total.log()).view(b, -1)


_OWN = {"rotary": _own_rotary, "cache": _own_cache, "attention": _own_attention}
_PLAIN = {"rotary": _plain_rotary, "cache": _plain_cache, "attention": _plain_attention}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _e4m3_table():
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(math.nan if (c & 127) == 127 else -v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _nearest(x, bits, emin, top):
    """Float64 values rounded (ties to even) to `bits` stored mantissa bits,
    smallest normal exponent emin, saturated to `top`."""
    e = (torch.frexp(x)[1] - 1).clamp(min=emin) - bits
    step = torch.exp2(e.double())
    return ((x / step).round() * step).clamp(-top, top)


def _round_trip(x, fmt):
    """bf16 rows -> the float64 values that the cache stands for."""
    x = x.double()
    if fmt == "bf16":
        return x
    if fmt == "fp8_token":
        top = x.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, (top / torch.full_like(top, 448.0)).float().double(), 1.0)   # the scale is an f32
        return _nearest((x / s).float().double(), 3, -6, 448.0) * s                            # and so is the quotient
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    e = torch.log2(torch.where(top > 0, top, 1.0)).floor()               # bf16 values: never within an ulp below 2^n
    e = torch.where(top > 0, (e - (8 if fmt == "mxfp8" else 2)).clamp(-127, 127), 0.0)
    s = torch.exp2(e)
    y = _nearest(g / s, 3, -6, 448.0) if fmt == "mxfp8" else _nearest(g / s, 1, 0, 6.0)
    return (y * s).flatten(-2)


def _sequence(s, case, i, lo, n, tables):
    """Float64 K and V [heads, n - lo, d] of sequence i's tokens lo .. n - 1."""
    fmt, ps, d, hk = case["fmt"], case["page_size"], case["head_dim"], case["kv_heads"]
    code, scale = _code_bytes(fmt, d)
    t = torch.arange(lo, n, device=DEV)
    base = s["table"][i].long()[t // ps] * (hk * 2 * ps * (code + scale))
    base = base + torch.arange(hk, device=DEV)[:, None] * (2 * ps * (code + scale))
    out = []
    for which in (0, 1):
        rows = base + which * ps * code + (t % ps) * code
        raw = s["cache"][rows[..., None] + torch.arange(code, device=DEV)]
        sbase = base + 2 * ps * code + which * ps * scale
        if fmt == "bf16":
            x = raw.view(torch.bfloat16).double()
        elif fmt == "fp8_token":
            raws = s["cache"][(sbase + (t % ps) * 4)[..., None] + torch.arange(4, device=DEV)]
            x = tables[0][raw.int()] * raws.view(torch.float32).double()
        else:
            x = tables[0][raw.int()] if fmt == "mxfp8" else \
                tables[1][torch.stack((raw % 16, raw // 16), -1).flatten(-2).int()]
            grp = torch.arange(scale, device=DEV)
            off = (t % ps)[:, None] * scale + grp if which == 0 else grp * ps + (t % ps)[:, None]
            x = x * torch.exp2(s["cache"][sbase[..., None] + off].double() - 127).repeat_interleave(32, -1)
        out.append(x)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        r = case["rotary_dim"]
        z = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=DEV).expand(case["tokens"], r // 2),
                        s["positions"].double()[:, None] * s["inv_freq"] * (-1 if case["inverse"] else 1))[:, None]
        out = []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            first = slice(0, r // 2) if case["layout"] == "half" else slice(0, r, 2)
            second = slice(r // 2, r) if case["layout"] == "half" else slice(1, r, 2)
            w = torch.complex(x[..., first], x[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y)
        return tuple(out)
    if case["op"] == "cache":
        of = torch.empty(int(s["slots"].max()) + 1, dtype=torch.long, device=DEV)
        of[s["slots"]] = torch.arange(case["tokens"], device=DEV)
        rows = of[s["read_slots"]]
        return _round_trip(s["k"], case["fmt"])[rows], _round_trip(s["v"], case["fmt"])[rows]
    tables = _e4m3_table(), torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
    b, hk, d = case["batch"], case["kv_heads"], case["head_dim"]
    out = torch.zeros((b, case["q_heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, case["q_heads"]), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        m, total, acc = None, None, None
        for a in range(lo, n, 16384):
            k, v = _sequence(s, case, i, a, min(n, a + 16384), tables)
            x = (s["q"][i].double().view(hk, -1, 1, d) * s["scale"] * k[:, None]).sum(-1) if k.shape[1] < 8 else \
                torch.matmul(s["q"][i].double().view(hk, -1, d) * s["scale"], k.transpose(-1, -2).contiguous())
            part = torch.logsumexp(x, -1, keepdim=True)
            o = torch.matmul(torch.exp(x - part), v)
            if m is None:
                m, acc = part, o
            else:
                total = torch.logaddexp(m, part)
                acc, m = acc * torch.exp(m - total) + o * torch.exp(part - total), total
        if m is not None:
            out[i], lse[i] = acc.reshape(-1, d), m.reshape(-1)
    return out, lse
