"""Cases of the operators around a layer's products: the root-mean-square norm
with the residual's addition and a quantized output, the routing of tokens to
experts, and the append of rotated keys and values to the paged cache.

``own`` chooses between the plain form (elementary torch operations in
float32, in float64 where a selection hangs on the last bits) and the
library's calls; both take what ``prepare`` returns.  ``exact`` states the
same results in float64, apart from the plain form.

Codes are returned as the values they stand for, without a copy: E4M3 codes
as ``float8_e4m3fn``, E8M0 scales as ``float8_e8m0fnu``.  MXFP4 takes the same
paths as MXFP8, but its packed pairs have no torch type that converts, so it
is not among the cases.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # before the qkv product of a single sequence's decode step: one token
        dict(name="norm step", op="norm", rows=1, size=4096, residual="bf16", fmt="fp8_token", offset=0.0),
        # a decode batch of 256 sequences, block-scaled activations
        dict(name="norm batch", op="norm", rows=256, size=7168, residual="bf16", fmt="fp8_group", offset=0.0),
        # an odd number of prompt tokens of an odd size, unquantized, the residual stream kept in f32, weights stored
        # as their distance from one
        dict(name="norm odd", op="norm", rows=3001, size=4100, residual="f32", fmt="bf16", offset=1.0),
        # a long prompt, activations quantized in blocks of 32
        dict(name="norm mx", op="norm", rows=8192, size=2048, residual="bf16", fmt="mxfp8", offset=0.0),
        # the largest: a long prompt of a wide model
        dict(name="norm prompt", op="norm", rows=16384, size=8192, residual="bf16", fmt="fp8_token", offset=0.0),
        # a decode batch among many experts in groups, balanced by a bias, some of its rows padding
        dict(name="route step", op="route", tokens=32, experts=256, topk=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype="f32", masked=0, padding=5),
        # a prompt among few experts
        dict(name="route few", op="route", tokens=4096, experts=8, topk=2, score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renormalize=True, scale=1.0, dtype="f32", masked=0, padding=0),
        # a long prompt, router logits in bf16 (equal ones are common), a few experts switched off
        dict(name="route bf16", op="route", tokens=16384, experts=128, topk=8, score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renormalize=True, scale=1.0, dtype="bf16", masked=3, padding=0),
        # an odd number of prompt tokens, many experts in groups with a bias
        dict(name="route groups", op="route", tokens=16381, experts=256, topk=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype="f32", masked=0, padding=0),
        # the new tokens of a decode step of 64 sequences
        dict(name="append step", op="append", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128,
             layout="half", norm=False, page_size=16, fmt="fp8_token", max_pos=32768),
        # an odd number of prompt tokens, wide heads, q and k normed per head first, part of each head turned in
        # adjacent pairs, kept in bf16
        dict(name="append normed", op="append", tokens=5003, q_heads=16, kv_heads=4, head_dim=256, rotary_dim=64,
             layout="interleaved", norm=True, page_size=32, fmt="bf16", max_pos=1 << 20),
        # a long prompt
        dict(name="append prompt", op="append", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128,
             layout="half", norm=False, page_size=64, fmt="mxfp8", max_pos=131072),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "append"])
    if op == "norm":
        fmt = rng.choice(["bf16", "fp8_token", "mxfp8", "fp8_group"])
        step = {"bf16": 1, "fp8_token": 8, "mxfp8": 32, "fp8_group": 128}[fmt]
        size = step * _log_int(rng, max(1, 64 // step), 16384 // step)
        return dict(op=op, rows=_log_int(rng, 1, min(16384, (1 << 26) // size)), size=size,
                    residual=rng.choice(["none", "bf16", "bf16", "f32"]), fmt=fmt, offset=rng.choice([0.0, 0.0, 1.0]))
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 72, 128, 160, 256, 384, 512])
        groups = rng.choice([1, 1, 4, 8]) if experts % 8 == 0 and experts >= 64 else 1
        kept = 1 if groups == 1 else rng.randint(1, groups)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts,
                    topk=min(rng.choice([1, 2, 4, 6, 8, 10]), experts // groups * kept),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, topk_groups=kept,
                    group_score=rng.choice(["max", "top2"]), renormalize=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "f32"]), masked=rng.choice([0, 0, 2]),
                    padding=rng.choice([0, 0, 1]))
    head_dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8]) if head_dim < 256 else rng.choice([1, 2, 4])
    return dict(op=op, tokens=_log_int(rng, 1, 8192), q_heads=kv_heads * rng.choice([1, 2, 4, 5]), kv_heads=kv_heads,
                head_dim=head_dim, rotary_dim=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4, 24]),
                layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.4,
                page_size=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["bf16", "fp8_token", "mxfp8"]),
                max_pos=_log_int(rng, 2048, 1 << 20))


# bytes of the codes of d values and of their scales
def _code_bytes(fmt, d):
    return {"bf16": 2 * d, "fp8_token": d, "fp8_group": d, "mxfp8": d}[fmt], \
        {"bf16": 0, "fp8_token": 4, "fp8_group": 4 * (d // 128), "mxfp8": d // 32}[fmt]


def work(case):
    if case["op"] == "norm":
        n, k = case["rows"], case["size"]
        stream = {"none": 0, "bf16": 4, "f32": 8}[case["residual"]]        # read and written
        return {"bytes": n * (k * (2 + stream) + sum(_code_bytes(case["fmt"], k))) + 2 * k, "flops": 8 * n * k}
    if case["op"] == "route":
        n, e = case["tokens"], case["experts"]
        return {"bytes": n * (e * (2 if case["dtype"] == "bf16" else 4) + 8 * case["topk"]) + (4 * e if case["bias"] else 0),
                "flops": 8 * n * e}
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    turned = t * (hq + hk)
    return {"bytes": t * (4 * hq * d + 2 * hk * (2 * d + sum(_code_bytes(case["fmt"], d))) + 16) + 4 * case["rotary_dim"],
            "flops": turned * (3 * case["rotary_dim"] + (4 * d if case["norm"] else 0))}


# ---------------------------------------------------------------------------
# inputs

def _page_unit(fmt, ps, d):
    """Bytes of one head of one page: K codes, V codes, K scales, V scales."""
    code, scale = _code_bytes(fmt, d)
    return ps * code, ps * scale, 2 * ps * (code + scale)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "norm":
        n, k = case["rows"], case["size"]
        x = normal(n, k)
        x[:, ::97] *= 6.0                              # a few channels stand out
        s = dict(case=case, x=x.to(torch.bfloat16), residual=None, weight=(1.0 - case["offset"] + 0.1 * normal(k)).to(torch.bfloat16))
        if case["residual"] != "none":
            r = normal(n, k).mul_(3.0)
            s["residual"] = r if case["residual"] == "f32" else r.to(torch.bfloat16)
        return s
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        x = normal(t, e).mul_(1.5)
        if case["masked"]:
            x[:, torch.randperm(e, generator=g, device=DEV)[:case["masked"]]] = -math.inf
        if case["padding"]:
            x[t - min(t, case["padding"]):] = -math.inf
        return dict(case=case, logits=x.to(torch.bfloat16) if case["dtype"] == "bf16" else x,
                    bias=normal(e).mul_(0.05) if case["bias"] else None)
    d, t, hq, hk, ps, fmt = (case[n] for n in ("head_dim", "tokens", "q_heads", "kv_heads", "page_size", "fmt"))
    # q, k and v as they come out of one product
    qkv = normal(t, hq + 2 * hk, d)
    qkv[:, hq:hq + hk, ::32] *= 4.0                    # keys have channels that stand out
    qkv = qkv.to(torch.bfloat16)
    # a decode step: tokens of as many sequences; a prompt: consecutive positions, page after page
    if t <= 256:
        pos = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV)
    else:
        pos = (torch.randint(0, case["max_pos"], (1,), generator=g, device=DEV) + torch.arange(t, device=DEV)) % case["max_pos"]
    pages = -(-t // ps) + 3
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:t] if t <= 256 else \
        (torch.randperm(pages, generator=g, device=DEV)[:, None] * ps + torch.arange(ps, device=DEV)).flatten()[:t].contiguous()
    slots[t // 2] = -1 if t > 4 else slots[t // 2]     # a token that another device holds
    r = case["rotary_dim"]
    inv_freq = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(DEV)
    norms = [(1.0 + 0.1 * normal(d)).to(torch.bfloat16) for _ in range(2)] if case["norm"] else [None, None]
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], positions=pos, slots=slots,
                inv_freq=inv_freq, q_norm=norms[0], k_norm=norms[1], pages=pages,
                cache=torch.zeros(pages * hk * _page_unit(fmt, ps, d)[2], dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------------------
# one pass

def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case)
    return _PLAIN[case["op"]](state, case)


def _norm_outputs(y, fmt, residual):
    """What a norm returns, codes and scales as their values."""
    if fmt != "bf16":
        q, sc = y
        y = (q.view(torch.float8_e4m3fn), sc.view(torch.float8_e8m0fnu) if fmt == "mxfp8" else sc)
    return y if residual is None else (y, residual)


def _own_norm(s, case):
    import quantized_gemm_packed_amd as hum
    r = hum.rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"], act_fmt=case["fmt"],
                     weight_offset=case["offset"])
    return _norm_outputs(r, case["fmt"], None) if s["residual"] is None else _norm_outputs(r[0], case["fmt"], r[1])


def _own_route(s, case):
    import quantized_gemm_packed_amd as hum
    return hum.moe_route(s["logits"], case["topk"], score=case["score"], bias=s["bias"], num_groups=case["groups"],
                         topk_groups=case["topk_groups"], group_score=case["group_score"],
                         renormalize=case["renormalize"], scale=case["scale"])


def _own_append(s, case):
    import quantized_gemm_packed_amd as hum
    if "own_desc" not in s:                            # the handle a program keeps with its cache
        s["own_desc"] = hum.make_kv_desc(case["fmt"], s["pages"], case["page_size"], case["kv_heads"], case["head_dim"])
    q = hum.rotary_kv_write(s["own_desc"], s["cache"], s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                            layout=case["layout"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    return q, _cache_values(s, case)


def _quantize(y, fmt):
    """float32 rows -> E4M3 codes and scales (f32 per row or per 128, E8M0 per 32)."""
    group = {"fp8_token": y.shape[-1], "fp8_group": 128, "mxfp8": 32}[fmt]
    g = y.unflatten(-1, (-1, group))
    top = g.abs().amax(-1, keepdim=True)
    if fmt == "mxfp8":
        e = torch.where(top > 0, (torch.frexp(top)[1] - 9 + 127).clamp(0, 254), 127)
        z = g * torch.exp2((127 - e).double()).float()
        sc = e.to(torch.uint8)
    else:
        sc = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))
        z = g / sc
    codes = z.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2), sc.squeeze(-1)


def _plain_norm(s, case):
    h = s["x"].float()
    out = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out = h.to(s["residual"].dtype)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * (s["weight"].float() + case["offset"])
    if case["fmt"] == "bf16":
        return _norm_outputs(y.to(torch.bfloat16), "bf16", out)
    q, sc = _quantize(y, case["fmt"])
    return _norm_outputs((q, sc[:, 0] if case["fmt"] == "fp8_token" else sc), case["fmt"], out)


def _plain_route(s, case):
    x, k = s["logits"].double(), case["topk"]
    t, e = x.shape
    live = x > -math.inf
    if case["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        p = p / p.sum(-1, keepdim=True).clamp(min=1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    # scores rise with their logits: without a bias these are compared, which no rounding makes equal
    order = x if s["bias"] is None else p + s["bias"].double()
    order = torch.where(live, order, -math.inf)
    if case["groups"] > 1:
        g, n = case["groups"], e // case["groups"]
        if case["group_score"] == "max" or n == 1:
            of = order.view(t, g, n).amax(-1)
        else:
            best = (p if s["bias"] is None else order).masked_fill(~live, -math.inf).view(t, g, n).sort(-1, descending=True)[0]
            of = best[..., 0] + torch.where(best[..., 1] > -math.inf, best[..., 1], 0.0)
        kept = torch.zeros((t, g), dtype=torch.bool, device=DEV)
        kept.scatter_(1, of.sort(dim=-1, descending=True, stable=True)[1][:, :case["topk_groups"]], True)
        order = order.masked_fill(~kept.repeat_interleave(n, 1), -math.inf)
    best, ids = order.sort(dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    w = torch.where(best > -math.inf, p.gather(1, ids), 0.0)
    if case["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(best > -math.inf, ids, -1).int(), (w * case["scale"]).float()


def _rows_of(units, fmt, ps, d):
    """Page units [..., unit] -> K codes, K scales, V codes, V scales, each [..., ps, bytes]."""
    nc, ns, _ = _page_unit(fmt, ps, d)
    kc, vc, ks, vs = units.split([nc, nc, ns, ns], -1)
    kc, vc, ks = (t.unflatten(-1, (ps, -1)) if t.shape[-1] else t.unsqueeze(-2) for t in (kc, vc, ks))
    # the scale bytes of V's 32-blocks lie by block, then by token
    vs = vs.unflatten(-1, (ps, -1)) if fmt == "fp8_token" else \
        vs.unflatten(-1, (-1, ps)).transpose(-1, -2) if ns else vs.unsqueeze(-2)
    return kc, ks, vc, vs


def _cache_values(s, case):
    """The cache's codes and scales as the values they stand for: views of it."""
    fmt, ps, d = case["fmt"], case["page_size"], case["head_dim"]
    units = s["cache"].view(s["pages"], case["kv_heads"], -1)
    nc = _page_unit(fmt, ps, d)[0]
    codes = units[..., :2 * nc].view(torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn)
    if fmt == "bf16":
        return (codes,)
    return codes, units[..., 2 * nc:].view(torch.float32 if fmt == "fp8_token" else torch.float8_e8m0fnu)


def _plain_append(s, case):
    r, fmt, ps, d = case["rotary_dim"], case["fmt"], case["page_size"], case["head_dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        if case["layout"] == "half":
            x0, x1 = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat((x0 * c - x1 * n, x0 * n + x1 * c), -1)
        else:
            x0, x1 = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack((x0 * c - x1 * n, x0 * n + x1 * c), -1).flatten(-2)
        return torch.cat((z, y[..., r:]), -1)

    rows = _rows_of(s["cache"].view(s["pages"], case["kv_heads"], -1), fmt, ps, d)
    live = torch.nonzero((s["slots"] >= 0) & (s["slots"] < s["pages"] * ps)).flatten()
    page, at = s["slots"][live] // ps, s["slots"][live] % ps
    for y, (codes, scales) in ((turn(s["k"], s["k_norm"]), rows[:2]), (s["v"].float(), rows[2:])):
        y = y[live]
        if fmt == "bf16":
            codes[page, :, at] = y.to(torch.bfloat16).view(torch.uint8)
            continue
        q, sc = _quantize(y, fmt)
        codes[page, :, at] = q
        scales[page, :, at] = sc.contiguous().view(torch.uint8)
    return turn(s["q"], s["q_norm"]).to(torch.bfloat16), _cache_values(s, case)


_OWN = {"norm": _own_norm, "route": _own_route, "append": _own_append}
_PLAIN = {"norm": _plain_norm, "route": _plain_route, "append": _plain_append}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _codes(y, fmt):
    """Float64 rows [..., k] -> what the codes round (as bf16 outputs are stated before their rounding) [..., k] and
    the scales [..., scales]."""
    k = y.shape[-1]
    n = {"fp8_token": k, "fp8_group": 128, "mxfp8": 32}[fmt]
    top = y.abs().view(*y.shape[:-1], k // n, n).max(-1)[0]
    if fmt == "mxfp8":
        s = torch.exp2((torch.log2(torch.where(top > 0, top, 256.0)).floor() - 8).clamp(-127, 127))
    else:
        s = torch.where(top > 0, top / 448.0, 1.0)
    return (y / s.repeat_interleave(n, -1)).clamp(-448.0, 448.0), s


def _normed(h, w):
    return w * h / (h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = _normed(h, s["weight"].double() + case["offset"])
        if case["fmt"] != "bf16":
            y = _codes(y, case["fmt"])
            y = (y[0], y[1].squeeze(-1) if case["fmt"] == "fp8_token" else y[1])
        return y if s["residual"] is None else (y, h)
    if case["op"] == "route":
        out = []
        for x in s["logits"].double().split(max(1, (1 << 26) // case["experts"] ** 2)):
            p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)).nan_to_num(0.0) if case["score"] == "softmax" else torch.sigmoid(x)
            live = x > -math.inf
            key = (x if s["bias"] is None else p + s["bias"].double()).masked_fill(~live, -math.inf)

            def ranks(v):              # how many come before each one
                before = v[:, None, :] > v[:, :, None]
                i = torch.arange(v.shape[1], device=DEV)
                return (before | ((v[:, None, :] == v[:, :, None]) & (i[None, :] < i[:, None]))).sum(-1)

            if case["groups"] > 1:
                n = x.shape[1] // case["groups"]
                two = case["group_score"] == "top2" and n > 1
                v = (p.masked_fill(~live, -math.inf) if two and s["bias"] is None else key).unflatten(1, (case["groups"], n))
                first, at = v.max(-1)
                if two:
                    second = v.scatter(-1, at[..., None], -math.inf).amax(-1)
                    first = torch.where(second > -math.inf, first + second, first)
                key = key.masked_fill((ranks(first) >= case["topk_groups"]).repeat_interleave(n, 1), -math.inf)
            rank = ranks(key)
            place = torch.arange(case["topk"], device=DEV)
            hit = (rank[:, None, :] == place[:, None]) & (key > -math.inf)[:, None, :]
            w = (hit * p[:, None, :]).sum(-1)
            if case["renormalize"]:
                w = (w / w.sum(-1, keepdim=True)).nan_to_num(0.0)
            out.append(w * case["scale"])
        return None, torch.cat(out)
    r, d, ps, hk, fmt = (case[n] for n in ("rotary_dim", "head_dim", "page_size", "kv_heads", "fmt"))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV).expand(case["tokens"], r // 2),
                       s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    first = slice(0, r // 2) if case["layout"] == "half" else slice(0, r, 2)
    second = slice(r // 2, r) if case["layout"] == "half" else slice(1, r, 2)
    done = []
    for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
        y = x.double() if w is None else _normed(x.double(), w.double())
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        done.append(y)
    q, kv = done[0], (done[1], s["v"].double())
    keep = s["slots"] >= 0
    page, at = s["slots"][keep] // ps, s["slots"][keep] % ps
    codes = torch.zeros((s["pages"], hk, 2, ps, d), dtype=torch.float64, device=DEV)
    scales = []
    for which in (0, 1):
        c, sc = (kv[which], None) if fmt == "bf16" else _codes(kv[which], fmt)
        codes[page, :, which, at] = c[keep]
        if fmt != "bf16":
            empty = 0.0 if fmt == "fp8_token" else 2.0 ** -127          # what zero bytes stand for
            of = torch.full((s["pages"], hk, ps, sc.shape[-1]), empty, dtype=torch.float64, device=DEV)
            of[page, :, at] = sc[keep]
            scales.append((of.transpose(-1, -2) if which and fmt == "mxfp8" else of).flatten(-2))
    codes = codes.view(s["pages"], hk, -1)
    return q, ((codes,) if fmt == "bf16" else (codes, torch.cat(scales, -1)))
