"""CPU checks of the norm, the routing and the rotated append: refusals before
any launch, from the C ABI and from the binding."""
import ctypes

import pytest
import torch

import quantized_gemm_packed_amd as hum

P = ctypes.c_void_p
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return hum.load_library()


def _norm(lib, m=4, k=256, fmt=hum.ACT_BF16, rdt=hum.BF16, wdt=hum.BF16, eps=1e-6, off=0.0, x=P(BIG), ldx=256, res=None,
          ldr=256, reso=None, ldro=256, w=P(64), out=P(2 * BIG), ldo=256, q=None, s=None):
    d = hum.NormDesc(fmt, rdt, wdt, eps, off)
    return lib.hum_rms_norm(ctypes.addressof(d), m, k, x, ldx, res, ldr, reso, ldro, w, out, ldo, q, s, None)


def test_norm_abi_refusals(lib):
    n = lambda **kw: _norm(lib, **kw)  # noqa: E731
    assert n(m=0) == 0 and n(m=0, x=None, w=None, out=None) == 0
    assert n(m=-1) == 1 and n(k=0) == 1 and n(k=65537) == 2 and n(m=1 << 40) == 2
    assert n(fmt=5) == 1 and n(fmt=-1) == 1 and n(rdt=hum.INT8) == 2 and n(wdt=hum.E4M3) == 2
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert n(eps=bad) == 1
    assert n(off=float("inf")) == 1 and n(off=float("nan")) == 1
    assert n(x=None) == 1 and n(w=None) == 1 and n(out=None) == 1
    assert n(res=P(3 * BIG)) == 1 and n(reso=P(3 * BIG)) == 1            # one without the other
    assert n(q=P(4 * BIG), s=P(5 * BIG)) == 1                            # codes of bf16
    c = dict(fmt=hum.ACT_MXFP8, q=P(4 * BIG), s=P(5 * BIG))
    for bad in (dict(q=None), dict(s=None), dict(q=P(4 * BIG + 4))):
        assert n(**{**c, **bad}) == 1
    assert n(fmt=hum.ACT_FP8_TOKEN, q=P(4 * BIG), s=P(5 * BIG + 2)) == 1
    for fmt, k in ((hum.ACT_FP8_TOKEN, 252), (hum.ACT_MXFP8, 240), (hum.ACT_MXFP4, 240), (hum.ACT_FP8_GROUP, 192)):
        assert n(fmt=fmt, k=k, q=P(4 * BIG), s=P(5 * BIG)) == 2
    assert n(x=P(BIG + 1)) == 1 and n(out=P(BIG - 1)) == 1 and n(w=P(65)) == 1 and n(w=P(66), wdt=hum.F32) == 1
    assert n(res=P(3 * BIG + 2), reso=P(3 * BIG + 2), rdt=hum.F32) == 1


def test_norm_overlaps_refused(lib):
    n = lambda **kw: _norm(lib, **kw)  # noqa: E731
    row = 512
    assert n(out=P(BIG + row)) == 1                                       # one row on
    assert n(out=P(BIG), ldo=512) == 1                                    # x's place with other strides
    assert n(out=P(BIG + 4 * row - 2)) == 1                               # the last element
    assert n(ldo=128) == 1                                                # rows of out over one another
    assert n(w=P(2 * BIG + 64)) == 1
    r = dict(res=P(3 * BIG), reso=P(4 * BIG))
    assert n(**{**r, "reso": P(2 * BIG + row)}) == 1                      # residual_out and out
    assert n(**{**r, "reso": P(3 * BIG + row)}) == 1
    assert n(res=P(3 * BIG), reso=P(BIG), rdt=hum.F32) == 1               # f32 in x's place
    assert n(res=P(3 * BIG), reso=P(BIG), out=P(BIG)) == 1                # both in x's place
    c = dict(fmt=hum.ACT_FP8_TOKEN, out=None, q=P(4 * BIG), s=P(5 * BIG))
    for bad in (dict(q=P(BIG + 8)), dict(s=P(BIG + 8)), dict(s=P(4 * BIG + 1020)), dict(q=P(64))):
        assert n(**{**c, **bad}) == 1


def test_norm_binding_refusals(lib):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    x, w = bf(4, 256), bf(256)
    for kw, msg in ((dict(x=x.float()), "x must be"), (dict(x=x[0]), "2-D"), (dict(x=x.t()), "contiguous"),
                    (dict(weight=bf(255)), "weight"), (dict(weight=w.half()), "weight"), (dict(weight=bf(1, 256)), "weight"),
                    (dict(residual=x.half()), "residual"), (dict(residual=bf(4, 128)), "residual"),
                    (dict(residual_out=x), "residual_out without"),
                    (dict(residual=x, residual_out=x.float()), "residual_out"),
                    (dict(residual=x, residual_out=bf(1, 256).expand(4, 256)), "expanded"),
                    (dict(act_fmt="other"), "act_fmt"), (dict(act_fmt=7), "act_fmt"),
                    (dict(act_fmt="mxfp8", out=x), "with_bf16"), (dict(out=bf(4, 128)), "out"),
                    (dict(x=bf(4, 0), weight=bf(0)), "columns|device"), (dict(), "device tensor"), (dict(x=None), "x must be")):
        a = dict(x=x, weight=w)
        a.update(kw)
        with pytest.raises((ValueError, hum.HumError), match=msg):
            hum.rms_norm(**a)


def _route(lib, t=4, x=P(BIG), ld=16, bias=None, ids=P(2 * BIG), w=P(3 * BIG), **kw):
    f = dict(logits_dtype=hum.F32, num_experts=16, topk=2, score=0, num_groups=1, topk_groups=1, group_score=0, renormalize=1,
             scale=1.0)
    f.update(kw)
    d = hum.RouteDesc(**f)
    return lib.hum_moe_route(ctypes.addressof(d), t, x, ld, bias, ids, w, None)


def test_route_abi_refusals(lib):
    r = lambda **kw: _route(lib, **kw)  # noqa: E731
    assert r(t=0) == 0 and r(t=0, x=None) == 0 and lib.hum_moe_route(None, 0, None, 0, None, None, None, None) == 1
    assert r(t=-1) == 1 and r(t=1 << 24) == 2 and r(logits_dtype=hum.INT8) == 2
    assert r(num_experts=0) == 2 and r(num_experts=513) == 2 and r(topk=0) == 1 and r(topk=17) == 1
    assert r(num_experts=128, topk=65) == 1 and r(score=2) == 1 and r(group_score=2) == 1 and r(renormalize=2) == 1
    assert r(num_groups=0) == 1 and r(num_groups=3) == 1 and r(num_groups=4, topk_groups=5) == 1 and r(topk_groups=0) == 1
    assert r(num_experts=512, num_groups=128) == 1
    assert r(scale=float("nan")) == 1 and r(scale=float("inf")) == 1
    assert r(x=None) == 1 and r(ids=None) == 1 and r(w=None) == 1
    assert r(x=P(BIG + 2)) == 1 and r(bias=P(66)) == 1 and r(ids=P(2 * BIG + 1)) == 1 and r(w=P(3 * BIG + 2)) == 1
    assert r(w=P(2 * BIG + 28)) == 1 and r(ids=P(BIG + 32)) == 1 and r(w=P(BIG - 28)) == 1 and r(bias=P(2 * BIG + 28)) == 1


def test_route_binding_refusals(lib):
    x = torch.zeros(4, 16)
    for kw, msg in ((dict(logits=x.double()), "logits"), (dict(logits=x[0]), "2-D"), (dict(logits=x.t()), "contiguous"),
                    (dict(topk=0), "topk"), (dict(topk=17), "topk"), (dict(score="other"), "score"),
                    (dict(group_score="sum"), "group_score"), (dict(bias=x[0].double()), "bias"), (dict(bias=x[0, :8]), "bias"),
                    (dict(topk_ids=torch.zeros(4, 2)), "topk_ids"), (dict(topk_ids=torch.zeros((4, 3), dtype=torch.int32)), "topk_ids"),
                    (dict(topk_weights=torch.zeros(4, 4)[:, ::2]), "topk_weights"),
                    (dict(topk_weights=torch.zeros(1, 2).expand(4, 2)), "topk_weights"), (dict(), "device tensor")):
        a = dict(logits=x, topk=2)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            hum.moe_route(**a)
    with pytest.raises((ValueError, TypeError)):
        hum.moe_route(x, 1.5)


def _append(lib, rot=None, kv=None, norm=None, nb=None, t=4, c=P(BIG), pos=P(64), f=P(1024), s=P(4096), q=P(2 * BIG), qs=(128, 64),
            qo=P(3 * BIG), qos=(128, 64), k=P(4 * BIG), ks=(64, 64), v=P(5 * BIG), vs=(64, 64)):
    r = dict(dtype=hum.BF16, layout=0, head_dim=64, rotary_dim=64, num_q_heads=2, num_kv_heads=1, inverse=0, factor=1.0)
    r.update(rot or {})
    d = kv or hum.make_kv_desc("bf16", 4, 16, 1, 64)
    r = hum.RotaryDesc(**r)
    nb = nb if nb is not None else 4 * 16 * 64 * 4
    return lib.hum_rotary_kv_write(ctypes.addressof(r), ctypes.addressof(d), None if norm is None else ctypes.addressof(norm),
                                   c, nb, t, pos, f, s, q, *qs, qo, *qos, k, *ks, v, *vs, None)


def test_append_abi_refusals(lib):
    a = lambda **kw: _append(lib, **kw)  # noqa: E731
    assert a(t=0) == 0 and a(t=0, c=None, q=None) == 0
    assert a(t=-1) == 1 and a(t=1 << 24) == 2
    assert a(rot=dict(dtype=hum.F32)) == 2 and a(rot=dict(layout=2)) == 1 and a(rot=dict(head_dim=128)) == 1
    assert a(rot=dict(rotary_dim=63)) == 1 and a(rot=dict(rotary_dim=66)) == 1 and a(rot=dict(rotary_dim=0)) == 1
    assert a(rot=dict(num_kv_heads=2)) == 1 and a(rot=dict(num_q_heads=-1)) == 1 and a(rot=dict(num_q_heads=4097)) == 1
    assert a(rot=dict(inverse=1)) == 1 and a(kv=hum.make_kv_desc("fp8_group", 4, 16, 1, 64)) == 2
    for name in ("c", "pos", "f", "s", "q", "qo", "k", "v"):
        assert a(**{name: None}) == 1, name
    assert a(nb=4 * 16 * 64 * 4 - 1) == 3 and a(c=P(BIG + 8)) == 1
    assert a(pos=P(68)) == 1 and a(f=P(1028)) == 1 and a(s=P(4100)) == 1 and a(k=P(4 * BIG + 1)) == 1 and a(q=P(2 * BIG + 1)) == 1
    n = lambda **kw: hum.HeadNorm(**{**dict(q_weight=1 << 40, k_weight=1 << 41, weight_dtype=hum.BF16, eps=1e-6, weight_offset=0.0), **kw})  # noqa: E731
    assert a(norm=n(eps=0.0)) == 1 and a(norm=n(eps=float("nan"))) == 1 and a(norm=n(weight_offset=float("inf"))) == 1
    assert a(norm=n(weight_dtype=hum.INT8)) == 2 and a(norm=n(q_weight=(1 << 40) + 1)) == 1
    assert a(norm=n(k_weight=(1 << 40) + 2, weight_dtype=hum.F32)) == 1


def test_append_overlaps_refused(lib):
    a = lambda **kw: _append(lib, **kw)  # noqa: E731
    size = 4 * 16 * 64 * 4
    assert a(qo=P(2 * BIG + 128)) == 1 and a(qo=P(2 * BIG), qos=(64, 256)) == 1 and a(qos=(64, 64)) == 1
    assert a(qo=P(4 * BIG)) == 1 and a(qo=P(5 * BIG + 64)) == 1 and a(qo=P(BIG + size - 2)) == 1
    assert a(k=P(BIG + 128)) == 1 and a(v=P(BIG)) == 1 and a(q=P(BIG + size - 2)) == 1
    assert a(pos=P(3 * BIG)) == 1 and a(s=P(3 * BIG + 8)) == 1 and a(f=P(3 * BIG + 16)) == 1
    assert a(pos=P(BIG)) == 1 and a(s=P(BIG + 8)) == 1 and a(f=P(BIG + 16)) == 1
    n = hum.HeadNorm(q_weight=3 * BIG + 64, k_weight=None, weight_dtype=hum.BF16, eps=1e-6, weight_offset=0.0)
    assert a(norm=n) == 1


def test_append_binding_refusals(lib):
    d = hum.make_kv_desc("mxfp8", 4, 16, 2, 64)
    cache = torch.zeros(hum.kv_cache_bytes(d), dtype=torch.uint8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q, k = bf(3, 4, 64), bf(3, 2, 64)
    pos, s, f = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    w = bf(64)
    for kw, msg in ((dict(cache=cache.int()), "cache"), (dict(q=q.float()), "q must"), (dict(q=bf(2, 4, 64)), "q must"),
                    (dict(k=bf(3, 1, 64)), "k must"), (dict(v=bf(3, 2, 32)), "v must"), (dict(positions=pos.int()), "positions"),
                    (dict(slots=s[:2]), "slots"), (dict(inv_freq=f.float()), "inv_freq"), (dict(layout="other"), "layout"),
                    (dict(q_norm=w.half()), "q_norm"), (dict(k_norm=bf(32)), "k_norm"), (dict(q_norm=w, k_norm=w.float()), "k_norm"),
                    (dict(q=None, q_norm=w), "q_norm without"), (dict(q=None, q_out=q), "q_out without"),
                    (dict(q_out=bf(3, 4, 32)), "q_out"), (dict(q_out=bf(1, 4, 64).expand(3, 4, 64)), "expanded"),
                    (dict(q=q.transpose(1, 2)), "shape|contiguous"), (dict(), "device tensor")):
        a = dict(cache=cache, q=q, k=k, v=k, positions=pos, inv_freq=f, slots=s)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            hum.rotary_kv_write(d, **a)
    with pytest.raises(ValueError, match="KvDesc"):
        hum.rotary_kv_write(hum.TileConfig(), cache, q, k, k, pos, f, s)


def test_empty_calls_launch_nothing(lib):
    """m = 0 and T = 0 pass the checks of everything but the device."""
    assert _norm(lib, m=0, fmt=hum.ACT_FP8_TOKEN) == 0
    assert _route(lib, t=0, ids=None, w=None) == 0
