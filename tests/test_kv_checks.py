"""CPU checks of the decode-step operators: sizes, frequencies, and refusals
before any launch (rotary, the paged cache, the attention over it)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return hum.load_library()


@pytest.mark.parametrize("fmt", ["bf16", "fp8_token", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_bytes_are_the_documented_layout(lib, fmt, d):
    desc = hum.make_kv_desc(fmt, 7, 32, 3, d)
    assert hum.kv_cache_bytes(desc) == oracle.attention.Cache(fmt, 7, 32, 3, d).buf.size


@pytest.mark.parametrize("bad", [dict(fmt="fp8_group"), dict(head_dim=96), dict(page_size=8), dict(page_size=48),
                                 dict(page_size=512), dict(num_kv_heads=0), dict(num_kv_heads=1025),
                                 dict(num_pages=0), dict(num_pages=-1), dict(num_pages=1 << 31)])
def test_cache_descriptions_refused(lib, bad):
    kw = dict(fmt="bf16", num_pages=4, page_size=16, num_kv_heads=2, head_dim=64)
    kw.update(bad)
    with pytest.raises(hum.HumError):
        hum.kv_cache_bytes(hum.make_kv_desc(**kw))


def test_inv_freq_values(lib):
    f, a = hum.rotary_inv_freq(64, 10000.0)
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    assert f.dtype == torch.float64 and a == 1.0
    g, _ = hum.rotary_inv_freq(64, scaling="linear", factor=8.0)
    np.testing.assert_allclose(g.numpy(), f.numpy() / 8, rtol=1e-14)
    # NTK: the fastest pair keeps its frequency, the slowest is divided by the factor
    g, _ = hum.rotary_inv_freq(64, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and abs(g[-1] / f[-1] * 8 - 1) < 1e-12 and (g[:-1] > g[1:]).all()
    # YaRN: pairs of 32 turns or more over the original length keep theirs, of less than one are divided
    g, a = hum.rotary_inv_freq(64, scaling="yarn", factor=8.0, original_len=4096)
    turns = 4096 * f.numpy() / (2 * math.pi)
    ratio = (g / f).numpy()
    assert (ratio[turns > 32 * 10000 ** (1 / 32)] == 1.0).all()
    np.testing.assert_allclose(ratio[turns < 10000 ** (-1 / 32)], 1 / 8, rtol=1e-12)
    assert (ratio[:-1] >= ratio[1:] - 1e-15).all() and abs(a - (0.1 * math.log(8) + 1)) < 1e-6


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="ntk", rotary_dim=2, factor=2.0),
                                dict(scaling="yarn", factor=2.0),
                                dict(scaling="yarn", factor=2.0, original_len=64, fast_turns=1, slow_turns=1)])
def test_inv_freq_refusals(lib, kw):
    kw.setdefault("rotary_dim", 64)
    with pytest.raises(hum.HumError):
        hum.rotary_inv_freq(**kw)


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def test_rotary_binding_refusals(lib):
    q, k = _bf(4, 8, 64), _bf(4, 2, 64)
    pos, f = torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    for bad, msg in ((dict(positions=pos.int()), "positions"), (dict(positions=pos[:3]), "positions"),
                     (dict(inv_freq=f.float()), "inv_freq"), (dict(q=q.half()), "q must"), (dict(k=k.float()), "k must"),
                     (dict(k=_bf(5, 2, 64)), "shape"), (dict(k=_bf(4, 2, 32)), "shape"), (dict(q=q[0]), "3-D"),
                     (dict(layout="other"), "layout"), (dict(q_out=_bf(4, 8, 32)), "q_out"),
                     (dict(q=q.transpose(1, 2)), "shape|contiguous"),
                     (dict(q_out=_bf(1, 8, 64).expand(4, 8, 64)), "expanded"), (dict(), "device tensor")):
        args = dict(q=q, k=k, positions=pos, inv_freq=f)
        args.update(bad)
        with pytest.raises(ValueError, match=msg):
            hum.rotary(**args)


def test_rotary_abi_refusals(lib):
    def call(t=4, dtype=hum.BF16, layout=0, d=64, r=64, hq=2, hk=1, inv=0, x=P(64), y=P(128), same_strides=True):
        desc = hum.RotaryDesc(dtype, layout, d, r, hq, hk, inv, 1.0)
        ys = 128 if same_strides else 256
        return lib.hum_rotary(ctypes.addressof(desc), t, P(16), P(16), x, 128, 64, y, ys, 64, P(256), 64, 64, P(512),
                              64, 64, None)
    assert call(t=-1) == 1 and call(t=1 << 24) == 2 and call(dtype=hum.INT8) == 2 and call(layout=2) == 1
    assert call(d=0) == 2 and call(d=1025) == 2 and call(r=63) == 1 and call(r=66) == 1 and call(r=0) == 1
    assert call(hq=-1) == 1 and call(inv=2) == 1 and call(x=None) == 1 and call(x=P(65)) == 1
    assert call(x=P(64), y=P(64), same_strides=False) == 1
    assert call(y=P(256)) == 1 and call(y=P(512)) == 1 and call(x=P(512), y=P(64)) == 1   # k, k's output, q = k's output
    assert call(t=0) == 0 and lib.hum_rotary(None, 0, *[None] * 2, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0,
                                             None) == 1


def test_cache_binding_refusals(lib):
    d = hum.make_kv_desc("mxfp8", 4, 16, 2, 64)
    cache = torch.zeros(hum.kv_cache_bytes(d), dtype=torch.uint8)
    k, s = _bf(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for args, msg in (((cache.int(), k, k, s), "cache"), ((cache, k.float(), k, s), "k must"),
                      ((cache, k, _bf(3, 1, 64), s), "v must"), ((cache, k, k, s.int()), "slots"),
                      ((cache, k, k, s[:2]), "slots"), ((cache[::2], k, k, s), "cache"), ((cache, k, k, s), "device")):
        with pytest.raises(ValueError, match=msg):
            hum.kv_write(d, *args)
    with pytest.raises(ValueError, match="slots"):
        hum.kv_read(d, cache, s.view(1, 3))
    with pytest.raises(ValueError, match="k_out"):
        hum.kv_read(d, cache, s, k_out=_bf(2, 2, 64))
    with pytest.raises(ValueError, match="device"):
        hum.kv_read(d, cache, s)


def test_cache_abi_refusals(lib):
    d = hum.make_kv_desc("mxfp8", 4, 16, 2, 64)
    a, nb = ctypes.addressof(d), hum.kv_cache_bytes(d)
    w = lambda **k: lib.hum_kv_write(a, k.get("c", P(64)), k.get("nb", nb), k.get("t", 3), k.get("s", P(8)),  # noqa: E731
                                     k.get("k", P(64)), 128, 64, P(64), 128, 64, None)
    assert w(c=None) == 1 and w(c=P(72)) == 1 and w(nb=nb - 1) == 3 and w(t=-1) == 1 and w(s=None) == 1
    assert w(k=None) == 1 and w(k=P(65)) == 1 and w(t=1 << 40) == 2 and w(t=0) == 0
    r = lambda ko=P(64), vo=P(128): lib.hum_kv_read(a, P(64), nb, 3, P(8), ko, vo, None)  # noqa: E731
    assert r(ko=None) == 1 and r(vo=P(72)) == 1 and r(vo=P(64)) == 1


def test_attention_binding_refusals(lib):
    d = hum.make_kv_desc("bf16", 4, 16, 2, 64)
    cache = torch.zeros(hum.kv_cache_bytes(d), dtype=torch.uint8)
    ok = dict(cache=cache, q=_bf(3, 4, 64), block_table=torch.zeros((3, 2), dtype=torch.int32),
              seq_lens=torch.zeros(3, dtype=torch.int32))
    for bad, msg in ((dict(q=_bf(3, 4, 128)), "q must"), (dict(q=torch.zeros(3, 4, 64)), "q must"),
                     (dict(q=_bf(3, 64)), "3-D"), (dict(block_table=ok["block_table"].long()), "block_table"),
                     (dict(block_table=ok["block_table"][:2]), "block_table"),
                     (dict(seq_lens=ok["seq_lens"].long()), "seq_lens"), (dict(seq_lens=ok["seq_lens"][:1]), "seq_lens"),
                     (dict(out=_bf(3, 4, 32)), "out"), (dict(cache=cache.float()), "cache"), (dict(), "device tensor")):
        args = dict(ok)
        args.update(bad)
        with pytest.raises(ValueError, match=msg):
            hum.kv_attention(d, **args)


def test_attention_abi_refusals(lib):
    d = hum.make_kv_desc("bf16", 4, 16, 2, 64)
    a, nb = ctypes.addressof(d), hum.kv_cache_bytes(d)
    need = hum.kv_attention_workspace_bytes(d, 4, 3, 2)

    def call(nb=nb, hq=4, b=3, q=P(64), tab=P(64), mp=2, lens=P(64), win=0, scale=1.0, out=P(64), ws=P(256), wsb=need,
             c=P(64)):
        return lib.hum_kv_attention(a, c, nb, hq, b, q, 256, 64, tab, 2, mp, lens, win, scale, out, None, ws, wsb, None)
    assert call(nb=nb - 1) == 3 and call(hq=5) == 1 and call(hq=0) == 1 and call(b=-1) == 1
    assert call(q=None) == 1 and call(q=P(65)) == 1 and call(tab=None) == 1 and call(lens=None) == 1
    assert call(out=None) == 1 and call(out=P(72)) == 1 and call(c=P(72)) == 1 and call(mp=-1) == 1
    assert call(mp=1 << 30) == 1 and call(win=-1) == 1 and call(scale=float("nan")) == 1
    assert call(b=65535, mp=1 << 24) == 2 and call(b=65536) == 1      # tiles past 32 bits, too many sequences
    assert call(scale=float("inf")) == 1 and call(ws=None) == 1 and call(wsb=need - 1) == 3 and call(b=0) == 0
    for bad in (dict(num_q_heads=3), dict(batch=-1), dict(max_pages=-1)):
        kw = dict(num_q_heads=4, batch=3, max_pages=2)
        kw.update(bad)
        with pytest.raises(hum.HumError):
            hum.kv_attention_workspace_bytes(d, **kw)


def test_binding_refuses_what_is_no_tensor_or_description(lib):
    d = hum.make_kv_desc("bf16", 4, 16, 2, 64)
    cache = torch.zeros(hum.kv_cache_bytes(d), dtype=torch.uint8)
    k, s = _bf(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for bad in (None, [1, 2], np.zeros(4)):
        with pytest.raises(ValueError, match="slots must be a"):
            hum.kv_write(d, cache, k, k, bad)
        with pytest.raises(ValueError, match="k must be a"):
            hum.kv_write(d, cache, bad, k, s)
        with pytest.raises(ValueError, match="cache must be a"):
            hum.kv_read(d, bad, s)
        with pytest.raises(ValueError, match="positions must be a"):
            hum.rotary(k, None, bad, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="KvDesc"):
        hum.kv_write(hum.TileConfig(), cache, k, k, s)
    with pytest.raises(TypeError):
        hum.kv_write(None, cache, k, k, s)
    q, tab, n = _bf(3, 4, 64), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        hum.kv_attention(d, cache, q, tab, n, workspace=torch.zeros(8))
    with pytest.raises(ValueError, match="seq_lens must have shape"):
        hum.kv_attention(d, cache, q, tab, n.view(3, 1))
    with pytest.raises(ValueError, match="rows must be contiguous"):
        hum.kv_attention(d, cache, q, torch.zeros((3, 4), dtype=torch.int32)[:, ::2], n)
    with pytest.raises(ValueError, match="layout"):
        hum.rotary(k, None, s, torch.zeros(32, dtype=torch.float64), layout=0)
    with pytest.raises(ValueError, match="negated"):
        hum.rotary(torch._neg_view(k.float()), None, s, torch.zeros(32, dtype=torch.float64))
    with pytest.raises((ValueError, TypeError)):
        hum.kv_attention(d, cache, q, tab, n, window=1.5)


def test_addresses_that_a_kernel_cannot_read_are_refused(lib):
    d = hum.make_kv_desc("bf16", 4, 16, 2, 64)
    a, nb, need = ctypes.addressof(d), hum.kv_cache_bytes(d), hum.kv_attention_workspace_bytes(d, 4, 3, 2)

    def attn(tab=P(64), lens=P(64), lse=None, scale=1.0):
        return lib.hum_kv_attention(a, P(64), nb, 4, 3, P(64), 256, 64, tab, 2, 2, lens, 0, scale, P(64), lse, P(256),
                                    need, None)
    assert attn(tab=P(66)) == 1 and attn(lens=P(65)) == 1 and attn(lse=P(66)) == 1
    assert attn(scale=3e38) == 1                                     # infinite in base 2
    assert lib.hum_kv_write(a, P(64), nb, 3, P(12), P(64), 128, 64, P(64), 128, 64, None) == 1
    # outputs of 3 x 2 x 64 bf16 = 768 bytes that share their last or first 16
    assert lib.hum_kv_read(a, P(64), nb, 3, P(8), P(1024), P(1024 + 752), None) == 1
    assert lib.hum_kv_read(a, P(64), nb, 3, P(8), P(1024 + 752), P(1024), None) == 1
    assert lib.hum_kv_read(a, P(64), nb, 3, P(12), P(1024), P(4096), None) == 1
    r = hum.RotaryDesc(hum.BF16, 0, 64, 64, 2, 0, 0, 1.0)
    for pos, freq in ((P(20), P(16)), (P(16), P(20))):
        assert lib.hum_rotary(ctypes.addressof(r), 4, pos, freq, P(64), 128, 64, P(4096), 128, 64, None, 0, 0, None, 0, 0,
                              None) == 1
