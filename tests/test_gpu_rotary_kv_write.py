"""GPU: rotary positions and the append to the cache in one launch: the bits of
the two calls where these round alike, the float64 oracle where k is rounded
once, head norms, slots and strides.

Bounds: a coefficient is off by 2^-23 or so of one (its function's last bits),
two products and their sum round in f32: the turned pair is off by less than
2^-21 of its length; a head norm (a lane sums 8 squares, 5 steps) adds less
than 2^-20 of it.  The angle a itself is an f64 on both sides: the oracle rounds
position * inv_freq once, the kernel rounds inv_freq / 2 pi (its constant and
its product) and the product with the position: together 4 roundings of 2^-53,
2^-51 |a| radians (which only positions past 2^28 make more than 2^-23)."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
from gpu_util import bf16_bits_of, f64
from test_gpu_rms_norm import half_step

pytestmark = pytest.mark.gpu
A, L = oracle.attention, oracle.layer
FMTS = ["bf16", "fp8_token", "mxfp8", "mxfp4"]


class Case:
    def __init__(self, seed, fmt, t, hq, hk, d, r, ps=16, layout="half", max_pos=100000, skip=True):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.t, self.hq, self.hk, self.d, self.r, self.ps, self.layout = fmt, t, hq, hk, d, r, ps, layout
        x = torch.randn(t, hq + 2 * hk, d, generator=g)
        x[:, hq:hq + hk, ::16] *= 4
        self.qkv = x.to(torch.bfloat16).cuda()
        self.pages = -(-t // ps) + 2
        self.slots = torch.randperm(self.pages * ps, generator=g)[:t].cuda()
        if skip and t > 2:
            self.slots[1], self.slots[t // 2] = -1, self.pages * ps
        self.pos = torch.randint(0, max_pos, (t,), generator=g).cuda()
        self.freq = hum.rotary_inv_freq(r)[0].cuda()
        self.desc = hum.make_kv_desc(fmt, self.pages, ps, hk, d)
        self.w = [(1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2)]

    def split(self):
        return self.qkv.split([self.hq, self.hk, self.hk], 1)

    def cache(self, fill=0xA5):
        return torch.full((hum.kv_cache_bytes(self.desc),), fill, dtype=torch.uint8, device="cuda")

    def run(self, cache, qkv=None, **kw):
        q, k, v = qkv or self.split()
        kw = {**dict(layout=self.layout), **kw}
        return hum.rotary_kv_write(self.desc, cache, q if self.hq else None, k, v, self.pos, self.freq, self.slots, **kw)

    def apart(self, cache, factor=1.0, qk=None):
        q, k, v = self.split()
        q, k = qk or (q, k)
        q, k = hum.rotary(q, k, self.pos, self.freq, layout=self.layout, factor=factor)
        hum.kv_write(self.desc, cache, k, v, self.slots)
        return q

    def units(self, cache):
        """K codes, V codes, scales of K, of V: bytes [pages, hk, ...]."""
        row, sc = A.row_bytes(self.fmt, self.d)
        u = cache.cpu().numpy().reshape(self.pages, self.hk, -1)
        n, m = self.ps * row, self.ps * sc
        return u[..., :n], u[..., n:2 * n], u[..., 2 * n:2 * n + m], u[..., 2 * n + m:]

    def check(self, q_out, cache, factor=1.0, q_norm=None, k_norm=None, eps=1e-6, offset=0.0, err=2.0 ** -21):
        """Everything against the oracle, from a cache that held 0xA5."""
        q, k, v = (f64(x) for x in self.split())
        pos, freq = self.pos.cpu().numpy(), self.freq.cpu().numpy()
        out = []
        for x, w in ((q, q_norm), (k, k_norm)):
            y = x if w is None or not x.size else L.rms_norm(x, f64(w), np.float32(eps), weight_offset=offset)[0]
            z = A.rotary(y, pos, freq, self.layout, factor) if x.size else y
            i0 = np.arange(self.r // 2) if self.layout == "half" else np.arange(0, self.r, 2)
            i1 = i0 + (self.r // 2 if self.layout == "half" else 1)
            size = np.abs(y)
            if x.size:
                size = size.copy()
                size[..., i0] = size[..., i1] = abs(factor) * np.hypot(y[..., i0], y[..., i1])
            e = np.full(self.d, err + (2.0 ** -20 if w is not None else 0.0))
            e = np.tile(e, (self.t, 1, 1))
            e[..., i0] += np.abs(pos[:, None, None] * freq) * 2.0 ** -51
            e[..., i1] += np.abs(pos[:, None, None] * freq) * 2.0 ** -51
            out.append((z, size * e))
        if self.hq:
            z, e = out[0]
            assert (np.abs(f64(q_out) - z) <= e + (np.abs(z) + e) * 2.0 ** -8).all()
        z, e = out[1]
        kc, vc, ks, vs = self.units(cache)
        ref = A.Cache(self.fmt, self.pages, self.ps, self.hk, self.d, fill=0xA5)
        ref.write(self.slots.cpu().numpy(), np.zeros((self.t, self.hk, self.d), np.uint16), bf16_bits_of(self.split()[2]))
        rc = ref.buf.reshape(self.pages, self.hk, -1)
        row, sc = A.row_bytes(self.fmt, self.d)
        n, m = self.ps * row, self.ps * sc
        assert np.array_equal(vc, rc[..., n:2 * n]) and np.array_equal(vs, rc[..., 2 * n + m:])
        slots = self.slots.cpu().numpy()
        live = (slots >= 0) & (slots < self.pages * self.ps)
        page, at = slots[live] // self.ps, slots[live] % self.ps
        codes, scales = kc.reshape(self.pages, self.hk, self.ps, row).copy(), ks.reshape(self.pages, self.hk, self.ps, sc).copy()
        got, gs = codes[page, :, at], scales[page, :, at]                 # [n, hk, bytes]
        codes[page, :, at], scales[page, :, at] = 0xA5, 0xA5
        assert (codes == 0xA5).all() and (scales == 0xA5).all(), "untouched slots"
        z, e = z[live], e[live]
        if self.fmt == "bf16":
            y = A.row_values(got.reshape(-1, row), gs.reshape(got.shape[0] * self.hk, 0), "bf16").reshape(z.shape)
            assert (np.abs(y - z) <= e + (np.abs(z) + e) * 2.0 ** -8).all()
            return
        c = oracle.formats.decode_e2m1(oracle.formats.unpack_nibbles(got.reshape(-1, row))) if self.fmt == "mxfp4" else \
            oracle.formats.decode_e4m3(got)
        c = c.reshape(z.shape)
        nb = self.d if self.fmt == "fp8_token" else 32
        amax = np.abs(z).reshape(*z.shape[:2], -1, nb).max(-1)
        ea = e.reshape(*z.shape[:2], -1, nb).max(-1)
        if self.fmt == "fp8_token":
            s = np.ascontiguousarray(gs).view(np.float32).astype(np.float64)
            assert (np.abs(s - amax / 448) <= ea / 448 + amax / 448 * 2.0 ** -23).all()
        else:
            f = oracle.quant.mxfp8_exponent if self.fmt == "mxfp8" else oracle.quant.mxfp4_exponent
            assert ((gs == f(amax)) | (gs == f(amax + ea)) | (gs == f(np.maximum(amax - ea, 0)))).all()
            s = np.ldexp(1.0, gs.astype(np.int64) - 127)
        s = np.repeat(s, nb, -1)
        top = 6.0 if self.fmt == "mxfp4" else 448.0
        v = np.clip(z / s, -top, top)
        slack = e / s + np.abs(v) * 2.0 ** -22
        tol = half_step(np.minimum(np.abs(v) + slack, top), self.fmt) + slack
        assert (np.abs(c - v) <= tol).all(), (np.abs(c - v) - tol).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,hq,hk,d,r,ps", [(1, 2, 1, 64, 64, 16), (3, 0, 2, 128, 128, 16), (33, 8, 2, 128, 64, 32), (5, 5, 5, 64, 2, 256),
                                            (70, 3, 1, 256, 256, 16), (9, 7, 3, 256, 24, 64), (17, 16, 4, 128, 20, 128), (300, 32, 8, 64, 16, 16),
                                            (600, 4, 4, 128, 128, 64), (40, 64, 1, 64, 62, 16)])
def test_append(fmt, t, hq, hk, d, r, ps, layout):
    c = Case(t + d, fmt, t, hq, hk, d, r, ps, layout)
    cache = c.cache()
    q = c.run(cache)
    c.check(q, cache)
    # the two calls: q bit for bit; v's bytes, and in bf16 k's too
    two = c.cache()
    q2 = c.apart(two)
    if hq:
        assert torch.equal(q, q2)
    else:
        assert q is None
    if fmt == "bf16":
        assert torch.equal(cache, two)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,r", [(64, 64), (128, 128), (128, 48), (256, 64), (256, 18)])
def test_append_with_head_norms(fmt, d, r, layout):
    c = Case(d + r, fmt, 37, 6, 3, d, r, 16, layout)
    for wdt in (torch.bfloat16, torch.float32):
        qn, kn = (w.to(wdt) for w in c.w)
        for kw in (dict(q_norm=qn, k_norm=kn), dict(k_norm=kn), dict(q_norm=qn), dict(q_norm=qn - 1, k_norm=kn - 1, weight_offset=1.0, eps=0.5)):
            cache = c.cache()
            q = c.run(cache, **kw)
            c.check(q, cache, q_norm=kw.get("q_norm"), k_norm=kw.get("k_norm"), eps=kw.get("eps", 1e-6), offset=kw.get("weight_offset", 0.0))


def test_factor_and_far_positions():
    for fmt in ("bf16", "fp8_token"):
        c = Case(4, fmt, 50, 4, 2, 128, 128, max_pos=1 << 40)
        c.pos[:3] = torch.tensor([0, -5, -(1 << 40)])
        cache, two = c.cache(), c.cache()
        q = c.run(cache, factor=1.25)
        c.check(q, cache, factor=float(np.float32(1.25)))
        assert torch.equal(q, c.apart(two, 1.25))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_same_bits_at_every_alignment(layout):
    for fmt in FMTS:
        for d, r in ((128, 128), (64, 32)):
            c = Case(11, fmt, 21, 4, 2, d, r, 16, layout)
            want_cache = c.cache()
            want = c.run(want_cache, k_norm=c.w[1])
            for off, pad in ((1, 0), (2, 2), (4, 4), (8, 8), (0, 3)):
                parts = []
                for x in c.split():
                    b = torch.full((c.t * x.shape[1] * (d + pad) + off,), 3.0, dtype=torch.bfloat16, device="cuda")
                    y = b[off:].view(c.t, x.shape[1], d + pad)[..., :d]
                    y.copy_(x)
                    parts.append(y)
                out = torch.full((c.t * c.hq * (d + pad) + off,), 9.0, dtype=torch.bfloat16, device="cuda")
                view = out[off:].view(c.t, c.hq, d + pad)[..., :d]
                cache = c.cache()
                got = c.run(cache, qkv=parts, k_norm=c.w[1], q_out=view)
                assert got is view and torch.equal(view, want) and torch.equal(cache, want_cache), (fmt, off, pad)
                view.fill_(9.0)
                assert (out == 9).all()


def test_in_place_and_slices_of_one_buffer():
    for layout in ("half", "interleaved"):
        for r in (128, 40):
            c = Case(12, "mxfp8", 200, 8, 2, 128, r, 16, layout)
            cache, other = c.cache(), c.cache()
            want = c.run(cache)
            q, k, v = c.split()
            got = c.run(other, q_out=q)
            assert got is q and torch.equal(q, want) and torch.equal(cache, other)


def test_nothing_past_the_slots_is_written():
    """Every slot outside: the cache stays as it is, q is turned all the same."""
    c = Case(13, "fp8_token", 40, 4, 2, 64, 64)
    c.slots[:] = torch.tensor([-1, c.pages * c.ps, -(1 << 62), 1 << 62] * 10)
    cache = c.cache()
    q = c.run(cache)
    assert (cache == 0xA5).all()
    assert torch.equal(q, hum.rotary(c.split()[0], None, c.pos, c.freq)[0])


def test_infinities_and_nans_stay_in_their_rows():
    for fmt in FMTS:
        c = Case(14, fmt, 8, 2, 2, 64, 64, skip=False)
        clean = c.cache()
        q0 = c.run(clean)
        c.qkv[3, 0, 5], c.qkv[3, 2, 7], c.qkv[3, 4, 1] = float("nan"), float("inf"), float("nan")
        cache = c.cache()
        q = c.run(cache)
        keep = [i for i in range(8) if i != 3]
        assert torch.equal(q[keep], q0[keep]) and torch.equal(q[3, 1], q0[3, 1])
        a, b = (hum.kv_read(c.desc, x, c.slots[keep]) for x in (cache, clean))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_every_bit_pattern_of_v_reaches_a_bf16_cache():
    """Signaling NaNs too: v is copied there, as by the two calls."""
    c = Case(17, "bf16", 256, 1, 2, 128, 128, skip=False)
    c.qkv.view(torch.int16)[:, 3:] = torch.arange(-32768, 32768, dtype=torch.int32).view(256, 2, 128).to(torch.int16).cuda()
    cache, two = c.cache(), c.cache()
    c.run(cache)
    c.apart(two)
    assert torch.equal(cache, two)
    assert torch.equal(hum.kv_read(c.desc, cache, c.slots)[1].view(torch.int16), c.split()[2].contiguous().view(torch.int16))


def test_pages_at_the_far_end_of_a_large_cache():
    """Slots whose bytes lie past 4 GiB."""
    c = Case(15, "bf16", 6, 2, 8, 128, 128, 256)
    pages = 4200                                            # 1 MiB each
    c.desc = hum.make_kv_desc("bf16", pages, 256, 8, 128)
    cache = torch.zeros(hum.kv_cache_bytes(c.desc), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    c.slots = torch.tensor([0, 4097 * 256 + 3, pages * 256 - 1, 4100 * 256, 255, 4199 * 256], device="cuda")
    c.run(cache)
    k, v = hum.kv_read(c.desc, cache, c.slots)
    _, kr, vr = c.split()
    assert torch.equal(v, vr) and torch.equal(k, hum.rotary(c.split()[0], kr, c.pos, c.freq)[1])
    assert cache.view(pages, -1).any(1).nonzero().flatten().tolist() == [0, 4097, 4100, 4199]


def test_empty():
    c = Case(16, "bf16", 4, 2, 1, 64, 64)
    cache = c.cache()
    q, k, v = (x[:0] for x in c.split())
    out = hum.rotary_kv_write(c.desc, cache, q, k, v, c.pos[:0], c.freq, c.slots[:0])
    assert out.shape == (0, 2, 64) and (cache == 0xA5).all()
