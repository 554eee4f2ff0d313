"""GPU: the root-mean-square norm with residual and quantized output against
the float64 oracle.

Bounds.  h = x + residual is one f32 sum (2^-24).  A thread sums up to 64
squares, then 6 steps over its wave and up to 16 waves: positive terms, at most
86 roundings, 43 of them in the root; 1/k, its product, eps, the root and the
division add 4, two products and the weight's sum 3 to y: y is off by less than
(1 + 43 + 4 + 3 + 8) 2^-24 < 2^-18 of itself (weights whose sum with the offset
cancels are not drawn).  Its rounding adds half a step: 2^-8 of the value in
bf16, and in a code's own grid."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth
from gpu_util import f64

pytestmark = pytest.mark.gpu
L = oracle.layer
EPS = 2.0 ** -18
FMTS = ["fp8_token", "fp8_group", "mxfp8", "mxfp4"]


def _inputs(seed, m, k, res="bf16", wdt="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * scale
    x[:, ::37] *= 8
    r = None if res is None else torch.randn(m, k, generator=g) * 2 * scale
    w = 1 + 0.2 * torch.randn(k, generator=g)
    x = x.to(torch.bfloat16)
    r = r if r is None or res == "f32" else r.to(torch.bfloat16)
    w = w if wdt == "f32" else w.to(torch.bfloat16)
    return [None if t is None else t.cuda() for t in (x, r, w)]


def _near(got, ref, what=""):
    """bf16 against float64."""
    d = np.abs(f64(got) - ref)
    assert (d <= np.abs(ref) * (EPS + 2.0 ** -8) + 2.0 ** -133).all(), (what, (d / np.abs(ref).clip(1e-300)).max())


def half_step(v, fmt):
    """Half the distance of neighbouring codes at |v|."""
    bits, emin = (3, -6) if fmt != "mxfp4" else (1, 0)
    e = np.maximum(np.frexp(np.abs(v))[1] - 1, emin)
    return 2.0 ** (e - bits - 1)


def check_codes(codes, scales, ref, fmt, eps=EPS, what=""):
    """Codes and scales against the float64 rows that they stand for."""
    m, k = ref.shape
    c = codes.cpu().numpy()
    c = oracle.formats.decode_e2m1(oracle.formats.unpack_nibbles(c)) if fmt == "mxfp4" else oracle.formats.decode_e4m3(c)
    assert c.shape == ref.shape, what
    n = {"fp8_token": k, "fp8_group": 128}.get(fmt, 32)
    amax = np.abs(ref).reshape(m, k // n, n).max(2)
    s = scales.cpu().numpy().reshape(m, k // n)
    if fmt.startswith("mx"):
        e = oracle.quant.mxfp8_exponent(amax) if fmt == "mxfp8" else oracle.quant.mxfp4_exponent(amax)
        ok = s == e
        # a maximum within the error of a power of two may lie on its other side
        for side in (1 - 2 * eps, 1 + 2 * eps):
            ok |= s == (oracle.quant.mxfp8_exponent(amax * side) if fmt == "mxfp8" else oracle.quant.mxfp4_exponent(amax * side))
        assert ok.all(), what
        sc = np.ldexp(1.0, s.astype(np.int64) - 127)
    else:
        want = np.where(amax > 0, amax / 448.0, 1.0)
        assert (np.abs(s - want) <= want * (eps + 2.0 ** -24) + 2.0 ** -149).all(), what
        sc = s.astype(np.float64)
    top = 6.0 if fmt == "mxfp4" else 448.0
    v = ref / np.repeat(sc, n, 1)
    slack = np.abs(v) * (eps + 2.0 ** -22)
    # (the half step of the larger side: a value within the error of a power of two may round on its other side)
    v1 = np.clip(v, -top, top)
    tol = half_step(np.minimum(np.abs(v1) + slack, top), fmt) + slack
    d = np.abs(c - v1)
    assert (d <= tol).all(), (what, np.argwhere(d > tol)[:4], d.max())


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 2), (5, 7), (1, 63), (4, 64), (9, 500), (2, 512), (2, 513), (7, 2048), (3, 2056),
                                 (1, 4096), (5, 4100), (2, 8191), (3, 8192), (1, 8200), (2, 16384), (2, 20000), (1, 32768),
                                 (2, 40001), (1, 65536)])
def test_norm_bf16(m, k, res):
    x, r, w = _inputs(m * 7 + k, m, k, res)
    got = hum.rms_norm(x, w, residual=r)
    y, h = L.rms_norm(f64(x), f64(w), np.float32(1e-6), None if r is None else f64(r))
    if r is None:
        _near(got, y)
        return
    _near(got[0], y)
    assert got[1].dtype == r.dtype
    assert torch.equal(got[1], (x.float() + r.float()).to(r.dtype))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("res,wdt,offset", [(None, "bf16", 0.0), ("bf16", "f32", 1.0), ("f32", "bf16", 0.0)])
@pytest.mark.parametrize("m,k", [(1, 128), (6, 256), (5, 512), (3, 640), (1, 2048), (4, 4096), (2, 7168), (1, 8192), (2, 12800),
                                 (1, 20480), (1, 65536)])
def test_norm_quantized(fmt, m, k, res, wdt, offset):
    x, r, w = _inputs(m * 5 + k, m, k, res, wdt)
    w = w - offset
    got = hum.rms_norm(x, w, eps=1e-5, residual=r, act_fmt=fmt, weight_offset=offset)
    (q, s), h = got if r is not None else (got, None)
    y, hh = L.rms_norm(f64(x), f64(w), np.float32(1e-5), None if r is None else f64(r), offset)
    check_codes(q, s, y, fmt)
    if r is not None:
        assert torch.equal(h, (x.float() + r.float()).to(r.dtype))
    q2, s2, b = hum.rms_norm(x, w, eps=1e-5, act_fmt=fmt, weight_offset=offset, with_bf16=True) if r is None else \
        hum.rms_norm(x, w, eps=1e-5, residual=r, act_fmt=fmt, weight_offset=offset, with_bf16=True)[0]
    assert torch.equal(q, q2) and torch.equal(s, s2)
    _near(b, y)


@pytest.mark.parametrize("fmt,k", [("fp8_token", 8), ("fp8_token", 1000), ("fp8_token", 520), ("mxfp8", 32), ("mxfp4", 32),
                                   ("mxfp8", 544), ("mxfp4", 2080), ("fp8_group", 128), ("fp8_group", 640)])
def test_norm_quantized_odd_sizes(fmt, k):
    x, r, w = _inputs(k, 11, k)
    (q, s), _ = hum.rms_norm(x, w, residual=r, act_fmt=fmt)
    check_codes(q, s, L.rms_norm(f64(x), f64(w), np.float32(1e-6), f64(r))[0], fmt)


def test_codes_are_the_quantizers_of_the_same_values():
    """Where y is a bf16 value, the codes are hum_quant_act's of it: rows of +-1 with weights of powers of two, whose
    root mean square is 1 (eps below half an ulp)."""
    g = np.random.default_rng(5)
    for k in (256, 4096):
        x = torch.from_numpy(g.choice([-1.0, 1.0], (9, k))).to(torch.bfloat16).cuda()
        w = torch.from_numpy(2.0 ** g.integers(-6, 5, k)).to(torch.bfloat16).cuda()
        for fmt in FMTS:
            q, s, y = hum.rms_norm(x, w, eps=1e-12, act_fmt=fmt, with_bf16=True)
            q2, s2 = hum.quant_act(fmt, y)
            assert torch.equal(y, x * w) and torch.equal(q, q2) and torch.equal(s, s2), fmt


@pytest.mark.parametrize("k", [96, 1000, 4096, 9000])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_same_bits_at_every_alignment_and_batch(k, res):
    """Strides, offsets and the number of rows change no bit; what lies between the rows stays."""
    m = 6
    x, r, w = _inputs(k, m, k, res)
    fmt = "fp8_token" if k % 8 == 0 else None
    run = lambda *a, **kw: hum.rms_norm(*a, **kw)  # noqa: E731
    want = run(x, w, residual=r)
    wq = None if fmt is None else run(x, w, residual=r, act_fmt=fmt)

    def spread(t, off, extra):
        b = torch.full((m * (k + extra) + off + 8,), 7.0, dtype=t.dtype, device="cuda")
        v = b[off:off + m * (k + extra)].view(m, k + extra)[:, :k]
        v.copy_(t)
        return b, v

    for off, extra in ((1, 0), (2, 2), (4, 4), (0, 1), (8, 24), (3, 5)):
        _, xv = spread(x, off, extra)
        rv = None if r is None else spread(r, off, extra)[1]
        wv = torch.cat([w.new_zeros(off), w])[off:]
        buf, out = spread(torch.zeros_like(x), off, extra)
        kw = {}
        if r is not None:
            rb, kw["residual_out"] = spread(torch.zeros_like(r), off, extra)
        got = run(xv, wv, residual=rv, out=out, **kw)
        if r is None:
            assert got is out and torch.equal(out, want), (off, extra)
        else:
            assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1]), (off, extra)
            kw["residual_out"].fill_(7.0)
            assert (rb == 7).all()
        out.fill_(7.0)
        assert (buf == 7).all(), "between the rows"
        if fmt:
            got = run(xv, wv, residual=rv, act_fmt=fmt)
            for a, b in zip((got if r is None else got[0]), (wq if r is None else wq[0])):
                assert torch.equal(a, b)
    for i in range(m):
        one = run(x[i:i + 1], w, residual=None if r is None else r[i:i + 1])
        assert torch.equal(one if r is None else one[0], (want if r is None else want[0])[i:i + 1])


def test_in_place():
    x, r, w = _inputs(3, 50, 1032)
    want = hum.rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    y, h = hum.rms_norm(x1, w, residual=r1, residual_out=r1, out=x1)
    assert y is x1 and h is r1 and torch.equal(x1, want[0]) and torch.equal(r1, want[1])
    x1, r1 = x.clone(), r.clone()
    hum.rms_norm(x1, w, residual=r1, residual_out=x1, out=r1)              # each in the other's place
    assert torch.equal(r1, want[0]) and torch.equal(x1, want[1])
    x1 = x.clone()
    (q, s), h = hum.rms_norm(x1, w, residual=x1, residual_out=x1, act_fmt="fp8_token")
    assert torch.equal(h, (x.float() * 2).to(torch.bfloat16))
    y = L.rms_norm(2 * f64(x), f64(w), np.float32(1e-6))[0]
    check_codes(q, s, y, "fp8_token")


def test_broadcast_rows():
    """An input may be expanded: the same row for every token."""
    x, r, w = _inputs(8, 5, 640)
    got = hum.rms_norm(x[:1].expand(5, 640), w, residual=r)
    want = hum.rms_norm(x[:1].repeat(5, 1), w, residual=r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", ["bf16"] + FMTS)
def test_rows_of_zeros_and_of_extremes(fmt):
    k = 1024
    x = torch.zeros(8, k)
    g = torch.Generator().manual_seed(2)
    n = torch.randn(k, generator=g)
    x[1] = n * 2.0 ** 50
    x[2] = n * 2.0 ** -60
    x[3] = n * 2.0 ** -120          # y far below eps: 2^-110, and its codes' scales too
    x[4, 17] = 3.0                  # one value
    x[5] = n
    x[6] = n
    x = x.to(torch.bfloat16)
    w = torch.ones(k, dtype=torch.bfloat16)
    y = L.rms_norm(f64(x), f64(w), np.float32(1e-6))[0]
    bad = x.clone()
    bad[5, 3], bad[6, 900] = float("inf"), float("nan")
    for rows in (x, bad):
        got = hum.rms_norm(rows.cuda(), w.cuda(), act_fmt=fmt)
        keep = [0, 1, 2, 3, 4, 7] + ([5, 6] if rows is x else [])
        if fmt == "bf16":
            _near(got[keep], y[keep])
            if rows is bad:
                assert torch.isnan(got[5, 3]) and torch.isnan(got[6]).all()
        else:
            check_codes(got[0][keep], got[1][keep], y[keep], fmt)
            if rows is bad:                                       # visible in every scale
                s = got[1].view(8, -1)[5:7]
                assert (s == 255).all() if fmt.startswith("mx") else torch.isnan(s).all()


def test_many_rows():
    """More rows than workgroups at once, a wave a row and a workgroup a row."""
    for m, k in ((70001, 64), (20011, 600)):
        x, r, w = _inputs(m, m, k)
        y, h = hum.rms_norm(x, w, residual=r)
        ref, hh = L.rms_norm(f64(x), f64(w), np.float32(1e-6), f64(r))
        _near(y, ref)
        assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("m,k,fmt", [((4 << 20) + 5, 8, "fp8_token"), ((4 << 20) + 5, 9, "bf16"), ((1 << 20) + 3, 544, "mxfp8")])
def test_more_rows_than_a_grid_has(m, k, fmt):
    """Workgroups that take several rows: the same bits as those rows alone."""
    g = torch.Generator("cuda").manual_seed(m)
    x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(k, generator=g, device="cuda").to(torch.bfloat16)
    y = hum.rms_norm(x, w, residual=x, act_fmt=fmt)
    at = torch.cat([torch.arange(300), torch.arange(m - 300, m), torch.randint(0, m, (2000,), generator=torch.Generator().manual_seed(1))]).cuda()
    z = hum.rms_norm(x[at], w, residual=x[at], act_fmt=fmt)
    assert torch.equal(y[1][at], z[1])
    for a, b in zip(y[0] if fmt != "bf16" else y[:1], z[0] if fmt != "bf16" else z[:1]):
        assert torch.equal(a[at], b)
    part = 1 << 18
    for i in (0, m - part):                               # every row of both ends: sums of squares near one
        v = hum.rms_norm(x[i:i + part], torch.ones_like(w), residual=x[i:i + part])[0].float()
        assert ((v * v).mean(1) - 1).abs().max() < 0.02


def test_empty():
    x, r, w = _inputs(1, 0, 256)
    y, h = hum.rms_norm(x, w, residual=r)
    assert y.shape == h.shape == (0, 256)
    q, s = hum.rms_norm(x, w, act_fmt="mxfp4")
    assert q.shape == (0, 128) and s.shape == (0, 8)


def test_linear_takes_the_codes():
    """The codes are the activations of every product that takes them quantized."""
    k, n, m = 512, 96, 5
    x, r, w = _inputs(4, m, k)
    for fmt, (wd, gran, gs, sd) in (("fp8_token", ("e4m3", "channel", 0, "f32")), ("mxfp8", ("e2m1", "group", 32, "e8m0")),
                                    ("mxfp4", ("e2m1", "group", 32, "e8m0")), ("fp8_group", ("e4m3", "block", 128, "f32"))):
        g = synth.rng(9)
        codes = g.integers(0, 256, (1, n, k // 2 if wd == "e2m1" else k)).astype(np.uint8)
        if wd == "e4m3":
            codes = np.where((codes & 0x7F) == 0x7F, 0x30, codes).astype(np.uint8)
        shape = {"channel": (1, n, 1), "group": (1, n, k // 32), "block": (1, -(-n // 128), k // 128)}[gran]
        sc = g.integers(120, 130, shape).astype(np.uint8) if sd == "e8m0" else g.uniform(0.5, 1, shape).astype(np.float32)
        d = hum.make_desc(wd, gran, gs, sd, n, k, act_fmt=fmt)
        packed = hum.prepare_weight(d, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
        q, s, y = hum.rms_norm(x, w, act_fmt=fmt, with_bf16=True)
        a, b = f64(hum.linear(d, packed, q, a_scales=s)), f64(hum.linear(d, packed, y))
        # the two differ by codes of y that its rounding to bf16 moves over a border: few
        assert np.linalg.norm(a - b) <= 0.02 * np.linalg.norm(b), fmt
