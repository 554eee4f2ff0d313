"""GPU: the paged key-value cache (bytes bit for bit against the oracle) and
the attention over it (against float64).

Tolerance of the attention, from its arithmetic: probabilities (times an FP8
row's scale) are rounded to bf16 before the product with V, at most 2^-8 of
each, and the result once more: 2^-8 (sum_t p_t |v_t| + |out|).  Scores are
f32 sums of D products whose magnitudes add up to B = max_t scale sum |q k|:
a relative error of the probabilities of at most d = (D + 16) 2^-24 (1 + B) +
2^-20 (exponential), and f32 sums over n tokens add n 2^-24; both count twice,
above and below the division.  lse is off by at most d + n 2^-24 + 2^-22
|lse|."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth

pytestmark = pytest.mark.gpu
A = oracle.attention
FMTS = ["bf16", "fp8_token", "mxfp8", "mxfp4"]


def _bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _kv(seed, t, h, d):
    g = synth.rng(seed)
    out = []
    for _ in range(2):
        x = g.standard_normal((t, h, d)).astype(np.float32) * np.exp2(g.standard_normal((t, h, 1)) * 2).astype(np.float32)
        if t > 3:
            x[0] = 0.0
            x[1] *= 1e30
            x[2] *= 1e-30
            x[3, :, :32] = 0.0
            x[3, :, 40] = -0.0
        out.append(synth.bf16_bits(x))
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,h,d,ps", [(1, 1, 64, 16), (37, 3, 128, 16), (200, 8, 64, 64), (65, 2, 256, 128),
                                      (129, 5, 128, 256)])
def test_cache_bytes_and_round_trip(fmt, t, h, d, ps):
    print(f"case kv {fmt} {t} {h} {d} {ps}", flush=True)
    kb, vb = _kv(t + d, t, h, d)
    pages = -(-t // ps) + 2
    g = np.random.default_rng(t)
    slots = g.permutation(pages * ps)[:t].astype(np.int64)
    if t > 8:
        slots[4], slots[5], slots[6] = -1, pages * ps, 1 << 40    # none of these is written
    ref = A.Cache(fmt, pages, ps, h, d, fill=0xA5)
    ref.write(slots, kb, vb)
    desc = hum.make_kv_desc(fmt, pages, ps, h, d)
    cache = torch.full((hum.kv_cache_bytes(desc),), 0xA5, dtype=torch.uint8, device="cuda")
    qkv = torch.cat([torch.zeros((t, 2, d), dtype=torch.bfloat16, device="cuda"), _bf(kb), _bf(vb)], 1)
    sl = torch.from_numpy(slots).cuda()
    hum.kv_write(desc, cache, qkv[:, 2:2 + h], qkv[:, 2 + h:], sl)
    assert np.array_equal(cache.cpu().numpy(), ref.buf.reshape(-1))
    k, v = hum.kv_read(desc, cache, sl)
    for got, which in ((k, 0), (v, 1)):
        want = torch.from_numpy(ref.rows(slots, which)).to(torch.bfloat16)
        # the code times the scale is one f32 product, exact in float64, rounded to bf16 by way of f32
        want2 = torch.from_numpy(ref.rows(slots, which).astype(np.float32)).to(torch.bfloat16)
        same = (got.cpu() == want) | (got.cpu() == want2)
        assert same.all()
    # the same rows two bytes off 16-byte alignment
    flat = torch.zeros(t * 2 * h * d + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(t, 2 * h, d)
    odd.copy_(qkv[:, 2:])
    cache2 = torch.full_like(cache, 0xA5)
    hum.kv_write(desc, cache2, odd[:, :h], odd[:, h:], sl)
    assert torch.equal(cache, cache2)


@pytest.mark.parametrize("exponent", [0, -69, -71, -126, 120, 127])
def test_fp8_rows_of_every_quotient(exponent):
    """Every bf16 mantissa over every scale's: rows whose maximum has each of
    the 128 mantissas and whose other values are all bf16 down to 2^-13 of it,
    both signs, so that no quotient near a rounding border is missed; exponents
    on both sides of where the division changes its form."""
    vals = ((np.arange(13 * 128, dtype=np.int64)) + ((exponent + 127 - 12) << 7))
    vals = vals[vals >= 0]
    rows = []
    for m in range(128):
        top = ((exponent + 127) << 7) + m
        low = vals[vals <= top]
        low = np.concatenate([low, low + 0x8000, [0x8000, 0]])
        pad = -len(low) % 127
        low = np.concatenate([low, np.zeros(pad, np.int64)]).reshape(-1, 127)
        rows.append(np.concatenate([np.full((len(low), 1), top), low], 1))
    x = np.concatenate(rows).astype(np.uint16)
    t = len(x)
    desc = hum.make_kv_desc("fp8_token", -(-t // 16), 16, 1, 128)
    ref, _ = A.quantize_rows(x, "fp8_token")
    cache = torch.zeros(hum.kv_cache_bytes(desc), dtype=torch.uint8, device="cuda")
    xb = _bf(x).view(t, 1, 128)
    hum.kv_write(desc, cache, xb, xb, torch.arange(t, device="cuda"))
    unit = cache.view(-1, 2 * 16 * 132).cpu().numpy()
    for which in (0, 1):
        got = unit[:, which * 16 * 128:(which + 1) * 16 * 128].reshape(-1, 128)[:t]
        assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    scales = unit[:, 2 * 16 * 128:2 * 16 * 128 + 64].copy().view(np.float32).reshape(-1)[:t]
    assert np.array_equal(scales, A.quantize_rows(x, "fp8_token")[1].view(np.float32).reshape(-1))


def test_cache_empty_call_and_repeated_reads():
    desc = hum.make_kv_desc("fp8_token", 2, 16, 1, 64)
    cache = torch.zeros(hum.kv_cache_bytes(desc), dtype=torch.uint8, device="cuda")
    e = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    s0 = torch.zeros(0, dtype=torch.int64, device="cuda")
    hum.kv_write(desc, cache, e, e, s0)
    assert hum.kv_read(desc, cache, s0)[0].shape == (0, 1, 64)
    x = torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16)
    hum.kv_write(desc, cache, x, x, torch.tensor([17], device="cuda"))
    k, v = hum.kv_read(desc, cache, torch.tensor([17, -5, 17, 32], device="cuda"))
    assert torch.equal(k[0], k[2]) and torch.equal(k, v) and not k[1].any() and not k[3].any() and k[0].any()


class Case:
    """A cache with sequences of the given lengths on scattered pages; every
    byte that no token owns is 0xFF (NaN in E4M3, E8M0, f32 and bf16)."""

    def __init__(self, seed, fmt, lens, hq, hk, d, ps, max_pages=None, missing=()):
        g = np.random.default_rng(seed)
        self.fmt, self.hq, self.d, self.ps = fmt, hq, d, ps
        need = [-(-n // ps) for n in lens]
        self.pages = sum(need) + 2
        mp = max(need + [1]) if max_pages is None else max_pages
        ids = g.permutation(self.pages)
        self.table = np.full((len(lens), mp), 0x7FFFFFFF, np.int32)     # never read, or skipped
        self.cache = A.Cache(fmt, self.pages, ps, hk, d, fill=0xFF)
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            t = np.arange(n)
            if n:
                slots = self.table[b][t // ps].astype(np.int64) * ps + t % ps
                kb = synth.bf16_bits((g.standard_normal((n, hk, d)) * 1.5).astype(np.float32))
                vb = synth.bf16_bits((g.standard_normal((n, hk, d)) + 0.5).astype(np.float32))
                self.cache.write(slots, kb, vb)
        for b, i in missing:
            self.table[b, i] = -1
        self.lens = np.array(lens, np.int32)
        self.qb = synth.bf16_bits(g.standard_normal((len(lens), hq, d)).astype(np.float32))
        self.q = oracle.formats.decode_bf16(self.qb)
        self.desc = hum.make_kv_desc(fmt, self.pages, ps, hk, d)
        self.dev = dict(cache=torch.from_numpy(self.cache.buf.reshape(-1)).cuda(), q=_bf(self.qb),
                        block_table=torch.from_numpy(self.table).cuda(), seq_lens=torch.from_numpy(self.lens).cuda())

    def run(self, **kw):
        return hum.kv_attention(self.desc, **{**self.dev, **kw})

    def check(self, got, scale=None, window=0, what=""):
        out, lse = (x.double().cpu().numpy() for x in got)
        ref, rl, mag, big = A.attention(self.cache, self.q, self.table, self.lens,
                                        float(np.float32(self.d ** -0.5 if scale is None else scale)), window)
        n = self.lens.max() if len(self.lens) else 0
        d = (self.d + 16) * 2.0 ** -24 * (1 + big) + 2.0 ** -20 + n * 2.0 ** -24
        tol = 2.0 ** -8 * (mag + np.abs(ref)) + 2 * d[..., None] * mag
        assert np.isfinite(out).all(), what
        assert (np.abs(out - ref) <= tol).all(), (what, (np.abs(out - ref) / np.maximum(tol, 1e-30)).max())
        fin = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse), ~fin), what
        assert (np.abs(lse[fin] - rl[fin]) <= d[fin] + 2.0 ** -22 * np.abs(rl[fin])).all(), what


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,hq,hk,d,ps", [
    ([1], 1, 1, 64, 16), ([0, 1, 31, 32, 33, 127, 128, 129], 8, 2, 128, 16), ([700, 0, 513], 4, 4, 64, 64),
    ([300, 77], 16, 1, 256, 32), ([65, 1023], 20, 1, 128, 128), ([259], 12, 2, 128, 256), ([5] * 9, 40, 2, 64, 16)])
def test_attention(fmt, lens, hq, hk, d, ps):
    print(f"case attention {fmt} {lens} {hq} {hk} {d} {ps}", flush=True)
    c = Case(sum(lens) + hq, fmt, lens, hq, hk, d, ps)
    got = c.run(return_lse=True)
    c.check(got, what="all tokens")
    again = c.run(return_lse=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    for w in (1, 50):
        c.check(c.run(return_lse=True, window=w), window=w, what=f"window {w}")
    out = torch.full((len(lens), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert c.run(out=out) is out and torch.equal(out, got[0])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_attention_missing_pages_and_empty_rows(fmt):
    """Pages outside the cache take no part; a sequence of only such pages is
    an empty row."""
    c = Case(11, fmt, [100, 64, 200, 16], 4, 2, 64, 16, missing=[(0, 1), (0, 6), (1, 0), (1, 1), (1, 2), (1, 3), (2, 0)])
    got = c.run(return_lse=True)
    c.check(got, what="missing pages")
    assert not got[0][1].any() and torch.isneginf(got[1][1]).all()
    c.check(c.run(return_lse=True, window=4), window=4, what="window in a missing page")


def test_attention_lengths_are_clamped_and_strides_are_any():
    c = Case(12, "bf16", [90, 40, 10], 6, 2, 64, 16)
    over = torch.tensor([90, 1 << 30, -7], dtype=torch.int32, device="cuda")
    c2 = Case(12, "bf16", [90, 48, 10], 6, 2, 64, 16)  # (48: whole pages, so a longer length adds no stale token)
    # q as a slice of a fused product, two bytes off alignment; a table with a row stride
    flat = torch.zeros(3 * 10 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    q = flat[1:].view(3, 10, 64)[:, 3:9]
    q.copy_(c.dev["q"])
    wide = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + c.table.shape[1]] = c.dev["block_table"]
    table = wide[:, 4:4 + c.table.shape[1]]
    c.check(c.run(return_lse=True, q=q, block_table=table), what="strided")
    assert c2.table.shape[1] == 6
    got = c2.run(return_lse=True, seq_lens=over)
    c2.lens = np.array([90, 96, 0])                    # the second row's further entries name no page
    c2.check(got, what="clamped")


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_large_scores_and_scale(fmt):
    """Scores in the hundreds (their differences decide which token wins), a
    negative and a zero scale."""
    c = Case(13, fmt, [150, 400], 4, 1, 128, 32)
    for s in (1.0, -0.3, 0.0):
        c.check(c.run(return_lse=True, scale=s), scale=s, what=f"scale {s}")


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_attention_mx_scales_at_their_ends(fmt):
    """Values whose E8M0 scales are near and at the smallest code, and large ones."""
    c = Case(19, fmt, [64, 33], 4, 2, 128, 16)
    g = np.random.default_rng(20)
    for b, n in enumerate((64, 33)):
        t = np.arange(n)
        slots = c.table[b][t // 16].astype(np.int64) * 16 + t % 16
        e = g.integers(-126, -100, (n, 2, 4)).repeat(32, -1)
        k = synth.bf16_bits(np.ldexp(g.standard_normal((n, 2, 128)), np.where(e < -120, e, 0)).astype(np.float32))
        v = synth.bf16_bits(np.ldexp(g.standard_normal((n, 2, 128)), np.where(e % 2 == 0, 100, 90)).astype(np.float32))
        c.cache.write(slots, k, v)
    scales = c.cache.buf[:, :, 2 * 16 * c.cache.row:2 * 16 * c.cache.row + 16 * 4]
    assert (scales == 0).any()
    c.dev["cache"] = torch.from_numpy(c.cache.buf.reshape(-1)).cuda()
    c.check(c.run(return_lse=True), what="scales")


@pytest.mark.parametrize("fmt,d,n", [("fp8_token", 128, 20011), ("bf16", 64, 20011), ("mxfp4", 64, 60001)])
def test_attention_long_sequence(fmt, d, n):
    """One key-value head: its tiles are cut into as many parts as there are
    workgroups (joined in groups, then the groups)."""
    c = Case(14, fmt, [n, 3], 8, 1, d, 64)
    c.check(c.run(return_lse=True), what="long")
    c.check(c.run(return_lse=True, window=12345), window=12345, what="long window")


@pytest.mark.parametrize("fmt,lens,hq,hk,d", [("fp8_token", [20011, 3], 40, 1, 128), ("bf16", [900, 0, 65], 1024, 1, 64),
                                              ("mxfp4", [1, 2500], 66, 2, 256), ("mxfp8", [3000] * 3, 200, 1, 128)])
def test_attention_many_query_heads_per_kv_head(fmt, lens, hq, hk, d):
    """Blocks of 16 query heads that read the same share of the cache, cut
    into parts and joined separately, the last block ragged."""
    print(f"case heads {fmt} {lens} {hq} {hk} {d}", flush=True)
    c = Case(21, fmt, lens, hq, hk, d, 32)
    got = c.run(return_lse=True)
    c.check(got, what="heads")
    c.check(c.run(return_lse=True, window=700), window=700, what="heads, window")
    again = c.run(return_lse=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_attention_batches_of_many_lengths():
    """Sequences more than lanes, workgroups that end inside a head, between
    heads and between sequences; also the head tiles of more than 16 query
    heads per key-value head, one of them ragged."""
    g = np.random.default_rng(16)
    for lens, hq, hk in ((list(g.integers(0, 400, 150)), 6, 3), (list(g.integers(0, 300, 70)), 36, 1)):
        c = Case(17, "bf16", [int(n) for n in lens], hq, hk, 64, 16)
        c.check(c.run(return_lse=True), what=f"{len(lens)} sequences")
        c.check(c.run(return_lse=True, window=100), window=100, what=f"{len(lens)} sequences, window")


@pytest.mark.parametrize("lens", [[40, 700], [5000, 300]])
def test_attention_nan_reaches_what_it_takes_part_in(lens):
    """A NaN among the values that take part: in a V element, that element of
    the heads that share it; in a K element or a query, their whole rows.
    Everything else keeps its bits."""
    c = Case(18, "bf16", lens, 4, 2, 64, 16)
    want, wl = c.run(return_lse=True)

    def poisoned(which, elem):
        buf = c.dev["cache"].clone().view(c.pages, 2, -1).view(torch.bfloat16)
        page, at = int(c.table[0, 1]), 3                       # token 19 of sequence 0, key-value head 1
        buf[page, 1, (which * 16 + at) * 64 + elem] = float("nan")
        return c.run(return_lse=True, cache=buf.view(torch.uint8).view(-1))

    out, lse = poisoned(1, 7)
    exp = want.clone()
    exp[0, 2:, 7] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(exp)) and torch.equal(out.nan_to_num(), exp.nan_to_num())
    assert torch.equal(lse, wl)
    out, lse = poisoned(0, 7)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[1], want[1])
    q = c.dev["q"].clone()
    q[1, 3] = float("nan")
    out, lse = c.run(return_lse=True, q=q)
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, :3], want[1, :3])


def test_attention_no_sequences_and_no_pages():
    c = Case(15, "bf16", [20], 4, 2, 64, 16)
    e = c.run(return_lse=True, q=c.dev["q"][:0], block_table=c.dev["block_table"][:0], seq_lens=c.dev["seq_lens"][:0])
    assert e[0].shape == (0, 4, 64) and e[1].shape == (0, 4)
    out, lse = c.run(return_lse=True, block_table=c.dev["block_table"][:, :0])
    assert not out.any() and torch.isneginf(lse).all()


def test_attention_cache_past_32_bit_offsets():
    """Pages whose bytes lie beyond 2^32 from the cache's start."""
    ps, hk, d = 256, 8, 128
    desc = hum.make_kv_desc("bf16", 5000, ps, hk, d)
    nb = hum.kv_cache_bytes(desc)
    assert nb // 5000 * 4500 > 1 << 32
    cache = torch.empty(nb, dtype=torch.uint8, device="cuda")
    x = torch.randn((300, hk, d), device="cuda").to(torch.bfloat16)
    y = torch.randn((300, hk, d), device="cuda").to(torch.bfloat16)
    t = torch.arange(300, device="cuda")
    big = torch.tensor([[4999, 4500]], dtype=torch.int32, device="cuda")
    small = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 32, d), device="cuda").to(torch.bfloat16)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    res = []
    for tab in (big, small):
        slots = tab[0].long()[t // ps] * ps + t % ps
        hum.kv_write(desc, cache, x, y, slots)
        k, v = hum.kv_read(desc, cache, slots)
        assert torch.equal(k, x) and torch.equal(v, y)
        res.append(hum.kv_attention(desc, cache, q, tab, n))
    assert torch.equal(*res)
