"""How exact the attention over the paged cache is, where that can be told
apart from its output's rounding.

Arithmetic.  A probability enters the second product as the sum of two bf16:
its rounding (off by at most 2^-8 of it) and the rounding of what that left
(2^-8 of that), 2^-16 of it in all.  Everything else is f32 and counted as in
the other attention tests: scores, exponentials and sums over n tokens are off
by d = (D + 16) 2^-24 (1 + B) + 2^-20 + n 2^-24 relative, above and below the
division; B = max_t scale sum |q k|.  The result is rounded to bf16 once.  So
  |out - ref| <= (2^-16 + 2 d) m + 2^-8 (|ref| + (2^-16 + 2 d) m),
m = sum_t p_t |v_t|.  Where V's signs cancel, |ref| is far below m, and the
first term is what counts."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth

A = oracle.attention
FMTS = ["bf16", "fp8_token", "mxfp8", "mxfp4"]


def _bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _filled(fmt, lens, hk, d, ps, k, v, order):
    """A cache that holds k, v [sum(lens), hk, d] on scattered pages, and its block table."""
    need = [-(-n // ps) for n in lens]
    c = A.Cache(fmt, sum(need) + 1, ps, hk, d, fill=0xFF)
    ids = order.permutation(sum(need) + 1)
    table = np.full((len(lens), max(need)), -1, np.int32)
    at = row = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        t = np.arange(n)
        c.write(table[b][t // ps].astype(np.int64) * ps + t % ps, synth.bf16_bits(k[row:row + n].astype(np.float32)),
                synth.bf16_bits(v[row:row + n].astype(np.float32)))
        row += n
    return c, table


def _cancelling(fmt, lens, hq, hk, d, ps, seed):
    """Tokens in pairs: keys that differ in one element, which the queries hardly see (scores within about 2^-7 of one
    another), and opposite values."""
    g = np.random.default_rng(seed)
    n = sum(lens)
    k = g.standard_normal((n // 2, hk, d)).repeat(2, 0)
    k[:, :, 0] = g.standard_normal((n, hk)) * 2
    v = (g.standard_normal((n // 2, hk, d)) + 0.3).repeat(2, 0)
    v[1::2] *= -1
    q = g.standard_normal((len(lens), hq, d)) * 0.5
    q[..., 0] = 0.05
    qb = synth.bf16_bits(q.astype(np.float32))
    return _filled(fmt, lens, hk, d, ps, k, v, g) + (qb,)


def _bound(ref, mag, big, d, n):
    e = 2.0 ** -16 + 2 * ((d + 16) * 2.0 ** -24 * (1 + big) + 2.0 ** -20 + n * 2.0 ** -24)[..., None]
    return e * mag + 2.0 ** -8 * (np.abs(ref) + e * mag)


CASES = [([2, 30, 64, 128, 34], 4, 2, 64, 16), ([130, 62], 16, 1, 128, 32), ([96, 200], 6, 2, 256, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,hq,hk,d,ps", CASES)
def test_oracle_with_probabilities_of_one_bf16_is_outside_the_bound(fmt, lens, hq, hk, d, ps):
    """The bound below tells the two apart: with the mistake planted in the oracle it is exceeded."""
    c, table, qb = _cancelling(fmt, lens, hq, hk, d, ps, sum(lens) + d)
    q = oracle.formats.decode_bf16(qb)
    lens = np.array(lens, np.int32)
    scale = float(np.float32(d ** -0.5))
    ref, _, mag, big = A.attention(c, q, table, lens, scale)
    tol = _bound(ref, mag, big, d, lens.max())
    worst = 0.0
    for b, n in enumerate(lens):
        t = np.arange(n)
        slots = table[b][t // ps].astype(np.int64) * ps + t % ps
        k, v = c.rows(slots, 0), c.rows(slots, 1)
        for h in range(hq):
            s = scale * (k[:, h // (hq // hk)] @ q[b, h])
            p = np.exp(s - s.max())
            one = oracle.formats.decode_bf16(synth.bf16_bits(p.astype(np.float32)))
            out = one @ v[:, h // (hq // hk)] / p.sum()
            worst = max(worst, (np.abs(out - ref[b, h]) / np.maximum(tol[b, h], 1e-30)).max())
    assert worst > 1.5, worst


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,hq,hk,d,ps", CASES)
def test_attention_keeps_sixteen_bits_of_a_probability(fmt, lens, hq, hk, d, ps):
    c, table, qb = _cancelling(fmt, lens, hq, hk, d, ps, sum(lens) + d)
    lens = np.array(lens, np.int32)
    desc = hum.make_kv_desc(fmt, c.buf.shape[0], ps, hk, d)
    out = hum.kv_attention(desc, torch.from_numpy(c.buf.reshape(-1)).cuda(), _bf(qb), torch.from_numpy(table).cuda(),
                           torch.from_numpy(lens).cuda()).double().cpu().numpy()
    ref, _, mag, big = A.attention(c, oracle.formats.decode_bf16(qb), table, lens, float(np.float32(d ** -0.5)))
    tol = _bound(ref, mag, big, d, lens.max())
    assert (np.abs(out - ref) <= tol).all(), (np.abs(out - ref) / np.maximum(tol, 1e-30)).max()
