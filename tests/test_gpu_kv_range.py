"""GPU: the attention over the paged cache at both ends of the range of values.
The bounds are those of test_gpu_kv_precision.py."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth
from test_gpu_kv_precision import A, FMTS, _bf, _bound, _filled

pytestmark = pytest.mark.gpu


# The largest value that every format keeps as it is: 2^127 in bf16 and E2M1 x E8M0; FP8 and MXFP8 round 2^127 to
# itself too (448 x scale holds 2^127 = 256 x 2^119).
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,hq,hk,d", [([1, 16, 300], 4, 2, 64), ([5000], 8, 1, 128), ([40, 900], 2, 1, 256),
                                          ([700], 40, 1, 64)])
def test_attention_of_the_largest_values_is_finite(fmt, lens, hq, hk, d):
    """Values of 2^127 in every token: sum_t p_t v_t is 2^127, however many tokens there are and in whatever order
    their scores rise, up to the roundings of p (2^-16), of sums of n (n 2^-24, above and below) and of the output."""
    ps = 16
    g = np.random.default_rng(3)
    n = sum(lens)
    k = np.zeros((n, hk, d))
    v = np.full((n, hk, d), 2.0 ** 127)
    v[:, :, 1::2] *= -1
    # scores rise by 5 (7.2 in base 2) from each 128 tokens to the next: the reference that probabilities are formed
    # against may lag behind by up to 8
    at = np.concatenate([np.arange(m) for m in lens])
    k[:, :, 0] = np.minimum(at // 128, 30)[:, None] * 5
    c, table = _filled(fmt, lens, hk, d, ps, k, v, g)
    lens = np.array(lens, np.int32)
    desc = hum.make_kv_desc(fmt, c.buf.shape[0], ps, hk, d)
    cache, tab, ln = torch.from_numpy(c.buf.reshape(-1)).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    want = np.where(np.arange(d) % 2 == 0, 2.0 ** 127, -2.0 ** 127)
    rel = 2.0 ** -16 + 2 * int(lens.max()) * 2.0 ** -24 + 2.0 ** -8
    for q0 in (0.0, 1.0):
        q = torch.zeros((len(lens), hq, d), dtype=torch.bfloat16, device="cuda")
        q[..., 0] = q0
        out = hum.kv_attention(desc, cache, q, tab, ln, scale=1.0).double().cpu().numpy()
        assert np.isfinite(out).all(), q0
        assert (np.abs(out - want) <= rel * 2.0 ** 127).all(), q0
        # and over a window, whose tokens bound the sums instead
        out = hum.kv_attention(desc, cache, q, tab, ln, scale=1.0, window=33).double().cpu().numpy()
        assert np.isfinite(out).all() and (np.abs(out - want) <= rel * 2.0 ** 127).all(), q0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,max_pages", [(3, 1), (2000, 200), (40, 1 << 20)])
def test_attention_of_small_values_keeps_its_precision(fmt, n, max_pages):
    """Values of about 2^-60, over tables that allow up to 2^24 tokens."""
    g = np.random.default_rng(4)
    hq, hk, d, ps = 4, 2, 64, 16
    k, v = g.standard_normal((n, hk, d)), (g.standard_normal((n, hk, d)) + 0.5) * 2.0 ** -60
    c, narrow = _filled(fmt, [n], hk, d, ps, k, v, g)
    qb = synth.bf16_bits(g.standard_normal((1, hq, d)).astype(np.float32))
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, :narrow.shape[1]] = torch.from_numpy(narrow).cuda()
    desc = hum.make_kv_desc(fmt, c.buf.shape[0], ps, hk, d)
    out, lse = hum.kv_attention(desc, torch.from_numpy(c.buf.reshape(-1)).cuda(), _bf(qb), table,
                                torch.tensor([n], dtype=torch.int32, device="cuda"), return_lse=True)
    ref, rl, mag, big = A.attention(c, oracle.formats.decode_bf16(qb), narrow, np.array([n]), float(np.float32(d ** -0.5)))
    out = out.double().cpu().numpy()
    assert (np.abs(out - ref) <= _bound(ref, mag, big, d, n)).all()
    e = (d + 16) * 2.0 ** -24 * (1 + big) + 2.0 ** -20 + n * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - rl) <= e + 2.0 ** -22 * np.abs(rl)).all()
