"""GPU: the attention's log-sum-exp where nothing but its own arithmetic is in
it: one token, whose score is the query's first element s, |s| <= 1.

s log2(e) is off by 2^-23 of it (the constant and the product, each rounded to
f32); the exponential of (at most) 0, the logarithm and their sum by an ulp of
values up to 2, at most 2^-23 each; the product with ln 2 (and the constant)
by 2^-23 of the result: 5 x 2^-23 in all, however many tokens the table allows."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8_token", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("max_pages", [1, 40, 1 << 20])
def test_lse_of_one_token(fmt, max_pages):
    b, hq, d = 256, 4, 64
    desc = hum.make_kv_desc(fmt, 1, 16, 1, d)
    k = torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = 1.0
    cache = torch.zeros(hum.kv_cache_bytes(desc), dtype=torch.uint8, device="cuda")
    hum.kv_write(desc, cache, k, k, torch.zeros(1, dtype=torch.int64, device="cuda"))
    k0 = float(hum.kv_read(desc, cache, torch.zeros(1, dtype=torch.int64, device="cuda"))[0][0, 0, 0])
    qb = synth.bf16_bits(np.random.default_rng(9).uniform(-1, 1, (b, hq, d)).astype(np.float32))
    table = torch.zeros((1, max_pages), dtype=torch.int32, device="cuda").expand(b, max_pages)
    _, lse = hum.kv_attention(desc, cache, torch.from_numpy(qb.view(np.int16)).cuda().view(torch.bfloat16), table,
                              torch.ones(b, dtype=torch.int32, device="cuda"), scale=1.0, return_lse=True)
    ref = oracle.formats.decode_bf16(qb)[..., 0] * k0
    assert k0 == 1.0
    assert (np.abs(lse.double().cpu().numpy() - ref) <= 5 * 2.0 ** -23).all()
