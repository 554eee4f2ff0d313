"""GPU: a rotary turn's bits go by its values alone, not by where they lie or
how wide the accesses are."""
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (80, 48)])
def test_rotary_bits_at_every_alignment(dtype, layout, d, r):
    t, hq, hk = 2000, 3, 2
    g = torch.Generator().manual_seed(d + r)
    x = torch.randn((t, hq + hk, d), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 20, (t,), generator=g).cuda()
    f, a = hum.rotary_inv_freq(r, scaling="yarn", factor=4.0, original_len=4096)
    f = f.cuda()
    want = hum.rotary(x[:, :hq], x[:, hq:], pos, f, layout=layout, factor=a)
    for odd in (1, 2, 4):
        buf = torch.empty(x.numel() + 8, dtype=dtype, device="cuda")
        y = buf[odd:odd + x.numel()].view(x.shape)
        y.copy_(x)
        for kw in ({}, dict(q_out=y[:, :hq], k_out=y[:, hq:])):
            got = hum.rotary(y[:, :hq], y[:, hq:], pos, f, layout=layout, factor=a, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (odd, bool(kw))
    # a token by itself, and the tokens in another order
    one = hum.rotary(x[777:778, :hq], x[777:778, hq:], pos[777:778], f, layout=layout, factor=a)
    assert torch.equal(one[0][0], want[0][777]) and torch.equal(one[1][0], want[1][777])
