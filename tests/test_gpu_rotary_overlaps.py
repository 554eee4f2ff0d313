"""GPU: rotary's outputs inside what it still reads are refused by the binding
too, and nothing is written then; neighbours that only interleave are not."""
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu


def test_shifted_views_are_refused_and_leave_their_buffer():
    buf = torch.randn((12, 6, 64), device="cuda").to(torch.bfloat16)
    before = buf.clone()
    f = hum.rotary_inv_freq(64)[0].cuda()
    pos = torch.arange(11, device="cuda")
    q, k = buf[:11, :4], buf[:11, 4:]
    flat = buf.view(-1)
    for kw in (dict(q_out=buf[1:, :4]), dict(q_out=buf[:11, 1:5]), dict(k_out=buf[:11, 3:5]), dict(k_out=buf[1:, 4:]),
               dict(q_out=flat[:11 * 4 * 64].view(11, 4, 64)), dict(q_out=flat[32:32 + 11 * 6 * 64].view(11, 6, 64)[:, :4]),
               dict(q_out=torch.empty(11 * 256, dtype=torch.bfloat16, device="cuda").as_strided((11, 4, 64), (64, 64, 1)))):
        with pytest.raises(hum.HumError, match="overlap|in place"):
            hum.rotary(q, k, pos, f, **kw)
    torch.cuda.synchronize()
    assert torch.equal(buf, before)


def test_outputs_that_interleave_with_inputs_are_taken():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((7, 12, 64), generator=g).cuda()
    f = hum.rotary_inv_freq(64)[0].cuda()
    pos = torch.arange(7, device="cuda") * 99
    q, k = x[:, 0:8:2], x[:, 8:10]
    wq, wk = hum.rotary(q, k, pos, f)
    yq, yk = hum.rotary(q, k, pos, f, q_out=x[:, 1:8:2], k_out=x[:, 10:])
    assert torch.equal(yq, wq) and torch.equal(yk, wk)
    assert torch.equal(x[:, 1:8:2], wq) and torch.equal(x[:, 10:], wk)
