"""GPU: rotary in place, q and k as slices of one buffer, on every access width
and layout; what the call is not given stays as it was."""
import numpy as np
import pytest
import torch

import quantized_gemm_packed_amd as hum
from test_gpu_rotary import _check

pytestmark = pytest.mark.gpu


def _fused(t, hq, hk, d, dtype, odd, by_head, seed):
    """q, k and v of one product with neighbours on every side, `odd` elements off 16-byte alignment: (buffer, q, k)."""
    heads = hq + 2 * hk + 2
    buf = torch.randn(t * heads * d + 8, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    x = buf[odd:odd + t * heads * d]
    x = x.view(heads, t, d).transpose(0, 1) if by_head else x.view(t, heads, d)
    return buf, x[:, 1:1 + hq], x[:, 1 + hq:1 + hq + hk]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("odd", [0, 1, 2, 4])
@pytest.mark.parametrize("t,hq,hk,d,r", [(5, 4, 2, 128, 128), (33, 8, 1, 128, 64), (300, 3, 3, 80, 40), (2, 1, 1, 64, 6)])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("which", ["both", "q", "k"])
def test_rotary_in_place(dtype, layout, odd, t, hq, hk, d, r, by_head, which):
    buf, q, k = _fused(t, hq, hk, d, dtype, odd, by_head, t + d)
    before, q0, k0 = buf.clone(), q.clone(), k.clone()
    pos = torch.arange(t) * 1234 - 777
    f, a = hum.rotary_inv_freq(r, scaling="yarn", factor=4.0, original_len=4096)
    yq, yk = hum.rotary(q, k, pos.cuda(), f.cuda(), layout=layout, factor=a, q_out=q if which != "k" else None,
                        k_out=k if which != "q" else None)
    for y, x, own in ((yq, q0, which != "k"), (yk, k0, which != "q")):
        _check(y, x, pos.numpy(), f.numpy(), layout, np.float32(a), False, which)
    # the same bits as out of place
    wq, wk = hum.rotary(q0, k0, pos.cuda(), f.cuda(), layout=layout, factor=a)
    assert torch.equal(yq, wq) and torch.equal(yk, wk)
    # everything but what was turned in place
    if which != "k":
        q.copy_(q0)
    if which != "q":
        k.copy_(k0)
    assert torch.equal(buf, before)
