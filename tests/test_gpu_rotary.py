"""GPU: rotary positions against the float64 oracle.

Tolerance: the angle reaches the f32 sine within 2^-24 of a turn's remainder,
so cos and sin carry at most 2 pi 2^-25 + 2 ulp, under 2^-21 in all, and
y = x0 c - x1 s adds three f32 roundings: 2^-20 a (|x0| + |x1|), then half a
step of the output type."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _check(y, x, pos, f, layout, factor, inverse, what):
    x64 = x.double().cpu().numpy()
    ref = oracle.attention.rotary(x64, pos, f, layout, factor, inverse)
    pair = np.abs(oracle.attention.rotary(np.abs(x64), np.zeros(len(pos)), f, layout, 1.0))
    r = 2 * len(f)
    i0 = np.arange(r // 2) if layout == "half" else np.arange(0, r, 2)
    i1 = i0 + (r // 2 if layout == "half" else 1)
    both = pair[..., i0] + pair[..., i1]
    tol = np.zeros_like(ref)
    tol[..., i0] = tol[..., i1] = 2.0 ** -20 * abs(factor) * both
    tol += HALF_STEP[x.dtype] * (np.abs(ref) + tol)
    got = y.double().cpu().numpy()
    assert np.array_equal(got[..., r:], x64[..., r:]), what
    assert (np.abs(got - ref) <= tol)[..., :r].all(), (what, np.abs(got - ref).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("t,hq,hk,d,r", [(1, 1, 1, 128, 128), (7, 32, 8, 128, 64), (300, 5, 1, 80, 40),
                                         (33, 3, 2, 64, 6), (2, 4, 4, 2, 2), (70, 4, 1, 80, 20), (70, 4, 1, 72, 24), (1500, 2, 1, 96, 96), (5, 2, 1, 1024, 1022),
                                         (3, 1, 1, 1023, 2)])
def test_rotary(dtype, layout, t, hq, hk, d, r):
    print(f"case rotary {dtype} {layout} {t} {hq} {hk} {d} {r}", flush=True)
    g = torch.Generator().manual_seed(t * d + r)
    qkv = torch.randn((t, hq + 2 * hk, d), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 20, (t,), generator=g)
    pos[0] = (1 << 20) - 1
    f, a = hum.rotary_inv_freq(r, scaling="yarn", factor=16.0, original_len=8192)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    yq, yk = hum.rotary(q, k, pos.cuda(), f.cuda(), layout=layout, factor=a)
    for y, x, n in ((yq, q, "q"), (yk, k, "k")):
        _check(y, x, pos.numpy(), f.numpy(), layout, np.float32(a), False, n)
    zq, _ = hum.rotary(yq, None, pos.cuda(), f.cuda(), layout=layout, factor=0.5, inverse=True)
    _check(zq, yq, pos.numpy(), f.numpy(), layout, 0.5, True, "inverse")


def test_rotary_in_place_odd_alignment_and_neighbours_untouched():
    """Rows two bytes off 16-byte alignment, turned in place inside a larger
    buffer whose other values stay as they were."""
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(9 * 300 + 1, generator=g).to(torch.bfloat16).cuda()
    before = buf.clone()
    x = buf[1:].view(9, 300)[:, 20:20 + 4 * 64].unflatten(1, (4, 64))
    ref_in = x.clone()
    pos = torch.arange(9, device="cuda") * 1000 - 4000     # negative positions turn back
    f, _ = hum.rotary_inv_freq(32)
    k = torch.zeros((9, 0, 64), dtype=torch.bfloat16, device="cuda")
    yq, _ = hum.rotary(x, k, pos, f.cuda(), q_out=x, k_out=k)
    _check(x, ref_in, pos.cpu().numpy(), f.numpy(), "half", 1.0, False, "in place")
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[1:].view(9, 300)[:, 20:20 + 4 * 64] = False
    assert torch.equal(buf[mask], before[mask]) and yq.data_ptr() == x.data_ptr()


def test_rotary_empty_and_many_tokens():
    f, _ = hum.rotary_inv_freq(64)
    e = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    q, k = hum.rotary(e, e, torch.zeros(0, dtype=torch.int64, device="cuda"), f.cuda())
    assert q.shape == (0, 4, 64)
    x = torch.randn((70001, 1, 64), device="cuda")
    pos = torch.arange(70001, device="cuda")
    y, _ = hum.rotary(x, None, pos, f.cuda())
    _check(y, x, pos.cpu().numpy(), f.numpy(), "half", 1.0, False, "many")


def test_rotary_gradient_against_differences():
    """<w, rotary(x)> changes along v as <rotary(w, inverse), v> says: linear
    in x, so one difference of step 1 is exact up to rounding."""
    g = torch.Generator().manual_seed(5)
    x, v, w = (torch.randn((17, 3, 64), generator=g).cuda() for _ in range(3))
    pos = torch.arange(17, device="cuda") * 777
    f, a = hum.rotary_inv_freq(48, scaling="yarn", factor=4.0, original_len=4096)
    f = f.cuda()
    diff = ((hum.rotary(x + v, None, pos, f, factor=a)[0] - hum.rotary(x, None, pos, f, factor=a)[0]).double()
            * w.double()).sum()
    grad = hum.rotary(w, None, pos, f, factor=a, inverse=True)[0].double()
    # every term's f32 roundings: about 2^-20 of |w| |x|, 17 * 3 * 64 terms
    tol = 2.0 ** -19 * float((w.abs().double() * (x.abs() + v.abs()).double()).sum()) * 2
    assert abs(float(diff - (grad * v.double()).sum())) <= tol
