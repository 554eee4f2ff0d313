"""GPU: the sines and cosines that a rotary turn multiplies with, to the last
bits of f32.

The pair (1, 0) turns into (cos, sin) with exact products, so an output is a
coefficient itself.  The reduced turn enters the f32 functions split into an
f32 and the rest of it, which is applied to first order: what is left is the
functions' own error (at most 4 ulp by their definition, an ulp being up to
2^-23 of the value) and half a step of the correction's sum, relative to the
VALUE also where it is small, next to a multiple of half a turn; the second
order of the rest, (2 pi 2^-26)^2 / 2 < 2^-46; and the float64 products that
form the angle, here and in the reference, each 2^-53 of it."""
import numpy as np
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_f32_coefficients(layout, inverse):
    g = np.random.default_rng(8)
    t, half = 4096, 32
    # angles up to 60 radians: every part of the turn, and its halves' neighbourhoods from 1e-1 down to 1e-6
    freq = np.concatenate([np.exp(g.uniform(np.log(1e-4), np.log(1.4e-2), half - 8)),
                           np.pi / 1000 * (1 + 10.0 ** -np.arange(1, 9))])
    pos = np.arange(t) - 10
    x = torch.zeros((t, 1, 2 * half), device="cuda")
    first = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    second = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    x[..., first] = 1.0
    y, _ = hum.rotary(x, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), layout=layout, inverse=inverse)
    y = y[:, 0].double().cpu().numpy()
    angle = pos[:, None] * freq * (-1 if inverse else 1)
    for got, ref, what in ((y[:, first], np.cos(angle), "cos"), (y[:, second], np.sin(angle), "sin")):
        tol = (4 * 2.0 ** -23 + 2.0 ** -24) * np.abs(ref) + 2.0 ** -46 + 2.0 ** -51 * np.abs(angle)
        assert (np.abs(got - ref) <= tol).all(), (what, (np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("factor", [1.0, 1.2772588])
def test_rotary_f32_is_as_exact_as_its_plain_form(layout, factor):
    """The plain form in f32, cosine and sine times the factor rounded once from float64, rounds four times to an
    output: two coefficients (their two shares of the output make up one rounding of it), two products (one), the sum.
    The kernel fuses a product with the sum: 2 1/2 roundings' variance where the plain form has 3, plus what the f32
    functions add to a correctly rounded coefficient; a factor rounded by itself would add one more.  Up to 0.8 of a
    rounding's variance is allowed to the functions: 3.3 / 3 = 1.05^2."""
    g = np.random.default_rng(10)
    t, half = 3001, 32
    factor = float(np.float32(factor))
    freq = 10000.0 ** (-np.arange(half) / half)
    pos = g.integers(0, 1 << 20, t)
    x = g.standard_normal((t, 4, 2 * half)).astype(np.float32)
    y, _ = hum.rotary(torch.from_numpy(x).cuda(), None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(),
                      layout=layout, factor=factor)
    y = y.cpu().numpy()
    angle = pos[:, None] * freq
    c, s = (np.cos(angle) * factor)[:, None], (np.sin(angle) * factor)[:, None]
    c32, s32 = c.astype(np.float32), s.astype(np.float32)
    first = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    second = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    x0, x1 = x[..., first], x[..., second]
    here = plain = 0.0
    for got, p, ref in ((y[..., first], x0 * c32 - x1 * s32, x0.astype(np.float64) * c - x1.astype(np.float64) * s),
                        (y[..., second], x0 * s32 + x1 * c32, x0.astype(np.float64) * s + x1.astype(np.float64) * c)):
        assert p.dtype == np.float32
        here += ((got - ref) ** 2).sum()
        plain += ((p - ref) ** 2).sum()
    assert here <= 3.3 / 3 * plain, (here / plain) ** 0.5
