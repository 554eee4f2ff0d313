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
