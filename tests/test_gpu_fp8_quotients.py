"""GPU: the FP8 codes and scales of float32 values are those of IEEE divisions,
bit for bit: scale = amax / 448, code = the nearest E4M3 value of y / scale,
ties to even.

Rows of +-1 make the norm's y its weights: their root mean square is 1 (a
power of two of them; eps vanishes beside 1)."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu
K = 65536
GRID = oracle.formats.decode_e4m3(np.arange(127, dtype=np.uint8))             # 0 .. 448
BORDERS = ((GRID[1:] + GRID[:-1]) / 2).astype(np.float32)                     # exact


def _weights(rng, exps):
    """[groups, 128] values, a maximum in each group, the others next to what the codes' borders stand for."""
    groups = K // 128
    amax = np.ldexp(1.0 + rng.integers(0, 1 << 23, groups) / 2.0 ** 23, rng.choice(exps, groups)).astype(np.float32)
    s = (amax / np.float32(448.0)).astype(np.float32)
    v = (rng.choice(BORDERS, (groups, 128)) * s[:, None]).astype(np.float32)
    bits = v.view(np.int32) + rng.integers(-3, 4, v.shape).astype(np.int32)    # a few units of the last place off
    v = np.minimum(np.maximum(bits, 0).astype(np.int32).view(np.float32), amax[:, None])
    v[:, 64] = (rng.random(groups) * amax).astype(np.float32)                  # any value, a zero, a tiny one
    v[:, 65], v[:, 66] = 0.0, amax * np.float32(2.0 ** -20)
    v[:, 7] = amax
    return v, amax


def _expected(v, amax):
    s = (amax / np.float32(448.0)).astype(np.float32)
    q = (v / s[:, None]).astype(np.float32).astype(np.float64)
    lo = np.clip(np.searchsorted(GRID, q, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    mid = (GRID[lo] + GRID[hi]) / 2
    up = (q > mid) | ((q == mid) & (lo % 2 == 1))
    return np.where(up, hi, lo).astype(np.uint8), s


@pytest.mark.parametrize("exps", [[0], list(range(-60, 60)), [-71, -70, -69, 119, 120, 121, 126], list(range(-100, -72))])
def test_codes_of_f32_values_are_those_of_divisions(exps):
    rng = np.random.default_rng(len(exps))
    for _ in range(24):
        v, amax = _weights(rng, exps)
        sign = rng.choice([-1.0, 1.0], K).astype(np.float32)
        x = torch.from_numpy(sign[None]).to(torch.bfloat16).cuda()
        w = torch.from_numpy(v.reshape(-1)).cuda()
        codes, s = _expected(v, amax)
        q, got = hum.rms_norm(x, w, eps=1e-12, act_fmt="fp8_group")
        assert np.array_equal(got.cpu().numpy()[0].view(np.int32), s.view(np.int32))
        q = q.cpu().numpy().reshape(codes.shape)
        want = codes | np.where(sign.reshape(codes.shape) < 0, 0x80, 0).astype(np.uint8)
        assert np.array_equal(q, want), np.argwhere(q != want)[:5]


@pytest.mark.parametrize("k", [128, 512, 4096])
def test_codes_of_rows_are_those_of_divisions(k):
    """A scale per row: the same rule over the whole row."""
    rng = np.random.default_rng(k)
    for _ in range(40):
        v, amax = _weights(rng, [0])
        v, amax = v[:k // 128] * (amax[0] / amax[:k // 128, None]), amax[:1]
        v = np.minimum(v, amax[0]).astype(np.float32).reshape(1, k)
        v[0, 7] = amax[0]
        codes, s = _expected(v, amax)
        q, got = hum.rms_norm(torch.ones(1, k, dtype=torch.bfloat16, device="cuda"), torch.from_numpy(v[0]).cuda(), eps=1e-12, act_fmt="fp8_token")
        assert got.cpu().numpy()[0] == s[0] and np.array_equal(q.cpu().numpy(), codes)
