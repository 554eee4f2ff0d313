"""CPU: rotary calls whose outputs overlap what other workgroups still read are
refused before any launch.  The addresses are never touched: every call here
ends in a refusal."""
import ctypes

import pytest

import quantized_gemm_packed_amd as hum

P = ctypes.c_void_p
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    return hum.load_library()


def _call(lib, q, k, qo, ko, t=4, hq=4, hk=2, d=64, dtype=None, r=64):
    """q, k, qo, ko: (address, token stride, head stride) in elements."""
    desc = hum.RotaryDesc(hum.BF16 if dtype is None else dtype, 0, d, r, hq, hk, 0, 1.0)
    a = lambda x: (P(x[0]), x[1], x[2])  # noqa: E731
    return lib.hum_rotary(ctypes.addressof(desc), t, P(8), P(8), *a(q), *a(qo), *a(k), *a(ko), None)


F = 8 * 64                       # a fused row: 4 query, 2 key and 2 value heads of 64
Q, K, V = (1 << 20, F, 64), ((1 << 20) + 4 * 128, F, 64), ((1 << 20) + 6 * 128, F, 64)
ELSE_Q, ELSE_K = (1 << 24, 256, 64), (1 << 25, 128, 64)


@pytest.mark.parametrize("what,qo,ko", [
    ("q shifted by one element", (Q[0] + 2, F, 64), ELSE_K), ("q shifted by a row", (Q[0] + F * 2, F, 64), ELSE_K),
    ("q shifted back by a head", (Q[0] - 128, F, 64), ELSE_K), ("the last of q in k", ((1 << 20) + 128, F, 64), ELSE_K),
    ("q packed where it was strided", (Q[0] + 128, 256, 64), ELSE_K),
    ("k where q is", ELSE_Q, ((1 << 20) + 3 * 128, F, 64)), ("k shifted in place", ELSE_Q, (K[0] + 64, F, 64)),
    ("outputs in one another", ELSE_Q, (ELSE_Q[0] + 2 * 128, 256, 64)), ("outputs' last rows", ELSE_Q, (ELSE_Q[0] + 3 * 512 + 384, 512, 64)),
    ("rows of an output", (1 << 24, 255, 64), ELSE_K), ("heads of an output", (1 << 24, 256, 63), ELSE_K),
    ("one row for all tokens", (1 << 24, 0, 64), ELSE_K), ("tokens backwards into q", (ELSE_Q[0], -(ELSE_Q[0] - Q[0]) // 2 // 3, 64), ELSE_K)])
def test_overlaps_refused(lib, what, qo, ko):
    assert _call(lib, Q, K, qo, ko) == INVALID, what
    assert lib.hum_last_error()


def test_overlap_of_the_largest_calls_refused(lib):
    assert _call(lib, Q, K, (Q[0] + 2 * F * ((1 << 24) - 2), F, 64), ELSE_K, t=(1 << 24) - 1) == INVALID
    # strides whose products pass 64 bits
    assert _call(lib, (1 << 20, 1 << 62, 1 << 61), (1 << 21, 1 << 62, 1 << 61), (1 << 20, 1 << 62, 1 << 60), (1 << 21, 1 << 62, 1 << 61)) == INVALID
