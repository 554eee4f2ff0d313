"""Pins of the attention oracle against something other than itself: complex
multiplication, invariants of the turn, brute-force sums, and joins of parts."""
import numpy as np
import pytest

import oracle
import synth

A = oracle.attention


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_is_complex_multiplication(layout):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 3, 12))
    f = np.array([1.0, 0.3, 0.01])
    pos = np.array([0, 1, 7, 1000, 123456])
    y = A.rotary(x, pos, f, layout, factor=1.25)
    i0, i1 = (np.arange(3), np.arange(3) + 3) if layout == "half" else (np.arange(0, 6, 2), np.arange(1, 6, 2))
    z = (x[..., i0] + 1j * x[..., i1]) * 1.25 * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., i0], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., i1], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    back = A.rotary(y, pos, f, layout, factor=1 / 1.25, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_rotary_inverse_is_the_gradient():
    """d/dx <w, rotary(x)> = rotary(w, inverse), against differences."""
    g = np.random.default_rng(2)
    x, w = g.standard_normal((2, 1, 8)), g.standard_normal((2, 1, 8))
    f, pos = np.array([0.7, 0.2]), np.array([3, 11])
    got = A.rotary(w, pos, f, "half", 1.5, inverse=True)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        diff = ((A.rotary(x + e, pos, f, "half", 1.5) - A.rotary(x - e, pos, f, "half", 1.5)) * w).sum() / 2e-6
        assert abs(diff - got[i]) < 1e-8


def test_rotary_scores_depend_on_the_distance():
    g = np.random.default_rng(3)
    q, k = g.standard_normal((2, 1, 1, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    a = (A.rotary(q, [5], f) * A.rotary(k, [2], f)).sum()
    b = (A.rotary(q, [1005], f) * A.rotary(k, [1002], f)).sum()
    assert abs(a - b) < 1e-9


@pytest.mark.parametrize("fmt,step", [("bf16", 0.0), ("fp8_token", 2.0 ** -4), ("mxfp8", 2.0 ** -3), ("mxfp4", 0.25)])
def test_cache_rows_are_near_what_was_written(fmt, step):
    g = synth.rng(4)
    c = A.Cache(fmt, 3, 16, 2, 64)
    k, v = synth.bf16_normal(g, (5, 2, 64)), synth.bf16_normal(g, (5, 2, 64))
    slots = np.array([0, 47, -1, 17, 48])               # the third and the last are outside
    c.write(slots, k, v)
    for which, bits in ((0, k), (1, v)):
        x = oracle.formats.decode_bf16(bits)
        y = c.rows(slots, which)
        assert not y[2].any() and not y[4].any()
        for i in (0, 1, 3):
            top = np.abs(x[i]).max(-1, keepdims=True)
            # half a step of the element (of a block's elements near zero: far less than half a step of top / 4);
            # the MX rule clips what it scales into [448, 512) or (6, 8): up to 1/8 or 1/4 of the element
            assert (np.abs(y[i] - x[i]) <= step * np.maximum(np.abs(x[i]), top / 4)).all()
    assert not c.buf[0, :, c.row:c.ps * c.row].any()    # no other K row of page 0 was touched


def test_attention_against_brute_force_and_joined_parts():
    g = synth.rng(5)
    c = A.Cache("bf16", 8, 16, 2, 64)
    k, v = synth.bf16_normal(g, (128, 2, 64)), synth.bf16_normal(g, (128, 2, 64))
    c.write(np.arange(128), k, v)
    q = g.standard_normal((3, 4, 64))
    table = np.array([[3, 1, 5], [0, -1, 2], [7, 6, 4]], np.int32)
    lens = np.array([40, 48, 0], np.int32)
    out, lse, _, _ = A.attention(c, q, table, lens, 0.125)
    assert not out[2].any() and np.isneginf(lse[2]).all()
    kf, vf = oracle.formats.decode_bf16(k), oracle.formats.decode_bf16(v)
    order = [list(range(48, 64)) + list(range(16, 32)) + list(range(80, 88)),
             list(range(0, 16)) + list(range(32, 48))]
    for b in (0, 1):
        for h in range(4):
            e = [np.exp(0.125 * sum(q[b, h, d] * kf[t, h // 2, d] for d in range(64))) for t in order[b]]
            want = sum(w * vf[t, h // 2] for w, t in zip(e, order[b])) / sum(e)
            np.testing.assert_allclose(out[b, h], want, atol=1e-12)
            assert abs(lse[b, h] - np.log(sum(e))) < 1e-12
    # a window and what lies before it join to the whole
    wo, wl, _, _ = A.attention(c, q[:1], table[:1], lens[:1], 0.125, window=13)
    po, pl, _, _ = A.attention(c, q[:1], table[:1], lens[:1] - 13, 0.125)
    tot = np.logaddexp(wl, pl)
    np.testing.assert_allclose(wo * np.exp(wl - tot)[..., None] + po * np.exp(pl - tot)[..., None], out[:1], atol=1e-12)
