"""GPU: the rotated append where a wave moves several rows one after another
(prompts): the same bits as the same tokens in small calls, whose waves have
one row of each lane, and those against the float64 oracle.

A call slices a token's rows (q's heads, k's, v's; 64 / (head_dim / 8) of them
side by side) over waves until there are 512 workgroups of four: from 2045
tokens on a wave has all rows of its token, with a few hundred it has some of
them, below that one each."""
import pytest
import torch

import quantized_gemm_packed_amd as hum
from test_gpu_rotary_kv_write import FMTS, Case

pytestmark = pytest.mark.gpu

# t, q heads, kv heads, head size: rows that are no multiple of what lies side by side (13 of 4, 9 of 2, 22 of 8),
# and a call between the two ends (80 rows of 4 in 7 slices)
SHAPES = [(2051, 7, 3, 128), (2051, 5, 2, 256), (2050, 16, 3, 64), (300, 64, 8, 128)]
SMALL = 23


def _in_small_calls(c, cache, **kw):
    q, k, v = c.split()
    out = []
    for i in range(0, c.t, SMALL):
        at = slice(i, i + SMALL)
        out.append(hum.rotary_kv_write(c.desc, cache, q[at] if c.hq else None, k[at], v[at], c.pos[at], c.freq, c.slots[at],
                                       layout=c.layout, **kw))
    return torch.cat(out) if c.hq else None


def _unaligned(x, off, pad):
    b = torch.full((x.shape[0] * x.shape[1] * (x.shape[2] + pad) + off,), 3.0, dtype=x.dtype, device="cuda")
    y = b[off:].view(x.shape[0], x.shape[1], x.shape[2] + pad)[..., :x.shape[2]]
    y.copy_(x)
    return b, y


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts_get_the_bits_of_small_calls(shape, fmt, layout):
    t, hq, hk, d = shape
    for r in (d, d // 2, 20):
        c = Case(t + d + r, fmt, t, hq, hk, d, r, 64, layout)
        for norms in ({}, dict(q_norm=c.w[0], k_norm=c.w[1])):
            few = c.cache()
            want = _in_small_calls(c, few, **norms)
            cache = c.cache()
            q = c.run(cache, **norms)
            assert torch.equal(q, want) and torch.equal(cache, few), (r, "aligned")
            # rows at odd places and strides
            parts = [_unaligned(x, 1, 3)[1] for x in c.split()]
            buf, out = _unaligned(torch.zeros_like(want), 1, 5)
            cache = c.cache()
            got = c.run(cache, qkv=parts, q_out=out, **norms)
            assert got is out and torch.equal(out, want) and torch.equal(cache, few), (r, "unaligned")
            out.fill_(3.0)
            assert (buf[1:] == 3).all() and buf[0] == 3
            # in q's own place, aligned and not
            cache = c.cache()
            assert c.run(cache, qkv=parts, q_out=parts[0], **norms) is parts[0]
            assert torch.equal(parts[0], want) and torch.equal(cache, few), (r, "in place, unaligned")
            mine, cache = c.qkv.clone(), c.cache()
            own = mine.split([hq, hk, hk], 1)
            c.run(cache, qkv=own, q_out=own[0], **norms)
            assert torch.equal(own[0], want) and torch.equal(cache, few), (r, "in place")
            assert torch.equal(mine[:, hq:], c.qkv[:, hq:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", FMTS)
def test_prompts_without_queries(fmt, layout):
    c = Case(5, fmt, 2049, 0, 5, 128, 96, 16, layout)
    cache, few = c.cache(), c.cache()
    assert c.run(cache, k_norm=c.w[1]) is None
    _in_small_calls(c, few, k_norm=c.w[1])
    assert torch.equal(cache, few)


@pytest.mark.parametrize("fmt,layout,norm", [("bf16", "interleaved", True), ("fp8_token", "half", True), ("mxfp8", "half", False),
                                             ("mxfp4", "interleaved", False)])
def test_prompts_against_the_oracle(fmt, layout, norm):
    for t, hq, hk, d, r in ((2051, 7, 3, 128, 128), (300, 64, 8, 128, 64), (2047, 3, 1, 256, 24)):
        c = Case(t, fmt, t, hq, hk, d, r, 32, layout)
        cache = c.cache()
        norms = dict(q_norm=c.w[0], k_norm=c.w[1]) if norm else {}
        c.check(c.run(cache, **norms), cache, **norms)
