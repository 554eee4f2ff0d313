"""GPU: routing weights are float64's, rounded once.

Bounds: a score is an exponential over a sum (or one over one and an
exponential), both in float64: the sum's terms are off by less than 2^-32 of
themselves (the polynomial in them), all else by a few 2^-53.  The weight's one rounding
to float32 adds half a step: 2^-24 of the value, below 2^-126 half of the
subnormals' 2^-149.  Together less than (2^-24 + 2^-30) of the weight, 2^-150."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu
L = oracle.layer


def _check(x, topk, **kw):
    bias = kw.get("bias")
    ids, w = hum.moe_route(x, topk, **kw)
    ri, rw = L.route(x.double().cpu().numpy(), topk, **dict(kw, bias=None if bias is None else bias.double().cpu().numpy()))
    assert (ids.cpu().numpy() == ri).all()
    d = np.abs(w.double().cpu().numpy() - rw)
    tol = np.abs(rw) * (2.0 ** -24 + 2.0 ** -30) + 2.0 ** -150
    assert (d <= tol).all(), (d / tol).max()


def _rows(e, seed):
    """Scores spread, near one another, ruled by one or two, far apart, at the ends of float32's range."""
    g = torch.Generator().manual_seed(seed)
    n = lambda t: torch.randn(t, e, generator=g)  # noqa: E731
    two = n(30) - 5
    two[:, 0], two[:, e // 2] = 3.0, 3.0 - torch.rand(30, generator=g)
    rows = [n(150) * 1.5, n(60) * 0.01 + 40, n(30) * 8, two, n(20) * 60 - 300, torch.linspace(-1, 1, e).expand(2, e) * 3e38,
            torch.zeros(1, e), torch.full((1, e), -3e38), torch.full((1, e), -float("inf"))]
    x = torch.cat(rows)
    x[5:9, ::3] = -float("inf")
    x[9, 1:] = -float("inf")
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm,scale", [(False, 1.0), (False, 2.5), (True, 1.0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k", [(1, 1), (8, 2), (60, 4), (64, 14), (129, 8), (256, 8), (300, 8), (512, 10), (128, 16)])
def test_weights_are_rounded_once(e, k, score, renorm, scale, dtype):
    x = _rows(e, e).to(dtype).cuda()
    if score == "sigmoid" and renorm:           # (rows of scores below float64's range have no quotient)
        x = x[(x.max(1)[0] > -600).cpu() | (x == -float("inf")).all(1).cpu()]
    bias = (torch.randn(e, generator=torch.Generator().manual_seed(k)) * 0.05).cuda()
    for kw in ({}, dict(bias=bias)):
        _check(x, k, score=score, renormalize=renorm, scale=scale, **kw)


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,k", [(64, 8, 3, 6), (72, 8, 3, 6), (160, 8, 3, 6), (256, 8, 4, 8), (512, 32, 8, 8)])
def test_weights_of_groups_are_rounded_once(e, groups, kept, k, score, gs):
    x = _rows(e, e + 1)[:300].cuda()
    for kw in ({}, dict(bias=(torch.randn(e, generator=torch.Generator().manual_seed(3)) * 0.05).cuda())):
        _check(x, k, score=score, renormalize=False, num_groups=groups, topk_groups=kept, group_score=gs, **kw)
