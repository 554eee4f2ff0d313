"""GPU: routing of rows that hold a NaN beside infinities or beside experts
that take no part."""
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu


def _row(e, at):
    x = torch.zeros(3, e, device="cuda")
    for i, v in at.items():
        x[1, i] = v
    return x


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [16, 256])
def test_a_nan_comes_before_infinity(e, score):
    inf, nan = float("inf"), float("nan")
    x = _row(e, {3: inf, 4: inf, 9: nan, 10: -nan})
    for bias in (None, torch.linspace(0.5, -0.5, e).cuda()):
        for k in (1, 2, 4, 15):
            ids, w = hum.moe_route(x, k, score=score, bias=bias, renormalize=False)
            ids = ids[1].tolist()
            assert ids[:2] == [9, 10][:k] and torch.isnan(w[1, :2]).all()
            if k > 3 and not (bias is not None and score == "sigmoid"):   # (sigmoids of infinity are 1, a bias may pass them)
                assert ids[2:4] == [3, 4]
            assert len(set(ids)) == k


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(32, 4), (36, 4), (256, 32)])
def test_a_group_with_a_nan_comes_before_those_with_infinities(e, groups, score, gs):
    inf, nan, n = float("inf"), float("nan"), e // groups
    x = _row(e, {0: inf, 1: inf, 2 * n + 3: nan, 3 * n: inf, 3 * n + 1: 5.0})
    for bias in (None, torch.zeros(e, device="cuda")):
        kw = dict(score=score, bias=bias, num_groups=groups, group_score=gs)
        ids, w = hum.moe_route(x, 1, topk_groups=1, **kw)
        assert ids[1, 0] == 2 * n + 3 and torch.isnan(w[1, 0])
        ids, w = hum.moe_route(x, 2, topk_groups=2, **kw)
        assert ids[1].tolist() == [2 * n + 3, 0]
