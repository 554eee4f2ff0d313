"""GPU: ids of -1 have weight 0 in rows that hold a NaN too."""
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [4, 15])
def test_nothing_left_beside_a_nan(k, score, renorm):
    x = torch.full((3, 64), -float("inf"), device="cuda")
    x[0, 5] = x[1, 6] = float("nan")
    x[1, 2] = 1.0
    for bias in (None, torch.zeros(64, device="cuda")):
        ids, w = hum.moe_route(x, k, score=score, bias=bias, renormalize=renorm, scale=2.5)
        assert ids[0].tolist() == [5] + [-1] * (k - 1) and ids[1].tolist() == [6, 2] + [-1] * (k - 2)
        assert torch.isnan(w[0, 0]) and torch.isnan(w[1, 0]) and torch.isnan(w[1, 1]) == (renorm or score == "softmax")
        assert (w[ids < 0] == 0).all()
