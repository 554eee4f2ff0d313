"""GPU: values of the norm that are not finite though their rows are (a NaN or
infinity among the weights, products past float32's range) show in the scales:
of the row, the group or the block that holds them, and only there."""
import pytest
import torch

import quantized_gemm_packed_amd as hum

pytestmark = pytest.mark.gpu
FMTS = {"fp8_token": None, "fp8_group": 128, "mxfp8": 32, "mxfp4": 32}


def _not_a_number(s, fmt):
    return s == 255 if fmt.startswith("mx") else torch.isnan(s)


@pytest.mark.parametrize("what", ["nan", "inf", "inf times zero", "overflow"])
@pytest.mark.parametrize("wdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [256, 1024, 5120, 17408])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_not_finite_y(fmt, k, wdt, what):
    g = torch.Generator().manual_seed(k)
    x = torch.randn(5, k, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(k, generator=g)).to(wdt).cuda()
    at = k // 2 + 45
    x[:, at] = 0.0 if what == "inf times zero" else 2.0
    x[:, at + 1] = -3.0
    bad = w.clone()
    bad[at] = float("nan") if what == "nan" else 3e38 if what == "overflow" else float("inf")
    if what == "overflow":
        bad[at + 1] = 3e38
    for kw in ({}, dict(residual=x, residual_out=torch.empty_like(x))):
        run = lambda w: hum.rms_norm(x, w, act_fmt=fmt, with_bf16=True, **kw)  # noqa: E731
        (q, s, y), (q0, s0, y0) = (r[0] if kw else r for r in (run(bad), run(w)))
        assert not torch.isfinite(y[:, at]).any() and torch.isfinite(y0).all() and not _not_a_number(s0, fmt).any()
        n = FMTS[fmt] or k
        s, s0 = s.view(5, k // n), s0.view(5, k // n)
        q, q0 = q.view(5, k // n, -1), q0.view(5, k // n, -1)
        rest = torch.arange(k // n, device="cuda") != at // n
        assert _not_a_number(s[:, at // n], fmt).all()
        assert torch.equal(s[:, rest], s0[:, rest]) and torch.equal(q[:, rest], q0[:, rest])


@pytest.mark.parametrize("fmt", list(FMTS))
def test_the_largest_finite_y_has_a_scale(fmt):
    """Rows of +-1 (y is the weight): maxima up to float32's largest value are numbers."""
    x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.full((256,), torch.finfo(torch.float32).max, device="cuda")
    q, s = hum.rms_norm(x, w, eps=1e-12, act_fmt=fmt)
    assert not _not_a_number(s, fmt).any() and (torch.isfinite(s.float())).all()
