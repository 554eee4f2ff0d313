"""GPU: routing against the float64 oracle: ids equal, ties to the lowest
index, and weights within their derived bound.

Weights: scores may be formed in f32 from x - max(x) (half an ulp of it, which
enters the exponential as its own size: |x - max| 2^-24), with exp, sum,
quotient and scale at most 24 further roundings of 2^-24."""
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
    okw = dict(kw, bias=None if bias is None else bias.double().cpu().numpy())
    xs = x.double().cpu().numpy()
    ri, rw = L.route(xs, topk, **okw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    gi, gw = ids.cpu().numpy(), w.double().cpu().numpy()
    bad = np.argwhere(gi != ri)
    assert len(bad) == 0, (bad[:3], gi[bad[0][0]], ri[bad[0][0]])
    fin = np.where(np.isfinite(xs), xs, 0.0)
    spread = np.abs(fin).max(1, keepdims=True) + np.abs(fin.max(1, keepdims=True))
    tol = np.abs(rw) * (24 + spread) * 2.0 ** -24 + 2.0 ** -126
    assert (np.abs(gw - rw) <= tol).all(), np.abs(gw - rw).max()
    return ids, w


def _logits(seed, t, e, dtype, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(t, e, generator=g) * scale).to(dtype).cuda()


def _bias(seed, e, scale=0.05):
    return (torch.randn(e, generator=torch.Generator().manual_seed(seed)) * scale).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (3, 2, 1), (5, 5, 5), (70, 8, 2), (33, 16, 4), (9, 60, 4), (65, 64, 6), (17, 72, 64),
                                   (40, 128, 8), (4, 129, 1), (31, 160, 6), (66, 256, 8), (13, 384, 10), (12, 511, 3), (37, 512, 64)])
def test_route(t, e, k, score, dtype):
    x = _logits(t + e, t, e, dtype)
    for bias in (None, _bias(e, e)):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            _check(x, k, score=score, bias=bias, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,k", [(8, 4, 1, 2), (8, 8, 3, 3), (64, 8, 3, 6), (160, 8, 3, 6), (256, 8, 4, 8), (256, 4, 1, 10),
                                             (512, 64, 5, 8), (384, 2, 1, 16), (72, 8, 8, 4), (60, 4, 2, 40), (66, 3, 1, 30)])
def test_route_groups(e, groups, kept, k, score, gs):
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(e + groups, 45, e, dtype)
        for bias in (None, _bias(3, e)):
            _check(x, k, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_score=gs)


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,k", [(15, 15, 4, 3), (30, 15, 3, 6), (36, 12, 5, 8), (72, 8, 3, 6), (72, 4, 1, 14), (170, 10, 3, 8),
                                             (266, 14, 2, 10), (500, 4, 2, 8), (510, 2, 1, 12)])
def test_route_groups_of_any_size(e, groups, kept, k, score, gs):
    g = torch.Generator().manual_seed(e)
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(e + groups, 75, e, dtype)
        x = x.masked_fill((torch.rand(75, e, generator=g) < 0.1).cuda(), float("-inf"))
        x = x.masked_fill((torch.rand(75, groups, generator=g) < 0.3).repeat_interleave(e // groups, 1).cuda(), float("-inf"))
        low = torch.where(torch.rand(e, generator=g).cuda() < 0.5, torch.finfo(torch.float32).min, _bias(4, e))
        for bias in (None, _bias(3, e), low):
            _check(x, k, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    g = np.random.default_rng(0)
    for e, groups in ((16, 1), (256, 8), (500, 1)):
        x = torch.from_numpy(g.integers(-2, 3, (60, e)).astype(np.float32)).cuda()
        for bias in (None, torch.zeros(e, device="cuda"), torch.from_numpy(g.integers(-1, 2, e).astype(np.float32) / 4).cuda()):
            for gs in ("max", "top2"):
                _check(x, min(e, 12), score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2), group_score=gs)
    x = torch.zeros(3, 512, device="cuda")
    ids, w = _check(x, 64, score=score)
    assert torch.equal(ids.cpu(), torch.arange(64, dtype=torch.int32).expand(3, 64))


def test_zeros_of_either_sign_are_equal():
    g = np.random.default_rng(3)
    for e in (8, 64, 200):
        x = torch.from_numpy(np.where(g.random((60, e)) < 0.5, -1.0, np.copysign(0.0, g.random((60, e)) - 0.5)).astype(np.float32)).cuda()
        assert (torch.signbit(x) & (x == 0)).any()
        for dtype in (torch.float32, torch.bfloat16):
            for k in (1, 2, 5):
                for kw in ({}, dict(num_groups=4, topk_groups=2), dict(num_groups=4, topk_groups=2, group_score="top2"),
                           dict(score="sigmoid", bias=torch.full((e,), -0.0, device="cuda"))):
                    _check(x.to(dtype), k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_scores_are_told_apart(score):
    """Neighbouring f32 logits, at magnitudes where their f32 scores are equal: without a bias the larger logit comes
    first; with one the f64 sums decide."""
    g = np.random.default_rng(1)
    for base in (0.5, 3.0, 12.0, 20.0):
        v = np.float32(base) + np.arange(64, dtype=np.float32) * np.spacing(np.float32(base))
        x = np.stack([g.permutation(v) for _ in range(20)])
        x = torch.from_numpy(np.concatenate([x, g.standard_normal((20, 64)).astype(np.float32)], 1)).cuda()
        _check(x, 16, score=score)
        if base > 12:
            continue                 # (f64 sigmoids of neighbours are apart by less than their sum's rounding)
        for b in (0.0, 1.0):
            _check(x, 16, score=score, bias=torch.full((128,), b, device="cuda"))
            _check(x, 16, score=score, bias=torch.full((128,), b, device="cuda"), num_groups=4, topk_groups=2, group_score="top2")
    # sums of score and bias that f32 makes equal: biases undo most of the score's difference
    x = (torch.randn(50, 64, generator=torch.Generator().manual_seed(4)) * 2)
    x = x.sort(-1)[0][:1].repeat(50, 1) + 1e-3 * x
    s = torch.from_numpy(L.scores(x[:1].double().numpy(), score))[0]
    _check(x.cuda(), 8, score=score, bias=(s.mean() - s).float().cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_rows(score, dtype):
    x = _logits(6, 40, 64, dtype)
    x[:, 5] = -float("inf")
    x[3] = -float("inf")                              # nothing left
    x[4, 1:] = -float("inf")                          # one left
    x[5, 8:] = -float("inf")                          # one group left
    x[6] = torch.finfo(dtype).min                     # the lowest value is a value
    x[7, ::2] = torch.finfo(dtype).min
    x[8, :32] = -float("inf")
    x[9] *= 60
    for bias in (None, _bias(1, 64)):
        for groups, kept, gs in ((1, 1, "max"), (8, 3, "max"), (8, 3, "top2")):
            for renorm in (True, False):
                ids, w = _check(x, 10, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_score=gs, renormalize=renorm)
                assert (ids[3] == -1).all() and (w[3] == 0).all()
                assert ids[4, 0] == 0 and (ids[4, 1:] == -1).all()
                assert not torch.isnan(w).any()
    b = _bias(1, 64)
    b[7] = -float("inf")
    ids, _ = _check(x, 10, score=score, bias=b)
    assert (ids != 7).all()


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_the_lowest_value(score, gs):
    """float32's lowest value as a mask: two of them pass it in a group's sum,
    and yet such a group comes before one without experts."""
    low = torch.finfo(torch.float32).min
    for e, groups, kept, k in ((256, 8, 4, 8), (64, 8, 3, 6), (16, 4, 2, 6), (60, 4, 3, 20)):
        n = e // groups
        x = _logits(e, 80, e, torch.float32)
        g = torch.Generator().manual_seed(e)
        empty = torch.rand(80, groups, generator=g) < 0.3       # of each token
        x = x.masked_fill(empty.repeat_interleave(n, 1).cuda(), float("-inf"))
        x[3] = float("-inf")
        single = torch.rand(80, e, generator=g) < 0.2
        x = x.masked_fill(single.cuda(), float("-inf"))
        for masked in (torch.rand(e, generator=g) < 0.5, torch.arange(e) // n < groups - kept + 1, torch.arange(e) // n >= 1, torch.ones(e, dtype=torch.bool)):
            bias = torch.where(masked.cuda(), torch.full((e,), low, device="cuda"), _bias(e, e))
            _check(x, k, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_score=gs)
            bias = torch.where(masked.cuda(), -(2.0 + torch.rand(e, generator=g).cuda()) * 1e38, _bias(e, e))
            _check(x, k, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_score=gs)


def test_far_logits():
    """Scores far below f32's range: sigmoids renormalise all the same."""
    x = torch.full((4, 16), -200.0, device="cuda")
    x[:, 3] = -199.0
    x[1] = 500.0
    x[2] = torch.linspace(-300, 300, 16)
    x[3] = -3e38
    x[3, 2] = 3e38
    _check(x, 4, score="softmax")
    ids, w = hum.moe_route(x, 4, score="sigmoid")
    ri, rw = L.route(x.double().cpu().numpy(), 4, "sigmoid")
    assert (ids.cpu().numpy() == ri).all()
    np.testing.assert_allclose(w.double().cpu().numpy(), rw, rtol=1e-6, atol=1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinity_stay_visible_and_ids_valid(score):
    x = _logits(2, 30, 256, torch.float32)
    x[0, 9] = float("nan")
    x[1] = float("nan")
    x[2, 3] = float("inf")
    clean = x.clone()
    clean[:3] = 0
    for groups in (1, 8):
        for bias in (None, _bias(5, 256)):
            kw = dict(score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2), group_score="top2")
            ids, w = hum.moe_route(x, 8, **kw)
            a, b = hum.moe_route(clean, 8, **kw)
            assert torch.equal(ids[3:], a[3:]) and torch.equal(w[3:], b[3:])
            assert (ids >= 0).all() and (ids < 256).all() and all(len(set(r.tolist())) == 8 for r in ids)
            assert ids[0, 0] == 9 and torch.isnan(w[0]).all() and torch.isnan(w[1]).all()
            assert ids[2, 0] == 3 or bias is not None
            if score == "softmax":
                assert torch.isnan(w[2]).all()
            else:
                assert not torch.isnan(w[2]).any()


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_switched_off_experts_stay_off_beside_nans_and_infinities(score, groups):
    for e, k in ((16, 4), (256, 8), (64, 20)):
        x = _logits(e, 12, e, torch.float32)
        bias = _bias(7, e)
        off = torch.rand(e, generator=torch.Generator().manual_seed(e)) < 0.3
        off[5], off[6] = True, False
        bias[off.cuda()] = float("-inf")
        x[1, 6], x[2, 6], x[3, 5], x[4, 5] = float("inf"), float("nan"), float("inf"), float("nan")
        x[5, :] = float("nan")
        ids, _ = hum.moe_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2))
        ids = ids.cpu()
        assert (ids < e).all() and not off[ids.clamp(min=0).long()][ids >= 0].any()
        assert ids[2, 0] == 6
        if score == "softmax":  # (a sigmoid of infinity is 1, and a bias may put another before it)
            assert ids[1, 0] == 6
        assert torch.equal(ids[5][ids[5] >= 0], torch.arange(e)[~off][:int((ids[5] >= 0).sum())].int())


def test_strided_logits_and_given_outputs():
    for dtype in (torch.float32, torch.bfloat16):
        wide = _logits(3, 21, 300, dtype)
        for off, e in ((0, 128), (1, 64), (2, 256), (3, 60), (5, 8)):
            x = wide[:, off:off + e]
            want = hum.moe_route(x.contiguous(), 4)
            ids, w = torch.full((23, 4), 77, dtype=torch.int32, device="cuda"), torch.full((23, 4), 7.0, device="cuda")
            got = hum.moe_route(x, 4, topk_ids=ids[1:22], topk_weights=w[1:22])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert (ids[[0, 22]] == 77).all() and (w[[0, 22]] == 7).all()
        one = hum.moe_route(wide[:1].expand(5, 300), 3)
        assert torch.equal(one[0], hum.moe_route(wide[:1], 3)[0].expand(5, 3))
    ids, w = hum.moe_route(wide[:0], 3)
    assert ids.shape == w.shape == (0, 3)


def test_many_tokens():
    """A prompt's worth, the same bits as a token at a time would have."""
    x = _logits(9, 30000, 128, torch.bfloat16)
    ids, w = hum.moe_route(x, 8)
    part = [hum.moe_route(p, 8) for p in x.split(7777)]
    assert torch.equal(ids, torch.cat([p[0] for p in part])) and torch.equal(w, torch.cat([p[1] for p in part]))
    s = x[:4000].double().cpu().numpy()
    order = np.argsort(-s, axis=1, kind="stable")[:, :8]
    assert (ids[:4000].cpu().numpy() == order).all()


@pytest.mark.parametrize("e,k,kw,biased", [(8, 2, {}, False), (64, 6, {}, True), (256, 8, dict(score="sigmoid"), True), (130, 4, dict(score="sigmoid"), False),
                                           (256, 8, dict(score="sigmoid", num_groups=8, topk_groups=4, group_score="top2", scale=2.5), True),
                                           (160, 6, dict(num_groups=8, topk_groups=3, renormalize=False), False),
                                           (512, 14, dict(num_groups=16, topk_groups=5, group_score="top2"), False), (72, 15, dict(num_groups=8, topk_groups=3), True)])
def test_prompts_are_routed_as_their_tokens_alone(e, k, kw, biased):
    """Large calls and small ones run on workgroups of other sizes: the same bits, also of tokens that share a wave
    with others (near and equal logits among them)."""
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(e + k, 6003, e, dtype)
        x[::7] = x[::7].round()                          # ties
        x[1::9, : e // 2] = x[1::9, e // 2: e // 2 * 2] * (1 + 2.0 ** -23)
        x[5::100] = -float("inf")
        bias = _bias(k, e) if biased else None
        ids, w = hum.moe_route(x, k, bias=bias, **kw)
        at = 0
        for n in (1, 2, 3, 5, 63, 64, 65, 800, 4000, 1000):
            a, b = hum.moe_route(x[at:at + n], k, bias=bias, **kw)
            assert torch.equal(a, ids[at:at + n]) and torch.equal(b, w[at:at + n]), n
            at += n
        assert at == 6003
        _check(x[:120], k, bias=bias, **kw)
