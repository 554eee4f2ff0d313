"""CPU pins of the layer oracle (norm, routing) against closed forms, torch and brute force."""
import itertools

import numpy as np
import torch

import oracle

L = oracle.layer


def test_norm_closed_forms():
    w = np.array([1.0, 2.0, -1.0, 0.5])
    y, h = L.rms_norm(np.array([[3.0, 4.0, 0.0, 0.0]]), w, 0.0 + 1e-300)
    np.testing.assert_allclose(y, [[3 / 2.5, 8 / 2.5, 0, 0]], rtol=1e-15)
    y, h = L.rms_norm(np.ones((2, 4)), w, 3.0, residual=np.full((2, 4), -2.0), weight_offset=1.0)
    np.testing.assert_allclose(h, -np.ones((2, 4)))
    np.testing.assert_allclose(y, -np.tile(w + 1, (2, 1)) / 2)


def test_norm_is_scale_free_and_agrees_with_torch():
    g = np.random.default_rng(0)
    x, w = g.standard_normal((5, 96)), g.standard_normal(96)
    a = L.rms_norm(x, w, 1e-6)[0]
    b = torch.nn.functional.rms_norm(torch.from_numpy(x), (96,), torch.from_numpy(w), 1e-6).numpy()
    np.testing.assert_allclose(a, b, rtol=1e-12)
    np.testing.assert_allclose(L.rms_norm(8 * x, w, 64e-6)[0], a, rtol=1e-12)


def test_scores():
    x = np.array([[0.0, np.log(3.0), -np.inf, np.log(4.0)]])
    np.testing.assert_allclose(L.scores(x, "softmax"), [[1 / 8, 3 / 8, 0, 4 / 8]], rtol=1e-14)
    np.testing.assert_allclose(L.scores(x, "sigmoid"), [[1 / 2, 3 / 4, 0, 4 / 5]], rtol=1e-14)
    assert (L.scores(np.full((1, 3), -np.inf), "softmax") == 0).all()


def test_route_against_all_subsets():
    """Without groups the chosen set is the one of the largest sum of keys; ids come best first."""
    g = np.random.default_rng(1)
    for score in ("softmax", "sigmoid"):
        x, b = g.standard_normal((20, 7)), 0.3 * g.standard_normal(7)
        ids, w = L.route(x, 3, score, b, renormalize=False)
        s = L.scores(x, score)
        for i in range(20):
            best = max(itertools.combinations(range(7), 3), key=lambda c: sum(s[i, j] + b[j] for j in c))
            assert set(ids[i]) == set(best)
            k = s[i, ids[i]] + b[ids[i]]
            assert (k[:-1] > k[1:]).all()
            np.testing.assert_array_equal(w[i], s[i, ids[i]])
        ids2, w2 = L.route(x, 3, score, b, scale=2.5)
        np.testing.assert_array_equal(ids, ids2)
        np.testing.assert_allclose(w2.sum(1), 2.5, rtol=1e-14)


def test_route_ties_masks_and_groups():
    x = np.array([[1.0, 5.0, 5.0, 1.0, 0.0, 5.0], [-np.inf, 2.0, -np.inf, -np.inf, -np.inf, -np.inf], [-np.inf] * 6])
    ids, w = L.route(x, 2)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    # groups {0,1,2} {3,4,5}: the second has the best expert, the first the best two
    x = np.log(np.array([[3.0, 3.0, 1.0, 4.0, 1.0, 1.0]]))
    assert L.route(x, 2, num_groups=2, topk_groups=1, group_score="max")[0].tolist() == [[3, 4]]
    assert L.route(x, 2, num_groups=2, topk_groups=1, group_score="top2")[0].tolist() == [[0, 1]]
    assert L.route(x, 4, num_groups=2, topk_groups=1, group_score="max")[0].tolist() == [[3, 4, 5, -1]]
    assert L.route(x, 3, num_groups=2, topk_groups=2)[0].tolist() == [[3, 0, 1]]
    # the group's two best count, a group of one left counts that one
    x = np.log(np.array([[3.0, 0.0, 0.0, 2.0, 2.0, 0.0]]) + np.array([[0, -0.0, 0, 0, 0, 0]]) + 1e-300)
    x[x < -100] = -np.inf
    assert L.route(x, 1, "sigmoid", num_groups=2, topk_groups=1, group_score="top2")[0].tolist() == [[3]]
