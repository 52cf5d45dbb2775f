"""The float64 router: hand-worked rows, torch's softmax and topk where they apply, and the
gradient formula against central differences of the forward functions."""
import numpy as np
import pytest
import torch

from oracle import gate


def test_hand_worked_rows():
    # scores 0.5, 0.25, 0.25 (ln 2 apart): ties go to the lowest index
    x = np.log(np.array([[2.0, 1.0, 1.0]]))
    ids, w = gate.topk(x, 2, "softmax")
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = gate.topk(x, 2, "softmax", renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    # the bias moves the choice, not the weights
    ids, w = gate.topk(x, 1, "softmax", bias=[0.0, 0.0, 0.5], renorm=False)
    assert ids.tolist() == [[2]] and np.allclose(w, [[0.25]])
    # groups {0, 1}, {2, 3}: sigmoid(0) + sigmoid(0) = 1 beats sigmoid(2) + sigmoid(-9) < 1
    ids, w = gate.topk([[0.0, 0.0, 2.0, -9.0]], 2, "sigmoid", groups=2, topk_groups=1)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.5, 0.5]])
    # experts taken out are chosen last and weigh nothing; a row without experts too
    ids, w = gate.topk([[-np.inf, 0.0, np.nan, -np.inf], [-np.inf] * 4], 3, "softmax")
    assert ids.tolist() == [[1, 0, 2], [0, 1, 2]] and np.allclose(w, [[1, 0, 0], [0, 0, 0]])
    # one sequence of two rows, E = 2, K = 1, both choose expert 0: loss = 2 (1 P_0) with P_0 = 0.5
    loss, counts, coef = gate.balance(np.zeros((2, 2)), np.array([[0], [0]]), "softmax")
    assert np.isclose(loss, 1.0) and counts.tolist() == [[2, 0]] and np.allclose(coef, [[1.0, 0.0]])


@pytest.mark.parametrize("seed", [0, 1])
def test_against_torch(seed):
    x = np.random.default_rng(seed).standard_normal((50, 24))
    ids, w = gate.topk(x, 5, "softmax", renorm=False)
    top = torch.softmax(torch.from_numpy(x), 1).topk(5, dim=1)
    assert np.array_equal(ids, top.indices.numpy()) and np.allclose(w, top.values.numpy())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(3)
    n, e, k = 7, 6, 3
    x = rng.standard_normal((n, e))
    x[2, 4] = -np.inf   # an expert taken out
    off, mask = [0, 2, 2, 6], [1, 1, 0, 1, 1, 1, 1]
    ids = gate.topk(x, k, scoring)[0]
    gw, gl = rng.standard_normal((n, k)), 0.7
    coef = gate.balance(x, ids, scoring, off, mask, 0.3)[2]

    def total(y):
        w = np.take_along_axis(gate.scores(y, scoring), ids, axis=1)
        if renorm:
            w = w / w.sum(axis=1, keepdims=True)
        return float((2.0 * w * gw).sum()) + gl * gate.balance(y, ids, scoring, off, mask, 0.3)[0]

    got, mag = gate.backward(x, ids, scoring, gw, renorm, 2.0, gl, coef, off, mask)
    assert np.all(np.abs(got) <= mag * (1 + 1e-12))
    h = 1e-6
    for t in range(n):
        for i in range(e):
            if not np.isfinite(x[t, i]):
                assert got[t, i] == 0.0
                continue
            y, z = x.copy(), x.copy()
            y[t, i] += h
            z[t, i] -= h
            # central difference: truncation h^2 |f'''| / 6 < 1e-11, rounding 2^-53 |f| / h < 1e-9
            assert abs((total(y) - total(z)) / (2 * h) - got[t, i]) < 1e-7


def test_biases_without_a_value():
    """NaN and -inf in the bias rank an expert last and add nothing to its group; it keeps its score."""
    x = np.log(np.array([[4.0, 2.0, 1.0, 1.0]]))
    ids, w = gate.topk(x, 3, "softmax", bias=[np.nan, 0.0, -np.inf, 0.0], renorm=False)
    assert ids.tolist() == [[1, 3, 0]] and np.allclose(w, [[0.25, 0.125, 0.5]])
    ids, _ = gate.topk(x, 2, "softmax", bias=[0.0, 0.0, np.inf, np.nan])
    assert ids.tolist() == [[2, 0]]
    # group {0, 1} has the sum 0.25, {2, 3} of 0.125
    ids, _ = gate.topk(x, 2, "softmax", bias=[np.nan, 0.0, -np.inf, 0.0], groups=2, topk_groups=1)
    assert ids.tolist() == [[1, 0]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_of_an_expert_chosen_twice(scoring):
    """An id that stands twice in a row gets both gradients (differences of the weights)."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 5))
    ids, gw = np.array([[1, 1, 3], [2, 2, 2]]), rng.standard_normal((2, 3))

    def total(y):
        w = np.take_along_axis(gate.scores(y, scoring), ids, axis=1)
        return float((w / w.sum(axis=1, keepdims=True) * gw).sum())

    got, h = gate.backward(x, ids, scoring, gw)[0], 1e-6
    for t in range(2):
        for i in range(5):
            y, z = x.copy(), x.copy()
            y[t, i] += h
            z[t, i] -= h
            assert abs((total(y) - total(z)) / (2 * h) - got[t, i]) < 1e-7
