"""The float64 oracles of the norm and of the router's training side: closed
forms, and every gradient against central differences of its forward."""

import numpy as np
import pytest

from oracle import balance as ob
from oracle import norm as on

STEP = 1e-6
# Central differences in float64 of functions of order 1: the step's own error
# is O(STEP^2) ~ 1e-12 times a third derivative, the rounding 2^-53 / STEP ~
# 1e-10; inputs keep the third derivatives below 1e3.
TOL = 1e-7


def differences(f, x):
    """d f(x) / d x, element by element (f returns a number)."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += STEP
        b[i] -= STEP
        out[i] = (f(a) - f(b)) / (2 * STEP)
    return out


def test_norm_of_equal_values_is_the_weight():
    h, y = on.rms_norm(np.full((2, 5), -3.0), np.arange(5.0), 0.0)
    assert np.array_equal(h, np.full((2, 5), -3.0))
    assert np.allclose(y, -np.arange(5.0), rtol=1e-15)


def test_norm_of_zeros_is_zero():
    _, y = on.rms_norm(np.zeros((1, 4)), np.ones(4), 1e-6)
    assert np.array_equal(y, np.zeros((1, 4)))


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 16)])
def test_norm_gradient_against_differences(T, H):
    rng = np.random.default_rng(T * 100 + H)
    x, res, dy, dh = (rng.normal(size=(T, H)) for _ in range(4))
    w = rng.normal(size=H)
    eps = 1e-3

    def f(x, w):
        h, y = on.rms_norm(x, w, eps, res)
        return np.sum(dy * y) + np.sum(dh * h)

    g = on.rms_norm_grad(dy, x + res, w, eps, dh)
    assert np.allclose(g["dx"], differences(lambda v: f(v, w), x), atol=TOL)
    assert np.allclose(g["dw"], differences(lambda v: f(x, v), w), atol=TOL)


def test_balanced_routing_has_loss_one():
    # every expert is chosen equally often: the loss is sum of the mean
    # probabilities, which is one
    E, k = 6, 2
    ids = np.array([[i % E, (i + 1) % E] for i in range(E)])
    r = ob.balance_loss(np.random.default_rng(0).normal(size=(E, E)), ids, "softmax")
    assert np.array_equal(r["counts"], np.full((1, E), k))
    assert abs(r["losses"][0] - 1.0) < 1e-14
    assert r["tokens"].tolist() == [E, E, 1]


def test_one_expert_for_all_has_loss_e():
    lg = np.full((4, 5), -1e3)
    lg[:, 2] = 0.0
    r = ob.balance_loss(lg, np.full((4, 1), 2), "softmax")
    assert abs(r["losses"][0] - 5.0) < 1e-12 and abs(r["losses"][1]) < 1e-12


def test_sequences_masks_and_foreign_ids():
    lg = np.zeros((6, 4))
    ids = np.array([[0, 1], [1, -1], [3, 9], [2, 2], [0, 3], [0, 0]])
    r = ob.balance_loss(lg, ids, "sigmoid", offsets=[0, 2, 2, 5], mask=[1, 1, 0, 1, 1, 1])
    assert r["counts"].tolist() == [[1, 2, 0, 0], [0, 0, 0, 0], [1, 0, 2, 1]]
    assert r["tokens"].tolist() == [2, 0, 2, 4, 2]
    assert np.allclose(r["probs"][[0, 2]], 0.25) and np.all(r["probs"][1] == 0)
    assert np.isclose(r["losses"][1], np.log(4.0) ** 2)


def test_rows_of_minus_infinity():
    lg = np.array([[-np.inf, -np.inf], [0.0, -np.inf]])
    r = ob.balance_loss(lg, np.array([[0], [0]]), "softmax")
    assert np.allclose(r["probs"], [[0.5, 0.0]]) and r["losses"][1] == 0.0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(scoring, renormalize):
    rng = np.random.default_rng(7)
    T, E, k, scale = 5, 6, 3, 2.5
    lg = rng.normal(size=(T, E))
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    ids[1, 2] = -1           # a slot without an expert
    ids[2] = ids[2, 0]       # the same expert in every slot
    off, mask = [0, 2, 2, 4], [1, 0, 1, 1, 1]
    dw = rng.normal(size=(T, k))
    dl = np.array([0.7, 0.3])
    counts = ob.balance_loss(lg, ids, scoring, off, mask)["counts"]

    def f(v):
        r = ob.balance_loss(v, ids, scoring, off, mask)
        return np.dot(dl, r["losses"]) + np.sum(dw * ob.weights(v, ids, scoring, renormalize, scale))

    d, mag = ob.route_grad(lg, ids, scoring, renormalize, scale, dw, dl, counts, off, mask)
    assert np.allclose(d, differences(f, lg), atol=TOL)
    assert np.all(mag >= np.abs(d) - 1e-15)
    # each part alone
    a, _ = ob.route_grad(lg, ids, scoring, renormalize, scale, d_weights=dw)
    b, _ = ob.route_grad(lg, ids, scoring, renormalize, scale, None, dl, counts, off, mask)
    assert np.allclose(a + b, d, atol=1e-14)


def test_gate_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, gate, d, dx_in = rng.normal(size=(4, 5)), rng.normal(size=(3, 5)), rng.normal(size=(4, 3)), rng.normal(size=(4, 5))
    g = ob.gate_grad(x, gate, d, dx_in)
    f = lambda x, gate: np.sum(d * (x @ gate.T)) + np.sum(dx_in * x)  # noqa: E731
    assert np.allclose(g["dx"], differences(lambda v: f(v, gate), x), atol=TOL)
    assert np.allclose(g["d_gate"], differences(lambda v: f(x, v), gate), atol=TOL)
