"""The oracle of the vocabulary-parallel operators: its gradients against
central differences of its own forward values, and pinned small cases."""
import numpy as np
import pytest

from oracle import vocab as vo


def differences(f, x, h=1e-5):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        if not np.isfinite(x[i]):
            continue
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


# central differences: truncation ~ h^2 |f'''| / 6 < 1e-9, rounding ~ 1e-15 / h = 1e-10
TOL = 1e-8


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.0])
@pytest.mark.parametrize("with_entropy", [False, True])
def test_log_probs_gradient_against_differences(temperature, with_entropy):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 9)) * 2
    x[1, 3:6] = -np.inf
    tokens = np.array([0, 8, -1, 4])
    a = rng.normal(size=4)
    b = rng.normal(size=4) if with_entropy else None

    def value(y):
        o = vo.log_probs(y, tokens, temperature, 0)
        return (a * o["log_probs"]).sum() + (0 if b is None else (b * o["entropy"]).sum())

    got = vo.log_probs_backward(x, tokens, temperature, a, b)
    assert np.abs(got - differences(value, x)).max() < TOL


@pytest.mark.parametrize("known_sum", [False, True])
def test_distill_gradient_against_differences(known_sum):
    rng = np.random.default_rng(6)
    x = rng.normal(size=(4, 9)) * 2
    ids = np.array([[0, 3, 8], [2, 2, -1], [9, -1, -5], [1, 4, 7]])
    t = rng.normal(size=(4, 3))
    t[3, 1] = -np.inf
    lse = np.array([2.0, 1.5, 3.0, 2.5]) if known_sum else None
    w = np.array([0.5, -1.0, 2.0, 0.25])
    loss, got = vo.distill(x, ids, t, 0.8, lse, w)
    assert loss[2] == 0 and not got[2].any()
    assert np.abs(got - differences(lambda y: (w * vo.distill(y, ids, t, 0.8, lse, w)[0]).sum(), x)).max() < TOL


def test_pinned_values():
    x = np.log(np.array([[1.0, 2.0, 5.0, 2.0]]))
    o = vo.log_probs(x, [1], 1.0, 3)
    assert abs(o["log_probs"][0] - np.log(0.2)) < 1e-15
    assert abs(o["entropy"][0] + 0.1 * np.log(0.1) + 0.4 * np.log(0.2) + 0.5 * np.log(0.5)) < 1e-15
    assert o["top_ids"].tolist() == [[2, 1, 3]]  # equal values: the lower column first
    assert np.allclose(o["stats"], [[np.log(5.0), np.log(2.0)]])
    loss, _ = vo.distill(x, np.array([[1]]), np.array([[7.0]]), 1.0)
    assert abs(loss[0] + np.log(0.2)) < 1e-15  # one entry: cross entropy


def test_masked_rows():
    x = np.full((2, 4), -np.inf)
    x[1, 2] = 3.0
    o = vo.log_probs(x, [0, 2], 1.0, 2)
    assert o["log_probs"].tolist() == [-np.inf, 0.0] and o["entropy"].tolist() == [0.0, 0.0]
    assert o["top_ids"].tolist() == [[-1, -1], [2, -1]]
    assert not vo.log_probs_backward(x, [0, 2], 1.0, [1.0, 1.0], [1.0, 1.0]).any()
    loss, g = vo.distill(x, np.array([[0], [0]]), np.zeros((2, 1)), 1.0, None, [1.0, 1.0])
    assert np.isposinf(loss).all() and not g[0].any() and g[1].tolist() == [-1.0, 0.0, 1.0, 0.0]
