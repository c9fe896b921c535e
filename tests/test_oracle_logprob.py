"""The oracle of the token log probabilities: its gradient against central
differences, its values against plain sums, its rules row by row (CPU)."""
import numpy as np
import pytest

from oracle import logprob as O


@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.0])
def test_values(temperature):
    rng = np.random.default_rng(0)
    l = rng.normal(size=(6, 37)) * 3
    l[2, 5:20] = -np.inf
    t = np.array([0, 36, 4, -1, 7, 9])
    o = O.token_logprob(l, t, temperature, top=3)
    p = np.exp(l / temperature) / np.exp(l / temperature).sum(1, keepdims=True)
    for r in (0, 1, 2, 4, 5):
        assert np.isclose(o["logp"][r], np.log(p[r, t[r]]), rtol=1e-12)
        assert np.isclose(o["entropy"][r], -sum(x * np.log(x) for x in p[r] if x > 0), rtol=1e-12)
        assert o["top_ids"][r].tolist() == sorted(range(37), key=lambda i: (-p[r, i], i))[:3]
    assert o["logp"][3] == o["lse"][3] == o["entropy"][3] == 0 and (o["top_ids"][3] == -1).all()


def test_rows_of_masks_and_nan():
    l = np.zeros((4, 5))
    l[0] = -np.inf
    l[1] = np.finfo(np.float32).min
    l[2, 3] = np.nan
    l[3, 1:] = -np.inf
    o = O.token_logprob(l, np.array([0, 1, 2, 4]), top=2)
    assert o["lse"][0] == o["lse"][1] == -np.inf and o["entropy"][0] == 0
    assert np.isnan(o["logp"][2])
    assert o["lse"][3] == 0 and o["logp"][3] == -np.inf and o["top_ids"][3].tolist() == [0, -1]


@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_gradient_against_differences(temperature):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(4, 11)) * 2
    l[1, 3] = -np.inf
    t = np.array([2, 5, -1, 10])
    g, gh = rng.normal(size=4), rng.normal(size=4)

    def f(x):
        o = O.token_logprob(x, t, temperature)
        return (g * o["logp"] + gh * o["entropy"]).sum()

    o = O.token_logprob(l, t, temperature)
    d, _ = O.token_logprob_backward(l, t, o["lse"], g, o["entropy"], gh, temperature)
    for r in range(4):
        for i in range(11):
            if not np.isfinite(l[r, i]):
                assert d[r, i] == 0
                continue
            a, b = l.copy(), l.copy()
            a[r, i] += 1e-5
            b[r, i] -= 1e-5
            assert abs((f(a) - f(b)) / 2e-5 - d[r, i]) < 1e-8


def test_gradient_of_a_nearly_certain_target():
    """From the target's own log p: the row's sum is 0 to its last bit; from an lse rounded to fp32 1 - p is lost."""
    l = np.zeros((1, 9))
    l[0, 4] = 25.0
    t, one = np.array([4]), np.ones(1)
    o = O.token_logprob(l, t)
    rounded = np.float64(np.float32(o["lse"]))
    exact, _ = O.token_logprob_backward(l, t, o["lse"], one)
    d, _ = O.token_logprob_backward(l, t, rounded, one, logp=o["logp"])
    assert np.isclose(d[0, 4], exact[0, 4], rtol=1e-12) and np.isclose(d[0, 4], 8 * np.exp(-25), rtol=1e-9)
    assert O.token_logprob_backward(l, t, rounded, one)[0][0, 4] == 0
