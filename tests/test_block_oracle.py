"""Pins of the mixer's and optimizer's fp64 oracle: against the quadratic form of
linear attention, central differences, and a scalar AdamW."""
import numpy as np
import pytest

from oracle import block_oracle as O


def _inputs(lens, Hs, r, Dk, Dv, seed=0):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(q=n(T, Hs * r, Dk), k=n(T, Hs, Dk), v=n(T, Hs, Dv), do=n(T, Hs * r, Dv),
                S0=n(N, Hs, Dk, Dv), X=n(N, Hs, Dk, Dv),
                ld=-rng.uniform(0.01, 1.0, Hs))


def test_forward_is_the_decayed_quadratic_form():
    lens, Hs, r, Dk, Dv = [5, 0, 3], 2, 3, 4, 6
    x = _inputs(lens, Hs, r, Dk, Dv)
    o, S = O.linattn_forward(x["q"], x["k"], x["v"], x["ld"], lens, 0.7, x["S0"])
    start = 0
    for n, L in enumerate(lens):
        for h in range(Hs):
            lam = np.exp(x["ld"][h])
            k, v = x["k"][start:start + L, h], x["v"][start:start + L, h]
            for a in range(r):
                q = x["q"][start:start + L, h * r + a]
                for i in range(L):
                    want = lam ** (i + 1) * q[i] @ x["S0"][n, h]
                    for j in range(i + 1):
                        want = want + lam ** (i - j) * (q[i] @ k[j]) * v[j]
                    np.testing.assert_allclose(o[start + i, h * r + a], 0.7 * want, rtol=1e-12, atol=1e-12)
            want = lam ** L * x["S0"][n, h]
            for j in range(L):
                want = want + lam ** (L - 1 - j) * np.outer(k[j], v[j])
            np.testing.assert_allclose(S[n, h], want, rtol=1e-12, atol=1e-12)
        start += L


@pytest.mark.parametrize("name", ["q", "k", "v", "S0"])
def test_backward_matches_central_differences(name):
    """The loss sum(o * do) + sum(S_out * X) is linear in each operand alone, so central differences
    are exact up to rounding: 1e-16 * |loss| / h with h = 1e-2, |loss| < 1e3, below 1e-10."""
    lens, Hs, r, Dk, Dv = [4, 0, 1, 3], 2, 2, 3, 4
    x = _inputs(lens, Hs, r, Dk, Dv, seed=1)

    def loss(y):
        o, S = O.linattn_forward(y["q"], y["k"], y["v"], y["ld"], lens, 0.6, y["S0"])
        return float((o * y["do"]).sum() + (S * y["X"]).sum())

    grads = dict(zip(["q", "k", "v", "S0"], O.linattn_backward(
        x["do"], x["q"], x["k"], x["v"], x["ld"], lens, 0.6, x["S0"], x["X"])))
    rng = np.random.default_rng(2)
    flat = grads[name].reshape(-1)
    for i in rng.choice(flat.size, min(40, flat.size), replace=False):
        d = np.zeros(flat.size)
        d[i] = 1e-2
        d = d.reshape(x[name].shape)
        diff = (loss({**x, name: x[name] + d}) - loss({**x, name: x[name] - d})) / 2e-2
        assert abs(diff - flat[i]) < 1e-10, (i, diff, flat[i])


def test_adamw_update_by_hand():
    p, m, v = O.adamw_update(np.array([2.0]), np.array([0.5]), np.array([0.1]), np.array([0.04]), 3,
                             0.01, 0.9, 0.99, 1e-8, 0.1)
    m1, v1 = 0.9 * 0.1 + 0.1 * 0.5, 0.99 * 0.04 + 0.01 * 0.25
    want = 2.0 - 0.01 * 0.1 * 2.0 - 0.01 * (m1 / (1 - 0.729)) / (np.sqrt(v1 / (1 - 0.99 ** 3)) + 1e-8)
    np.testing.assert_allclose([p[0], m[0], v[0]], [want, m1, v1], rtol=1e-14)


def test_rounding_numbers_are_uniform_and_their_rounding_unbiased():
    n = 200_000
    for u in O.rounding_numbers(7, 101, 2, n):
        assert abs(u.mean() - 0.5) < 5 * np.sqrt(1 / 12 / n)
        hist = np.histogram(u, bins=16, range=(0, 1))[0]
        assert abs(hist - n / 16).max() < 5 * np.sqrt(n / 16)
    u = O.rounding_numbers(7, 101, 2, n)[0]
    x = np.full(n, 1.0 + 1 / 64)  # an eighth of the way between two E4M3 values
    got = O.round_stochastic(x, O.e4m3_unit(x), u)
    assert set(np.unique(got)) == {1.0, 1.125}
    assert abs(got.mean() - x[0]) < 5 * 0.125 * np.sqrt(0.125 * 0.875 / n)
