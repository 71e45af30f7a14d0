"""Pins of the fp64 oracle of routing, norm, convolution and scan: against central differences, closed forms and
hand-made rows."""
import numpy as np
import pytest

from oracle import mixer_oracle as O


def _slope(f, x, d, eps=1e-6):
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


def _check_gradients(f, inputs, grads, rng):
    """f(**inputs) is a number; its slope along a random direction of each input is the gradient's."""
    for name, g in grads.items():
        d = rng.standard_normal(inputs[name].shape)
        got = _slope(lambda v: f(**{**inputs, name: v}), inputs[name], d)
        np.testing.assert_allclose(got, (g * d).sum(), rtol=2e-6, atol=1e-7, err_msg=name)


def test_route_hand_made_rows():
    l = np.array([[3.0, 1.0, 2.0, 0.0, 2.5, 2.5, -1.0, 0.5]])
    idx, w, s = O.route(l, None, 3)
    assert idx.tolist() == [[0, 4, 5]]
    np.testing.assert_allclose(s[0], 1 / (1 + np.exp([-3.0, -2.5, -2.5])))
    np.testing.assert_allclose(w.sum(), 1.0)
    # groups of two: sums of both scores; the second group (2, 0) loses to (2.5, 2.5) and (3, 1)
    assert O.route(l, None, 2, groups=4, group_k=2)[0].tolist() == [[0, 4]]
    assert O.route(l, np.array([0, 0, 5, 5, 0, 0, 0, 0.0]), 2, groups=4, group_k=1)[0].tolist() == [[2, 3]]
    # a bias chooses and does not weigh
    idx, w, s = O.route(l, np.array([0, 0, 0, 0, 0, 0, 9.0, 0]), 1, renorm=False, scale=2.0)
    assert idx.tolist() == [[6]]
    np.testing.assert_allclose(w, 2 / (1 + np.exp(1.0)))


def test_route_masked_experts_come_last():
    l = np.array([[-np.inf, 1.0, -np.inf, 2.0]])
    idx, w, s = O.route(l, None, 4, "softmax")
    assert idx.tolist() == [[3, 1, 0, 2]]
    np.testing.assert_allclose(w[0, 2:], 0)
    np.testing.assert_allclose(w[0, :2], np.exp([2, 1]) / np.exp([2, 1]).sum())
    idx, w, s = O.route(np.full((1, 4), -np.inf), None, 2)
    assert idx.tolist() == [[0, 1]] and not w.any()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient(kind, renorm):
    rng = np.random.default_rng(1)
    l, g = rng.standard_normal((3, 12)), rng.standard_normal((3, 4))
    idx, w, s = O.route(l, None, 4, kind, renorm=renorm, scale=1.5)
    f = lambda l: (O.route(l, None, 4, kind, renorm=renorm, scale=1.5)[1] * g).sum()  # noqa: E731
    _check_gradients(f, dict(l=l), dict(l=O.route_backward(g, l, idx, w, s, kind, renorm, 1.5)), rng)


def test_renormalised_weights_of_tiny_scores():
    idx, w, s = O.route(np.array([[-800.0, -801.0, -900.0]]), None, 2)
    np.testing.assert_allclose(w[0], np.exp([0, -1]) / np.exp([0, -1]).sum(), rtol=1e-12)


def test_norm_gradient():
    rng = np.random.default_rng(2)
    u, w, dy, ds = (rng.standard_normal(s) for s in ((3, 10), (10,), (3, 10), (3, 10)))
    f = lambda u, w: (O.rmsnorm(u, w, 1e-3) * dy).sum() + (u * ds).sum()  # noqa: E731
    du, dw = O.rmsnorm_backward(dy, u, w, 1e-3, ds)
    _check_gradients(f, dict(u=u, w=w), dict(u=du, w=dw), rng)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_convolution(W, silu):
    rng = np.random.default_rng(W)
    lens, D = [5, 0, 1, 2], 3
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, w, b, st, dy, ds = n(8, D), n(D, W), n(D), n(4, W - 1, D), n(8, D), n(4, W - 1, D)
    y, out = O.conv(x, w, b, lens, silu, st)
    full = np.concatenate([st[0], x[:5]])
    p = np.stack([np.convolve(full[:, c], w[c, ::-1], "valid") for c in range(D)], 1) + b
    np.testing.assert_allclose(y[:5], p * O.sigmoid(p) if silu else p)
    np.testing.assert_allclose(out[1], st[1])

    def f(x, w, b, st):
        y, out = O.conv(x, w, b, lens, silu, st)
        return (y * dy).sum() + (out * ds).sum()
    dx, dw, db, dst = O.conv_backward(dy, x, w, b, lens, silu, st, ds)
    _check_gradients(f, dict(x=x, w=w, b=b, st=st), dict(x=dx, w=dw, b=db, st=dst), rng)


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("soft", [False, True])
def test_scan(G, soft):
    rng = np.random.default_rng(G)
    lens, D, S = [4, 0, 1, 3], 4, 4
    T, n = 8, lambda *s: rng.standard_normal(s)  # noqa: E731
    x = dict(u=n(T, D), delta=n(T, D), A=-np.exp(n(D, S)), B=n(T, G, S), C=n(T, G, S), skip=n(D), z=n(T, D),
             dt_bias=n(D), state=n(4, D, S))
    dy, X = n(T, D), n(4, D, S)
    if not soft:
        x["delta"], x["dt_bias"] = np.abs(x["delta"]), np.abs(x["dt_bias"])
    y, out = O.scan(lens=lens, soft=soft, **x)
    np.testing.assert_allclose(out[1], x["state"][1])
    # the closed form of the first sequence's last state
    dt = (O.softplus if soft else (lambda v: v))(x["delta"] + x["dt_bias"])
    want = np.exp(dt[:4].sum(0)[:, None] * x["A"]) * x["state"][0]
    for t in range(4):
        B = np.repeat(x["B"][t], D // G, axis=0)
        want = want + np.exp(dt[t + 1:4].sum(0)[:, None] * x["A"]) * (dt[t] * x["u"][t])[:, None] * B
    np.testing.assert_allclose(out[0], want, rtol=1e-12)
    f = lambda **v: (lambda r: (r[0] * dy).sum() + (r[1] * X).sum())(O.scan(lens=lens, soft=soft, **v))  # noqa: E731
    g = O.scan_backward(dy, lens=lens, soft=soft, d_state=X, **x)
    _check_gradients(f, x, {k: g["d_dt_bias" if k == "dt_bias" else "d_state_in" if k == "state" else "d" + k] for k in x}, rng)
