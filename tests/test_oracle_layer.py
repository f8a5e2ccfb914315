"""The oracle of the steps around the experts against hand-worked cases and differences."""
import numpy as np
import pytest

import oracle.layer_oracle as Y


def test_route_by_hand():
    l = np.log(np.array([[4.0, 1, 2, 3], [1, 1, 1, 1]]))
    idx, w = Y.route(l, 2)
    assert idx.tolist() == [[0, 3], [0, 1]] and np.allclose(w, [[4 / 7, 3 / 7], [0.5, 0.5]])
    assert np.allclose(Y.route(l, 2, renorm=False, scale=3.0)[1], [[1.2, 0.9], [0.75, 0.75]])
    # sigmoid(log x) = x / (1 + x); the bias moves the choice and not the weights
    idx, w = Y.route(l, 2, sigmoid=True, bias=[0, 0.5, 0, 0], renorm=False)
    assert idx.tolist() == [[1, 0], [1, 0]] and np.allclose(w, [[0.5, 0.8], [0.5, 0.5]])


def test_route_groups_by_hand():
    l = np.array([[9.0, 0, 0, 8, 7, 6]])
    assert Y.route(l, 2, groups=3, topk_groups=1)[0].tolist() == [[0, 1]]
    s = np.log(np.array([[8.0, 1, 5, 4, 3, 3]]))  # sums of sigmoids: 8/9 + 1/2, 5/6 + 4/5, 3/2
    assert Y.route(s, 2, sigmoid=True, groups=3, topk_groups=1, group_top=2)[0].tolist() == [[2, 3]]
    assert Y.route(s, 3, sigmoid=True, groups=3, topk_groups=1, group_top=2)[0].tolist() == [[2, 3, -1]]


def test_route_masks():
    n, inf = np.nan, np.inf
    idx, w = Y.route(np.array([[-inf, n, -inf], [n, 0, -inf], [inf, 1, inf]]), 2)
    assert idx.tolist() == [[-1, -1], [1, -1], [0, 2]]
    assert np.allclose(w, [[0, 0], [1, 0], [0.5, 0.5]])
    assert Y.route(np.zeros((1, 3)), 3, bias=[n, 1.0, -inf])[0].tolist() == [[1, -1, -1]]
    idx, w = Y.route(np.array([[-2000.0, -2001.0, -5000.0]]), 2, sigmoid=True)  # scores that 64 bits do not hold
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(sigmoid, renorm):
    rng = np.random.default_rng(3)
    l, g = rng.standard_normal((5, 7)), rng.standard_normal((5, 3))
    l[2, 4] = -np.inf
    idx = Y.route(l, 3, sigmoid)[0]
    idx[3] = [5, 5, -1]  # twice the same, and none
    got, mag = Y.route_backward(l, idx, g, sigmoid, renorm, 2.5)
    assert (np.abs(got) <= mag + 1e-15).all()
    for t in range(5):
        for e in range(7):
            if np.isfinite(l[t, e]):
                side = []
                for step in (1e-6, -1e-6):
                    x = l.copy()
                    x[t, e] += step
                    side.append((Y.chosen_weights(x, idx, sigmoid, renorm, 2.5) * g).sum())
                assert abs((side[0] - side[1]) / 2e-6 - got[t, e]) < 1e-8
            else:
                assert got[t, e] == 0


def test_norm_backward_against_differences():
    rng = np.random.default_rng(4)
    h, w, g, back = rng.standard_normal((3, 8)), rng.standard_normal(8), rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    f = lambda h, w: (Y.residual_norm(h, w, 1e-3)[1] * g).sum() + (h * back).sum()  # noqa: E731
    dh, _, dw, _ = Y.residual_norm_backward(g, h, w, Y.residual_norm(h, w, 1e-3)[0], back)
    for at in np.ndindex(3, 8):
        d = np.zeros((3, 8))
        d[at] = 1e-6
        assert abs((f(h + d, w) - f(h - d, w)) / 2e-6 - dh[at]) < 1e-8
    for c in range(8):
        d = np.zeros(8)
        d[c] = 1e-6
        assert abs((f(h, w + d) - f(h, w - d)) / 2e-6 - dw[c]) < 1e-8


@pytest.mark.parametrize("gelu", [False, True])
def test_glu_against_known_values_and_differences(gelu):
    if gelu:  # 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))
        g = np.linspace(-4, 4, 9)
        assert np.allclose(Y.gate(g, True)[0], 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))), atol=1e-15)
    else:
        assert np.allclose(Y.gate(np.array([0.0, np.log(3)]), False)[0], [0, 0.75 * np.log(3)])
    rng = np.random.default_rng(5)
    h, g = rng.standard_normal((4, 6)), rng.standard_normal((4, 3))
    got, mag = Y.glu_backward(h, g, gelu)
    assert (np.abs(got) <= mag * (1 + 1e-15)).all()
    for at in np.ndindex(4, 6):
        d = np.zeros((4, 6))
        d[at] = 1e-6
        assert abs(((Y.glu(h + d, gelu) - Y.glu(h - d, gelu)) * g).sum() / 2e-6 - got[at]) < 1e-8
    assert (Y.glu(np.array([[-80.0, 1.0]]), gelu) == 0).all()  # below 2^-100
