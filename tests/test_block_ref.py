"""The 64-bit references of the operators around the quantized products against differences and brute force."""
import numpy as np
import pytest

from tests import block_ref as ref

RNG = np.random.default_rng


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(sigmoid, renorm):
    rng = RNG(3)
    logits = rng.normal(size=(5, 12))
    logits[1, 3] = -np.inf
    ids, _, _ = ref.route(logits, 4, sigmoid, renorm)
    ids[2, 3] = -1
    dw = rng.normal(size=ids.shape)
    got = ref.route_backward(logits, ids, dw, sigmoid, renorm, 1.7)
    h = 1e-6
    for t, e in [(0, 0), (0, int(ids[0, 0])), (1, 4), (2, int(ids[2, 1])), (2, 7), (4, int(ids[4, 3]))]:
        a, b = logits.copy(), logits.copy()
        a[t, e] += h
        b[t, e] -= h
        diff = ((ref.route_weights(a, ids, sigmoid, renorm, 1.7) - ref.route_weights(b, ids, sigmoid, renorm, 1.7)) * dw).sum()
        # central differences: h^2 truncation and 1e-16 / h rounding of values of order 10
        assert abs(diff / (2 * h) - got[t, e]) < 1e-8
    assert got[1, 3] == 0.0


def test_route_of_closed_and_extreme_logits():
    inf = np.inf
    logits = np.array([[0.0, -inf, 1.0, np.nan], [-inf] * 4, [inf, 0.0, inf, 1.0], [-3e38, -3e38, -3e38, -3e38]])
    ids, w, _ = ref.route(logits, 3)
    assert ids.tolist() == [[2, 0, -1], [-1, -1, -1], [0, 2, 1], [0, 1, 2]]
    assert np.allclose(w[0], [np.e / (1 + np.e), 1 / (1 + np.e), 0]) and np.all(w[1] == 0)
    assert np.allclose(w[2], [0.5, 0.5, 0]) and np.allclose(w[3], 0.25)


@pytest.mark.parametrize("case", ["all", "no_post", "no_gate", "token_gate", "no_pre", "one_plus", "no_y"])
def test_block_norm_gradient_against_differences(case):
    rng = RNG(5)
    T, D, alpha, eps = 3, 8, 0.7, 1e-3
    x, y = rng.normal(size=(T, D)), rng.normal(size=(T, D))
    a = {"x": x, "y": None if case == "no_y" else y,
         "w_post": None if case in ("no_post", "no_y") else rng.normal(size=D),
         "gate": None if case in ("no_gate", "no_y") else rng.normal(size=(T, D) if case == "token_gate" else D),
         "w_pre": None if case == "no_pre" else rng.normal(size=D)}
    one_plus = case == "one_plus"
    dx_out = rng.normal(size=(T, D))
    dn = None if a["w_pre"] is None else rng.normal(size=(T, D))

    def loss(b):
        x1, n, _, _ = ref.block_norm(b["x"], b["y"], b["w_post"], b["gate"], b["w_pre"], alpha, eps, one_plus)
        return (x1 * dx_out).sum() + (0.0 if n is None else (n * dn).sum())

    got = ref.block_norm_backward(dx_out, dn, a["x"], a["y"], a["w_post"], a["gate"], a["w_pre"], alpha, eps, one_plus)
    h = 1e-5
    for name, v in a.items():
        if v is None:
            assert "d" + name not in got
            continue
        flat = np.empty(v.size)
        for i in range(v.size):
            up, down = dict(a), dict(a)
            up[name], down[name] = v.copy(), v.copy()
            up[name].flat[i] += h
            down[name].flat[i] -= h
            flat[i] = (loss(up) - loss(down)) / (2 * h)
        # third derivatives of order 100 times h^2, and 1e-15 / h of rounding
        np.testing.assert_allclose(got["d" + name].reshape(-1), flat, atol=1e-7)


def test_plan_by_hand():
    ids = np.array([[2, 0], [0, -1], [2, 7]])
    offsets, rows, pos = ref.plan(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert rows.tolist() == [1, 2, 0, 4, -1, -1]
    assert pos.tolist() == [[2, 0], [1, -1], [3, -1]]


def test_int8_rows_by_hand():
    q, s = ref.int8_rows(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1e-37, 0, 0, 0]], dtype=np.float32))
    assert q.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [0, 0, 0, 0]] and s.tolist() == [1.0, 0.0, 0.0]
