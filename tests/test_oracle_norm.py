"""Pins of the block-norm oracle: closed forms, and every gradient against central differences of
the forward in fp64. No GPU."""
import numpy as np
import pytest

from oracle import norm


def test_closed_forms():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    f = norm.forward(x, pre=norm.RMS, eps=0.5)
    assert np.allclose(f["h"][0], x[0] / np.sqrt(12.5 + 0.5)) and (f["h"][1] == 0).all()
    f = norm.forward(x, pre=norm.LAYER, eps=0.0, w_pre=np.array([2.0, 1.0]), b_pre=np.array([1.0, 0.0]))
    assert np.allclose(f["h"][0], [-1.0, 1.0])
    o = np.array([[1.0, -1.0], [2.0, 2.0]])
    gate = np.array([[0.5, 0.5], [2.0, 0.0]])
    f = norm.forward(x, o, gate, 1, 0.1, norm.NONE, norm.NONE)
    assert np.allclose(f["r"], 0.1 * x + gate * o) and np.array_equal(f["h"], f["r"])


@pytest.mark.parametrize("post", [norm.NONE, norm.RMS, norm.LAYER])
@pytest.mark.parametrize("pre", [norm.NONE, norm.RMS, norm.LAYER])
@pytest.mark.parametrize("rows", [0, 1, 2, 9])
def test_gradients_against_differences(post, pre, rows):
    rng = np.random.default_rng(7 * post + pre + 100 * rows)
    t, d, eps = 5, 6, 1e-2
    p = {"r": rng.standard_normal((t, d)), "o": rng.standard_normal((t, d)) + 0.3, "alpha": np.array(0.8)}
    if rows:
        p["gate"] = rng.standard_normal((-(-t // rows), d))
    if post:
        p["w_post"], p["b_post"] = rng.standard_normal(d), rng.standard_normal(d)
    if pre:
        p["w_pre"], p["b_pre"] = rng.standard_normal(d), rng.standard_normal(d)
    dh, dr = rng.standard_normal((t, d)), rng.standard_normal((t, d))

    def loss(q):
        f = norm.forward(**q, gate_rows=rows or 1, post=post, pre=pre, eps=eps)
        return (f["h"] * dh).sum() + (f["r"] * dr).sum()

    f = norm.forward(**p, gate_rows=rows or 1, post=post, pre=pre, eps=eps)
    b = norm.backward(p["r"], f["r"], dh, dr, p["o"], p.get("gate"), rows or 1, float(p["alpha"]), post, pre, f["post"], f["pre"],
                      p.get("w_post"), p.get("b_post"), p.get("w_pre"), p.get("b_pre"))
    names = {"r": "dr", "o": "do", "alpha": "dscale", "gate": "dgate", "w_post": "dw_post", "b_post": "db_post", "w_pre": "dw_pre", "b_pre": "db_pre"}
    for k, v in p.items():
        got, step = np.asarray(b[names[k]]), 1e-6
        for i in np.ndindex(v.shape):
            up, down = {**p, k: v.copy()}, {**p, k: v.copy()}
            up[k][i] += step
            down[k][i] -= step
            # central differences: truncation O(step^2) and rounding 2^-52 |loss| / step, both < 1e-6
            assert abs((loss(up) - loss(down)) / (2 * step) - got[i]) < 2e-6 * (1 + abs(got[i])), (k, i)
