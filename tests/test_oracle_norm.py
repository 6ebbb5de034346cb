"""Pins of the norm's oracle: hand-made rows, and its gradients against
central differences of the forward in float64 (CPU)."""

import numpy as np
import pytest

from oracle import norm as onorm


def test_hand_made_rows():
    x = np.zeros((2, 128), np.float32)
    x[0, 0] = 16.0     # mean square 2
    r = onorm.rmsnorm(x, None, np.full(128, 0.5, np.float32), 2.0)
    assert r["rstd"][0] == 0.5 and r["rstd"][1] == np.float32(1 / np.sqrt(2.0))
    assert r["y"][0, 0] == 4.0 and not r["y"][0, 1:].any() and not r["y"][1].any()
    assert r["scale"][1, 0] == 1.0 and not r["q"][1].any()
    assert r["scale"][0, 0] == np.float32(4.0 / 448)


def test_residual_is_rounded_once():
    x = np.full((1, 128), 1.0, np.float32)
    s = onorm.rmsnorm(x, np.full((1, 128), 2.0 ** -9, np.float32), np.ones(128, np.float32), 1e-6)["sum"]
    assert np.all(s == 1.0)     # a quarter step: to the even neighbour


@pytest.mark.parametrize("T,d", [(1, 128), (3, 256)])
def test_backward_against_differences(T, d):
    rng = np.random.default_rng(T * d)
    h, w, up, dres = (rng.standard_normal(s) for s in ((T, d), (d,), (T, d), (T, d)))
    eps = 0.1

    def loss(h, w):
        rs = 1.0 / np.sqrt((h * h).mean(1) + eps)
        return float((up * h * rs[:, None] * w).sum() + (dres * h).sum())

    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    dh, dw = onorm.rmsnorm_backward(up, h, w, rstd, dres)
    step = 1e-5
    for t, c in [(0, 0), (T - 1, d - 1), (T // 2, 7)]:
        e = np.zeros((T, d)); e[t, c] = step
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dh[t, c]) < 1e-7
    for c in (0, 5, d - 1):
        e = np.zeros(d); e[c] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[c]) < 1e-7


def test_grad_norm():
    assert onorm.grad_norm([np.array([3.0]), np.array([]), np.array([4.0])], 10.0) == (5.0, 1.0)
    assert onorm.grad_norm([np.array([3.0, 4.0])], 1.0) == (5.0, 0.2)
