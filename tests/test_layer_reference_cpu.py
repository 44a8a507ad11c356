"""The 64-bit definitions that the gated linear recurrence and the q/k norm with rotation are
tested against, themselves held to closed forms and central differences."""

from __future__ import annotations

import numpy as np
import pytest

import layer_reference as ref


def _case(T=9, D=4, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((2, T, D)), -g.random((2, T, D)) * 2, g.standard_normal((2, D)),
            g.standard_normal((2, T, D)), g.standard_normal((2, D)))


def test_recurrence_against_its_unrolled_sum():
    x, la, h0, _, _ = _case()
    h = ref.scan(x, la, h0)
    for t in range(9):
        want = np.exp(la[:, :t + 1].sum(1)) * h0
        for j in range(t + 1):
            want = want + np.exp(la[:, j + 1:t + 1].sum(1)) * x[:, j]
        np.testing.assert_allclose(h[:, t], want, rtol=1e-12, atol=1e-14)


def test_recurrence_limits():
    x, la, h0, _, _ = _case()
    np.testing.assert_allclose(ref.scan(x, 0 * la, h0), np.cumsum(x, 1) + h0[:, None], rtol=1e-12)
    np.testing.assert_array_equal(ref.scan(x, np.full_like(la, -np.inf), h0), x)


def test_recurrence_gradients_against_differences():
    x, la, h0, d, dT = _case()
    loss = lambda x, la, h0: (lambda h: (h * d).sum() + (h[:, -1] * dT).sum())(  # noqa: E731
        ref.scan(x, la, h0))
    grads = ref.scan_backward(x, la, d, h0, dT)
    for i, grad in enumerate(grads):
        for at in np.ndindex(grad.shape):
            args = [[a.copy() for a in (x, la, h0)] for _ in range(2)]
            args[0][i][at] += 1e-6
            args[1][i][at] -= 1e-6
            np.testing.assert_allclose(grad[at], (loss(*args[0]) - loss(*args[1])) / 2e-6,
                                       rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation_gradients_against_differences(norm, interleaved):
    g = np.random.default_rng(1)
    x, w = g.standard_normal((1, 3, 2, 16)), g.standard_normal(16)
    d = g.standard_normal((1, 2, 3, 16))
    f, pos = np.array([1.0, 0.3, 0.1, 0.01]), np.array([[0, 5, 1000]])
    args = (pos, f, norm, 1e-3, interleaved)
    loss = lambda x, w: (ref.qk_one(x, w, *args)[0] * d).sum()  # noqa: E731
    dx, _, dw, _ = ref.qk_one_backward(x, w, d, *args)
    for grad, i in ((dx, 0), (dw, 1)):
        for at in np.ndindex(grad.shape):
            up, down = [x.copy(), w.copy()], [x.copy(), w.copy()]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            np.testing.assert_allclose(grad[at], (loss(*up) - loss(*down)) / 2e-6, rtol=1e-6,
                                       atol=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    g = np.random.default_rng(2)
    q, k = g.standard_normal((2, 1, 1, 1, 24))
    f = np.array([1.0, 0.2, 0.05, 0.003])
    turn = lambda y, p: ref.rotate(y, np.array([[p]]), f, interleaved)  # noqa: E731
    np.testing.assert_allclose(np.linalg.norm(turn(q, 77)), np.linalg.norm(q), rtol=1e-12)
    np.testing.assert_array_equal(turn(q, 77)[..., 8:], q[..., 8:])
    np.testing.assert_allclose((turn(q, 77) * turn(k, 70)).sum(), (turn(q, 7) * k).sum(),
                               rtol=1e-10)
    np.testing.assert_allclose(ref.rotate(turn(q, 77), np.array([[77]]), f, interleaved, back=True),
                               q, rtol=1e-12, atol=1e-14)


def test_unit_rows():
    x = np.random.default_rng(3).standard_normal((1, 2, 3, 8))
    y, _ = ref.qk_one(x, None, None, None, "l2", 1e-12, False)
    np.testing.assert_allclose((y * y).sum(-1), 1.0, rtol=1e-9)
    y, _ = ref.qk_one(x, None, None, None, "rms", 1e-12, False)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-9)
