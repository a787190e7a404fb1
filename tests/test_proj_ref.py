"""The 64-bit forms of the operators between two recurrences (tests/proj_ref.py) against differences of a loss."""
import numpy as np
import pytest

from tests import proj_ref as R

EPS = 1e-5


def differences(loss, value, at, step=1e-6):
    out = []
    for i in at:
        keep = value.flat[i]
        value.flat[i] = keep + step
        up = loss()
        value.flat[i] = keep - step
        down = loss()
        value.flat[i] = keep
        out.append((up - down) / (2 * step))
    return np.array(out)


def test_linear_gradients_are_those_of_the_values_that_the_codes_stand_for():
    g = np.random.default_rng(0)
    xc, wc = g.integers(-127, 128, (5, 16)), g.integers(-127, 128, (7, 16))
    xs, ws, bias, dy = g.random(5) * 0.01, g.random(7) * 0.01, g.normal(size=7), g.normal(size=(5, 7))
    x, w = xc * xs[:, None], wc * ws[:, None]
    np.testing.assert_allclose(R.linear_fwd(xc, xs, wc, ws, bias), x @ w.T + bias, rtol=1e-12)
    loss = lambda: (dy * (x @ w.T + bias)).sum()  # noqa: E731
    for got, value in zip(R.linear_bwd(xc, xs, wc, ws, dy), (x, w, bias)):
        at = range(0, value.size, 3)
        np.testing.assert_allclose(got.flat[list(at)], differences(loss, value, at), rtol=1e-6, atol=1e-8)


CASES = [(act, first, post, pre, head, res) for act in (0, 1, 2) for first in (0, 1) for post in (0, 1) for pre in (0, 1)
         for head in (0, 16) for res in (0, 1) if not (first and act == 0) and not (head and not post)]


@pytest.mark.parametrize("act,first,post,pre,head,res", CASES)
def test_gate_norm_gradients(act, first, post, pre, head, res):
    g = np.random.default_rng(1)
    rows, d = 3, 32
    x, z, w_post, alpha = g.normal(size=(rows, d)), g.normal(size=(rows, d)), 1 + g.normal(size=head or d) * 0.2, g.normal(size=d)
    r, w_pre, dy, dh = g.normal(size=(rows, d)), 1 + g.normal(size=d) * 0.2, g.normal(size=(rows, d)), g.normal(size=(rows, d))
    args = lambda: (x, z if act else None, w_post if post else None, alpha, r if res else None, w_pre if pre else None, head,  # noqa: E731
                    EPS, act, first, post, pre)

    def loss():
        t, v, _ = R.gate_norm_fwd(*args())
        return (dy * v).sum() + (dh * t).sum()

    keep = R.gate_norm_fwd(*args())[2]
    grads = R.gate_norm_bwd(x, keep, dy, dh, first, post, pre)
    wanted = dict(zip(("dx", "dz", "dres", "dw_post", "dalpha", "dw_pre"), grads))
    for name, value, there in (("dx", x, 1), ("dz", z, act), ("dres", r, res), ("dw_post", w_post, post), ("dalpha", alpha, 1),
                               ("dw_pre", w_pre, pre)):
        if there:
            at = range(0, value.size, 5)
            np.testing.assert_allclose(wanted[name].flat[list(at)], differences(loss, value, at), rtol=2e-6, atol=1e-7)
