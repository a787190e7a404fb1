"""The 64-bit forms of the layer operators pinned: gradients against central differences and
float64 autograd, the scan against a closed form, the codecs against their formats."""
import numpy as np
import pytest
import torch

from tests import layer_ref as R


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def num_grad(f, v, eps=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        old = v[i]
        v[i] = old + eps
        up = f()
        v[i] = old - eps
        g[i] = (up - f()) / (2 * eps)
        v[i] = old
    return g


@pytest.mark.parametrize("T,W,act", [(5, 4, 1), (1, 3, 1), (2, 4, 0), (7, 2, 1)])
def test_conv_gradients(T, W, act):
    x, w, bias, s0 = rnd(1, T, 3), rnd(2, 3, W), rnd(3, 3), rnd(4, W - 1, 3)
    dy, dsT = rnd(5, T, 3), rnd(6, W - 1, 3)

    def loss():
        y, s = R.conv_fwd(x, w, bias, s0, act)
        return (y * dy).sum() + (s * dsT).sum()

    got = R.conv_bwd(x, w, bias, s0, dy, dsT, act)
    for g, v in zip(got, (x, w, bias, s0)):
        np.testing.assert_allclose(g, num_grad(loss, v), rtol=1e-6, atol=1e-8)


def test_conv_is_a_correlation():
    x, w = rnd(7, 9, 2), rnd(8, 2, 4)
    y, _ = R.conv_fwd(x, w, np.zeros(2), np.zeros((3, 2)), 0)
    for c in range(2):
        np.testing.assert_allclose(y[:, c], np.convolve(x[:, c], w[c, ::-1])[:9], rtol=1e-12)


def scan_case(T=6, H=4, G=2, N=3, P=2, sp=1):
    z, delta = R.steps(rnd(11, T, H), rnd(12, H), sp)
    if not sp:
        z = delta = np.abs(z)
    return dict(x=rnd(10, T, H, P), z=z, delta=delta, A=-np.abs(rnd(13, H)), b=rnd(14, T, G, N), c=rnd(15, T, G, N),
                D=rnd(16, H), S0=rnd(17, H, N, P), dy=rnd(18, T, H, P), dST=rnd(19, H, N, P))


@pytest.mark.parametrize("sp", [0, 1])
def test_scan_gradients_by_autograd(sp):
    k = scan_case(sp=sp)
    t = {n: torch.tensor(k[n], dtype=torch.float64, requires_grad=True) for n in ("x", "z", "A", "b", "c", "D", "S0")}
    delta = torch.nn.functional.softplus(t["z"]) if sp else t["z"]
    S, loss = t["S0"], 0.0
    of = torch.arange(4) // 2
    for i in range(6):
        S = torch.exp(delta[i] * t["A"])[:, None, None] * S + (delta[i][:, None] * t["b"][i][of])[:, :, None] * t["x"][i][:, None, :]
        y = (S * t["c"][i][of][:, :, None]).sum(1) + t["D"][:, None] * t["x"][i]
        loss = loss + (y * torch.tensor(k["dy"][i])).sum()
    (loss + (S * torch.tensor(k["dST"])).sum()).backward()
    got, _ = R.scan_bwd(k["x"], k["z"], k["delta"], k["A"], k["b"], k["c"], k["D"], k["S0"], k["dy"], k["dST"], sp)
    for n, m in (("dx", "x"), ("ddt", "z"), ("dA", "A"), ("db", "b"), ("dc", "c"), ("dD", "D"), ("dS0", "S0")):
        np.testing.assert_allclose(got[n], t[m].grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=n)
    np.testing.assert_allclose(got["ddt_bias"], t["z"].grad.numpy().sum(0), rtol=1e-10)


def test_scan_closed_form():
    """One head, d_k = d_v = 1: y_t = c_t sum_s exp(sum_{s < i <= t} Delta_i A) Delta_s b_s x_s."""
    k = scan_case(H=1, G=1, N=1, P=1)
    y, S, _ = R.scan_fwd(k["x"], k["delta"], k["A"], k["b"], k["c"], k["D"], np.zeros((1, 1, 1)))
    d, a = k["delta"][:, 0], k["A"][0]
    for t in range(6):
        want = sum(np.exp(a * d[s + 1:t + 1].sum()) * d[s] * k["b"][s, 0, 0] * k["x"][s, 0, 0] for s in range(t + 1))
        np.testing.assert_allclose(y[t, 0, 0], k["c"][t, 0, 0] * want + k["D"][0] * k["x"][t, 0, 0], rtol=1e-12)


def test_norm_gradients():
    h, w, dy, dres = rnd(21, 3, 8), rnd(22, 8), rnd(23, 3, 8), rnd(24, 3, 8)

    def loss():
        return (R.norm_fwd(h, w, 1e-3)[0] * dy).sum() + (h * dres).sum()

    dx, dw = R.norm_bwd(h, w, 1e-3, dy, dres)
    np.testing.assert_allclose(dx, num_grad(loss, h), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, num_grad(loss, w), rtol=1e-6, atol=1e-8)


def test_codecs():
    grid = R.e4m3_grid()
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(grid, bits)
    n = rnd(25, 4, 64) * 3
    v, s, _ = R.codec(n, 16, "e4m3")
    want = torch.tensor(n.reshape(4, 4, 16) / s[:, :, None]).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_allclose(v.reshape(4, 4, 16), want * s[:, :, None], rtol=1e-12)
    v, s, step = R.codec(n, 0, "int8")
    assert np.abs(v - n).max() <= 0.5 * step.max() * (1 + 1e-12) and s.shape == (4, 1)
    v, s, _ = R.codec(np.zeros((1, 16)), 16, "int8")
    assert s[0, 0] == 1 and not v.any()
