"""The operators between two recurrences in 64 bits, written from their definitions (numpy).

The magnitudes that tolerances scale with come from the same functions on absolute values.
"""
import numpy as np


# --------------------------------------------------------------------------- matrix product
def linear_fwd(xc, xs, wc, ws, bias):
    y = (xc.astype(np.float64) @ wc.astype(np.float64).T) * xs[:, None] * ws
    return y if bias is None else y + bias


def linear_bwd(xc, xs, wc, ws, dy):
    """dx, dweight, dbias."""
    xhat, what = xc * xs[:, None], wc * ws[:, None]
    return dy @ what, dy.T @ xhat, dy.sum(0)


# -------------------------------------------------------------------------- norms around a block
def gate(z, act):
    """act(z), its derivative, and the sum of the absolute values of the derivative's terms (silu's two
    cancel at z = -1.28)."""
    if act == 0:
        return np.ones_like(z), np.zeros_like(z), np.zeros_like(z)
    s = 1 / (1 + np.exp(-z))
    if act == 1:
        return z * s, s * (1 + z * (1 - s)), s * (1 + np.abs(z) * (1 - s))
    return s, s * (1 - s), s * (1 - s)


def gate_norm_fwd(x, z, w_post, alpha, res, w_pre, head, eps, act, first, post, pre, h=None):
    """t, v and what the backward needs; h: what the second norm reads (None: t)."""
    rows, d = x.shape
    head = head or d
    g, slope, terms = gate(z, act) if z is not None else (np.ones_like(x), np.zeros_like(x), np.zeros_like(x))
    u = x * g if first else x
    r1 = np.ones_like(x)
    wp = np.ones(d)
    if post:
        r1 = np.repeat(1 / np.sqrt((u ** 2).reshape(rows, -1, head).mean(2) + eps), head, 1)
        wp = np.tile(w_post, d // head) if w_post is not None else wp
    n = u * r1 * wp
    p = n if first else n * g
    a = alpha if alpha is not None else np.ones(d)
    t = a * p + (res if res is not None else 0)
    h = t if h is None else h
    r2, w2 = np.ones((rows, 1)), np.ones(d)
    if pre:
        r2 = 1 / np.sqrt((h ** 2).mean(1, keepdims=True) + eps)
        w2 = w_pre if w_pre is not None else w2
    v = h * r2 * w2 if pre else t
    return t, v, dict(g=g, slope=slope, terms=terms, u=u, r1=r1, wp=wp, n=n, p=p, a=a, h=h, r2=r2, w2=w2, head=head)


def gate_norm_bwd(x, keep, dy, dh, first, post, pre, mag=False):
    """dx, dz, dres, dw_post (per head column), dalpha, dw_pre.  mag: sums of the terms' absolute values."""
    k = {n: np.abs(v) for n, v in keep.items()} if mag else keep
    sign = 1.0 if mag else -1.0
    if mag:
        x, dy, k["slope"] = np.abs(x), np.abs(dy), k["terms"]
        dh = None if dh is None else np.abs(dh)
    rows, d = x.shape
    head = k["head"]
    G = dy
    if pre:
        c = dy * k["w2"]
        G = k["r2"] * (c + sign * k["h"] * k["r2"] ** 2 * (c * k["h"]).mean(1, keepdims=True))
    if dh is not None:
        G = G + dh
    dres, dalpha, dw_pre = G, (G * k["p"]).sum(0), (dy * k["h"] * k["r2"]).sum(0)
    G = G * k["a"]
    dz = G * k["n"] * k["slope"]
    if not first:
        G = G * k["g"]
    dw_post = (G * k["u"] * k["r1"]).sum(0).reshape(-1, head).sum(0)
    if post:
        c = G * k["wp"]
        m = np.repeat((c * k["u"]).reshape(rows, -1, head).mean(2), head, 1)
        G = k["r1"] * (c + sign * k["u"] * k["r1"] ** 2 * m)
    if first:
        dz = G * x * k["slope"]
        G = G * k["g"]
    return G, dz, dres, dw_post, dalpha, dw_pre
