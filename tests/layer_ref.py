"""The layer operators in 64 bits, written from their definitions, token by token (numpy).

Arrays carry one sequence: x [T, H, P], dt [T, H], b and c [T, G, N], S [H, N, P]; convolution
rows [T, C], states [W-1, C].  The magnitudes that tolerances scale with come from the same
functions on absolute values: every output is then the sum of its terms' absolute values.
"""
import numpy as np


def silu(z):
    return z / (1 + np.exp(-z))


def dsilu(z):
    s = 1 / (1 + np.exp(-z))
    return s * (1 + z * (1 - s))


# ------------------------------------------------------------------------------- convolution
def conv_pre(x, w, bias, s0):
    W = w.shape[1]
    z = np.concatenate([s0, x])
    return z, bias + sum(z[j:j + len(x)] * w[:, j] for j in range(W))


def conv_fwd(x, w, bias, s0, act):
    z, pre = conv_pre(x, w, bias, s0)
    return (silu(pre) if act else pre), z[len(x):]


def conv_bwd(x, w, bias, s0, dy, dsT, act, pre=None):
    """pre: the values at which act's derivative is taken (None: x's own)."""
    W, T = w.shape[1], len(x)
    z, p = conv_pre(x, w, bias, s0)
    p = p if pre is None else pre
    dp = dy * (np.abs(dsilu(p)) if pre is not None else dsilu(p)) if act else dy
    dz = np.zeros_like(z)
    dz[T:] += dsT
    for j in range(W):
        dz[j:j + T] += dp * w[:, j]
    dw = np.stack([(dp * z[j:j + T]).sum(0) for j in range(W)], 1)
    return dz[W - 1:], dw, dp.sum(0), dz[:W - 1]


# -------------------------------------------------------------------------------------- scan
def softplus(z):
    return np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))


def steps(dt, bias, sp):
    z = dt + bias
    return z, (softplus(z) if sp else z)


def scan_fwd(x, delta, A, b, c, D, S0):
    H, G = x.shape[1], b.shape[1]
    of = np.arange(H) // (H // G)
    S, y = S0.copy(), np.zeros_like(x)
    states = [S]
    for t in range(len(x)):
        S = np.exp(delta[t] * A)[:, None, None] * S + (delta[t][:, None] * b[t][of])[:, :, None] * x[t][:, None, :]
        states.append(S)
        y[t] = np.einsum("hnp,hn->hp", S, c[t][of]) + D[:, None] * x[t]
    return y, S, states


def scan_bwd(x, z, delta, A, b, c, D, S0, dy, dST, sp, A_sum=None):
    """A_sum: the rates in the decay's share of dDelta (|A| for magnitudes)."""
    H, G = x.shape[1], b.shape[1]
    rep = H // G
    of = np.arange(H) // rep
    A_sum = A if A_sum is None else A_sum
    _, _, states = scan_fwd(x, delta, A, b, c, D, S0)
    dS = dST.copy()
    dx, dd, rate = np.zeros_like(x), np.zeros_like(delta), np.zeros_like(delta)
    db, dc = np.zeros_like(b), np.zeros_like(c)
    for t in reversed(range(len(x))):
        a = np.exp(delta[t] * A)
        dc[t] = np.einsum("hnp,hp->hn", states[t + 1], dy[t]).reshape(G, rep, -1).sum(1)
        dS = dS + c[t][of][:, :, None] * dy[t][:, None, :]
        into = np.einsum("hnp,hn->hp", dS, b[t][of])
        dx[t] = delta[t][:, None] * into + D[:, None] * dy[t]
        db[t] = (delta[t][:, None] * np.einsum("hnp,hp->hn", dS, x[t])).reshape(G, rep, -1).sum(1)
        rate[t] = a * (dS * states[t]).sum((1, 2))
        dd[t] = (into * x[t]).sum(1)
        dS = a[:, None, None] * dS
    dd = dd + A_sum * rate
    sg = 1 / (1 + np.exp(-z)) if sp else np.ones_like(z)
    ddt = dd * sg
    return dict(dx=dx, ddt=ddt, dA=(rate * delta).sum(0), db=db, dc=dc, dD=(dy * x).sum((0, 2)), ddt_bias=ddt.sum(0),
                dS0=dS), rate


# -------------------------------------------------------------------------------------- norm
def norm_fwd(h, w, eps):
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h * r * w, r


def norm_bwd(h, w, eps, dy, dres):
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = dy * w
    return dres + r * (g - h * r * r * (g * h).mean(1, keepdims=True)), (dy * h * r).sum(0)


def e4m3_grid():
    """The non-negative finite values of 4 exponent and 3 mantissa bits."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) / 8 * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:-1])  # the last is NaN's code


def codec(n, group, kind):
    """(value stood for, scale, distance of n/s to the nearest rounding border) per element."""
    rows, d = n.shape
    g = group or d
    v = n.reshape(rows, d // g, g)
    s = np.abs(v).max(2, keepdims=True) / (127.0 if kind == "int8" else 448.0)
    s = np.where(s == 0, 1.0, s)
    q = v / s
    if kind == "int8":
        code = np.clip(np.rint(q), -127, 127)
        step = np.ones_like(q)
    else:
        grid = e4m3_grid()
        i = np.clip(np.searchsorted(grid, np.abs(q)), 1, len(grid) - 1)
        lo, hi = grid[i - 1], grid[i]
        up = (np.abs(q) - lo > hi - np.abs(q)) | ((np.abs(q) - lo == hi - np.abs(q)) & (i % 2 == 0))
        code = np.sign(q) * np.where(up, hi, lo)
        step = hi - lo
    return (code * s).reshape(rows, d), s[:, :, 0], (step * s).reshape(rows, d)
