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
