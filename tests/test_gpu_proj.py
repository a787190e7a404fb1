"""The operators between two recurrences on the GPU against their 64-bit forms (tests/proj_ref.py).

Tolerances, derived: an output may be off by half a step of its type (bf16 2^-8, fp32 2^-24 of the
value) plus a share of its magnitude, the sum of its terms' absolute values:
  product       the integer sum is exact; its conversion, two scales and the bias are four FP32
                roundings: 2^-22 of |product| + |bias|.
  gradients     a term's factor dy s is two FP32 roundings (2 x 2^-24) and then FP16, whose rounding
                is off by at most half a step, eps / 2 = 2^-11 of the value: one part for a bf16
                gradient, and for an FP32 one a second that rounds the first's remainder (at most
                2^-11) to 2^-11 of itself, 2^-22 together; a sum of n terms in FP32 is n roundings of at
                most 2^-23 (matrix cores may truncate), and the power of two is exact.
  dbias         FP32 sums of 64 terms (64 x 2^-24), then double.
"""
import numpy as np
import pytest
import torch

import quantized_state_qat_amd as la
from tests import proj_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: la.LA_BF16, F32: la.LA_F32}
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def draw(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, mag, share, name):
    half = HALF[got.dtype]
    got = np64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), name
    over = np.abs(got - want) - (half * 1.01 * np.abs(want) + share * mag + 1e-30)
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over.max() <= 0, (name, worst, got[worst], want[worst], mag[worst] if np.ndim(mag) else mag)


def wider(g, rows, width, extra, dtype, fill=None):
    """Rows of `width` inside wider rows: (whole, view)."""
    buf = draw(g, rows, width + extra, dtype=dtype) if fill is None else torch.full((rows, width + extra), fill, dtype=dtype, device="cuda")
    return buf, buf[:, :width]


# --------------------------------------------------------------------------- matrix product
def codes(g, rows, K, extra=0):
    c = torch.randint(-128, 128, (rows, K + extra), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    return c[:, :K], (torch.rand(rows, generator=g) * 0.02 + 1e-3).cuda()


LINEAR = [
    # M, N, K, y and dy, dx, dweight, extra columns of x, of y, bias
    (1, 1, 16, F32, F32, F32, 0, 0, F32),
    (1, 512, 2048, BF, BF, F32, 0, 0, None),
    (1, 33, 144, F32, BF, BF, 0, 0, BF),
    (2, 8, 64, BF, F32, F32, 16, 3, F32),
    (5, 1040, 80, BF, BF, BF, 0, 8, F32),
    (16, 264, 4096, BF, BF, F32, 0, 0, BF),
    (17, 2305, 48, F32, F32, F32, 48, 0, F32),
    (31, 65, 1040, BF, BF, F32, 0, 0, F32),
    (33, 96, 528, BF, F32, BF, 0, 0, None),
    (64, 64, 128, F32, F32, F32, 0, 0, None),
    (65, 130, 272, F32, BF, F32, 0, 2, F32),
    (127, 129, 112, BF, BF, BF, 0, 1, F32),
    (128, 200, 1040, BF, BF, F32, 0, 0, F32),
    (256, 2048, 256, BF, BF, F32, 0, 0, F32),
    (257, 255, 400, F32, F32, F32, 16, 5, BF),
    (777, 305, 1040, F32, F32, F32, 0, 0, F32),
    (1030, 776, 144, BF, BF, BF, 0, 0, F32),
    (2000, 24, 512, F32, F32, F32, 0, 0, None),
]


def linear_case(k):
    M, N, K, t, tx, tw, ex, ey, tb = LINEAR[k]
    g = gen(100 + k)
    xc, xs = codes(g, M, K, ex)
    wc, ws = codes(g, N, K)
    bias = draw(g, N, dtype=tb) if tb else None
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[tx], out_dtype=CODE[t], w_dtype=CODE[tb or F32], dw_dtype=CODE[tw],
                          ld_x=K + ex if ex else 0, ld_y=N + ey if ey else 0)
    return cfg, g, xc, xs, wc, ws, bias


@pytest.mark.parametrize("k", range(len(LINEAR)))
def test_linear_fwd(k):
    M, N, K, t, _, _, _, ey, _ = LINEAR[k]
    cfg, g, xc, xs, wc, ws, bias = linear_case(k)
    whole, y = wider(g, M, N, ey, t, fill=7.0)
    la.la_linear_fwd(cfg, xc, xs, wc, ws, bias, y)
    X, W, b = np64(xc), np64(wc), None if bias is None else np64(bias)
    want = R.linear_fwd(X, np64(xs), W, np64(ws), b)
    mag = np.abs(R.linear_fwd(X, np64(xs), W, np64(ws), None)) + (0 if b is None else np.abs(b))
    close(y, want, mag, 2.0 ** -22, "y")
    assert (whole[:, N:] == 7.0).all()  # the columns between the rows are not y's


@pytest.mark.parametrize("k", range(len(LINEAR)))
def test_linear_bwd(k):
    M, N, K, t, tx, tw, _, ey, _ = LINEAR[k]
    cfg, g, xc, xs, wc, ws, _ = linear_case(k)
    # magnitudes of tokens over eight binades
    dy = wider(g, M, N, ey, t)[1]
    dy.mul_((torch.exp2(torch.rand(M, 1, generator=g) * 8 - 14)).cuda().to(t))
    dx = torch.full((M, K), float("nan"), dtype=tx, device="cuda")
    dw = torch.full((N, K), float("nan"), dtype=tw, device="cuda")
    db = torch.full((N,), float("nan"), device="cuda")
    n = la.la_linear_bwd_workspace_bytes(cfg)
    ws_ = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # (NaN in every type)
    la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, dx, dw, db, ws_, n)
    args = [np64(v) for v in (xc, xs, wc, ws, dy)]
    want, mag = R.linear_bwd(*args), R.linear_bwd(*[np.abs(a) for a in args])
    held = lambda typ, terms: (2.0 ** -11 if typ is BF else 2.0 ** -22) + 2.0 ** -23 + terms * 2.0 ** -23  # noqa: E731
    close(dx, want[0], mag[0], held(tx, N), "dx")
    close(dw, want[1], mag[1], held(tw, M), "dweight")
    close(db, want[2], mag[2], 2.0 ** -18, "dbias")
    # each gradient alone is the same
    for k, out in enumerate((dx, dw, db)):
        again = torch.full_like(out, float("nan"))
        ws_.fill_(0xFF)
        la.la_linear_bwd(cfg, xc if k == 1 else None, xs if k == 1 else None, wc if k == 0 else None, ws if k == 0 else None, dy,
                         *[again if i == k else None for i in range(3)], ws_, n)
        assert torch.equal(again, out), k
