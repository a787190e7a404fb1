"""How many bits the layer operators hold between their inputs and outputs, by path, against the
64-bit forms (tests/layer_ref.py).

The scan's inputs here are positive and its sequences short: every output is a sum of few positive
terms, so an operand held in fewer bits than it should is not averaged away.  With T <= 5 tokens
and d_k = 16 a sum has at most T + 16 = 21 terms, 21 x 2^-24 < 2^-19 of it; a step, its decays and
their products with an operand are eight roundings or so more, 2^-21: 2^-18 with room for both.
Where an operand is two bf16 parts (y, dx, db and dc of bf16 inputs; 2^-17 each): 2^-16.
"""
import numpy as np
import pytest
import torch

import quantized_state_qat_amd as la
from tests import layer_ref as R
from tests.test_gpu_layer import BF, CODE, F32, Scan, close, draw, gen, np64

pytestmark = pytest.mark.gpu


class Positive(Scan):
    def __init__(self, *a, **k):
        super().__init__(*a, extra=0, **k)
        for t in (self.buf, self.dy, self.D, self.S0, self.dST):
            if t is not None:
                t.abs_()


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_scan_holds_its_operands(dtype, T, states):
    s = Positive(dtype, 3, T, 4, 2, 16, 64, states=states)
    w, m = s.reference(True)
    fine, parts = 2.0 ** -18, 2.0 ** -18 if dtype == F32 else 2.0 ** -16
    o = s.bwd()
    s.out = F32  # (the forward takes any output type)
    s.cfg.out_dtype = CODE[F32]
    y, ST = s.fwd()
    close(y.reshape(w["y"].shape), w["y"], m["y"], parts, "y")
    close(ST, w["S_T"], m["S_T"], fine, "S_T")
    for k in ("dx", "db", "dc"):
        close(o[k].reshape(w[k].shape), w[k], m[k], parts, k)
    for k in ("dS0", "dD", "ddt", "dA", "ddt_bias"):
        close(o[k].reshape(w[k].shape), w[k], m[k], fine, k)


@pytest.mark.parametrize("H,G,N,P", [(2, 1, 16, 64), (6, 2, 64, 192), (3, 3, 128, 128)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_first_tokens_decay_has_no_gradient_without_a_state(dtype, H, G, N, P):
    """One token and no state: its decay multiplies zeros, so dA is zero and ddt the step's own share,
    Delta's derivative times b.c x.dy.  Nothing of that product's rounding may reach dA."""
    s = Scan(dtype, 40, 1, H, G, N, P, states=False, extra=0, rate=16.0)
    o = s.bwd()
    assert not o["dA"].any()
    x, b, c, dy = (np64(t).reshape(40, n, -1) for t, n in ((s.x, H), (s.b, G), (s.c, G), (s.dy, H)))
    of = np.arange(H) // (H // G)
    z, _ = R.steps(np64(s.dt), np64(s.bias), 1)
    sg = 1 / (1 + np.exp(-z))
    want = (b * c).sum(2)[:, of] * (x * dy).sum(2) * sg
    mag = np.abs(b * c).sum(2)[:, of] * np.abs(x * dy).sum(2) * sg
    # two sums of at most 192 FP32 terms, a few roundings each
    close(o["ddt"].reshape(want.shape), want, mag, 2.0 ** -16, "ddt")
    close(o["ddt_bias"], want.sum(0), mag.sum(0), 2.0 ** -16, "ddt_bias")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_skip_gradient_is_summed_over_tokens_in_64_bits(dtype):
    """dy.x of a chunk's 64 tokens: 2^24 for one of them and 1 for each other, which an FP32 sum over
    the tokens loses (each by itself is exact); the sum of the exact values, rounded once."""
    for big in (0, 17, 63):
        s = Scan(dtype, 2, 130, 2, 1, 16, 64, extra=0)
        x, dy = torch.zeros(260, 2, 64, device="cuda"), torch.zeros(260, 2, 64, device="cuda")
        x[:, :, 5] = dy[:, :, 5] = 1.0
        x[64 + big, :, 5] = dy[64 + big, :, 5] = 2.0 ** 12
        s.x.copy_(x.reshape(260, -1))
        s.dy.copy_(dy.reshape(260, -1))
        want = float(np.float32(2.0 ** 24 + 259))
        assert (s.bwd()["dD"] == want).all()


def test_parameter_gradients_are_joined_in_64_bits():
    """Sums over tokens or rows of one 2^24 and ones that FP32 additions to it would lose.  A lane's
    own sum (32 tokens; the rows a grid apart) and a workgroup's are FP32 and rounded once: at most
    half a step of 2 each for the workgroup that holds the 2^24, and the result's own rounding."""
    T, C = 4096, 1024
    dy = torch.zeros(T, C, dtype=BF, device="cuda")
    dy[::32] = 1
    dy[1024 + 32] = 2.0 ** 24
    x, w = torch.ones(T, C, dtype=BF, device="cuda"), torch.ones(C, 2, device="cuda")
    cfg = la.ConvConfig(B=1, T=T, C=C, width=2, act=la.LA_ACT_NONE)
    n = la.la_conv_bwd_workspace_bytes(cfg)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(C, 2, device="cuda"), torch.empty(C, device="cuda")
    la.la_conv_bwd(cfg, x, w, None, None, dy, None, dx, dw, db, None, ws, n)
    want = 2.0 ** 24 + T // 32 - 1
    for got, v in ((db, want), (dw[:, 1], want), (dw[:, 0], want - 1)):  # (the first token has none before it)
        assert (got.double() - v).abs().max() <= 2, got.double() - v
    for rows, d in ((2048, 64), (512, 512)):  # 32 rows and 4 a workgroup, one for a lane
        h = torch.ones(rows, d, dtype=BF, device="cuda")
        dy = torch.ones(rows, d, dtype=BF, device="cuda")
        dy[100] = 2.0 ** 24
        cfg = la.NormConfig(rows=rows, d=d, eps=0.0)
        n = la.la_norm_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
        la.la_norm_bwd(cfg, h, None, dy, None, dx, dw, ws, n)
        assert (dw.double() - (2.0 ** 24 + rows - 1)).abs().max() <= 2, dw


def test_sigmoids_of_fp32_results_hold_for_large_arguments():
    """The convolution's SiLU and its derivative and the step's derivative, with FP32 results, over
    +-80: a sigmoid within 4 x 2^-23 of itself and four roundings more, 2^-20 of the terms."""
    n, C = 1024, 8
    x = torch.linspace(-80, 80, n * C, device="cuda").view(n, C)
    w = torch.zeros(C, 2, device="cuda")
    w[:, 1] = 1
    cfg = la.ConvConfig(B=1, T=n, C=C, width=2, x_dtype=CODE[F32])
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    la.la_conv_fwd(cfg, x, w, None, None, y)
    b = la.la_conv_bwd_workspace_bytes(cfg)
    ws = torch.empty(b, dtype=torch.uint8, device="cuda")
    la.la_conv_bwd(cfg, x, w, None, None, torch.ones_like(x), None, dx, dw, None, None, ws, b)
    v = np64(x)
    sg = 1 / (1 + np.exp(-v))
    close(y, v * sg, np.abs(v * sg), 2.0 ** -20, "y")
    close(dx, sg * (1 + v * (1 - sg)), sg * (1 + np.abs(v) * (1 - sg)), 2.0 ** -20, "dx")
    st, ys = torch.zeros(n, 1, C, device="cuda"), torch.empty_like(y)
    la.la_conv_step(la.ConvConfig(B=n, T=1, C=C, width=2, x_dtype=CODE[F32]), x, w, None, st, ys)
    assert torch.equal(ys, y)
    # the scan: one token of ones, b.c x.dy = 16 x 64 exactly
    H = 512
    dt = torch.linspace(-80, 80, H, device="cuda").view(1, H)
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    cfg = la.ScanConfig(B=1, T=1, H=H, G=1, d_k=16, d_v=64, x_dtype=CODE[F32], dt_dtype=CODE[F32], out_dtype=CODE[F32])
    b = la.la_scan_bwd_workspace_bytes(cfg)
    ws = torch.empty(b, dtype=torch.uint8, device="cuda")
    ddt, dA = torch.empty_like(dt), one(H)
    la.la_scan_bwd(cfg, one(1, H * 64), dt, -one(H), one(1, 16), one(1, 16), None, None, None, one(1, H * 64), None,
                   one(1, H * 64), ddt, dA, one(1, 16), one(1, 16), None, None, None, ws, b)
    want = 1024 / (1 + np.exp(-np64(dt)))
    close(ddt, want, want, 2.0 ** -20, "ddt")


def test_silu_at_infinities():
    """silu(inf) = inf, silu(-inf) = NaN as z / (1 + exp(-z)) has it, and NaN stays."""
    for dtype in (F32, BF):
        x = torch.tensor([float("inf"), float("-inf"), float("nan"), 300.0, -300.0, 0.0, -89.5, 89.5], device="cuda").to(dtype)
        w = torch.zeros(8, 2, device="cuda")
        w[:, 1] = 1
        y = torch.empty(1, 8, dtype=dtype, device="cuda")
        la.la_conv_fwd(la.ConvConfig(B=1, T=1, C=8, width=2, x_dtype=CODE[dtype]), x.view(1, 8), w, None, None, y)
        v = x.double()
        want = (v / (1 + torch.exp(-v))).to(dtype)
        assert torch.equal(y[0].isnan(), want.isnan())
        torch.testing.assert_close(y[0], want, rtol=0, atol=1e-30, equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rates_gradients_are_joined_in_64_bits(dtype):
    """Steps of 1 and a rate of 0: dA is the sum of (t - s) P_ts with P_ts = dy_t x_s.  x is 2^26 for
    token 0 and 1 for tokens 16 and 20, dy 2 for token 48 and -3 for token 32: the large terms cancel
    (48 x 2 = 32 x 3) and leave 32 x 2 - 16 x 3 + 28 x 2 - 12 x 3 = 36.  Row 48's sum 2 (2^26 + 2) and
    row 32's are not FP32 numbers; those of its 16 x 16 tiles are."""
    T, H = 64, 2
    x, dy, b = (torch.zeros(1, T, n, device="cuda") for n in (H * 64, H * 64, 16))
    x[0, 0, 5::64], x[0, 16, 5::64], x[0, 20, 5::64] = 2.0 ** 26, 1, 1
    dy[0, 48, 5::64], dy[0, 32, 5::64] = 2, -3
    b[:, :, 3] = 1
    x, dy, b = x.to(dtype), dy.to(dtype), b.to(dtype)
    cfg = la.ScanConfig(B=1, T=T, H=H, G=1, d_k=16, d_v=64, softplus=0, x_dtype=CODE[dtype], dt_dtype=CODE[F32], out_dtype=CODE[dtype])
    n = la.la_scan_bwd_workspace_bytes(cfg)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dt, A = torch.ones(1, T, H, device="cuda"), torch.zeros(H, device="cuda")
    ddt, dA = torch.empty_like(dt), torch.empty_like(A)
    la.la_scan_bwd(cfg, x, dt, A, b, b, None, None, None, dy, None, torch.empty_like(x), ddt, dA, torch.empty_like(b),
                   torch.empty_like(b), None, None, None, ws, n)
    assert (dA == 36).all(), dA
    # Delta_s: the column sums
    assert (ddt[0, 0] == -2.0 ** 26).all() and (ddt[0, 16] == -1).all() and (ddt[0, 20] == -1).all() and not ddt[0, 21:].any()
