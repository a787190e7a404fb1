"""The operators between two recurrences on the GPU where their values cancel, are not finite, or sizes reach
the larger tiles and later rows of a workgroup; against the 64-bit forms (tests/proj_ref.py) with the tolerances
derived in test_gpu_proj.py.
"""
import numpy as np
import pytest
import torch

import quantized_state_qat_amd as la
from tests import proj_ref as R
from tests.test_gpu_proj import BF, CODE, F32, close, codes, draw, gen, np64, wider

pytestmark = pytest.mark.gpu


def gradients(cfg, xc, xs, wc, ws, dy, tx, tw):
    """dx, dweight, dbias by the library."""
    n = la.la_linear_bwd_workspace_bytes(cfg)
    out = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in (((cfg.M, cfg.K), tx), ((cfg.N, cfg.K), tw), ((cfg.N,), F32))]
    la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, *out, torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n)
    return out


# --------------------------------------------------------------------------- matrix product
@pytest.mark.parametrize("t", [BF, F32])
def test_gradients_of_terms_that_cancel(t):
    """Two terms that differ in the 13th bit of their scales: what is left is exact in both parts of FP16 (the
    second's a subnormal one in the last token's row), in every product and in a bf16 result."""
    M, N, K = 40, 48, 32
    g = gen(1)
    a = torch.exp2(torch.randint(-6, 7, (M, N // 2), generator=g).float()) * (torch.randint(0, 2, (M, N // 2), generator=g) * 2 - 1)
    # dx: each pair of neighbouring channels has the same dy and opposite codes, in one column of its own
    dy = a.repeat_interleave(2, 1).cuda()
    dy[-1] = 2.0 ** -17
    dy[-1, 0:2] = 1.0
    ws = torch.ones(N, device="cuda")
    ws[::2] += 2.0 ** -12
    wc = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    pair = torch.arange(N // 2, device="cuda")
    wc[2 * pair, pair], wc[2 * pair + 1, pair] = 1, -1
    xc, xs = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[t], out_dtype=la.LA_F32, dw_dtype=CODE[t])
    dx = gradients(cfg, xc, xs, wc, ws, dy, t, t)[0]
    want = torch.zeros(M, K, device="cuda")
    want[:, :N // 2] = dy[:, ::2] * 2.0 ** -12
    assert torch.equal(dx.float(), want)
    # dweight: the same of neighbouring tokens
    dy = a.repeat_interleave(2, 1).T.contiguous()[:, :M].cuda()  # [N][M]: N tokens, M channels
    xs, ws = ws, torch.ones(M, device="cuda")
    xc, wc = wc, torch.zeros(M, K, dtype=torch.int8, device="cuda")
    cfg = la.LinearConfig(M=N, N=M, K=K, x_dtype=CODE[t], out_dtype=la.LA_F32, dw_dtype=CODE[t])
    dw = gradients(cfg, xc, xs, wc, ws, dy, t, t)[1]
    want = torch.zeros(M, K, device="cuda")
    want[:, :N // 2] = dy[::2].T * 2.0 ** -12
    assert torch.equal(dw.float(), want)


@pytest.mark.parametrize("M,N,K,t,tx,tw", [(300, 264, 144, BF, BF, BF), (65, 130, 272, F32, BF, F32), (33, 2000, 528, BF, F32, BF)])
def test_gradients_keep_22_bits_of_dy_under_every_type(M, N, K, t, tx, tw):
    """dy s: two FP32 roundings and two parts of FP16, 2^-22 + 2^-23 of the magnitude; n terms in FP32, each at most 2^-23."""
    g = gen(2)
    (xc, xs), (wc, ws) = codes(g, M, K), codes(g, N, K)
    dy = draw(g, M, N, dtype=t, scale=1e-3)
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[tx], out_dtype=CODE[t], dw_dtype=CODE[tw])
    got = gradients(cfg, xc, xs, wc, ws, dy, tx, tw)
    args = [np64(v) for v in (xc, xs, wc, ws, dy)]
    want, mag = R.linear_bwd(*args), R.linear_bwd(*[np.abs(v) for v in args])
    for name, terms, o, w, m in zip(("dx", "dweight"), (N, M), got, want, mag):
        close(o, w, m, 2.0 ** -22 + 2.0 ** -23 + terms * 2.0 ** -23, name)
