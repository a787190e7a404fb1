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


@pytest.mark.parametrize("tx,tw", [(BF, F32), (F32, BF)])
def test_gradients_of_empty_sums_look_at_no_operand(tx, tw):
    """Zeros, without codes, scales, dy or a workspace, and for the empty gradient's address too."""
    spare = torch.full((64,), 7.0, device="cuda")
    for M, N, K in ((0, 200, 272), (3000, 0, 80), (0, 1, 16), (1, 0, 2048)):
        out = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (((M, K), tx), ((N, K), tw), ((N,), F32))]
        cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[tx], dw_dtype=CODE[tw])
        la.la_linear_bwd(cfg, None, None, None, None, None, *[v if v.numel() else spare.data_ptr() for v in out], None, 0)
        assert all((v == 0).all() for v in out) and (spare == 7.0).all()


# ---------------------------------------------------------------------- norms around a block
def gate_gradients(cfg, s, dy, dh, t):
    """The backward's outputs by name, s the forward's arguments."""
    rows, d = dy.shape
    nan = lambda *shape, dtype=F32: torch.full(shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    h = nan(rows, d, dtype=t)
    la.la_gate_norm_fwd(cfg, *s.values(), h, None)
    out = dict(dx=nan(rows, d, dtype=t), dz=nan(rows, d, dtype=t) if cfg.gate else None, dres=nan(rows, d, dtype=t),
               dw_post=nan(cfg.head or d) if cfg.post else None, dalpha=nan(d), dw_pre=nan(d) if cfg.pre else None)
    n = la.la_gate_norm_bwd_workspace_bytes(cfg)
    la.la_gate_norm_bwd(cfg, s["x"], s["z"], s["w_post"], s["alpha"], h if cfg.pre else None, s["w_pre"], dy, dh, *out.values(),
                        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n)
    return h, out


@pytest.mark.parametrize("t,d,head", [(BF, 64, 16), (F32, 512, 0), (F32, 520, 0), (BF, 2048, 128), (F32, 5120, 0), (BF, 10240, 512)])
@pytest.mark.parametrize("act,first", [(0, 0), (1, 0), (2, 1)])
@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("pre", [0, 1])
def test_gate_norm_bwd_infinities_and_nan(t, d, head, act, first, post, pre):
    """They go where the formula takes them: without the norm after the block to their own element and not
    beyond, with it to their head or row, with the next norm to the row; never to another row."""
    rows, g = 5, gen(3)
    head = head if post else 0
    s = dict(x=draw(g, rows, d, dtype=t), z=draw(g, rows, d, dtype=t) if act else None, w_post=draw(g, head or d, dtype=F32) if post else None,
             alpha=draw(g, d, dtype=F32), residual=draw(g, rows, d, dtype=t), w_pre=draw(g, d, dtype=F32) if pre else None)
    dy, dh = draw(g, rows, d, dtype=t), draw(g, rows, d, dtype=t)
    cfg = la.GateNormConfig(rows=rows, d=d, head=head, eps=1e-5, gate=act, gate_first=first, post=post, pre=pre, x_dtype=CODE[t], out_dtype=CODE[t])
    clean = gate_gradients(cfg, s, dy, dh, t)[1]
    bad = {1: (8, float("inf")), 2: (d - 1, float("nan")), 3: (9, float("-inf"))}
    for r, (c, v) in bad.items():
        s["x"][r, c] = v
    h, out = gate_gradients(cfg, s, dy, dh, t)
    for name in ("dx", "dz", "dres"):
        if out[name] is not None:
            assert torch.equal(out[name][[0, 4]], clean[name][[0, 4]]), name
    if post:
        width = head or d
        for r, (c, _) in bad.items():
            at = c // width * width
            assert out["dx"][r, at:at + width].isnan().all()
            if not pre:
                keep = [k for k in range(d) if not at <= k < at + width]
                assert torch.equal(out["dx"][r, keep], clean["dx"][r, keep])
        return
    if pre:
        assert all(out["dx"][r].isnan().all() for r in bad)
        return
    with np.errstate(invalid="ignore"):
        keep = R.gate_norm_fwd(*[None if v is None else np64(v) for v in s.values()], 0, 1e-5, act, first, 0, 0)[2]
        want = R.gate_norm_bwd(np64(s["x"]), keep, np64(dy), np64(dh), first, 0, 0)
    for name, w in zip(("dx", "dz", "dres"), want):
        if out[name] is None:
            continue
        assert np.array_equal(np.isnan(w), np.isnan(np64(out[name]))), name  # (a gate of NaN times x: no NaN in z here)
        fine = np.isfinite(w)
        assert np.array_equal(w[~fine & ~np.isnan(w)], np64(out[name])[~fine & ~np.isnan(w)]), name
        assert torch.equal(out[name][torch.from_numpy(fine).cuda()], clean[name][torch.from_numpy(fine).cuda()]), name
