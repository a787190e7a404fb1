"""The operators between two recurrences on the GPU where their values cancel, are not finite, or sizes reach
the larger tiles and later rows of a workgroup; against the 64-bit forms (tests/proj_ref.py) with the tolerances
derived in test_gpu_proj.py.
"""
import numpy as np
import pytest
import torch

import quantized_state_qat_amd as la
from tests import proj_ref as R
from tests.proj_tiles import FORWARD, GRADIENTS
from tests.test_gpu_proj import BF, CODE, F32, close, codes, draw, gen, np64, two_norm, wider

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


# Every way of cutting the products (proj_tiles.py says which shape takes which), on operands without a zero block.
@pytest.mark.parametrize("M,N,K", [c[:3] for c in FORWARD])
@pytest.mark.parametrize("t", [BF, F32])
def test_forward_of_every_tiling(M, N, K, t):
    """Bit for bit: the sum is exact, its conversion, two products and an addition are rounded as written."""
    g = gen(M + N + K)
    (xc, xs), (wc, ws) = codes(g, M, K), codes(g, N, K)
    bias = draw(g, N, dtype=F32)
    whole, y = wider(g, M, N, 3, t, fill=7.0)
    la.la_linear_fwd(la.LinearConfig(M=M, N=N, K=K, out_dtype=CODE[t], ld_y=N + 3), xc, xs, wc, ws, bias, y)
    exact = torch.mm(xc.double(), wc.double().t().contiguous())
    assert torch.equal(y, (exact.float() * xs[:, None] * ws + bias).to(t))
    assert (whole[:, N:] == 7.0).all()
    tight = torch.full((M, N), float("nan"), dtype=t, device="cuda")
    la.la_linear_fwd(la.LinearConfig(M=M, N=N, K=K, out_dtype=CODE[t]), xc, xs, wc, ws, None, tight)
    assert torch.equal(tight, (exact.float() * xs[:, None] * ws).to(t))


@pytest.mark.parametrize("M,N,K,dx,dw", [c[:5] for c in GRADIENTS])
@pytest.mark.parametrize("t", [BF, F32])
def test_gradients_of_every_tiling(M, N, K, dx, dw, t):
    """Against 64-bit products on the GPU.  Beside each element's bound the 2-norm of what a result is off by: operands 2^-22 + 2^-23,
    a part's sum of n terms is n / 8 additions (16 products each, of two parts), each off by 2^-23 of a partial sum that grows
    to the result, its own rounding (2^-24, or 2^-9 on average for bf16)."""
    g = gen(M + N + K)
    (xc, xs), (wc, ws) = codes(g, M, K), codes(g, N, K)
    dy = draw(g, M, N, dtype=t) * torch.exp2(torch.randint(-8, 9, (M, 1), generator=g).float()).cuda().to(t)
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[t], out_dtype=CODE[t], dw_dtype=CODE[t])
    got = gradients(cfg, xc, xs, wc, ws, dy, t, t)
    d, x, w = dy.double(), xc.double() * xs.double()[:, None], wc.double() * ws.double()[:, None]
    half = 2.0 ** -8 if t is BF else 2.0 ** -24
    for name, o, a, b, n, parts in (("dx", got[0], d, w, N, dx[1]), ("dweight", got[1], d.t().contiguous(), x, M, dw[1])):
        want, mag = torch.mm(a, b), torch.mm(a.abs(), b.abs())
        off = (o.double() - want).abs()
        assert (off <= half * 1.01 * want.abs() + (2.0 ** -22 + 2.0 ** -23 + n * 2.0 ** -23) * mag).all(), name
        bound = 2.0 ** -22 + 2.0 ** -23 + n / parts / 8 * 2.0 ** -23 + half / 2
        assert off.norm() <= bound * want.norm(), (name, float(off.norm() / want.norm()), bound)
    # dbias: at most 64 terms in FP32, the rest in double
    off = (got[2].double() - d.sum(0)).abs()
    assert (off <= 2.0 ** -24 * d.sum(0).abs() + 64 * 2.0 ** -24 * d.abs().sum(0)).all()


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


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("codec", ["int8", "e4m3"])
@pytest.mark.parametrize("d,group", [(2048, 0), (512, 64), (4096, 128)])
def test_codes_of_a_row_are_the_codec_of_its_values(t, codec, d, group):
    """Without norms v is x itself: s = max / 127 (448) and code = rne(v / s), quotients rounded to FP32 as written,
    so every code is known (8 million values, some of them within 2^-23 of a tie)."""
    rows = (1 << 23) // d
    x = draw(gen(5), rows, d, dtype=t)
    cfg = la.GateNormConfig(rows=rows, d=d, post=0, qdq=la.LA_QDQ_INT8_GROUP if codec == "int8" else la.LA_QDQ_E4M3_TILE, group=group, x_dtype=CODE[t])
    c = torch.empty(rows, d, dtype=torch.int8 if codec == "int8" else torch.float8_e4m3fn, device="cuda")
    s = torch.empty(rows, d // (group or d), device="cuda")
    la.la_gate_norm_fwd(cfg, x, None, None, None, None, None, None, None, c, s)
    v = x.float().cpu().unflatten(1, (-1, group or d))
    scale = v.abs().amax(2) / (127.0 if codec == "int8" else 448.0)
    assert torch.equal(s.cpu(), scale)
    q = (v / scale[:, :, None]).flatten(1)
    if codec == "int8":
        assert torch.equal(c.cpu(), torch.round(q).to(torch.int8))
    else:  # (a zero's sign aside)
        assert torch.equal(c.cpu().float(), q.clamp(-448, 448).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("codec", ["int8", "e4m3"])
def test_codes_beside_the_residual_norm_s(t, codec):
    """The formula that both operators have, residual, norm and codes: h is the same, a scale within what the
    norms may be off by (2^-17, as the tolerances of the forward), and a code moves to its neighbour only where its
    quotient lies as near to the middle between the two."""
    rows, d = 1024, 2048
    g = gen(6)
    x, res, w = draw(g, rows, d, dtype=t), draw(g, rows, d, dtype=t, scale=3.0), draw(g, d, dtype=F32, scale=0.2) + 1
    qdq, top = (la.LA_QDQ_INT8_GROUP, 127) if codec == "int8" else (la.LA_QDQ_E4M3_TILE, 448)
    new = lambda dtype, *shape: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    ct = torch.int8 if codec == "int8" else torch.float8_e4m3fn
    h1, h2, c1, c2, s1, s2 = new(t, rows, d), new(t, rows, d), new(ct, rows, d), new(ct, rows, d), new(F32, rows), new(F32, rows)
    la.la_norm_fwd(la.NormConfig(rows=rows, d=d, eps=1e-6, qdq=qdq, group=0, x_dtype=CODE[t]), x, res, w, h1, None, c1, s1)
    la.la_gate_norm_fwd(la.GateNormConfig(rows=rows, d=d, eps=1e-6, post=0, pre=1, qdq=qdq, x_dtype=CODE[t]), x, None, None, None, res, w, h2, None, c2, s2)
    assert torch.equal(h1, h2)
    a, b = np64(s1), np64(s2)
    assert (np.abs(a - b) <= 2.0 ** -17 * a).all()
    h = np64(h1)
    q = h / np.sqrt((h ** 2).mean(1, keepdims=True) + 1e-6) * np64(w) / a[:, None]
    k1, k2 = np64(c1.float()), np64(c2.float())
    off = k1 != k2
    # either code is a nearest one of a quotient that far away
    step = 1.0 if codec == "int8" else np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -20))), -6) - 3)
    assert (np.abs(k1 - k2)[off] <= 2.0001 * np.broadcast_to(step, q.shape)[off]).all()
    assert (np.abs(np.abs(k1 - q) - np.abs(k2 - q))[off] <= 2 * 2.0 ** -16 * np.abs(q)[off]).all()
    assert off.mean() <= 2.0 ** -16 * top * 4


@pytest.mark.parametrize("d,head", [(64, 16), (512, 64), (520, 0), (2048, 128), (4096, 0), (16384, 0)])
def test_h_without_codes_is_rounded_stepwise(d, head):
    """As in front of codes: with squares whose sums are exact in any order, h is the formula's in FP32, operation by
    operation, and h of any values is the same with codes and without."""
    rows, g = 65, gen(7)
    x = (torch.exp2(torch.randint(-2, 3, (rows, d), generator=g).float()) * (torch.randint(0, 2, (rows, d), generator=g) * 2 - 1)).cuda().to(BF)
    w, al, res = draw(g, head or d, dtype=F32), draw(g, d, dtype=F32), draw(g, rows, d)
    h = torch.empty_like(x)
    cfg = la.GateNormConfig(rows=rows, d=d, head=head, eps=2.0 ** -6, pre=1)
    la.la_gate_norm_fwd(cfg, x, None, w, al, res, None, h, None)
    f = x.float().cpu().unflatten(-1, (-1, head or d))
    rms = ((f.double() ** 2).mean(-1, keepdim=True).float() + 2.0 ** -6).double().sqrt().float()
    p = ((f / rms) * w.cpu()).flatten(-2)
    assert torch.equal(h.cpu(), (res.float().cpu() + al.cpu() * p).to(BF))
    x, z, hs = draw(g, 4096, d), draw(g, 4096, d), []
    for qdq in (0, la.LA_QDQ_INT8_GROUP):
        hs.append(torch.empty_like(x))
        cfg = la.GateNormConfig(rows=4096, d=d, head=head, gate=la.LA_GATE_SILU, pre=1, qdq=qdq)
        la.la_gate_norm_fwd(cfg, x, z, w, al, None, None, hs[-1], None)
    assert torch.equal(*hs)


# The backward's workgroups walk rows a grid apart: 256 x 1 to 256 x 3 workgroups of a row, or of 4 to 32 rows up
# to 512 columns.  Each case has two whole rounds of them and a part of a third.
# type, rows, d, head, gate, first, post, pre, residual
WALKS = [
    (F32, 36001, 64, 16, 2, 0, 1, 1, 1),
    (BF, 52000, 64, 0, 1, 0, 1, 0, 0),
    (F32, 26003, 128, 128, 0, 0, 1, 1, 1),
    (BF, 9001, 256, 256, 1, 1, 1, 1, 0),
    (F32, 4500, 512, 64, 1, 0, 1, 1, 1),
    (F32, 6200, 512, 0, 0, 0, 0, 1, 1),
    (BF, 3500, 1024, 0, 0, 0, 1, 1, 1),
    (F32, 1300, 1152, 0, 1, 1, 1, 1, 1),
    (BF, 1700, 2048, 128, 2, 0, 1, 0, 0),
    (F32, 1701, 2048, 0, 0, 0, 0, 1, 1),
    (F32, 1100, 2048, 0, 1, 0, 1, 1, 1),
    (BF, 1100, 2304, 0, 0, 0, 1, 0, 1),
    (F32, 600, 4096, 32, 1, 0, 1, 1, 0),
    (BF, 600, 8192, 512, 1, 1, 1, 1, 1),
    (F32, 600, 8192, 0, 2, 0, 1, 1, 1),
    (F32, 530, 10240, 0, 0, 0, 1, 1, 1),
    (BF, 530, 16384, 64, 1, 0, 1, 1, 1),
]


@pytest.mark.parametrize("k", range(len(WALKS)))
def test_gate_norm_bwd_of_many_rows_a_workgroup(k):
    """Every row and the parameters' sums against 64 bits.  Tolerances as in test_gpu_proj.py; a lane's share of a
    sum is three rows, and up to 32 of them are joined in double."""
    t, rows, d, head, act, first, post, pre, res = WALKS[k]
    g = gen(700 + k)
    s = dict(x=draw(g, rows, d, dtype=t), z=draw(g, rows, d, dtype=t) if act else None,
             w_post=draw(g, head or d, dtype=F32, scale=0.2) + 1 if post else None, alpha=draw(g, d, dtype=F32, scale=0.5),
             residual=draw(g, rows, d, dtype=t, scale=2.0) if res else None, w_pre=draw(g, d, dtype=F32, scale=0.2) + 1 if pre else None)
    dy, dh = draw(g, rows, d, dtype=t), draw(g, rows, d, dtype=t) if res else None
    cfg = la.GateNormConfig(rows=rows, d=d, head=head, eps=1e-5, gate=act, gate_first=first, post=post, pre=pre, x_dtype=CODE[t], out_dtype=CODE[t])
    h, out = gate_gradients(cfg, s, dy, dh, t)
    sums = {n: np.zeros(out[n].numel()) for n in ("dw_post", "dalpha", "dw_pre") if out[n] is not None}
    mags = {n: np.zeros_like(v) for n, v in sums.items()}
    step = max(1, (1 << 22) // d)
    for a in range(0, rows, step):
        cut = slice(a, a + step)
        part = {n: None if v is None else np64(v[cut] if n in ("x", "z", "residual") else v) for n, v in s.items()}
        keep = R.gate_norm_fwd(*part.values(), head, 1e-5, act, first, post, pre, np64(h[cut]) if pre else None)[2]
        args = (part["x"], keep, np64(dy[cut]), None if dh is None else np64(dh[cut]), first, post, pre)
        want, mag = R.gate_norm_bwd(*args), R.gate_norm_bwd(*args, mag=True)
        for name, w, m in zip(out, want, mag):
            if name in sums:
                sums[name] += w
                mags[name] += m
            elif out[name] is not None:
                close(out[name][cut], w, m, 2.0 ** -15, name)
                two_norm(out[name][cut], w, 2.0 ** -20 * max(1.0, np.linalg.norm(m) / np.linalg.norm(w)), name)
    for name, w in sums.items():
        close(out[name], w, mags[name], 2.0 ** -15, name)
        # (independent errors of many rows: their share of a sum shrinks with the root of its terms)
        assert np.linalg.norm(np64(out[name]) - w) <= 2.0 ** -20 * np.linalg.norm(mags[name]), name


def test_parameter_sums_over_many_rows_are_not_all_fp32():
    """Behind 2^24 in the first rows, ones are lost in FP32 sums: of at most 128 rows, 2^-17 of the sum."""
    rows, d = 1 << 16, 8192
    x = torch.ones(rows, d, dtype=BF, device="cuda")
    dy = torch.ones(rows, d, dtype=BF, device="cuda")
    dy[:256] = 2.0 ** 24
    cfg = la.GateNormConfig(rows=rows, d=d, post=0)
    n = la.la_gate_norm_bwd_workspace_bytes(cfg)
    dalpha = torch.empty(d, device="cuda")
    la.la_gate_norm_bwd(cfg, x, None, None, None, None, None, dy, None, torch.empty_like(x), None, None, None, dalpha, None,
                        torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    want = 256 * 2.0 ** 24 + rows - 256
    assert ((dalpha.double() - want).abs() <= (2.0 ** -17 + 2.0 ** -24) * want).all()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("first", [0, 1])
def test_gates_far_from_zero(t, act, first):
    """The gate's derivative keeps its bits where the gate is all but open or shut: dz within 2^-15 of the magnitude as
    near zero, z over -60 to 60."""
    rows, d, g = 64, 512, gen(8)
    s = dict(x=draw(g, rows, d, dtype=t), z=torch.linspace(-60, 60, rows * d, device="cuda")[torch.randperm(rows * d, generator=g).cuda()].view(rows, d).to(t),
             w_post=None, alpha=None, residual=None, w_pre=None)
    dy = draw(g, rows, d, dtype=t)
    cfg = la.GateNormConfig(rows=rows, d=d, eps=1e-5, gate=act, gate_first=first, post=0, x_dtype=CODE[t], out_dtype=CODE[t])
    out = gate_gradients(cfg, s, dy, None, t)[1]
    keep = R.gate_norm_fwd(np64(s["x"]), np64(s["z"]), None, None, None, None, 0, 1e-5, act, first, 0, 0)[2]
    if act == 2:  # (64 bits lose 1 - s too, from z = 37 on all of it: the same by both sigmoids)
        z = np64(s["z"])
        keep["slope"] = keep["terms"] = 1 / (1 + np.exp(-z)) / (1 + np.exp(z))
    args = (np64(s["x"]), keep, np64(dy), None, first, 0, 0)
    want, mag = R.gate_norm_bwd(*args), R.gate_norm_bwd(*args, mag=True)
    for name, w, m in zip(("dx", "dz"), want, mag):
        close(out[name], w, m, 2.0 ** -15, name)
