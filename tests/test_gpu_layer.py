"""The layer operators on the GPU against their 64-bit forms (tests/layer_ref.py).

Tolerances, derived: an output may be off by half a step of its type (bf16 2^-8, fp32 2^-24 of
the value) plus a share of its magnitude, the sum of its terms' absolute values:
  convolution   up to 5 FP32 terms (5 x 2^-24) through silu and its derivative, whose slope is
                at most 1.1 and whose own error is a few 2^-23: 2^-20.
  scan          operands in two bf16 parts (2^-17 each, two in a product: 2^-16), at most 192
                terms a sum in FP32 (192 x 2^-24 < 2^-16), decays to a few 2^-22: 2^-14.  The
                rates' gradients are suffix sums over a chunk of terms that cancel: their
                magnitude is the chunk's sum of the terms' absolute values.  With bf16 inputs
                the pair products' factor enters dx, db and dc rounded to bf16 once, half a step
                of every term: 2^-8 more for these; and as such errors are independent, the
                2-norm of theirs and of the result's own rounding stays within 2^-8 of the
                result's (two errors uniform in +-2^-8 of a value: sqrt(2/3) 2^-8).
  norm          a row's mean and two products in FP32: 2^-19 (d <= 16384 terms, summed in
                pieces of at most 64 per lane).
"""
import numpy as np
import pytest
import torch

import quantized_state_qat_amd as la
from tests import layer_ref as R

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


def close(got, want, mag, share, name, dtype=None):
    half = HALF[dtype or got.dtype]
    got = np64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), name
    over = np.abs(got - want) - (half * 1.01 * np.abs(want) + share * mag + 1e-30)
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over.max() <= 0, (name, worst, got[worst], want[worst], mag[worst] if np.ndim(mag) else mag)


def spans(B, T, cu):
    return [(cu[i], cu[i + 1]) for i in range(B)] if cu is not None else [(i * T, (i + 1) * T) for i in range(B)]


def cu_tensor(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def strided(g, tokens, width, extra, dtype):
    """Rows of `width` inside wider rows: (view, ld)."""
    buf = draw(g, tokens, width + extra, dtype=dtype)
    return buf[:, 8:8 + width] if extra else buf, width + extra


# ------------------------------------------------------------------------------- convolution
CONV = [
    # dtype, B, T, cu, C, W, act, extra columns, bias, states, weights' dtype
    (BF, 2, 37, None, 64, 4, 1, 0, True, True, F32),
    (F32, 1, 130, None, 24, 3, 1, 16, True, True, F32),
    (BF, 3, 1, None, 2312, 4, 1, 0, True, True, BF),
    (BF, 2, 2, None, 72, 4, 0, 24, False, True, F32),
    (F32, 2, 3, None, 8, 2, 1, 0, True, False, BF),
    (BF, 6, 200, [3, 3, 40, 41, 43, 150, 190], 136, 4, 1, 8, True, True, F32),
    (F32, 4, 70, [0, 0, 70, 70, 70], 40, 3, 0, 0, False, True, F32),
    (BF, 1, 700, None, 264, 2, 1, 0, True, False, F32),
    (BF, 65, 300, [min(300, 4 * i) for i in range(66)], 16, 4, 1, 0, True, True, F32),
]


@pytest.mark.parametrize("dtype,B,T,cu,C,W,act,extra,bias,states,wt", CONV)
def test_conv(dtype, B, T, cu, C, W, act, extra, bias, states, wt):
    g = gen(C + T)
    tokens = T if cu is not None else B * T
    x, ld = strided(g, tokens, C, extra, dtype)
    w = draw(g, C, W, dtype=wt, scale=0.5)
    bv = draw(g, C, dtype=wt) if bias else None
    s0 = draw(g, B, W - 1, C, dtype=dtype) if states else None
    dsT = draw(g, B, W - 1, C, dtype=dtype) if states else None
    dy = draw(g, tokens, C, dtype=dtype)
    cfg = la.ConvConfig(B=B, T=T, C=C, width=W, act=act, x_dtype=CODE[dtype], w_dtype=CODE[wt], ld_x=ld if extra else 0)
    y = torch.full((tokens, C), 7.0, dtype=dtype, device="cuda")
    sT = torch.full((B, W - 1, C), float("nan"), dtype=dtype, device="cuda")
    la.la_conv_fwd(cfg, x, w, bv, s0, y, sT, cu_seqlens=cu_tensor(cu))
    dxb = torch.full((tokens, C + extra), 9.0, dtype=dtype, device="cuda")
    dx = dxb[:, 8:8 + C] if extra else dxb
    dw, db = torch.full((C, W), float("nan"), device="cuda"), torch.full((C,), float("nan"), device="cuda")
    ds0 = torch.full((B, W - 1, C), float("nan"), dtype=dtype, device="cuda")
    n = la.la_conv_bwd_workspace_bytes(cfg)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    la.la_conv_bwd(cfg, x, w, bv, s0, dy, dsT, dx, dw, db, ds0, ws, n, cu_seqlens=cu_tensor(cu))

    xn, wn, dyn = np64(x), np64(w), np64(dy)
    bn = np64(bv) if bias else np.zeros(C)
    zero = np.zeros((B, W - 1, C))
    s0n, dsn = (np64(s0), np64(dsT)) if states else (zero, zero)
    yr, ym, dxr, dxm = (np.zeros((tokens, C)) for _ in range(4))
    yr[:] = 7.0
    dwr, dwm, dbr, dbm = np.zeros((C, W)), np.zeros((C, W)), np.zeros(C), np.zeros(C)
    for b, (lo, hi) in enumerate(spans(B, T, cu)):
        yr[lo:hi], last = R.conv_fwd(xn[lo:hi], wn, bn, s0n[b], act)
        np.testing.assert_array_equal(np64(sT[b]), last)
        _, pre = R.conv_pre(xn[lo:hi], wn, bn, s0n[b])
        _, big = R.conv_pre(np.abs(xn[lo:hi]), np.abs(wn), np.abs(bn), np.abs(s0n[b]))
        ym[lo:hi] = big
        a, c, d, e = R.conv_bwd(xn[lo:hi], wn, bn, s0n[b], dyn[lo:hi], dsn[b], act)
        # the derivative moves with pre by at most half its error
        scale = (1.0 + big) if act else np.ones_like(big)
        am, cm, dm, em = R.conv_bwd(np.abs(xn[lo:hi]), np.abs(wn), np.abs(bn), np.abs(s0n[b]), np.abs(dyn[lo:hi]) * scale * 1.1,
                                    np.abs(dsn[b]), 0)
        dxr[lo:hi], dxm[lo:hi] = a, am
        dwr += c
        dwm += cm
        dbr += d
        dbm += dm
        close(ds0[b], e, em, 2.0 ** -20, f"dstate0[{b}]")
    close(y, yr, ym, 2.0 ** -20, "y")
    close(dx, dxr, dxm, 2.0 ** -20, "dx")
    sums = 2.0 ** -20 + 2.0 ** -24 * min(tokens, 512)  # sums over tokens: 32 a lane, then 8 and the workgroups
    close(dw, dwr, dwm, sums, "dweight")
    close(db, dbr, dbm, sums, "dbias")
    if extra:
        assert (dxb[:, :8] == 9).all() and (dxb[:, 8 + C:] == 9).all()


@pytest.mark.parametrize("cu", [None, [0, 7000, 7001, 9000]])
def test_conv_gradients_over_more_blocks_than_workgroups(cu):
    """9000 tokens by 32768 channels: a workgroup takes several of the token blocks."""
    g = gen(2)
    T, C, W = 9000, 32768, 4
    B = 1 if cu is None else 3
    x, dy, w = draw(g, T, 256, dtype=BF), draw(g, T, 256, dtype=BF), draw(g, 256, W, dtype=F32)
    wide = lambda t: t.repeat(1, C // 256).contiguous()  # noqa: E731
    cfg = la.ConvConfig(B=B, T=T, C=C, width=W, x_dtype=CODE[BF])
    n = la.la_conv_bwd_workspace_bytes(cfg)
    assert n <= 32 * C * (W + 1) * 4
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx = torch.empty(T, C, dtype=BF, device="cuda")
    dw, db = torch.empty(C, W, device="cuda"), torch.empty(C, device="cuda")
    la.la_conv_bwd(cfg, wide(x), w.repeat(C // 256, 1), None, None, wide(dy), None, dx, dw, db, None, ws, n,
                   cu_seqlens=cu_tensor(cu))
    for t in (dx.view(T, -1, 256).transpose(0, 1), dw.view(-1, 256, W), db.view(-1, 256)):
        assert torch.equal(t, t[:1].expand_as(t))  # the repeated channels agree in every bit
    xn, dyn, wn, zero = np64(x), np64(dy), np64(w), np.zeros((W - 1, 256))
    dwr, dwm, dbr, dbm = np.zeros((256, W)), np.zeros((256, W)), np.zeros(256), np.zeros(256)
    for lo, hi in spans(B, T, cu):
        dxr, c, d, _ = R.conv_bwd(xn[lo:hi], wn, np.zeros(256), zero, dyn[lo:hi], zero, 1)
        _, big = R.conv_pre(np.abs(xn[lo:hi]), np.abs(wn), np.zeros(256), zero)
        dxm, cm, dm, _ = R.conv_bwd(np.abs(xn[lo:hi]), np.abs(wn), np.zeros(256), zero, np.abs(dyn[lo:hi]) * (1.0 + big) * 1.1,
                                    zero, 0)
        close(dx[lo:hi, :256], dxr, dxm, 2.0 ** -20, "dx")
        dwr, dwm, dbr, dbm = dwr + c, dwm + cm, dbr + d, dbm + dm
    sums = 2.0 ** -20 + 2.0 ** -24 * 512
    close(dw[:256], dwr, dwm, sums, "dweight")
    close(db[:256], dbr, dbm, sums, "dbias")


def test_conv_gradients_of_no_sequences():
    cfg = la.ConvConfig(B=0, T=50, C=64, width=4)
    dw, db = torch.full((64, 4), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    w = torch.ones(64, 4, device="cuda")
    la.la_conv_bwd(cfg, None, w, None, None, None, None, None, dw, db, None, None, 0,
                   cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dtype,T,C,ld", [(BF, 50, 64, 0), (F32, 3, 8, 16), (BF, 70000, 264, 272)])
def test_conv_gradients_of_no_sequences_are_zero_rows(dtype, T, C, ld):
    cfg = la.ConvConfig(B=0, T=T, C=C, width=4, x_dtype=CODE[dtype], ld_x=ld)
    wide = torch.full((T, ld or C), 9.0, dtype=dtype, device="cuda")
    dw, db = torch.full((C, 4), 3.0, device="cuda"), torch.full((C,), 3.0, device="cuda")
    la.la_conv_bwd(cfg, None, torch.ones(C, 4, device="cuda"), None, None, None, None, wide[:, :C], dw, db, None, None, 0,
                   cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not wide[:, :C].any() and (wide[:, C:] == 9).all() and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype,B,C,W,pool", [(BF, 5, 264, 4, True), (F32, 1, 8, 2, True), (BF, 3, 2312, 3, False)])
def test_conv_step_continues_the_forward(dtype, B, C, W, pool):
    g = gen(B)
    T = 6
    x = draw(g, B, T, C, dtype=dtype)
    w, bv, s0 = draw(g, C, W, dtype=F32), draw(g, C, dtype=F32), draw(g, B, W - 1, C, dtype=dtype)
    full = la.ConvConfig(B=B, T=T, C=C, width=W, x_dtype=CODE[dtype])
    y, sT = torch.empty_like(x), torch.empty_like(s0)
    la.la_conv_fwd(full, x, w, bv, s0, y, sT)
    cfg = la.ConvConfig(B=B, T=1, C=C, width=W, x_dtype=CODE[dtype])
    if pool:
        state = draw(g, B + 3, W - 1, C, dtype=dtype)
        before = state.clone()
        slots = torch.arange(B + 1, 1, -1, dtype=torch.int32, device="cuda")
        state[slots.long()] = s0
        if B > 2:
            slots[1], slots[2] = 0, B + 3  # padding
    else:
        state, slots = s0.clone(), None
    for t in range(T):
        yt = torch.full((B, C), float("nan"), dtype=dtype, device="cuda")
        la.la_conv_step(cfg, x[:, t].contiguous(), w, bv, state, yt, slots=slots, n_slots=B + 3 if pool else 0)
        for b in range(B):
            if pool and B > 2 and b in (1, 2):
                assert not yt[b].any()
            else:
                assert torch.equal(yt[b], y[b, t]), (b, t)
    for b in range(B):
        if pool and B > 2 and b in (1, 2):
            continue
        assert torch.equal(state[int(slots[b]) if pool else b], sT[b])
    if pool:
        assert torch.equal(state[0], before[0])


# -------------------------------------------------------------------------------------- scan
class Scan:
    """One case's inputs, in slices of wider rows, and its 64-bit results."""

    def __init__(self, dtype, B, T, H, G, N, P, cu=None, sp=1, seed=0, states=True, params=True, extra=8, dtt=None, rate=4.0,
                 out=None):
        g = gen(1000 * T + 10 * H + N + seed)
        self.dtype, self.B, self.T, self.H, self.G, self.N, self.P, self.cu, self.sp = dtype, B, T, H, G, N, P, cu, sp
        self.states, self.params, self.out, self.dtt = states, params, out or dtype, dtt or dtype
        self.tokens = n = T if cu is not None else B * T
        self.wx, self.wb = H * P, G * N
        self.ld = self.wx + 2 * self.wb + extra
        self.buf = draw(g, n, self.ld, dtype=dtype, scale=0.7)
        self.x, self.b, self.c = self.cut(self.buf)
        self.dt = draw(g, n, H, dtype=self.dtt) if sp else draw(g, n, H, dtype=self.dtt).abs()
        self.A = -torch.rand(H, generator=g).cuda() * rate
        self.D = draw(g, H, dtype=F32) if params else None
        self.bias = draw(g, H, dtype=F32) - 2.0 if params and sp else None
        self.S0 = draw(g, B, H, N, P, dtype=F32) if states else None
        self.dST = draw(g, B, H, N, P, dtype=F32) if states else None
        self.dy = draw(g, n, H * P, dtype=self.out)
        self.cfg = la.ScanConfig(B=B, T=T, H=H, G=G, d_k=N, d_v=P, softplus=sp, x_dtype=CODE[dtype], dt_dtype=CODE[self.dtt],
                                 out_dtype=CODE[self.out], ld_x=self.ld, ld_b=self.ld, ld_c=self.ld)

    def cut(self, buf):
        return buf[:, :self.wx], buf[:, self.wx:self.wx + self.wb], buf[:, self.wx + self.wb:self.wx + 2 * self.wb]

    def fwd(self, stream=None):
        y = torch.full((self.tokens, self.H * self.P), 5.0, dtype=self.out, device="cuda")
        ST = torch.full((self.B, self.H, self.N, self.P), float("nan"), device="cuda")
        n = la.la_scan_workspace_bytes(self.cfg)
        ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
        la.la_scan_fwd(self.cfg, self.x, self.dt, self.A, self.b, self.c, self.D, self.bias, self.S0, y, ST,
                       ws if n else None, n, cu_seqlens=cu_tensor(self.cu), stream=stream)
        return y, ST

    def out_buffers(self):
        nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        buf = torch.full_like(self.buf, 9.0)
        dx, db, dc = self.cut(buf)
        return buf, dict(dx=dx, db=db, dc=dc, ddt=torch.full_like(self.dt, 9.0), dA=nan(self.H), dD=nan(self.H),
                         ddt_bias=nan(self.H), dS0=nan(self.B, self.H, self.N, self.P))

    def bwd_into(self, bufs):
        o = bufs[1]
        n = (la.la_scan_bwd_varlen_workspace_bytes if self.cu is not None else la.la_scan_bwd_workspace_bytes)(self.cfg)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        la.la_scan_bwd(self.cfg, self.x, self.dt, self.A, self.b, self.c, self.D, self.bias, self.S0, self.dy, self.dST, o["dx"],
                       o["ddt"], o["dA"], o["db"], o["dc"], o["dD"], o["ddt_bias"], o["dS0"], ws, n,
                       cu_seqlens=cu_tensor(self.cu))
        return o

    def bwd(self):
        bufs = self.out_buffers()
        o = self.bwd_into(bufs)
        assert (bufs[0][:, self.wx + 2 * self.wb:] == 9).all()
        return o

    def reference(self, backward):
        n, H, G, N, P = self.tokens, self.H, self.G, self.N, self.P
        x, b, c = np64(self.x).reshape(n, H, P), np64(self.b).reshape(n, G, N), np64(self.c).reshape(n, G, N)
        dy = np64(self.dy).reshape(n, H, P)
        A = np64(self.A)
        D = np64(self.D) if self.D is not None else np.zeros(H)
        z, delta = R.steps(np64(self.dt), np64(self.bias) if self.bias is not None else np.zeros(H), self.sp)
        zero = np.zeros((self.B, H, N, P))
        S0, dST = (np64(self.S0), np64(self.dST)) if self.states else (zero, zero)
        w = dict(y=np.full((n, H, P), 5.0), S_T=zero.copy())
        m = dict(y=np.zeros((n, H, P)), S_T=zero.copy())
        if backward:
            shapes = dict(dx=(n, H, P), db=(n, G, N), dc=(n, G, N), ddt=(n, H), dA=(H,), dD=(H,), ddt_bias=(H,), dS0=zero.shape)
            for k, s in shapes.items():
                w[k], m[k] = np.zeros(s), np.zeros(s)
        a = np.abs
        for i, (lo, hi) in enumerate(spans(self.B, self.T, self.cu)):
            r = slice(lo, hi)
            w["y"][r], w["S_T"][i], _ = R.scan_fwd(x[r], delta[r], A, b[r], c[r], D, S0[i])
            m["y"][r], m["S_T"][i], _ = R.scan_fwd(a(x[r]), a(delta[r]), A, a(b[r]), a(c[r]), a(D), a(S0[i]))
            if not backward:
                continue
            got, _ = R.scan_bwd(x[r], z[r], delta[r], A, b[r], c[r], D, S0[i], dy[r], dST[i], self.sp)
            big, _ = R.scan_bwd(a(x[r]), z[r], a(delta[r]), A, a(b[r]), a(c[r]), a(D), a(S0[i]), a(dy[r]), a(dST[i]), self.sp,
                                A_sum=a(A))
            # the rates' gradients: suffix sums of y.dy - x.dx (without D) over a chunk, and the state's part at its end
            T = hi - lo
            yn, S_end, st = R.scan_fwd(a(x[r]), a(delta[r]), A, a(b[r]), a(c[r]), 0 * D, a(S0[i]))
            dxn = big["dx"] - a(D)[:, None] * a(dy[r])
            terms = (yn * a(dy[r])).sum(2) + (dxn * a(x[r])).sum(2)
            chunk = np.zeros((T, H))
            for t0 in range(0, T, 64):
                t1 = min(T, t0 + 64)
                # <S_end, dS_end> of the chunk: the sums of b, x against the gradient that leaves it
                endS = st[t1]
                nxt = R.scan_bwd(a(x[r])[t1:], z[r][t1:], a(delta[r])[t1:], A, a(b[r])[t1:], a(c[r])[t1:], a(D), endS,
                                 a(dy[r])[t1:], a(dST[i]), self.sp, A_sum=a(A))[0]["dS0"]
                chunk[t0:t1] = terms[t0:t1].sum(0) + (endS * nxt).sum((1, 2))
            sg = 1 / (1 + np.exp(-z[r])) if self.sp else 1.0
            extra = dict(ddt=a(A) * chunk * sg, dA=(a(delta[r]) * chunk).sum(0), ddt_bias=(a(A) * chunk * sg).sum(0))
            for k in shapes:
                v, u = got[k], big[k] + extra.get(k, 0.0)
                if k in ("dA", "dD", "ddt_bias"):
                    w[k] += v
                    m[k] += u
                elif k == "dS0":
                    w[k][i], m[k][i] = v, u
                else:
                    w[k][r], m[k][r] = v, u
        return w, m

    def check(self, backward=True):
        w, m = self.reference(backward)
        y, ST = self.fwd()
        share = 2.0 ** -14
        close(y.reshape(w["y"].shape), w["y"], m["y"], share, "y")
        close(ST, w["S_T"], m["S_T"], share, "S_T")
        if not backward:
            return
        o = self.bwd()
        for k, t in o.items():
            if k == "dD" and self.D is None or k == "ddt_bias" and self.bias is None:
                pass  # written all the same
            once = 2.0 ** -8 if self.dtype == BF and k in ("dx", "db", "dc") else 0.0
            close(t.reshape(w[k].shape), w[k], m[k], share + once, k)
            if once and t.numel() >= 1024:
                assert np.linalg.norm(np64(t).reshape(w[k].shape) - w[k]) <= 2.0 ** -8 * np.linalg.norm(w[k]), k


SCAN = [
    # dtype, B, T, H, G, d_k, d_v, more
    (BF, 2, 1, 2, 1, 16, 64, {}),
    (BF, 1, 2, 3, 3, 32, 64, {}),
    (BF, 2, 63, 4, 2, 64, 64, {}),
    (BF, 1, 64, 2, 1, 128, 128, {}),
    (BF, 2, 65, 4, 1, 128, 64, {}),
    (BF, 1, 130, 5, 1, 64, 192, dict(states=False)),
    (BF, 1, 200, 2, 2, 16, 64, dict(params=False)),
    (BF, 1, 100, 2, 1, 128, 64, dict(sp=0, rate=0.5)),
    (BF, 1, 150, 2, 1, 64, 64, dict(rate=30.0)),
    (F32, 2, 1, 2, 1, 64, 64, {}),
    (F32, 1, 65, 4, 2, 16, 64, {}),
    (F32, 1, 130, 2, 1, 128, 128, {}),
    (F32, 2, 90, 3, 1, 32, 64, dict(sp=0, rate=0.5, states=False)),
    (BF, 1, 70, 2, 1, 64, 64, dict(dtt=F32)),
    (BF, 6, 300, 2, 1, 64, 64, dict(cu=[2, 2, 66, 67, 131, 260, 290])),
    (F32, 3, 80, 2, 2, 32, 64, dict(cu=[0, 80, 80, 80])),
    (BF, 3, 200, 4, 1, 128, 128, dict(cu=[0, 0, 129, 200])),
    (BF, 1, 700, 2, 1, 32, 64, {}),     # few heads: the walks cut into segments / chunks
    (F32, 1, 1025, 1, 1, 16, 64, {}),
    (BF, 3, 1200, 1, 1, 16, 64, dict(cu=[0, 900, 900, 1190])),
    (BF, 4, 70, 64, 2, 16, 64, {}),     # many heads: a workgroup walks a sequence
]


@pytest.mark.parametrize("H", [2, 1])
def test_scan_of_many_short_sequences(H):
    """200 ragged sequences, some empty, tokens before and behind them (H = 1: a workgroup a chunk)."""
    lens = torch.randint(0, 41, (200,), generator=gen(7)).tolist()
    lens[17], lens[18], lens[199] = 130, 0, 64
    cu = np.concatenate([[5], 5 + np.cumsum(lens)]).tolist()
    Scan(BF, 200, cu[-1] + 300, H, 1, 16, 64, cu=cu).check()


@pytest.mark.parametrize("B,T,H,G,N,P,more", [
    (32, 70, 16, 1, 32, 64, {}), (33, 65, 16, 2, 128, 64, {}), (16, 66, 16, 1, 64, 128, {}), (18, 130, 15, 5, 16, 128, {}),
    (1, 4096, 16, 2, 16, 64, {}), (2, 4130, 4, 1, 128, 128, dict(cu=[0, 4100, 4125])), (2, 4200, 8, 1, 64, 64, dict(cu=[0, 0, 4200])),
    (1, 4097, 18, 2, 32, 64, {}),
])
def test_scan_two_tiles_a_workgroup(B, T, H, G, N, P, more):
    """Many heads, or few cut into many segments: a workgroup takes 128 columns of a head or two heads
    of 64 (the last one: an odd number of heads a group, one tile again)."""
    Scan(BF, B, T, H, G, N, P, **more).check(backward=False)


@pytest.mark.parametrize("dtt,H", [(BF, 3), (BF, 4), (F32, 3)])
def test_scan_steps_in_wider_rows(dtt, H):
    """dt and ddt as the first columns of rows of 7 (bf16: rows that start in the middle of a word)."""
    class Wide(Scan):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            wide = torch.full((self.tokens, 7), float("nan"), dtype=self.dtt, device="cuda")
            wide[:, :H] = self.dt
            self.dt, self.cfg.ld_dt = wide[:, :H], 7

        def out_buffers(self):
            buf, o = super().out_buffers()
            self.wide = torch.full((self.tokens, 7), 9.0, dtype=self.dtt, device="cuda")
            o["ddt"] = self.wide[:, :H]
            return buf, o

    s = Wide(BF, 2, 131, H, 1, 32, 64, dtt=dtt)
    s.check()
    assert (s.wide[:, H:] == 9).all()


def test_scan_nan_step_reaches_its_own_head_from_its_token_on():
    s = Scan(BF, 1, 200, 2, 1, 64, 64)
    s.dt[70, 1] = float("nan")
    y, ST = s.fwd()
    y = y.view(200, 2, 64)
    assert y[:, 0].isfinite().all() and y[:70, 1].isfinite().all() and y[70:, 1].isnan().all()
    assert ST[0, 0].isfinite().all() and ST[0, 1].isnan().all()


@pytest.mark.parametrize("dtype,B,T,H,G,N,P,more", SCAN)
def test_scan(dtype, B, T, H, G, N, P, more):
    Scan(dtype, B, T, H, G, N, P, **more).check()


def test_scan_mixed_output_dtypes():
    Scan(BF, 1, 100, 2, 1, 64, 64, out=F32).check(backward=False)
    Scan(F32, 1, 100, 2, 1, 64, 64, out=BF).check(backward=False)


def test_scan_steps_that_vanish_and_explode():
    """Delta = 0 leaves the state; a very negative rate empties it within a token."""
    k = Scan(BF, 1, 130, 2, 1, 64, 64, sp=0)
    k.dt[:65] = 0
    k.dt[100] = 200.0
    k.A[:] = -5.0
    k.check()


def test_scan_without_tokens():
    for cu, T in ((None, 0), ([0, 0, 0], 4)):
        k = Scan(BF, 2, max(T, 1), 2, 1, 64, 64, cu=[0, 0, 0])
        k.cfg.T = T
        k.cu = cu
        y, ST = k.fwd()
        assert torch.equal(ST, k.S0) and (y == 5).all()
        o = k.bwd()
        assert torch.equal(o["dS0"], k.dST)
        for n in ("dA", "dD", "ddt_bias"):
            assert not o[n].any()
        if T:
            assert not o["dx"].any() and not o["ddt"].any() and not o["db"].any() and not o["dc"].any()


@pytest.mark.parametrize("dtype,B,T,H,G,cu", [(BF, 0, 70, 3, 1, [0]), (F32, 0, 300, 4, 2, [0]), (BF, 0, 1, 16, 1, [0]),
                                              (BF, 2, 70, 0, 3, None), (F32, 2, 70, 0, 1, [0, 5, 60])])
def test_scan_gradients_of_no_sequences_or_heads_are_zero(dtype, B, T, H, G, cu):
    N, P = 32, 64
    tokens = T if cu is not None else B * T
    wx, wb = H * P, G * N
    ld = wx + 2 * wb + 8
    cfg = la.ScanConfig(B=B, T=T, H=H, G=G, d_k=N, d_v=P, x_dtype=CODE[dtype], dt_dtype=CODE[dtype], out_dtype=CODE[dtype],
                        ld_x=ld, ld_b=ld, ld_c=ld, ld_dt=H + 5)
    buf, ddt = (torch.full((tokens, w), 9.0, dtype=dtype, device="cuda") for w in (ld, H + 5))
    sums = [torch.full((H,), 3.0, device="cuda") if H else None for _ in range(3)]
    A = torch.ones(max(H, 1), device="cuda")
    la.la_scan_bwd(cfg, None, None, A, None, None, None, None, None, None, None, buf[:, :wx] if H else None,
                   ddt[:, :H] if H else None, sums[0], buf[:, wx:wx + wb], buf[:, wx + wb:wx + 2 * wb], sums[1], sums[2], None,
                   None, 0, cu_seqlens=cu_tensor(cu))
    assert not buf[:, :wx + 2 * wb].any() and (buf[:, wx + 2 * wb:] == 9).all()
    assert not ddt[:, :H].any() and (ddt[:, H:] == 9).all()
    assert not any(t is not None and t.any() for t in sums)


@pytest.mark.parametrize("B,H,G,N,P,dtype", [(1, 2, 1, 16, 64, BF), (3, 4, 2, 32, 64, F32), (2, 3, 1, 64, 192, BF),
                                             (5, 16, 1, 128, 128, BF), (40, 16, 1, 64, 64, F32), (70, 16, 2, 16, 128, BF)])
def test_scan_step(B, H, G, N, P, dtype):
    g = gen(B + H)
    cfg = la.ScanConfig(B=B, T=1, H=H, G=G, d_k=N, d_v=P, x_dtype=CODE[dtype], dt_dtype=CODE[dtype], out_dtype=CODE[dtype])
    x, b, c = draw(g, B, H, P, dtype=dtype), draw(g, B, G, N, dtype=dtype), draw(g, B, G, N, dtype=dtype)
    dt, A, D, bias = draw(g, B, H, dtype=dtype), -torch.rand(H, generator=g).cuda() * 4, draw(g, H, dtype=F32), draw(g, H, dtype=F32)
    pool = draw(g, B + 3, H, N, P, dtype=F32)
    slots = (torch.randperm(B + 2, generator=g)[:B] + 1).to(torch.int32).cuda()
    if B > 2:
        slots[1], slots[2] = 0, B + 3
    before = pool.clone()
    y = torch.full((B, H, P), float("nan"), dtype=dtype, device="cuda")
    la.la_scan_step(cfg, x, dt, A, b, c, D, bias, pool, y, slots=slots, n_slots=B + 3)
    _, delta = R.steps(np64(dt), np64(bias), 1)
    touched = set()
    for i in range(B):
        s = int(slots[i])
        if s <= 0 or s >= B + 3:
            assert not y[i].any()
            continue
        touched.add(s)
        want, S, _ = R.scan_fwd(np64(x[i:i + 1]), delta[i:i + 1], np64(A), np64(b[i:i + 1]), np64(c[i:i + 1]), np64(D), np64(before[s]))
        mag, Sm, _ = R.scan_fwd(*(np.abs(v) for v in (np64(x[i:i + 1]), delta[i:i + 1])), np64(A), np.abs(np64(b[i:i + 1])),
                                np.abs(np64(c[i:i + 1])), np.abs(np64(D)), np.abs(np64(before[s])))
        close(y[i], want[0], mag[0], 2.0 ** -17, "y")  # at most 129 FP32 terms
        close(pool[s], S, Sm, 2.0 ** -21, "S")
    for s in range(B + 3):
        if s not in touched:
            assert torch.equal(pool[s], before[s])
    if B <= 3:  # without slots: the states in order
        st = before[:B].clone()
        y2 = torch.empty_like(y)
        la.la_scan_step(cfg, x, dt, A, b, c, D, bias, st, y2)
        i = 0
        pool2 = before.clone()
        one = torch.zeros(B, dtype=torch.int32, device="cuda")
        one[i] = 1
        pool2[1] = before[0]
        la.la_scan_step(cfg, x, dt, A, b, c, D, bias, pool2, y, slots=one, n_slots=B + 3)
        assert torch.equal(y2[0], y[0]) and torch.equal(pool2[1], st[0])


@pytest.mark.parametrize("given,means", [([-5, 60, 400], [0, 60, 150]), ([0, 200, 300], [0, 150, 150])])
def test_boundaries_are_clamped(given, means):
    """Boundaries outside the packing are moved to its ends."""
    T = 150
    g = gen(3)
    x, w, dy = draw(g, T, 64), draw(g, 64, 4, dtype=F32), draw(g, T, 64)
    cc = la.ConvConfig(B=2, T=T, C=64, width=4)
    s = Scan(BF, 2, T, 2, 1, 32, 64, cu=given)
    results = []
    for cu in (given, means):
        y = torch.full_like(x, 5.0)
        sT = torch.empty(2, 3, 64, dtype=BF, device="cuda")
        dx, dw = torch.full_like(x, 5.0), torch.empty(64, 4, device="cuda")
        n = la.la_conv_bwd_workspace_bytes(cc)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        la.la_conv_fwd(cc, x, w, None, None, y, sT, cu_seqlens=cu_tensor(cu))
        la.la_conv_bwd(cc, x, w, None, None, dy, None, dx, dw, None, None, ws, n, cu_seqlens=cu_tensor(cu))
        s.cu = cu
        results.append([y, sT, dx, dw, *s.fwd(), *(t.clone() for t in s.bwd().values())])
    for a, b in zip(*results):
        assert torch.equal(a, b)


# -------------------------------------------------------------------------------------- norm
NORM = [
    # dtype, rows, d, codec, group, out, weights, residual
    (BF, 5, 8, "none", 0, BF, F32, True), (BF, 3, 64, "int8", 0, BF, F32, True), (F32, 7, 96, "int8", 16, F32, F32, True),
    (BF, 9, 128, "e4m3", 128, BF, BF, True), (BF, 4, 256, "int8", 64, F32, F32, False), (F32, 2, 520, "e4m3", 0, F32, None, True),
    (BF, 33, 1024, "e4m3", 32, F32, F32, True), (BF, 6, 2048, "int8", 128, BF, F32, True), (BF, 3, 2056, "none", 0, F32, F32, True),
    (F32, 2, 4096, "int8", 0, F32, BF, True), (BF, 2, 8192, "e4m3", 16, BF, F32, True), (BF, 2, 16384, "none", 0, F32, F32, True),
    (BF, 1, 16384, "int8", 32, F32, F32, True), (BF, 1000, 72, "none", 0, BF, F32, True),
]


@pytest.mark.parametrize("dtype,rows,d,kind,group,out,wt,residual", NORM)
def test_norm(dtype, rows, d, kind, group, out, wt, residual):
    g = gen(rows + d)
    x = draw(g, rows, d, dtype=dtype)
    res = draw(g, rows, d, dtype=dtype, scale=3.0) if residual else None
    w = draw(g, d, dtype=wt) if wt is not None else None
    x[0] = 0
    if residual:
        res[0] = 0  # a row of zeros
    eps = 1e-5
    qdq = {"none": la.LA_QDQ_NONE, "int8": la.LA_QDQ_INT8_GROUP, "e4m3": la.LA_QDQ_E4M3_TILE}[kind]
    cfg = la.NormConfig(rows=rows, d=d, eps=eps, qdq=qdq, group=group, x_dtype=CODE[dtype], w_dtype=CODE[wt or F32],
                        out_dtype=CODE[out])
    ro, y = torch.empty_like(x), torch.empty(rows, d, dtype=out, device="cuda")
    codes = scales = None
    if kind != "none":
        codes = torch.empty(rows, d, dtype=torch.int8 if kind == "int8" else torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(rows, d // (group or d), device="cuda")
    la.la_norm_fwd(cfg, x, res, w, ro, y, codes, scales)
    h = (x.float() + res.float()).to(dtype) if residual else x
    assert torch.equal(ro, h)
    hn, wn = np64(h), np64(w) if w is not None else np.ones(d)
    n, _ = R.norm_fwd(hn, wn, eps)
    tol = 2.0 ** -19
    if kind == "none":
        close(y, n, np.abs(n), tol, "y")
    else:
        v, s, step = R.codec(n, group, kind)
        close(scales, s, s, tol, "scales")
        # a value next to a rounding border may take the neighbouring code: one step, at most one in 2000
        # (borders are a step apart, the error is below 2^-18 of 127 or 448 steps: 2 x 448 x 2^-18 = 1 in 290 at most)
        got = np64(y)
        off = np.abs(got - v) - (HALF[out] * 1.01 * np.abs(v) + 2 * tol * np.abs(v) + 1e-30)
        assert (off <= 1.01 * step).all() and (off > 0).mean() <= 1 / 290
        stood = np64(codes.float()) * np.repeat(np64(scales), group or d, 1)
        np.testing.assert_array_less(np.abs(got - stood), HALF[out] * 1.01 * np.abs(stood) + 2.0 ** -23 * np.abs(stood) + 1e-30)
    # backward
    dy, dres = draw(g, rows, d, dtype=out), draw(g, rows, d, dtype=dtype)
    dx, dw = torch.empty_like(x), torch.full((d,), float("nan"), device="cuda")
    nb = la.la_norm_bwd_workspace_bytes(cfg)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    la.la_norm_bwd(cfg, h, w, dy, dres, dx, dw, ws, nb)
    dxr, dwr = R.norm_bwd(hn, wn, eps, np64(dy), np64(dres))
    a = np.abs
    r = 1 / np.sqrt((hn * hn).mean(1, keepdims=True) + eps)
    gm = a(np64(dy) * wn)
    mag = a(np64(dres)) + r * (gm + a(hn) * r * r * (gm * a(hn)).mean(1, keepdims=True))
    close(dx, dxr, mag, tol, "dx")
    close(dw, dwr, (a(np64(dy)) * a(hn) * r).sum(0), tol + rows * 2.0 ** -24, "dweight")
    # without the optional tensors, in place
    same = dres.clone()
    la.la_norm_bwd(cfg, h, w, dy, same, same, None, None, 0)
    assert torch.equal(same, dx)
    y2, x2 = torch.empty_like(y), x.clone()
    la.la_norm_fwd(cfg, x2, res, w, x2, y2)
    assert torch.equal(x2, ro) and torch.equal(y2, y)


@pytest.mark.parametrize("kind,group", [("int8", 64), ("int8", 0), ("e4m3", 0), ("e4m3", 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 2048, 4096])
def test_norm_codes_are_the_same_for_every_type_of_values(d, dtype, kind, group):
    rows = 2000
    g = gen(d)
    x, res, w = draw(g, rows, d, dtype=dtype), draw(g, rows, d, dtype=dtype, scale=3.0), draw(g, d, dtype=F32)
    qdq = la.LA_QDQ_INT8_GROUP if kind == "int8" else la.LA_QDQ_E4M3_TILE
    got = []
    for out in (F32, BF, None):
        cfg = la.NormConfig(rows=rows, d=d, qdq=qdq, group=group, x_dtype=CODE[dtype], out_dtype=CODE[out or BF])
        y = torch.empty(rows, d, dtype=out, device="cuda") if out else None
        codes = torch.empty(rows, d, dtype=torch.int8 if kind == "int8" else torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(rows, d // (group or d), device="cuda")
        la.la_norm_fwd(cfg, x, res, w, None, y, codes, scales)
        got.append((codes.view(torch.uint8), scales, y))
    for codes, scales, _ in got[1:]:
        assert torch.equal(codes, got[0][0]) and torch.equal(scales, got[0][1])
    assert torch.equal(got[0][2].to(BF), got[1][2])


def test_norm_keeps_infinities_and_nan_in_their_rows():
    for qdq in (la.LA_QDQ_NONE, la.LA_QDQ_INT8_GROUP, la.LA_QDQ_E4M3_TILE):
        x = torch.ones(4, 256, dtype=BF, device="cuda")
        x[1, 3], x[2, 7] = float("nan"), float("inf")
        cfg = la.NormConfig(rows=4, d=256, eps=0.0, qdq=qdq, group=0)
        y = torch.empty_like(x)
        la.la_norm_fwd(cfg, x, None, None, None, y)
        ones = torch.ones(256, dtype=BF, device="cuda")
        assert torch.equal(y[0], ones) and torch.equal(y[3], ones)
        assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7])


@pytest.mark.parametrize("kind", ["none", "int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 16, 64, 128])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [256, 2048, 4096])
def test_norm_infinities_and_nan_by_the_formula(d, dtype, out, group, kind):
    """NaN exactly where torch's float64 formula has it: values, scales, codes."""
    g = gen(d + group)
    x, w = draw(g, 9, d, dtype=dtype), 1 + draw(g, d, dtype=F32, scale=0.1)
    nan, inf = float("nan"), float("inf")
    x[1, 3], x[2, d - 1], x[3, 0], x[4, 70], x[6, :] = nan, inf, -inf, nan, inf
    x[7, 5], x[7, d // 2] = inf, nan
    if dtype == F32:
        w[130] = inf  # an infinite product: an infinite scale
    qdq = {"none": la.LA_QDQ_NONE, "int8": la.LA_QDQ_INT8_GROUP, "e4m3": la.LA_QDQ_E4M3_TILE}[kind]
    cfg = la.NormConfig(rows=9, d=d, eps=1e-5, qdq=qdq, group=group if kind != "none" else 0, x_dtype=CODE[dtype], out_dtype=CODE[out])
    y = torch.empty(9, d, dtype=out, device="cuda")
    codes = scales = None
    width = cfg.group or d
    if kind != "none":
        codes = torch.empty(9, d, dtype=torch.int8 if kind == "int8" else torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(9, d // width, device="cuda")
    la.la_norm_fwd(cfg, x, None, w, None, y, codes, scales)
    h = x.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * w.double()
    if kind == "none":
        assert torch.equal(y.isnan(), n.isnan()) and torch.equal(y.isinf(), n.isinf())
        return
    v = n.view(9, -1, width)
    s = v.abs().amax(2, keepdim=True) / (127.0 if kind == "int8" else 448.0)  # (amax keeps NaN)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = v / s
    q = torch.round(q).clamp(-127, 127) if kind == "int8" else q.clamp(-448, 448)
    want, q = (q * s).view(9, d), q.view(9, d)
    assert torch.equal(scales.isnan(), s[:, :, 0].isnan()) and torch.equal(scales.isinf(), s[:, :, 0].isinf())
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    if kind == "int8":
        assert not codes[q.isnan()].any()
    else:
        assert torch.equal(codes.float().isnan(), q.isnan())


# ----------------------------------------------------------------------------- run together
class Layer:
    """norm (8-bit) -> projection -> convolution -> scan -> projection, as a hybrid stack runs them."""

    def __init__(self, d=256, H=4, G=1, N=64, P=64, seed=5):
        g = gen(seed)
        self.d, self.H, self.G, self.N, self.P = d, H, G, N, P
        self.C = H * P + 2 * G * N
        self.W = self.C + 8  # the projection's rows: the convolution's channels, dt, unused (a multiple of 16 bytes)
        self.w, self.cw, self.cb = 1 + draw(g, d, dtype=F32, scale=0.1), draw(g, self.C, 4, dtype=F32, scale=0.4), draw(g, self.C, dtype=F32, scale=0.1)
        self.win, self.wout = draw(g, d, self.W, scale=d ** -0.5), draw(g, H * P, d, scale=(H * P) ** -0.5)
        self.A, self.D, self.bias = -torch.rand(H, generator=g).cuda() * 4, draw(g, H, dtype=F32), draw(g, H, dtype=F32) - 2

    def prefill(self, x, res, B, T, cu=None):
        n = x.shape[0]
        h, y = torch.empty_like(x), torch.empty_like(x)
        codes, scales = torch.empty(n, self.d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(n, 1, device="cuda")
        la.la_norm_fwd(la.NormConfig(rows=n, d=self.d, qdq=la.LA_QDQ_E4M3_TILE), x, res, self.w, h, y, codes, scales)
        proj = y @ self.win
        z, cs = torch.empty(n, self.C, dtype=BF, device="cuda"), torch.zeros(B, 3, self.C, dtype=BF, device="cuda")
        la.la_conv_fwd(la.ConvConfig(B=B, T=T, C=self.C, width=4, ld_x=self.W), proj[:, :self.C], self.cw, self.cb, None, z, cs, cu_seqlens=cu)
        cfg = la.ScanConfig(B=B, T=T, H=self.H, G=self.G, d_k=self.N, d_v=self.P, ld_x=self.C, ld_b=self.C, ld_c=self.C, ld_dt=self.W)
        o, S = torch.zeros(n, self.H * self.P, dtype=BF, device="cuda"), torch.zeros(B, self.H, self.N, self.P, device="cuda")
        nb = la.la_scan_workspace_bytes(cfg)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
        i, j = self.H * self.P, self.H * self.P + self.G * self.N
        la.la_scan_fwd(cfg, z[:, :i], proj[:, self.C:self.C + self.H], self.A, z[:, i:j], z[:, j:], self.D, self.bias, None, o, S, ws, nb, cu_seqlens=cu)
        return o @ self.wout, h, cs, S

    def step(self, x, res, cs, S):
        B = x.shape[0]
        h, y = torch.empty_like(x), torch.empty_like(x)
        la.la_norm_fwd(la.NormConfig(rows=B, d=self.d, qdq=la.LA_QDQ_E4M3_TILE), x, res, self.w, h, y)
        proj = y @ self.win
        z, o = torch.empty(B, self.C, dtype=BF, device="cuda"), torch.empty(B, self.H * self.P, dtype=BF, device="cuda")
        la.la_conv_step(la.ConvConfig(B=B, T=1, C=self.C, width=4, ld_x=self.W), proj[:, :self.C], self.cw, self.cb, cs, z)
        i, j = self.H * self.P, self.H * self.P + self.G * self.N
        cfg = la.ScanConfig(B=B, T=1, H=self.H, G=self.G, d_k=self.N, d_v=self.P, ld_x=self.C, ld_b=self.C, ld_c=self.C, ld_dt=self.W)
        la.la_scan_step(cfg, z[:, :i], proj[:, self.C:self.C + self.H], self.A, z[:, i:j], z[:, j:], self.D, self.bias, S, o)
        return o @ self.wout, h


def test_layer_prompt_then_tokens():
    """A prompt of T tokens followed by single tokens equals one prompt of all of them, dense and packed."""
    m, g = Layer(), gen(6)
    B, T, more = 3, 70, 4
    x, res = draw(g, B, T + more, m.d), draw(g, B, T + more, m.d)
    full, _, cs_full, S_full = m.prefill(x.reshape(-1, m.d), res.reshape(-1, m.d), B, T + more)
    full = full.reshape(B, T + more, -1)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    px, pr = x[:, :T].reshape(-1, m.d).contiguous(), res[:, :T].reshape(-1, m.d).contiguous()
    out, _, cs, S = m.prefill(px, pr, B, B * T, cu=cu)
    # a bf16 result of the same inputs, computed with sums in another order: a step of its type
    torch.testing.assert_close(out.reshape(B, T, -1), full[:, :T], rtol=2 ** -6, atol=2 ** -6)
    for t in range(more):
        o, _ = m.step(x[:, T + t].contiguous(), res[:, T + t].contiguous(), cs, S)
        torch.testing.assert_close(o, full[:, T + t], rtol=2 ** -6, atol=2 ** -6)
    # the states hold bf16 roundings of the convolution's outputs, some of them one step apart
    assert torch.equal(cs, cs_full) or (cs.float() - cs_full.float()).abs().max() < 0.1
    assert (S - S_full).norm() <= 2 ** -7 * S_full.norm()


def test_calls_repeat_bit_for_bit_and_on_other_streams():
    k = Scan(BF, 1, 700, 2, 1, 32, 64)
    y, ST = k.fwd()
    a = k.bwd()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y1, S1 = k.fwd()
        b = k.bwd()
    with torch.cuda.stream(other):
        y2, S2 = k.fwd()
        c = k.bwd()
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(ST, S1) and torch.equal(y, y2) and torch.equal(ST, S2)
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), n


def test_captured_layer_replays():
    m, g = Layer(), gen(8)
    B = 2
    x, res = draw(g, B * 130, m.d), draw(g, B * 130, m.d)
    tx, tr = draw(g, B, m.d), draw(g, B, m.d)
    _, _, cs0, S0 = m.prefill(x, res, B, 130)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up
        m.prefill(x, res, B, 130)
        m.step(tx, tr, cs0.clone(), S0.clone())
    torch.cuda.current_stream().wait_stream(side)
    cs, S = cs0.clone(), S0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h, cs_p, S_p = m.prefill(x, res, B, 130)
        o, hs = m.step(tx, tr, cs, S)
    for i in range(4):
        x.copy_(draw(gen(20 + i), B * 130, m.d))
        tx.copy_(draw(gen(30 + i), B, m.d))
        cs_e, S_e = cs.clone(), S.clone()
        graph.replay()
        torch.cuda.synchronize()
        e_out, e_h, e_cs, e_S = m.prefill(x, res, B, 130)
        e_o, _ = m.step(tx, tr, cs_e, S_e)
        torch.cuda.synchronize()
        for a, b in ((out, e_out), (h, e_h), (cs_p, e_cs), (S_p, e_S), (o, e_o), (cs, cs_e), (S, S_e)):
            assert torch.equal(a, b), i


def test_captured_backward_replays():
    k = Scan(BF, 2, 140, 2, 1, 64, 64)
    g = gen(9)
    n, C = 2 * 140, 64
    x, w, dy = draw(g, n, C), draw(g, C, 4, dtype=F32), draw(g, n, C)
    cc = la.ConvConfig(B=2, T=140, C=C, width=4)
    nc = la.NormConfig(rows=n, d=C)

    def run():
        o = k.bwd_into(k.out_buffers())
        dx, dw, ds = torch.empty_like(x), torch.empty_like(w), torch.empty(2, 3, C, dtype=BF, device="cuda")
        b = la.la_conv_bwd_workspace_bytes(cc)
        la.la_conv_bwd(cc, x, w, None, None, dy, None, dx, dw, None, ds, torch.empty(b, dtype=torch.uint8, device="cuda"), b)
        nx, nw = torch.empty_like(x), torch.empty(C, device="cuda")
        b = la.la_norm_bwd_workspace_bytes(nc)
        la.la_norm_bwd(nc, x, None, dy, None, nx, nw, torch.empty(b, dtype=torch.uint8, device="cuda"), b)
        return [o[i] for i in sorted(o)] + [dx, dw, ds, nx, nw]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(3):
        x.copy_(draw(gen(40 + i), n, C))
        k.buf.copy_(draw(gen(50 + i), *k.buf.shape))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, run()):
            assert torch.equal(a, b), i


def test_binding_refuses_layouts():
    x = torch.zeros(2, 8, 64, dtype=BF, device="cuda")
    w = torch.zeros(64, 4, device="cuda")
    cfg = la.ConvConfig(B=2, T=8, C=64, width=4)
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="strides"):
        la.la_conv_fwd(cfg, x.transpose(0, 1), w, None, None, y)
    with pytest.raises(ValueError, match="holds 512"):
        la.la_conv_fwd(cfg, x[:1], w, None, None, y)
    with pytest.raises(ValueError, match="dtype"):
        la.la_conv_fwd(cfg, x.float(), w, None, None, y)
    with pytest.raises(ValueError, match="contiguous"):
        la.la_conv_fwd(cfg, x, torch.zeros(4, 64, device="cuda").t(), None, None, y)
    wide = torch.zeros(2, 8, 96, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="strides"):
        la.la_conv_fwd(cfg, wide[..., :64], w, None, None, y)
    la.la_conv_fwd(la.ConvConfig(B=2, T=8, C=64, width=4, ld_x=96), wide[..., 8:72], w, None, None, y)
    with pytest.raises(ValueError, match="GPU"):
        la.la_conv_fwd(cfg, x, w.cpu(), None, None, y)


@pytest.mark.parametrize("qdq,own,other", [(la.LA_QDQ_INT8_GROUP, torch.int8, torch.float8_e4m3fn),
                                           (la.LA_QDQ_E4M3_TILE, torch.float8_e4m3fn, torch.int8)])
def test_binding_takes_codes_of_the_quantizers_type(qdq, own, other):
    x, cfg = draw(gen(3), 4, 64), la.NormConfig(rows=4, d=64, qdq=qdq)
    got = []
    for t in (own, torch.uint8):
        codes = torch.empty(4, 64, dtype=t, device="cuda")
        la.la_norm_fwd(cfg, x, None, None, None, None, codes)
        got.append(codes.view(torch.uint8))
    assert torch.equal(*got) and got[0].any()
    for t in (other, torch.float8_e5m2, torch.bool, torch.float16):
        with pytest.raises(ValueError, match="codes has dtype"):
            la.la_norm_fwd(cfg, x, None, None, None, None, torch.empty(4, 64, dtype=t, device="cuda"))


def test_binding_takes_tensors_after_addresses_and_nulls():
    g = gen(4)
    x, w, st, y = draw(g, 2, 64), draw(g, 64, 4, dtype=F32), draw(g, 2, 3, 64), torch.empty(2, 64, dtype=BF, device="cuda")
    bias, want, first = draw(g, 64, dtype=F32), torch.empty_like(y), st.clone()
    cfg = la.ConvConfig(B=2, T=1, C=64, width=4)
    la.la_conv_step(cfg, x, w, bias, first, want)
    la.la_conv_step(cfg, x.data_ptr(), w.data_ptr(), bias, st.data_ptr(), y.data_ptr())
    assert torch.equal(y, want) and torch.equal(st, first)
    nc = la.NormConfig(rows=2, d=64, qdq=la.LA_QDQ_INT8_GROUP)
    scales, other = torch.empty(2, 1, device="cuda"), torch.empty(2, 1, device="cuda")
    la.la_norm_fwd(nc, x, None, None, None, None, None, scales)
    la.la_norm_fwd(nc, x.data_ptr(), None, None, None, None, None, other)
    assert torch.equal(scales, other)
    dST, dS0, dA = draw(g, 1, 2, 16, 64, dtype=F32), torch.empty(1, 2, 16, 64, device="cuda"), torch.ones(2, device="cuda")
    la.la_scan_bwd(la.ScanConfig(B=1, T=0, H=2, G=1, d_k=16, d_v=64), None, None, None, None, None, None, None, None, None, dST,
                   None, None, dA, None, None, None, None, dS0, None, 0)
    assert torch.equal(dS0, dST) and not dA.any()


# ----------------------------------------------------------------------- offsets past 32 bits
def zeros(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_convolution_and_norm_past_32_bits():
    """The last rows of tensors of more than 2^31 elements, the rest zeros: bit for bit what the
    rows alone give."""
    g = gen(11)
    T, C, n = 935000, 2304, 200
    assert T * C > 1 << 31
    x, w = zeros(T, C), draw(g, C, 4, dtype=F32)
    x[-n:] = draw(g, n, C)
    y, sT = zeros(T, C), zeros(1, 3, C)
    la.la_conv_fwd(la.ConvConfig(B=1, T=T, C=C, width=4), x, w, None, None, y, sT)
    tail, small = x[-n:].clone(), la.ConvConfig(B=1, T=n, C=C, width=4)
    yn, sn = zeros(n, C), zeros(1, 3, C)
    la.la_conv_fwd(small, tail, w, None, None, yn, sn)
    assert torch.equal(y[-n:], yn) and torch.equal(sT, sn)
    dxs, dws = [], []
    for cfg, xs in ((la.ConvConfig(B=1, T=T, C=C, width=4), x), (small, tail)):
        b = la.la_conv_bwd_workspace_bytes(cfg)
        ws = torch.empty(b, dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(xs), zeros(C, 4, dtype=F32)
        la.la_conv_bwd(cfg, xs, w, None, None, xs, None, dx, dw, None, None, ws, b)  # dy = x
        dxs.append(dx[-n:].clone())
        dws.append(dw)
        del dx
    assert torch.equal(*dxs)
    # the weights' sums take other orders: each an FP32 sum of at most 200 nonzero terms
    big = (tail.float().abs().amax(0) ** 2 * 1.1 * n * 2.0 ** -24 * n)[:, None]
    assert ((dws[0] - dws[1]).abs() <= big).all()
    del x, y
    rows, d = 263000, 8192
    assert rows * d > 1 << 31
    x = zeros(rows, d)
    x[-3:] = draw(g, 3, d)
    y, codes, scales = zeros(rows, d), zeros(rows, d, dtype=torch.uint8), zeros(rows, d // 64, dtype=F32)
    cfg = la.NormConfig(rows=rows, d=d, eps=1e-6, qdq=la.LA_QDQ_INT8_GROUP, group=64)
    la.la_norm_fwd(cfg, x, None, None, x, y, codes, scales)
    cfg.rows = 3
    t, yt, ct, st = x[-3:].clone(), zeros(3, d), zeros(3, d, dtype=torch.uint8), zeros(3, d // 64, dtype=F32)
    la.la_norm_fwd(cfg, t, None, None, t, yt, ct, st)
    assert torch.equal(y[-3:], yt) and torch.equal(codes[-3:], ct) and torch.equal(scales[-3:], st)
    assert not codes[0].any() and (scales[0] == 1).all()
    cfg = la.NormConfig(rows=rows, d=d, eps=1e-6)
    dx = torch.empty_like(x)
    la.la_norm_bwd(cfg, x, None, y, None, dx, None, None, 0)
    cfg.rows = 3
    dt = torch.empty_like(t)
    la.la_norm_bwd(cfg, t, None, yt, None, dt, None, None, 0)
    assert torch.equal(dx[-3:], dt) and not dx[0].any()


def test_scan_past_32_bits():
    """A packing of more than 2^31 elements whose last sequence begins behind them."""
    s = Scan(BF, 1, 200, 16, 1, 16, 128, states=False)
    T = (1 << 31) // (s.H * s.P) + 300
    def wide(t):  # noqa: E306
        big = zeros(T, t.shape[1], dtype=t.dtype)
        big[-200:] = t
        return big
    buf, dt, dy = wide(s.buf), wide(s.dt), wide(s.dy)
    x, b, c = s.cut(buf)
    cfg = la.ScanConfig(B=2, T=T, H=s.H, G=s.G, d_k=s.N, d_v=s.P, softplus=1, ld_x=s.ld, ld_b=s.ld, ld_c=s.ld)
    cu = cu_tensor([0, T - 200, T])
    n = max(la.la_scan_workspace_bytes(cfg), la.la_scan_bwd_varlen_workspace_bytes(cfg))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y, ST = zeros(T, s.H * s.P), torch.empty(2, s.H, s.N, s.P, device="cuda")
    la.la_scan_fwd(cfg, x, dt, s.A, b, c, s.D, s.bias, None, y, ST, ws, n, cu_seqlens=cu)
    dbuf = torch.empty_like(buf)
    dx, db, dc = s.cut(dbuf)
    o = dict(ddt=torch.empty_like(dt), dA=zeros(s.H, dtype=F32), dD=zeros(s.H, dtype=F32), ddt_bias=zeros(s.H, dtype=F32))
    la.la_scan_bwd(cfg, x, dt, s.A, b, c, s.D, s.bias, None, dy, None, dx, o["ddt"], o["dA"], db, dc, o["dD"], o["ddt_bias"],
                   None, ws, n, cu_seqlens=cu)
    w, m = s.reference(True)
    share, once = 2.0 ** -14, 2.0 ** -8
    close(y[-200:].reshape(w["y"].shape), w["y"], m["y"], share, "y")
    close(ST[1:], w["S_T"], m["S_T"], share, "S_T")
    for k, t in dict(dx=dx, db=db, dc=dc).items():
        close(t[-200:].reshape(w[k].shape), w[k], m[k], share + once, k)
    close(o["ddt"][-200:], w["ddt"], m["ddt"], share, "ddt")
    for k in ("dA", "dD", "ddt_bias"):
        close(o[k], w[k], m[k], share, k)
    assert not y[0].any() and not ST[0].any() and not dx[0].any() and not o["ddt"][0].any()


def test_state_pools_past_32_bits():
    """A live slot behind 2^32 bytes (and 2^31 elements) of a pool."""
    g = gen(12)
    H, N, P, n = 8, 64, 64, 66000
    assert (n - 1) * H * N * P > 1 << 31
    x, dt, b, c = draw(g, 1, H * P), draw(g, 1, H), draw(g, 1, N), draw(g, 1, N)
    A, S = -torch.rand(H, generator=g).cuda(), draw(g, 1, H, N, P, dtype=F32)
    cfg = la.ScanConfig(B=1, T=1, H=H, G=1, d_k=N, d_v=P, softplus=1)
    pool = zeros(n, H, N, P, dtype=F32)
    pool[n - 1] = S[0]
    y, yp = zeros(1, H * P), zeros(1, H * P)
    slot = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    la.la_scan_step(cfg, x, dt, A, b, c, None, None, pool, yp, slots=slot, n_slots=n)
    la.la_scan_step(cfg, x, dt, A, b, c, None, None, S, y)
    assert y.any() and torch.equal(y, yp) and torch.equal(pool[n - 1], S[0]) and not pool[:2].any()
    del pool
    C, W, n = 8192, 4, 90000
    assert (n - 1) * (W - 1) * C > 1 << 31
    x, w, st = draw(g, 1, C), draw(g, C, W, dtype=F32), draw(g, 1, W - 1, C)
    cfg = la.ConvConfig(B=1, T=1, C=C, width=W)
    pool = zeros(n, W - 1, C)
    pool[n - 1] = st[0]
    y, yp = zeros(1, C), zeros(1, C)
    slot[0] = n - 1
    la.la_conv_step(cfg, x, w, None, pool, yp, slots=slot, n_slots=n)
    la.la_conv_step(cfg, x, w, None, st, y)
    assert y.any() and torch.equal(y, yp) and torch.equal(pool[n - 1], st[0]) and not pool[:2].any()


def test_scan_gradients_without_tokens_past_32_bits():
    """T = 0: more than 2^32 elements of the states' gradient pass through."""
    B, H, N, P = 4097, 64, 128, 128
    assert B * H * N * P > 1 << 32
    cfg = la.ScanConfig(B=B, T=0, H=H, G=1, d_k=N, d_v=P)
    dST, dS0 = torch.ones(B, H, N, P, device="cuda"), zeros(B, H, N, P, dtype=F32)
    dST[-1] = draw(gen(1), H, N, P, dtype=F32)
    dA = torch.ones(H, device="cuda")
    la.la_scan_bwd(cfg, None, None, None, None, None, None, None, None, None, dST, None, None, dA, None, None, None, None, dS0,
                   None, 0)
    assert torch.equal(dS0[-1], dST[-1]) and (dS0[:-1].amin(dim=(1, 2, 3)) == 1).all() and not dA.any()


@pytest.mark.parametrize("cu", [None, [0, 0, 0], [0, 1, 1]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_conv_of_no_or_one_token_passes_its_states(dtype, cu):
    """Sequences shorter than the state: its later rows move up, and their gradient comes back."""
    g = gen(13)
    T, C, W = cu[-1] if cu else 0, 40, 4
    x, w, s0, dsT = draw(g, T, C, dtype=dtype), draw(g, C, W, dtype=F32), draw(g, 2, W - 1, C, dtype=dtype), draw(g, 2, W - 1, C, dtype=dtype)
    cfg = la.ConvConfig(B=2, T=T, C=C, width=W, x_dtype=CODE[dtype])
    y, sT, dx, ds0, dw = torch.empty_like(x), torch.empty_like(s0), torch.empty_like(x), torch.empty_like(s0), torch.ones(C, W, device="cuda")
    la.la_conv_fwd(cfg, x, w, None, s0, y, sT, cu_seqlens=cu_tensor(cu))
    n = la.la_conv_bwd_workspace_bytes(cfg)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    la.la_conv_bwd(cfg, x, w, None, s0, torch.zeros_like(x), dsT, dx, dw, None, ds0, ws, n, cu_seqlens=cu_tensor(cu))
    assert not dw.any() and torch.equal(sT[1], s0[1]) and torch.equal(ds0[1], dsT[1])
    if T:
        assert torch.equal(sT[0], torch.cat([s0[0, 1:], x])) and torch.equal(dx, dsT[0, 2:])
        assert torch.equal(ds0[0, 1:], dsT[0, :2]) and not ds0[0, 0].any()
    else:
        assert torch.equal(sT, s0) and torch.equal(ds0, dsT)
