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
    (1500, 2001, 144, BF, BF, F32, 0, 0, F32),
    (3000, 3100, 208, BF, F32, BF, 16, 4, F32),
    (2900, 3333, 80, F32, BF, BF, 0, 0, None),
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


# ---------------------------------------------------------------------- norms around a block
# Tolerances: a row's mean in FP32 is at most 64 terms a lane and a tree of 10, (74 x 2^-24) of its
# magnitude, half of it in a root; the gate within (|z| + 2) 2^-23 (|z| < 8: 2^-19); a handful of products:
# 2^-17 forward.  The backward takes two such means after each other and products of both: 2^-15 of the
# magnitude.  The parameters' sums add FP32 sums over a workgroup's rows (at most 16 here): 2^-15 too.  As such
# errors are independent, the 2-norm of what FP32 results are off by is far smaller: 2^-20 of the result's.
GATE = [
    # type, y's type, weights' type, rows, d, head, gate, first, post, pre, residual, alpha, extra columns of x, z
    (BF, BF, F32, 1, 8, 0, 1, 0, 1, 1, 1, 1, 0, 0),
    (BF, BF, F32, 4, 2048, 128, 1, 0, 1, 0, 0, 0, 0, 0),
    (F32, F32, F32, 33, 64, 16, 2, 0, 1, 1, 1, 1, 8, 16),
    (BF, F32, BF, 7, 520, 0, 0, 0, 1, 1, 1, 1, 0, 0),
    (F32, BF, F32, 5, 1024, 512, 1, 1, 1, 1, 1, 0, 0, 8),
    (BF, BF, BF, 65, 256, 256, 2, 0, 1, 0, 0, 1, 16, 0),
    (F32, F32, F32, 31, 504, 0, 1, 1, 1, 1, 0, 1, 0, 0),
    (BF, BF, F32, 9, 4096, 32, 1, 0, 1, 0, 0, 0, 0, 4096),
    (BF, BF, F32, 6, 16384, 0, 1, 0, 1, 1, 1, 1, 0, 0),
    (F32, F32, F32, 3, 16384, 64, 2, 0, 1, 1, 1, 1, 0, 0),
    (F32, F32, F32, 17, 200, 0, 1, 0, 0, 0, 0, 0, 0, 0),
    (BF, BF, F32, 300, 2048, 0, 0, 0, 1, 1, 1, 1, 0, 0),
    (F32, F32, F32, 40, 128, 0, 0, 0, 0, 1, 1, 1, 0, 0),
    (F32, F32, F32, 2, 8192, 128, 1, 0, 1, 1, 1, 1, 0, 0),
    (BF, F32, F32, 12, 6144, 0, 2, 1, 1, 0, 1, 1, 0, 0),
    (F32, F32, F32, 1000, 512, 64, 1, 0, 1, 1, 1, 1, 0, 0),
    (F32, F32, F32, 11, 32, 32, 0, 0, 1, 0, 0, 0, 0, 0),
    (BF, BF, F32, 21, 1024, 0, 1, 0, 1, 1, 1, 1, 0, 0),
    (F32, F32, F32, 13, 1152, 128, 2, 0, 1, 1, 1, 1, 0, 0),
    (BF, F32, F32, 19, 2304, 256, 1, 1, 1, 1, 1, 1, 8, 0),
    (F32, F32, BF, 800, 2056, 0, 0, 0, 1, 1, 1, 1, 0, 0),
    (BF, BF, F32, 10, 8192, 512, 1, 0, 1, 1, 1, 1, 0, 0),
    (BF, BF, F32, 7, 10240, 0, 0, 0, 1, 1, 1, 1, 0, 0),
]


def gate_case(k, **codec):
    t, o, tw, rows, d, head, act, first, post, pre, res, alpha, ex, ez = GATE[k]
    g = gen(300 + k)
    s = dict(x=wider(g, rows, d, ex, t)[1], z=wider(g, rows, d, ez, t)[1] if act else None,
             w_post=draw(g, head or d, dtype=tw, scale=0.2).add_(1.0) if post else None,
             alpha=draw(g, d, dtype=tw, scale=0.5) if alpha else None, residual=draw(g, rows, d, dtype=t, scale=2.0) if res else None,
             w_pre=draw(g, d, dtype=tw, scale=0.2).add_(1.0) if pre else None)
    cfg = la.GateNormConfig(rows=rows, d=d, head=head, eps=1e-5, gate=act, gate_first=first, post=post, pre=pre, x_dtype=CODE[t],
                            w_dtype=CODE[tw], out_dtype=CODE[o], ld_x=d + ex if ex else 0, ld_z=d + ez if ez else 0, **codec)
    return cfg, g, s


def gate_ref(k, s, h):
    _, _, _, _, _, head, act, first, post, pre = GATE[k][:10]
    return R.gate_norm_fwd(*[None if v is None else np64(v) for v in s.values()], head, 1e-5, act, first, post, pre,
                           None if h is None or not pre else np64(h))


def two_norm(got, want, bound, name):
    if got.dtype is F32 and np.abs(want).max() > 0:
        e = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
        assert e <= bound, (name, e)


@pytest.mark.parametrize("k", range(len(GATE)))
def test_gate_norm_fwd(k):
    t, o, _, rows, d = GATE[k][:5]
    cfg, g, s = gate_case(k)
    h = torch.full((rows, d), float("nan"), dtype=t, device="cuda")
    y = torch.full((rows, d), float("nan"), dtype=o, device="cuda")
    la.la_gate_norm_fwd(cfg, *s.values(), h, y)
    want_t, want_v, keep = gate_ref(k, s, h)
    res = 0 if s["residual"] is None else np.abs(np64(s["residual"]))
    mag = np.abs(keep["a"] * keep["p"]) + res
    close(h, want_t, mag, 2.0 ** -17, "h")
    close(y, want_v, np.abs(want_v) if cfg.pre else mag, 2.0 ** -17, "y")
    two_norm(y, want_v, 2.0 ** -20, "y")
    # in place, and each output alone
    if s["residual"] is not None:
        both = s["residual"].clone()
        la.la_gate_norm_fwd(cfg, *{**s, "residual": both}.values(), both, None)
        assert torch.equal(both, h)
    y2 = torch.full_like(y, float("nan"))
    la.la_gate_norm_fwd(cfg, *s.values(), None, y2)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("codec", ["int8", "e4m3"])
@pytest.mark.parametrize("k", range(len(GATE)))
def test_gate_norm_codes(k, codec):
    t, o, _, rows, d = GATE[k][:5]
    fits = [0] + [n for n in (16, 32, 64, 128) if d % n == 0]
    group = fits[k % len(fits)]
    cfg, g, s = gate_case(k, qdq=la.LA_QDQ_INT8_GROUP if codec == "int8" else la.LA_QDQ_E4M3_TILE, group=group)
    h = torch.empty(rows, d, dtype=t, device="cuda")
    y = torch.empty(rows, d, dtype=o, device="cuda")
    typ = torch.int8 if codec == "int8" else torch.float8_e4m3fn
    codes = torch.empty(rows, d, dtype=typ, device="cuda")
    scales = torch.full((rows, d // (group or d)), float("nan"), device="cuda")
    la.la_gate_norm_fwd(cfg, *s.values(), h, y, codes, scales)
    _, v, keep = gate_ref(k, s, h)
    width = group or d
    res = 0 if s["residual"] is None else np.abs(np64(s["residual"]))
    err = 2.0 ** -17 * (np.abs(v) if cfg.pre else np.abs(keep["a"] * keep["p"]) + res)
    top = np.abs(v).reshape(rows, -1, width).max(2)
    slack = err.reshape(rows, -1, width).max(2)
    sc = np64(scales)
    assert (np.abs(sc - top / (127 if codec == "int8" else 448)) <= slack / (127 if codec == "int8" else 448) + 2.0 ** -23 * sc).all()
    value = codes.float() * scales.repeat_interleave(width, 1)
    assert torch.equal(value.to(o), y)
    wide = np.repeat(sc, width, 1)
    # half a step: of the integers, or of E4M3's three bits of mantissa (2^-4 of the value; 2^-10 below the smallest normal)
    step = 0.5 * wide if codec == "int8" else np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * wide)
    assert (np.abs(np64(value) - v) <= step * 1.0001 + err).all()
    # without y and in the other type
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    la.la_gate_norm_fwd(cfg, *s.values(), None, None, c2.view(torch.uint8), s2)
    other = la.GateNormConfig(*[getattr(cfg, n) for n, _ in cfg._fields_])
    other.out_dtype = 1 - cfg.out_dtype
    c3, s3 = torch.empty_like(codes), torch.empty_like(scales)
    la.la_gate_norm_fwd(other, *s.values(), None, torch.empty(rows, d, dtype=F32 if o is BF else BF, device="cuda"), c3, s3)
    for c, q in ((c2, s2), (c3, s3)):
        assert torch.equal(c.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(q, scales)


@pytest.mark.parametrize("k", range(len(GATE)))
def test_gate_norm_bwd(k):
    t, o, _, rows, d, head, act, first, post, pre, res = GATE[k][:11]
    cfg, g, s = gate_case(k)
    h = torch.empty(rows, d, dtype=t, device="cuda")
    la.la_gate_norm_fwd(cfg, *s.values(), h, None)
    dy = draw(g, rows, d, dtype=o)
    dh = draw(g, rows, d, dtype=t) if res else None
    nan = lambda *shape, dtype=F32: torch.full(shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    dx = nan(rows, cfg.ld_x or d, dtype=t)[:, :d]
    dz = nan(rows, cfg.ld_z or d, dtype=t)[:, :d] if act else None
    dres = nan(rows, d, dtype=t)
    out = dict(dx=dx, dz=dz, dres=dres, dw_post=nan(head or d) if post else None, dalpha=nan(d), dw_pre=nan(d) if pre else None)
    n = la.la_gate_norm_bwd_workspace_bytes(cfg)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    args = (s["x"], s["z"], s["w_post"], s["alpha"], h if pre else None, s["w_pre"], dy, dh)
    la.la_gate_norm_bwd(cfg, *args, *out.values(), ws, n)
    keep = gate_ref(k, s, h)[2]
    x64, dy64, dh64 = np64(s["x"]), np64(dy), None if dh is None else np64(dh)
    want = R.gate_norm_bwd(x64, keep, dy64, dh64, first, post, pre)
    mag = R.gate_norm_bwd(x64, keep, dy64, dh64, first, post, pre, mag=True)
    for (name, got), w, m in zip(out.items(), want, mag):
        if got is not None:
            close(got, w, m, 2.0 ** -15, name)
            two_norm(got, w, 2.0 ** -20 * max(1.0, np.linalg.norm(m) / np.linalg.norm(w)), name)
    # dres in dh's place, and without what may be missing
    both = dh.clone() if dh is not None else None
    dx2 = torch.empty(rows, cfg.ld_x or d, dtype=t, device="cuda")[:, :d]
    la.la_gate_norm_bwd(cfg, *args[:7], both, dx2, None, both, None, None, None, None, 0)
    assert torch.equal(dx2, dx) and (both is None or torch.equal(both, dres))


def test_linear_extremes():
    """The integer sum at its largest, scales of zero, infinity and NaN, all tokens' counts around the tiles."""
    K = 65536
    xc = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    wc = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    wc[1], wc[2, ::2] = 127, 0
    xs, ws = torch.tensor([1.0, 0.0, 2.0 ** -30], device="cuda"), torch.ones(5, device="cuda")
    y = torch.empty(3, 5, device="cuda")
    la.la_linear_fwd(la.LinearConfig(M=3, N=5, K=K, out_dtype=la.LA_F32), xc, xs, wc, ws, None, y)
    exact = (xc.cpu().long() @ wc.cpu().long().T).double() * xs.cpu().double()[:, None]
    assert torch.equal(y.cpu(), exact.float())
    for M in (3, 70, 130):
        xc, xs = codes(gen(1), M, 64)
        wc, ws = codes(gen(2), 200, 64)
        clean = torch.empty(M, 200, device="cuda")
        cfg = la.LinearConfig(M=M, N=200, K=64, out_dtype=la.LA_F32)
        la.la_linear_fwd(cfg, xc, xs, wc, ws, None, clean)
        xs[M - 1], ws[7], ws[8] = float("nan"), float("inf"), float("nan")
        y = torch.empty_like(clean)
        la.la_linear_fwd(cfg, xc, xs, wc, ws, None, y)
        keep = [n for n in range(200) if n not in (7, 8)]
        assert torch.equal(y[:M - 1][:, keep], clean[:M - 1][:, keep])  # nothing leaves its row or column
        assert y[M - 1].isnan().all() and y[:, 8].isnan().all() and not y[:, 7].isfinite().any()


@pytest.mark.parametrize("tx,tw", [(BF, BF), (F32, F32)])
def test_linear_bwd_infinities_stay_in_their_rows(tx, tw):
    M, N, K = 150, 140, 96
    xc, xs = codes(gen(3), M, K)
    wc, ws = codes(gen(4), N, K)
    wc[wc == 0] = 1
    xc[xc == 0] = 1
    cfg = la.LinearConfig(M=M, N=N, K=K, out_dtype=la.LA_F32, x_dtype=CODE[tx], dw_dtype=CODE[tw])
    n = la.la_linear_bwd_workspace_bytes(cfg)
    ws_ = torch.empty(n, dtype=torch.uint8, device="cuda")

    def grads(dy):
        out = torch.empty(M, K, dtype=tx, device="cuda"), torch.empty(N, K, dtype=tw, device="cuda"), torch.empty(N, device="cuda")
        la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, *out, ws_, n)
        return out

    dy = draw(gen(5), M, N, dtype=F32)
    dy[20] = 0.0   # a token without a gradient
    dy[:, 30] = 0.0
    clean = grads(dy)
    assert (clean[0][20] == 0).all() and (clean[1][30] == 0).all() and clean[2][30] == 0
    dy[3, 5], dy[90, 100] = float("inf"), float("nan")
    dx, dw, db = grads(dy)
    rows, cols = [m for m in range(M) if m not in (3, 90)], [k for k in range(N) if k not in (5, 100)]
    assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dw[cols], clean[1][cols]) and torch.equal(db[cols], clean[2][cols])
    # one infinity times codes that are not zero is an infinity of their sign
    assert torch.equal(dx[3].float(), torch.sign(wc[5].float()) * float("inf")) and torch.equal(dw[5].float(), torch.sign(xc[3].float()) * float("inf"))
    assert dx[90].isnan().all() and dw[100].isnan().all() and db[5] == float("inf") and db[100].isnan()


def test_linear_bwd_keeps_the_bits_of_its_type():
    """Errors of the operands are independent: the 2-norm of a bf16 gradient's stays that of its own rounding
    (2^-8 / sqrt(12) to 2^-8 / sqrt(3) of a value, a little less than 2^-9.2 on average over a binade; 2^-9 with
    the operands' 2^-11), of an FP32 one's below 2^-20."""
    M, N, K = 1000, 640, 528
    xc, xs = codes(gen(6), M, K)
    wc, ws = codes(gen(7), N, K)
    dy = draw(gen(8), M, N, scale=1e-4) * torch.exp(draw(gen(9), M, 1, dtype=F32)).to(BF)
    for tx, bound in ((BF, 2.0 ** -9), (F32, 2.0 ** -20)):
        cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=CODE[tx], dw_dtype=CODE[tx])
        n = la.la_linear_bwd_workspace_bytes(cfg)
        dx, dw = torch.empty(M, K, dtype=tx, device="cuda"), torch.empty(N, K, dtype=tx, device="cuda")
        la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, dx, dw, None, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
        for got, want in zip((dx, dw), R.linear_bwd(*[np64(v) for v in (xc, xs, wc, ws, dy)])):
            assert np.linalg.norm(np64(got) - want) <= bound * np.linalg.norm(want)


def test_linear_without_tokens_or_channels():
    for M, N in ((0, 40), (40, 0)):
        cfg = la.LinearConfig(M=M, N=N, K=64, out_dtype=la.LA_F32, x_dtype=la.LA_F32)
        xc, xs = codes(gen(1), M, 64)
        wc, ws = codes(gen(2), N, 64)
        n = la.la_linear_bwd_workspace_bytes(cfg)
        out = [torch.full(s, 7.0, device="cuda") for s in ((M, 64), (N, 64), (N,))]
        la.la_linear_bwd(cfg, xc, xs, wc, ws, torch.empty(M, N, device="cuda"), *out, torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n)
        assert all((v == 0).all() for v in out)


def test_linear_past_32_bits():
    M, N, K, ld = (1 << 20) + 3, 4104, 16, 4112
    xc = torch.zeros(M, ld, dtype=torch.int8, device="cuda")
    xc[-200:, :K] = codes(gen(1), 200, K)[0]
    wc, ws = codes(gen(2), N, K)
    xs = torch.ones(M, device="cuda")
    y = torch.empty(M, N, dtype=BF, device="cuda")
    la.la_linear_fwd(la.LinearConfig(M=M, N=N, K=K, ld_x=ld), xc[:, :K], xs, wc, ws, None, y)
    want = (xc[-200:, :K].float() @ wc.float().T * ws).to(BF)
    assert torch.equal(y[-200:], want) and (y[0] == 0).all()
    del y
    # the backward: rows of dx and of the laid out operands past 2^32 elements
    M, N, K = 1 << 19, 24, 8320
    xc = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    xc[-64:] = codes(gen(3), 64, K)[0]
    wc, ws = codes(gen(4), N, K)
    dy = torch.zeros(M, N, device="cuda")
    dy[-64:] = draw(gen(5), 64, N, dtype=F32)
    xs = torch.full((M,), 0.01, device="cuda")
    cfg = la.LinearConfig(M=M, N=N, K=K, out_dtype=la.LA_F32)
    n = la.la_linear_bwd_workspace_bytes(cfg)
    dx, dw = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(N, K, device="cuda")
    la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, dx, dw, None, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    args = [np64(xc[-64:]), np64(xs[-64:]), np64(wc), np64(ws), np64(dy[-64:])]
    want, mag = R.linear_bwd(*args), R.linear_bwd(*[np.abs(a) for a in args])
    close(dx[-64:], want[0], mag[0], 2.0 ** -11 + 25 * 2.0 ** -23, "dx")
    close(dw, want[1], mag[1], 2.0 ** -22 + 65 * 2.0 ** -23, "dweight")
    assert (dx[:64] == 0).all()


def test_gate_norm_past_32_bits():
    rows, d = (1 << 18) + 77, 16384
    x = torch.zeros(rows, d, dtype=BF, device="cuda")
    x[-3:] = draw(gen(1), 3, d)
    w = draw(gen(2), d, dtype=F32)
    codes_, scales = torch.empty(rows, d, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    la.la_gate_norm_fwd(la.GateNormConfig(rows=rows, d=d, pre=0, qdq=la.LA_QDQ_INT8_GROUP), x, None, w, None, None, None, None, None, codes_, scales)
    c3, s3 = torch.empty(3, d, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    la.la_gate_norm_fwd(la.GateNormConfig(rows=3, d=d, pre=0, qdq=la.LA_QDQ_INT8_GROUP), x[-3:], None, w, None, None, None, None, None, c3, s3)
    assert torch.equal(codes_[-3:], c3) and torch.equal(scales[-3:], s3) and (codes_[:3] == 0).all() and (scales[:3] == 1).all()
    dy = x  # (any values)
    dx = torch.empty_like(x)
    la.la_gate_norm_bwd(la.GateNormConfig(rows=rows, d=d), x, None, w, None, None, None, dy, None, dx, None, None, None, None, None, None, 0)
    d3 = torch.empty_like(x[-3:])
    la.la_gate_norm_bwd(la.GateNormConfig(rows=3, d=d), x[-3:], None, w, None, None, None, dy[-3:], None, d3, None, None, None, None, None, None, 0)
    assert torch.equal(dx[-3:], d3) and (dx[:3] == 0).all()


@pytest.mark.parametrize("d,head", [(64, 16), (520, 0), (2048, 128), (4096, 0), (16384, 0)])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("codec", ["none", "int8", "e4m3"])
def test_gate_norm_infinities_and_nan(d, head, t, codec):
    """They stay in their row, reach its head or the row by the formula, and codes are defined."""
    qdq = dict(none=la.LA_QDQ_NONE, int8=la.LA_QDQ_INT8_GROUP, e4m3=la.LA_QDQ_E4M3_TILE)[codec]
    cfg = la.GateNormConfig(rows=5, d=d, head=head, gate=la.LA_GATE_SIGMOID, qdq=qdq, x_dtype=CODE[t], out_dtype=la.LA_F32)
    x, z = draw(gen(1), 5, d, dtype=t), draw(gen(2), 5, d, dtype=t)
    x[1] = 0.0
    z[4, :3] = torch.tensor([float("inf"), float("-inf"), -200.0]).to(t)

    def run():
        y = torch.empty(5, d, device="cuda")
        c = torch.empty(5, d, dtype=torch.uint8, device="cuda") if qdq else None
        s = torch.empty(5, device="cuda") if qdq else None
        la.la_gate_norm_fwd(cfg, x, z, None, None, None, None, None, y, c, s)
        return y, c, s

    clean = run()
    assert clean[0].isfinite().all() and (clean[0][1] == 0).all() and (clean[0][4, 1:3] == 0).all()
    x[2, 8], x[3, 8] = float("nan"), float("inf")
    y, c, s = run()
    for a, b in zip((y, c, s), clean):
        assert a is None or all(torch.equal(a[r], b[r]) for r in (0, 1, 4))
    assert y[2, 8].isnan() and y[3, 8].isnan()  # inf / rms(inf)
    if codec != "none":
        assert s[2].isnan() and s[3].isnan() and y[2].isnan().all() and ((c[2] == 0) if codec == "int8" else (c[2] & 0x7F) == 0x7F).all()  # (E4M3 has a NaN of each sign)
    else:
        width = head or d
        assert y[2, :width].isnan().all() and (y[3, :8] == 0).all() and (width == d or y[2:4, width:].isfinite().all())


# ------------------------------------------------------------------------------ used together
def layer(s, cfgs):
    """A layer from the recurrence's output to the next one's projected input: gated norm to codes, output
    projection, join to the residual stream and codes, input projection."""
    g, o, j, i = cfgs
    la.la_gate_norm_fwd(g, s["o"], s["z"], s["w_o"], None, None, None, None, None, s["c0"], s["s0"])
    la.la_linear_fwd(o, s["c0"], s["s0"], s["wo"][0], s["wo"][1], None, s["y0"])
    la.la_gate_norm_fwd(j, s["y0"], None, s["w_post"], s["alpha"], s["res"], s["w_pre"], s["h"], None, s["c1"], s["s1"])
    la.la_linear_fwd(i, s["c1"], s["s1"], s["wi"][0], s["wi"][1], None, s["y1"])


def layer_case(rows, H=4, hd=64, model=512, out=776):
    g = gen(11)
    d = H * hd

    def weight(n, k):
        w = draw(g, n, k, scale=k ** -0.5)
        c, s = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        la.la_gate_norm_fwd(la.GateNormConfig(rows=n, d=k, post=0, qdq=la.LA_QDQ_INT8_GROUP), w, None, None, None, None, None, None, None, c, s)
        return c, s

    e = lambda *shape, dtype=BF: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(o=draw(g, rows, d), z=draw(g, rows, d), w_o=draw(g, hd, dtype=F32, scale=0.1) + 1, wo=weight(model, d), wi=weight(out, model),
             w_post=draw(g, model, dtype=F32, scale=0.1) + 1, alpha=draw(g, model, dtype=F32, scale=0.1) + 0.5, res=draw(g, rows, model, scale=2.0),
             w_pre=draw(g, model, dtype=F32, scale=0.1) + 1, c0=e(rows, d, dtype=torch.int8), s0=e(rows, dtype=F32), y0=e(rows, model),
             h=e(rows, model), c1=e(rows, model, dtype=torch.int8), s1=e(rows, dtype=F32), y1=e(rows, out))
    cfgs = (la.GateNormConfig(rows=rows, d=d, head=hd, gate=la.LA_GATE_SILU, qdq=la.LA_QDQ_INT8_GROUP),
            la.LinearConfig(M=rows, N=model, K=d),
            la.GateNormConfig(rows=rows, d=model, pre=1, qdq=la.LA_QDQ_INT8_GROUP),
            la.LinearConfig(M=rows, N=out, K=model))
    return s, cfgs


@pytest.mark.parametrize("rows", [1, 5, 300])
def test_layer_in_8_bits(rows):
    """Against the same path in 64 bits with its own rounding to codes: 8-bit steps of independent errors, each
    1/254 of a row's largest value at most, about 1% of a result's root mean square in each of two products."""
    s, cfgs = layer_case(rows)
    layer(s, cfgs)
    v = {k: np64(t) for k, t in s.items() if torch.is_tensor(t)}
    wo, wi = [np64(c) * np64(sc)[:, None] for c, sc in (s["wo"], s["wi"])]
    n0 = R.gate_norm_fwd(v["o"], v["z"], v["w_o"], None, None, None, 64, 1e-6, 1, 0, 1, 0)[1]
    t, n1, _ = R.gate_norm_fwd(n0 @ wo.T, None, v["w_post"], v["alpha"], v["res"], v["w_pre"], 0, 1e-6, 0, 0, 1, 1)
    for got, want, bound in (("h", t, 0.01), ("y1", n1 @ wi.T, 0.03)):
        e = np.linalg.norm(v[got] - want) / np.linalg.norm(want)
        assert e <= bound, (got, e)
    # the pieces, from the codes that the GPU has
    close(s["y0"], R.linear_fwd(v["c0"], v["s0"], np64(s["wo"][0]), np64(s["wo"][1]), None), np.abs(v["y0"]), 2.0 ** -22, "y0")
    close(s["y1"], R.linear_fwd(v["c1"], v["s1"], np64(s["wi"][0]), np64(s["wi"][1]), None), np.abs(v["y1"]), 2.0 ** -22, "y1")


def test_layer_captured_and_on_another_stream():
    s, cfgs = layer_case(37)
    layer(s, cfgs)
    outs = ("c0", "s0", "y0", "h", "c1", "s1", "y1")
    want = {k: s[k].clone() for k in outs}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in outs:
        s[k].zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(s, cfgs)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s[k], want[k]) for k in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(s, cfgs)
    for r in range(3):
        for k in outs:
            s[k].zero_()
        s["o"].mul_(2.0 if r == 1 else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: s[k].clone() for k in outs}
        layer(s, cfgs)
        assert all(torch.equal(s[k], got[k]) for k in outs), r


@pytest.mark.parametrize("t", [BF, F32])
def test_training_step_captured(t):
    """Forward and backward of both operators in one graph, replayed with new gradients among eager work."""
    M, N, K = 333, 264, 512
    g = gen(21)
    xc, xs = codes(g, M, K)
    wc, ws = codes(g, N, K)
    cfg = la.LinearConfig(M=M, N=N, K=K, out_dtype=CODE[t], x_dtype=CODE[t])
    gate = la.GateNormConfig(rows=M, d=N, gate=la.LA_GATE_SILU, pre=1, x_dtype=CODE[t], out_dtype=CODE[t])
    z, res, dv, dh = (draw(g, M, N, dtype=t) for _ in range(4))
    wp, al, w2 = (draw(g, N, dtype=F32, scale=0.1) + 1 for _ in range(3))
    n1, n2 = la.la_linear_bwd_workspace_bytes(cfg), la.la_gate_norm_bwd_workspace_bytes(gate)
    ws1, ws2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (n1, n2))
    e = lambda *shape, dtype=t: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    out = dict(y=e(M, N), h=e(M, N), v=e(M, N), dy=e(M, N), dz=e(M, N), dres=e(M, N), dwp=e(N, dtype=F32), dal=e(N, dtype=F32), dw2=e(N, dtype=F32),
               dx=e(M, K), dw=e(N, K, dtype=F32), db=e(N, dtype=F32))

    def step():
        la.la_linear_fwd(cfg, xc, xs, wc, ws, None, out["y"])
        la.la_gate_norm_fwd(gate, out["y"], z, wp, al, res, w2, out["h"], out["v"])
        la.la_gate_norm_bwd(gate, out["y"], z, wp, al, out["h"], w2, dv, dh, out["dy"], out["dz"], out["dres"], out["dwp"], out["dal"], out["dw2"], ws2, n2)
        la.la_linear_bwd(cfg, xc, xs, wc, ws, out["dy"], out["dx"], out["dw"], out["db"], ws1, n1)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        dv.copy_(draw(gen(30 + r), M, N, dtype=t, scale=10.0 ** -r))
        step()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in out.items()}
        for v in out.values():
            v.fill_(float("nan"))
        ws1.fill_(0xFF), ws2.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in out), r
    assert all(v.isfinite().all() for v in out.values())


def test_two_streams_with_workspaces_of_their_own():
    M, N, K = 700, 520, 272
    streams = [torch.cuda.Stream() for _ in range(2)]
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=la.LA_F32)
    n = la.la_linear_bwd_workspace_bytes(cfg)
    cases = []
    for k in range(2):
        xc, xs = codes(gen(40 + k), M, K)
        wc, ws = codes(gen(50 + k), N, K)
        dy = draw(gen(60 + k), M, N)
        outs = [[torch.empty(s, device="cuda") for s in ((M, K), (N, K), (N,))] for _ in range(2)]
        cases.append((xc, xs, wc, ws, dy, outs, torch.empty(n, dtype=torch.uint8, device="cuda")))
        la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, *outs[0], cases[-1][-1], n)
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (xc, xs, wc, ws, dy, outs, space) in zip(streams, cases):
            la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, *outs[1], space, n, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for c in cases for a, b in zip(*c[5]))


@pytest.mark.parametrize("M,N", [(192, 512), (130, 520)])
@pytest.mark.parametrize("t", [BF, F32])
def test_linear_bwd_other_rows_beside_an_infinity(M, N, t):
    """Largest magnitudes are the finite values' in whole blocks of rows and columns and in parts of them."""
    K = 64
    g = gen(11)
    (xc, xs), (wc, ws) = codes(gen(3), M, K), codes(gen(4), N, K)
    # (magnitudes over 2^40: a maximum lost or taken too high leaves nothing of the values)
    dy = (draw(g, M, N, dtype=F32) * torch.exp2(torch.randint(-20, 21, (M, 1), generator=g).float()).cuda()).to(t)
    dy[3, 5], dy[65, 300], dy[129, N - 1] = float("inf"), float("-inf"), float("nan")
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=la.LA_F32, out_dtype=CODE[t], dw_dtype=la.LA_F32)
    n = la.la_linear_bwd_workspace_bytes(cfg)
    dx, dw, db = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    la.la_linear_bwd(cfg, xc, xs, wc, ws, dy, dx, dw, db, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    rows, cols = [m for m in range(M) if m not in (3, 65, 129)], [c for c in range(N) if c not in (5, 300, N - 1)]
    for a, bad in ((dx, (3, 65, 129)), (dw, (5, 300, N - 1))):
        assert not any(a[i].isfinite().any() for i in bad)
    held = dy.clone()
    held[~held.isfinite()] = 0.0
    args = [np64(xc), np64(xs), np64(wc), np64(ws), np64(held)]
    want, mag = R.linear_bwd(*args), R.linear_bwd(*[np.abs(a) for a in args])
    close(dx[rows], want[0][rows], mag[0][rows], 2.0 ** -22 + (N + 2) * 2.0 ** -23, "dx")
    # a column's smaller rows: 2^-29 of its largest value
    top = (np.abs(args[4]) * args[1][:, None]).max(0)[:, None] * np.abs(args[0]).sum(0) * 2.0 ** -29
    close(dw[cols], want[1][cols], mag[1][cols] + top[cols], 2.0 ** -22 + (M + 2) * 2.0 ** -23, "dweight")
    assert db[cols].isfinite().all() and not db[[5, 300, N - 1]].isfinite().any()


@pytest.mark.parametrize("d,head", [(64, 0), (512, 64), (520, 0), (2048, 0), (4096, 128), (16384, 0)])
@pytest.mark.parametrize("codec", [la.LA_QDQ_INT8_GROUP, la.LA_QDQ_E4M3_TILE])
def test_gate_norm_h_before_codes_is_rounded_stepwise(d, head, codec):
    """With squares whose sums are exact in any order, h is the formula's in FP32, operation by operation."""
    rows, g = 65, gen(12)
    x = (torch.exp2(torch.randint(-2, 3, (rows, d), generator=g).float()) * (torch.randint(0, 2, (rows, d), generator=g) * 2 - 1)).cuda()
    w, al = (draw(g, n, dtype=F32) for n in (head or d, d))
    x, res = x.to(BF), draw(g, rows, d)
    h, y = torch.empty_like(x), torch.empty_like(x)
    codes_, scales = torch.empty(rows, d, dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    cfg = la.GateNormConfig(rows=rows, d=d, head=head, eps=2.0 ** -6, pre=1, qdq=codec)
    la.la_gate_norm_fwd(cfg, x, None, w, al, res, None, h, y, codes_, scales)
    f = x.float().cpu().unflatten(-1, (-1, head or d))
    # the mean is rounded once (520 columns), and the root: 53 bits, 2 x 24 + 2 or more, round to FP32's own root
    # (the vectorised FP32 root on the CPU is not it: 12 of 65 rows of 2048 a bit off)
    rms = ((f.double() ** 2).mean(-1, keepdim=True).float() + 2.0 ** -6).double().sqrt().float()
    p = ((f / rms) * w.cpu()).flatten(-2)
    assert torch.equal(h.cpu(), (res.float().cpu() + al.cpu() * p).to(BF))
