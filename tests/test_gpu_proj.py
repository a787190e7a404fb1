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
