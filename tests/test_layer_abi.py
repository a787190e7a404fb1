"""The layer operators' C ABI on the host (no GPU): exports, refusals before any HIP call, empty
calls, and the binding's own checks."""
import os
import re
import sys

import pytest
import torch

import quantized_state_qat_amd as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never dereferenced


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "la_layer.h")).read()
    names = sorted(set(re.findall(r"^\s*(?:la_status|size_t)\s+(la_\w+)\s*\(", text, re.M)))
    assert names == sorted(["la_conv_fwd", "la_conv_bwd", "la_conv_step", "la_conv_bwd_workspace_bytes", "la_scan_fwd",
                            "la_scan_bwd", "la_scan_step", "la_scan_workspace_bytes", "la_scan_bwd_workspace_bytes",
                            "la_scan_bwd_varlen_workspace_bytes",
                            "la_norm_fwd", "la_norm_bwd", "la_norm_bwd_workspace_bytes"])
    lib = la.load_library()
    for n in names:
        assert hasattr(lib, n) and hasattr(la, n), n


def refused(call, status, word):
    with pytest.raises(la.LaError) as e:
        call()
    assert e.value.status == status and word in str(e.value), str(e.value)


# ------------------------------------------------------------------------------- convolution
def conv(**kw):
    return la.ConvConfig(**{**dict(B=2, T=8, C=64, width=4), **kw})


def conv_fwd(cfg, **p):
    q = {**dict(x=FAKE, weight=FAKE, bias=None, state0=None, y=FAKE, state_T=None, cu_seqlens=None), **p}
    la.la_conv_fwd(cfg, q["x"], q["weight"], q["bias"], q["state0"], q["y"], q["state_T"], cu_seqlens=q["cu_seqlens"],
                   stream=0)


@pytest.mark.parametrize("kw,status,word", [
    (dict(B=-1), la.LA_ERR_INVALID_ARG, "size"), (dict(C=0), la.LA_ERR_INVALID_ARG, "size"),
    (dict(C=60), la.LA_ERR_UNSUPPORTED, "multiple of 8"), (dict(C=1 << 21), la.LA_ERR_UNSUPPORTED, "2^20"),
    (dict(width=1), la.LA_ERR_UNSUPPORTED, "width"), (dict(width=5), la.LA_ERR_UNSUPPORTED, "width"),
    (dict(act=2), la.LA_ERR_INVALID_ARG, "act"), (dict(x_dtype=7), la.LA_ERR_INVALID_ARG, "x_dtype"),
    (dict(w_dtype=-1), la.LA_ERR_INVALID_ARG, "w_dtype"), (dict(ld_x=32), la.LA_ERR_INVALID_ARG, "shorter"),
    (dict(ld_y=68), la.LA_ERR_ALIGNMENT, "16 bytes"), (dict(B=1 << 20, T=1 << 20), la.LA_ERR_UNSUPPORTED, "elements"),
    (dict(B=65536), la.LA_ERR_UNSUPPORTED, "65535"), (dict(T=(1 << 30) + 1), la.LA_ERR_UNSUPPORTED, "2^30"),
])
def test_conv_refuses_configs(kw, status, word):
    refused(lambda: conv_fwd(conv(**kw)), status, word)
    assert la.la_conv_bwd_workspace_bytes(conv(**kw)) == 0


@pytest.mark.parametrize("kw", [dict(B=32768, T=1, C=131072), dict(B=65528, T=16, C=65544), dict(B=65535, T=17, C=61672)])
def test_conv_refuses_grids_of_two_to_the_32(kw):
    """Width 4: three rows of the final states and a walk for every 16 tokens, 16 bytes of channels each."""
    cfg = conv(x_dtype=la.LA_F32, **kw)
    assert cfg.B * (-(-cfg.T // 16) + 3) * (cfg.C // 4) > (1 << 32) - 512
    refused(lambda: conv_fwd(cfg), la.LA_ERR_UNSUPPORTED, "elements")


def test_conv_refuses_pointers():
    refused(lambda: conv_fwd(conv(), x=None), la.LA_ERR_INVALID_ARG, "x is NULL")
    refused(lambda: conv_fwd(conv(), weight=FAKE + 4), la.LA_ERR_ALIGNMENT, "weight")
    refused(lambda: conv_fwd(conv(), state0=FAKE, state_T=FAKE), la.LA_ERR_INVALID_ARG, "state_T")
    refused(lambda: conv_fwd(conv(), cu_seqlens=FAKE + 8), la.LA_ERR_ALIGNMENT, "cu_seqlens")
    conv_fwd(conv(B=0), x=None, weight=None, y=None)
    n = la.la_conv_bwd_workspace_bytes(conv())
    args = [FAKE] * 3 + [None, FAKE, None, FAKE, FAKE, None, None]
    refused(lambda: la.la_conv_bwd(conv(), *args, FAKE, n - 1, stream=0), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: la.la_conv_bwd(conv(), *args, None, n, stream=0), la.LA_ERR_WORKSPACE, "workspace")
    args[7] = None
    refused(lambda: la.la_conv_bwd(conv(), *args, FAKE, n, stream=0), la.LA_ERR_INVALID_ARG, "dweight")
    refused(lambda: la.la_conv_step(conv(T=2), FAKE, FAKE, None, FAKE, FAKE, stream=0), la.LA_ERR_INVALID_ARG, "T == 1")
    refused(lambda: la.la_conv_step(conv(T=1), FAKE, FAKE, None, FAKE, FAKE, slots=FAKE, n_slots=0, stream=0),
            la.LA_ERR_INVALID_ARG, "n_slots")
    la.la_conv_step(conv(T=1, B=0), None, None, None, None, None, stream=0)


# -------------------------------------------------------------------------------------- scan
def scan(**kw):
    return la.ScanConfig(**{**dict(B=2, T=8, H=4, G=2, d_k=64, d_v=64), **kw})


def scan_fwd(cfg, **p):
    q = {**dict(x=FAKE, dt=FAKE, A=FAKE, b=FAKE, c=FAKE, D=None, dt_bias=None, S0=None, y=FAKE, S_T=None, ws=None, n=0), **p}
    la.la_scan_fwd(cfg, q["x"], q["dt"], q["A"], q["b"], q["c"], q["D"], q["dt_bias"], q["S0"], q["y"], q["S_T"], q["ws"],
                   q["n"], stream=0)


@pytest.mark.parametrize("kw,status,word", [
    (dict(T=-1), la.LA_ERR_INVALID_ARG, "size"), (dict(G=0), la.LA_ERR_INVALID_ARG, "size"),
    (dict(G=3), la.LA_ERR_INVALID_ARG, "divide"), (dict(d_k=48), la.LA_ERR_UNSUPPORTED, "d_k"),
    (dict(d_k=256), la.LA_ERR_UNSUPPORTED, "d_k"), (dict(d_v=32), la.LA_ERR_UNSUPPORTED, "d_v"),
    (dict(d_v=8192), la.LA_ERR_UNSUPPORTED, "d_v"), (dict(softplus=2), la.LA_ERR_INVALID_ARG, "softplus"),
    (dict(x_dtype=2), la.LA_ERR_INVALID_ARG, "x_dtype"), (dict(dt_dtype=2), la.LA_ERR_INVALID_ARG, "dt_dtype"),
    (dict(out_dtype=2), la.LA_ERR_INVALID_ARG, "out_dtype"), (dict(ld_x=128), la.LA_ERR_INVALID_ARG, "shorter"),
    (dict(ld_b=132), la.LA_ERR_ALIGNMENT, "16 bytes"), (dict(ld_c=64), la.LA_ERR_INVALID_ARG, "shorter"),
    (dict(ld_dt=3), la.LA_ERR_INVALID_ARG, "ld_dt"), (dict(B=70000), la.LA_ERR_UNSUPPORTED, "65535"),
    (dict(B=65535, H=65534), la.LA_ERR_UNSUPPORTED, "too many"), (dict(T=(1 << 30) + 1), la.LA_ERR_UNSUPPORTED, "2^30"),
    (dict(H=65534, d_v=192), la.LA_ERR_UNSUPPORTED, "2^23"), (dict(ld_x=(1 << 23) + 8), la.LA_ERR_UNSUPPORTED, "2^23"),
    (dict(ld_c=(1 << 23) + 8), la.LA_ERR_UNSUPPORTED, "2^23"), (dict(ld_dt=(1 << 23) + 1), la.LA_ERR_UNSUPPORTED, "2^23"),
])
def test_scan_refuses_configs(kw, status, word):
    refused(lambda: scan_fwd(scan(**kw)), status, word)
    assert la.la_scan_workspace_bytes(scan(**kw)) == 0 and la.la_scan_bwd_workspace_bytes(scan(**kw)) == 0


def test_scan_refuses_pointers():
    refused(lambda: scan_fwd(scan(), A=None), la.LA_ERR_INVALID_ARG, "A is NULL")
    refused(lambda: scan_fwd(scan(), c=FAKE + 2), la.LA_ERR_ALIGNMENT, "c is")
    refused(lambda: scan_fwd(scan(), S0=FAKE, S_T=FAKE), la.LA_ERR_INVALID_ARG, "S_T")
    long = scan(B=1, T=4096)
    n = la.la_scan_workspace_bytes(long)
    assert n > 0
    refused(lambda: scan_fwd(long), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: scan_fwd(long, ws=FAKE, n=n - 1), la.LA_ERR_WORKSPACE, "workspace")
    scan_fwd(scan(B=0), x=None, dt=None, A=None, b=None, c=None, y=None)
    n = la.la_scan_bwd_workspace_bytes(scan())
    assert n > 0
    bwd = lambda cfg, ws, n: la.la_scan_bwd(cfg, *[FAKE] * 5, None, None, None, FAKE, None, *[FAKE] * 5, None, None,  # noqa: E731
                                            None, ws, n, stream=0)
    refused(lambda: bwd(scan(), FAKE, n - 1), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: bwd(scan(out_dtype=la.LA_F32), FAKE, n), la.LA_ERR_UNSUPPORTED, "out_dtype")
    refused(lambda: la.la_scan_step(scan(), *[FAKE] * 5, None, None, FAKE, FAKE, stream=0), la.LA_ERR_INVALID_ARG, "T == 1")
    refused(lambda: la.la_scan_step(scan(T=1), *[FAKE] * 5, None, None, FAKE, FAKE, slots=FAKE, n_slots=-1, stream=0),
            la.LA_ERR_INVALID_ARG, "n_slots")


def test_packed_workspaces_do_not_grow_with_the_sequences():
    """64 sequences of one packing of 2^18 tokens: about the states of one sequence of them."""
    one, many = scan(B=1, T=1 << 18), scan(B=64, T=1 << 18)
    n1, n64 = la.la_scan_bwd_varlen_workspace_bytes(one), la.la_scan_bwd_varlen_workspace_bytes(many)
    assert n1 <= n64 <= 1.02 * n1 and n64 <= la.la_scan_bwd_workspace_bytes(many)
    # two FP32 states of 64 x 64 a head at each of 4096 + 65 slots, and 4 KB beside them
    assert n64 <= (4096 + 65) * 4 * (2 * 64 * 64 * 4 + 4096)
    assert la.la_conv_bwd_workspace_bytes(conv(B=4096, T=1 << 20, C=4096)) <= 256 << 20
    args = [FAKE] * 5 + [None, None, None, FAKE, None, *[FAKE] * 5, None, None, None]
    refused(lambda: la.la_scan_bwd(many, *args, FAKE, n64 - 1, cu_seqlens=FAKE, stream=0), la.LA_ERR_WORKSPACE, "workspace")


def test_backward_refuses_what_its_grids_cannot_hold():
    args = [FAKE] * 5 + [None, None, None, FAKE, None, *[FAKE] * 5, None, None, None, FAKE]
    for kw, cu in ((dict(B=64, T=1 << 23), None), (dict(T=1 << 28), FAKE)):
        refused(lambda: la.la_scan_bwd(scan(**kw), *args, 1 << 62, cu_seqlens=cu, stream=0), la.LA_ERR_UNSUPPORTED, "2^23")
        assert la.la_scan_bwd_workspace_bytes(scan(**kw)) == 0


@pytest.mark.parametrize("kw", [dict(B=128, T=1, H=65535), dict(B=1, T=64 * 65535, H=128), dict(B=65535, T=1, H=128)])
def test_backward_needs_its_workspace_where_only_the_dense_layout_fits(kw):
    """B sequences of T tokens just below the limit on chunks, which a packing of them would pass."""
    cfg = scan(G=1, d_k=16, **kw)
    args = [FAKE] * 5 + [None, None, None, FAKE, None, *[FAKE] * 5, None, None, None]
    states = 2 * cfg.B * -(-cfg.T // 64) * cfg.H * 16 * 64 * 4
    n = la.la_scan_bwd_workspace_bytes(cfg)
    assert n >= states and la.la_scan_bwd_varlen_workspace_bytes(cfg) == 0
    for ws, given in ((None, 0), (FAKE, 0), (FAKE, n - 1)):
        refused(lambda: la.la_scan_bwd(cfg, *args, ws, given, stream=0), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: la.la_scan_bwd(cfg, *args, FAKE, n, cu_seqlens=FAKE, stream=0), la.LA_ERR_UNSUPPORTED, "2^23")


def test_no_sequences_need_no_tensors():
    """B = 0 with boundaries and a packed length."""
    la.la_conv_fwd(conv(B=0), None, None, None, None, None, None, cu_seqlens=FAKE, stream=0)
    la.la_scan_fwd(scan(B=0), None, None, None, None, None, None, None, None, None, None, None, 0, cu_seqlens=FAKE, stream=0)
    assert la.la_conv_bwd_workspace_bytes(conv(B=0, T=4096)) == 0


# -------------------------------------------------------------------------------------- norm
def norm(**kw):
    return la.NormConfig(**{**dict(rows=4, d=256), **kw})


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), la.LA_ERR_INVALID_ARG, "size"), (dict(d=0), la.LA_ERR_INVALID_ARG, "size"),
    (dict(d=12), la.LA_ERR_UNSUPPORTED, "multiple of 8"), (dict(d=16392), la.LA_ERR_UNSUPPORTED, "16384"),
    (dict(rows=1 << 24, d=4096), la.LA_ERR_UNSUPPORTED, "rows"), (dict(rows=1 << 29, d=8), la.LA_ERR_UNSUPPORTED, "rows"),
    (dict(eps=-1.0), la.LA_ERR_INVALID_ARG, "eps"), (dict(eps=float("nan")), la.LA_ERR_INVALID_ARG, "eps"),
    (dict(qdq=5), la.LA_ERR_INVALID_ARG, "qdq"), (dict(qdq=la.LA_QDQ_INT8_GROUP, group=8), la.LA_ERR_UNSUPPORTED, "group"),
    (dict(qdq=la.LA_QDQ_E4M3_TILE, group=64, d=96), la.LA_ERR_INVALID_ARG, "divide"),
    (dict(x_dtype=3), la.LA_ERR_INVALID_ARG, "x_dtype"), (dict(w_dtype=3), la.LA_ERR_INVALID_ARG, "w_dtype"),
    (dict(out_dtype=3), la.LA_ERR_INVALID_ARG, "out_dtype"),
])
def test_norm_refuses_configs(kw, status, word):
    refused(lambda: la.la_norm_fwd(norm(**kw), FAKE, None, None, FAKE, FAKE, stream=0), status, word)
    assert la.la_norm_bwd_workspace_bytes(norm(**kw)) == 0


def test_norm_refuses_grids_of_two_to_the_32():
    """d = 8: workgroups of 32 rows by 8 lanes."""
    for rows in ((1 << 29) - 31, (1 << 29) - 1):
        assert -(-rows // 32) * 256 == 1 << 32
        refused(lambda: la.la_norm_fwd(norm(rows=rows, d=8), FAKE, None, None, FAKE, FAKE, stream=0), la.LA_ERR_UNSUPPORTED, "rows")


def test_norm_refuses_pointers():
    refused(lambda: la.la_norm_fwd(norm(), None, None, None, FAKE, FAKE, stream=0), la.LA_ERR_INVALID_ARG, "x is NULL")
    refused(lambda: la.la_norm_fwd(norm(), FAKE, None, None, FAKE, FAKE, codes=FAKE, stream=0), la.LA_ERR_INVALID_ARG,
            "quantizer")
    refused(lambda: la.la_norm_fwd(norm(), FAKE, FAKE + 8, None, FAKE, FAKE, stream=0), la.LA_ERR_ALIGNMENT, "residual")
    la.la_norm_fwd(norm(rows=0), None, None, None, None, None, stream=0)
    n = la.la_norm_bwd_workspace_bytes(norm())
    refused(lambda: la.la_norm_bwd(norm(), FAKE, None, FAKE, None, FAKE, FAKE, FAKE, n - 1, stream=0), la.LA_ERR_WORKSPACE,
            "workspace")


def test_null_configs():
    lib = la.load_library()
    for f in ("la_conv_fwd", "la_conv_bwd", "la_conv_step", "la_scan_fwd", "la_scan_bwd", "la_scan_step", "la_norm_fwd",
              "la_norm_bwd"):
        fn = getattr(lib, f)
        assert fn(None, *[0 if t is not None and t.__name__ in ("c_int", "c_ulong") else None for t in fn.argtypes[1:]]) == \
            la.LA_ERR_INVALID_ARG, f
        assert b"cfg is NULL" in lib.la_last_error()


# ------------------------------------------------------------------------- the binding's checks
def test_binding_refuses_tensors():
    host = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        la.la_conv_fwd(conv(), host, FAKE, None, None, FAKE, stream=0)
    with pytest.raises(ValueError, match="weight must be a GPU tensor"):
        la.la_conv_fwd(conv(), FAKE, torch.zeros(64, 4), None, None, FAKE, stream=0)


def test_binding_is_whole_once_it_looks_initialised(monkeypatch):
    """What another thread's call sees between any two lines of the first call's initialisation."""
    from quantized_state_qat_amd import layers
    for name, value in (("_torch", None), ("_types", ()), ("_current", None)):
        monkeypatch.setattr(layers, name, value)
    lines = []

    def trace(frame, event, arg):
        if frame.f_code is not layers._library.__code__:
            return None
        lines.append(frame.f_lineno)
        assert layers._torch is None or (len(layers._types) == 2 and callable(layers._current)), frame.f_lineno
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        layers._library()
    finally:
        sys.settrace(before)
    assert len(set(lines)) >= 6 and layers._torch is torch
