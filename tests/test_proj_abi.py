"""The C ABI of the operators between two recurrences on the host (no GPU): exports, refusals before
any HIP call, empty calls, and the binding's own checks."""
import os
import re

import pytest
import torch

import quantized_state_qat_amd as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never dereferenced


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "la_proj.h")).read()
    names = set(re.findall(r"^\s*(?:la_status|size_t)\s+(la_\w+)\s*\(", text, re.M))
    assert {"la_linear_fwd", "la_linear_bwd", "la_linear_bwd_workspace_bytes"} <= names
    lib = la.load_library()
    for n in names:
        assert hasattr(lib, n) and hasattr(la, n), n


def refused(call, status, word):
    with pytest.raises(la.LaError) as e:
        call()
    assert e.value.status == status and word in str(e.value), str(e.value)


# --------------------------------------------------------------------------- matrix product
def linear(**kw):
    return la.LinearConfig(**{**dict(M=8, N=64, K=64), **kw})


def linear_fwd(cfg, **p):
    q = {**dict(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, bias=None, y=FAKE), **p}
    la.la_linear_fwd(cfg, q["xc"], q["xs"], q["wc"], q["ws"], q["bias"], q["y"], stream=0)


def linear_bwd(cfg, space, n, **p):
    q = {**dict(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, db=None), **p}
    la.la_linear_bwd(cfg, q["xc"], q["xs"], q["wc"], q["ws"], q["dy"], q["dx"], q["dw"], q["db"], space, n, stream=0)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), la.LA_ERR_INVALID_ARG, "size"), (dict(N=-1), la.LA_ERR_INVALID_ARG, "size"),
    (dict(K=0), la.LA_ERR_INVALID_ARG, "size"), (dict(K=40), la.LA_ERR_UNSUPPORTED, "multiple of 16"),
    (dict(K=65552), la.LA_ERR_UNSUPPORTED, "65536"), (dict(M=(1 << 24) + 1), la.LA_ERR_UNSUPPORTED, "2^24"),
    (dict(N=(1 << 24) + 1), la.LA_ERR_UNSUPPORTED, "2^24"), (dict(M=1 << 20, N=1 << 16), la.LA_ERR_UNSUPPORTED, "tiles"),
    (dict(x_dtype=2), la.LA_ERR_INVALID_ARG, "x_dtype"), (dict(out_dtype=-1), la.LA_ERR_INVALID_ARG, "out_dtype"),
    (dict(w_dtype=2), la.LA_ERR_INVALID_ARG, "w_dtype"), (dict(dw_dtype=5), la.LA_ERR_INVALID_ARG, "dw_dtype"),
    (dict(ld_x=48), la.LA_ERR_INVALID_ARG, "shorter"), (dict(ld_x=72), la.LA_ERR_ALIGNMENT, "16 bytes"),
    (dict(ld_x=-16), la.LA_ERR_INVALID_ARG, "shorter"), (dict(ld_x=(1 << 22) + 16), la.LA_ERR_UNSUPPORTED, "2^22"),
    (dict(ld_y=63), la.LA_ERR_INVALID_ARG, "shorter"),
])
def test_linear_refuses_configs(kw, status, word):
    refused(lambda: linear_fwd(linear(**kw)), status, word)
    refused(lambda: linear_bwd(linear(**kw), FAKE, 1 << 40), status, word)
    assert la.la_linear_bwd_workspace_bytes(linear(**kw)) == 0


def test_linear_refuses_pointers():
    for p in ("xc", "xs", "wc", "ws", "y"):
        refused(lambda: linear_fwd(linear(), **{p: None}), la.LA_ERR_INVALID_ARG, "is NULL")
        refused(lambda: linear_fwd(linear(), **{p: FAKE + 4}), la.LA_ERR_ALIGNMENT, "aligned")
    refused(lambda: linear_fwd(linear(), bias=FAKE + 2), la.LA_ERR_ALIGNMENT, "bias")
    for kw in (dict(M=0), dict(N=0)):
        linear_fwd(linear(**kw), xc=None, xs=None, wc=None, ws=None, y=None)
    n = la.la_linear_bwd_workspace_bytes(linear())
    assert n > 0
    refused(lambda: linear_bwd(linear(), FAKE, n - 1), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: linear_bwd(linear(), None, n), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: linear_bwd(linear(), FAKE + 8, n), la.LA_ERR_ALIGNMENT, "workspace")
    refused(lambda: linear_bwd(linear(), FAKE, n, dy=None), la.LA_ERR_INVALID_ARG, "dy is NULL")
    for p in ("xc", "xs", "wc", "ws"):  # each is needed by one gradient alone
        refused(lambda: linear_bwd(linear(), FAKE, n, **{p: None}), la.LA_ERR_INVALID_ARG, "is NULL")
    for p in ("dx", "dw", "db"):
        refused(lambda: linear_bwd(linear(), FAKE, n, **{p: FAKE + 4}), la.LA_ERR_ALIGNMENT, "aligned")
    linear_bwd(linear(), FAKE, n, dx=None, dw=None)
    for kw in (dict(M=(1 << 19) + 1), dict(N=(1 << 19) + 1, M=1)):
        assert la.la_linear_bwd_workspace_bytes(linear(**kw)) == 0
        refused(lambda: linear_bwd(linear(**kw), FAKE, 1 << 50), la.LA_ERR_UNSUPPORTED, "2^19")


def test_linear_backward_without_tokens_or_channels_needs_nothing():
    """Nothing to sum: no workspace, so no operand is laid out for the products, whose codes may be NULL."""
    for kw in (dict(M=0), dict(N=0), dict(M=0, N=0), dict(M=0, N=1 << 19, K=65536), dict(N=0, M=1 << 19)):
        assert la.la_linear_bwd_workspace_bytes(linear(**kw)) == 0
        linear_bwd(linear(**kw), None, 0, xc=None, xs=None, wc=None, ws=None, dy=None, dx=None, dw=None)
    assert la.la_linear_bwd_workspace_bytes(linear(M=1, N=1, K=16)) > 0


def test_linear_binding_refuses_tensors():
    cfg = linear()
    xc, xs = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU tensor"):
        la.la_linear_fwd(cfg, xc, xs, FAKE, FAKE, None, FAKE, stream=0)


# ---------------------------------------------------------------------- norms around a block
def gate(**kw):
    return la.GateNormConfig(**{**dict(rows=8, d=256, gate=la.LA_GATE_SILU, pre=1), **kw})


FWD = dict(x=FAKE, z=FAKE, w_post=FAKE, alpha=FAKE, residual=FAKE, w_pre=FAKE, h=FAKE, y=FAKE, codes=None, scales=None)
BWD = dict(x=FAKE, z=FAKE, w_post=FAKE, alpha=FAKE, h=FAKE, w_pre=FAKE, dy=FAKE, dh=FAKE, dx=FAKE, dz=FAKE, dres=FAKE,
           dw_post=FAKE, dalpha=FAKE, dw_pre=FAKE)


def gate_fwd(cfg, **p):
    la.la_gate_norm_fwd(cfg, *{**FWD, **p}.values(), stream=0)


def gate_bwd(cfg, space, n, **p):
    la.la_gate_norm_bwd(cfg, *{**BWD, **p}.values(), space, n, stream=0)


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), la.LA_ERR_INVALID_ARG, "size"), (dict(d=0), la.LA_ERR_INVALID_ARG, "size"),
    (dict(d=100), la.LA_ERR_UNSUPPORTED, "multiple of 8"), (dict(d=16392), la.LA_ERR_UNSUPPORTED, "16384"),
    (dict(rows=1 << 30, d=16384), la.LA_ERR_UNSUPPORTED, "too many rows"), (dict(head=8), la.LA_ERR_UNSUPPORTED, "head"),
    (dict(head=48), la.LA_ERR_UNSUPPORTED, "head"), (dict(head=1024, d=1024), la.LA_ERR_UNSUPPORTED, "head"),
    (dict(head=512), la.LA_ERR_INVALID_ARG, "divide"), (dict(eps=-1.0), la.LA_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), la.LA_ERR_INVALID_ARG, "eps"), (dict(gate=3), la.LA_ERR_INVALID_ARG, "gate"),
    (dict(gate_first=2), la.LA_ERR_INVALID_ARG, "gate_first"), (dict(post=-1), la.LA_ERR_INVALID_ARG, "post"),
    (dict(pre=2), la.LA_ERR_INVALID_ARG, "pre"), (dict(gate=0, gate_first=1), la.LA_ERR_INVALID_ARG, "needs a gate"),
    (dict(x_dtype=2), la.LA_ERR_INVALID_ARG, "x_dtype"), (dict(w_dtype=2), la.LA_ERR_INVALID_ARG, "w_dtype"),
    (dict(out_dtype=2), la.LA_ERR_INVALID_ARG, "out_dtype"), (dict(ld_x=248), la.LA_ERR_INVALID_ARG, "shorter"),
    (dict(ld_z=260), la.LA_ERR_ALIGNMENT, "16 bytes"), (dict(qdq=3), la.LA_ERR_INVALID_ARG, "qdq"),
    (dict(qdq=1, group=48), la.LA_ERR_UNSUPPORTED, "group"), (dict(qdq=1, group=128, d=192), la.LA_ERR_INVALID_ARG, "divide"),
])
def test_gate_norm_refuses_configs(kw, status, word):
    refused(lambda: gate_fwd(gate(**kw)), status, word)
    refused(lambda: gate_bwd(gate(**kw), FAKE, 1 << 40), status, word)
    assert la.la_gate_norm_bwd_workspace_bytes(gate(**kw)) == 0


@pytest.mark.parametrize("d,lanes", [(64, 8), (72, 16), (256, 32), (512, 64), (520, 128), (1032, 192), (2048, 256), (2304, 384), (16384, 256)])
def test_gate_norm_refuses_grids_of_two_to_the_32(d, lanes):
    """A row has that many threads, and a grid whole workgroups of 256, or of the row's threads."""
    most = min(((1 << 32) - 1) // lanes - 31, (1 << 31) - 1)  # (most + 31) lanes < 2^32
    assert la.la_gate_norm_bwd_workspace_bytes(gate(rows=most, d=d)) > 0 and -(-most * lanes // max(lanes, 256)) * max(lanes, 256) < 1 << 32
    if most < (1 << 31) - 1:
        refused(lambda: gate_fwd(gate(rows=most + 1, d=d)), la.LA_ERR_UNSUPPORTED, "too many rows")


def test_linear_backward_refuses_grids():
    cfg = linear(M=1 << 19, N=1 << 16)
    assert la.la_linear_bwd_workspace_bytes(cfg) == 0
    refused(lambda: linear_bwd(cfg, FAKE, 1 << 60), la.LA_ERR_UNSUPPORTED, "2^23")
    assert la.la_linear_bwd_workspace_bytes(linear(M=1 << 19, N=(1 << 16) - 64, K=65536)) > 0


@pytest.mark.parametrize("d,rpw", [(8, 32), (64, 32), (128, 16), (256, 8), (512, 4), (520, 1), (2048, 1), (4096, 1), (16384, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(gate=0), dict(pre=0)])
def test_gate_norm_backward_sums_128_rows_at_most(d, rpw, kw):
    """The workspace has three rows of sums a workgroup, which walks rows of its own that many at a time."""
    for rows in (1, 77, 5000, 32768, 1 << 20, (1 << 23) + 5):
        groups = la.la_gate_norm_bwd_workspace_bytes(gate(rows=rows, d=d, **kw)) / (12 * d)
        assert groups == int(groups) and groups * rpw * 128 >= rows
        assert groups * rpw < rows + rpw  # none without rows
        assert groups * rpw * 64 < rows or groups <= 1536  # (several rounds of resident workgroups are of more rows than half of that)


def test_gate_norm_refuses_pointers():
    for p in FWD:
        refused(lambda: gate_fwd(gate(qdq=1), **{p: FAKE + 8}), la.LA_ERR_ALIGNMENT, "aligned")
    n = la.la_gate_norm_bwd_workspace_bytes(gate())
    for p in BWD:
        refused(lambda: gate_bwd(gate(), FAKE, n, **{p: FAKE + 8}), la.LA_ERR_ALIGNMENT, "aligned")
    for p in ("x", "z"):
        refused(lambda: gate_fwd(gate(), **{p: None}), la.LA_ERR_INVALID_ARG, "is NULL")
    for p in ("x", "z", "h", "dy", "dx"):
        refused(lambda: gate_bwd(gate(), FAKE, n, **{p: None}), la.LA_ERR_INVALID_ARG, "is NULL")
    refused(lambda: gate_fwd(gate(gate=0)), la.LA_ERR_INVALID_ARG, "z needs")
    refused(lambda: gate_fwd(gate(post=0)), la.LA_ERR_INVALID_ARG, "w_post needs")
    refused(lambda: gate_fwd(gate(pre=0)), la.LA_ERR_INVALID_ARG, "w_pre needs")
    refused(lambda: gate_fwd(gate(), codes=FAKE), la.LA_ERR_INVALID_ARG, "quantizer")
    refused(lambda: gate_bwd(gate(gate=0), FAKE, n, z=None), la.LA_ERR_INVALID_ARG, "dz needs")
    refused(lambda: gate_bwd(gate(post=0), FAKE, n, w_post=None), la.LA_ERR_INVALID_ARG, "dw_post needs")
    refused(lambda: gate_bwd(gate(pre=0), FAKE, n, w_pre=None), la.LA_ERR_INVALID_ARG, "dw_pre needs")
    refused(lambda: gate_bwd(gate(), FAKE, n - 1), la.LA_ERR_WORKSPACE, "workspace")
    refused(lambda: gate_bwd(gate(), None, n), la.LA_ERR_WORKSPACE, "workspace")
    gate_fwd(gate(rows=0), **{k: None for k in FWD})
