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


def test_linear_binding_refuses_tensors():
    cfg = linear()
    xc, xs = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU tensor"):
        la.la_linear_fwd(cfg, xc, xs, FAKE, FAKE, None, FAKE, stream=0)
