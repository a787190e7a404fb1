"""Binding of the operators between two recurrences (include/la_proj.h): the matrix product of 8-bit
codes with scales, and the norms around a block with its gate and residual scale.

Arguments are checked and marshalled as in the layer operators' binding.
"""
from __future__ import annotations

import ctypes

from . import layers as _layers
from .layers import _BF16, _F32, _Config, _call, _code_type, _dtype, _gpu, _library, _rows, _tight, _workspace

LA_GATE_NONE, LA_GATE_SILU, LA_GATE_SIGMOID = 0, 1, 2


class LinearConfig(_Config):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "x_dtype", "out_dtype", "w_dtype", "dw_dtype", "ld_x", "ld_y")]

    def __init__(self, M, N, K, x_dtype=_BF16, out_dtype=_BF16, w_dtype=_F32, dw_dtype=_F32, ld_x=0, ld_y=0):
        super().__init__(M, N, K, x_dtype, out_dtype, w_dtype, dw_dtype, ld_x, ld_y)


class GateNormConfig(_Config):
    _fields_ = [("rows", ctypes.c_int32), ("d", ctypes.c_int32), ("head", ctypes.c_int32), ("eps", ctypes.c_float)] + [
        (n, ctypes.c_int32) for n in ("gate", "gate_first", "post", "pre", "qdq", "group", "x_dtype", "w_dtype", "out_dtype",
                                      "ld_x", "ld_z")]

    def __init__(self, rows, d, head=0, eps=1e-6, gate=LA_GATE_NONE, gate_first=0, post=1, pre=0, qdq=0, group=0, x_dtype=_BF16,
                 w_dtype=_F32, out_dtype=_BF16, ld_x=0, ld_z=0):
        super().__init__(rows, d, head, eps, gate, gate_first, post, pre, qdq, group, x_dtype, w_dtype, out_dtype, ld_x, ld_z)


def declare(lib) -> None:
    """ctypes signatures of the operators between two recurrences."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    for name, cfg, args in (
            ("la_linear_fwd", LinearConfig, [vp] * 7),
            ("la_linear_bwd", LinearConfig, [vp] * 9 + [sz, vp]),
            ("la_gate_norm_fwd", GateNormConfig, [vp] * 11),
            ("la_gate_norm_bwd", GateNormConfig, [vp] * 15 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(cfg)] + args
    for name, cfg in (("la_linear_bwd_workspace_bytes", LinearConfig), ("la_gate_norm_bwd_workspace_bytes", GateNormConfig)):
        f = getattr(lib, name)
        f.restype, f.argtypes = sz, [ctypes.POINTER(cfg)]


# ----------------------------------------------- matrix product in 8-bit integers with scales
def _codes(gpu, t, name, rows, width, ld):
    """Address of rows of INT8 codes, held as int8 or uint8."""
    torch = _layers._torch
    return _rows(gpu, t, name, rows, width, ld, torch.uint8 if getattr(t, "dtype", None) is torch.uint8 else torch.int8)


def _linear_inputs(gpu, cfg, x_codes, x_scales, w_codes, w_scales):
    f32 = _dtype(_F32)
    return (_codes(gpu, x_codes, "x_codes", cfg.M, cfg.K, cfg.ld_x), _tight(gpu, x_scales, "x_scales", cfg.M, f32),
            _codes(gpu, w_codes, "w_codes", cfg.N, cfg.K, 0), _tight(gpu, w_scales, "w_scales", cfg.N, f32))


def la_linear_fwd(cfg: LinearConfig, x_codes, x_scales, w_codes, w_scales, bias, y, stream=None) -> None:
    """y = s_x s_w (c_x c_w^T) + bias, of INT8 codes (int8 or uint8) and float32 scales."""
    lib = _library()
    gpu = _gpu(x_codes, x_scales, w_codes, w_scales, y, bias)
    _call(gpu, stream, lib.la_linear_fwd, cfg, *_linear_inputs(gpu, cfg, x_codes, x_scales, w_codes, w_scales),
          _tight(gpu, bias, "bias", cfg.N, _dtype(cfg.w_dtype)), _rows(gpu, y, "y", cfg.M, cfg.N, cfg.ld_y, _dtype(cfg.out_dtype)))


def la_linear_bwd_workspace_bytes(cfg: LinearConfig) -> int:
    return _library().la_linear_bwd_workspace_bytes(cfg)


def la_linear_bwd(cfg: LinearConfig, x_codes, x_scales, w_codes, w_scales, dy, dx, dweight, dbias, workspace, ws_bytes: int,
                  stream=None) -> None:
    """Straight-through gradients of la_linear_fwd; each of dx, dweight and dbias (float32) may be None."""
    lib = _library()
    gpu = _gpu(x_codes, x_scales, w_codes, w_scales, dy, dx, dweight, dbias, workspace)
    _call(gpu, stream, lib.la_linear_bwd, cfg, *_linear_inputs(gpu, cfg, x_codes, x_scales, w_codes, w_scales),
          _rows(gpu, dy, "dy", cfg.M, cfg.N, cfg.ld_y, _dtype(cfg.out_dtype)), _tight(gpu, dx, "dx", cfg.M * cfg.K, _dtype(cfg.x_dtype)),
          _tight(gpu, dweight, "dweight", cfg.N * cfg.K, _dtype(cfg.dw_dtype)), _tight(gpu, dbias, "dbias", cfg.N, _dtype(_F32)),
          _workspace(gpu, workspace, ws_bytes), int(ws_bytes))


# ------------------------------------------- norms around a block, its gate and residual scale
def _gate_inputs(gpu, cfg, x, z, w_post, alpha):
    xt, wt = _dtype(cfg.x_dtype), _dtype(cfg.w_dtype)
    return (_rows(gpu, x, "x", cfg.rows, cfg.d, cfg.ld_x, xt), _rows(gpu, z, "z", cfg.rows, cfg.d, cfg.ld_z, xt),
            _tight(gpu, w_post, "w_post", cfg.head or cfg.d, wt), _tight(gpu, alpha, "alpha", cfg.d, wt))


def la_gate_norm_fwd(cfg: GateNormConfig, x, z, w_post, alpha, residual, w_pre, h, y, codes=None, scales=None,
                     stream=None) -> None:
    """h = residual + alpha p, p the gated norm of x, and y = h's norm (or h), with a quantizer its codes
    (uint8, or int8 for INT8 and float8_e4m3fn for E4M3) and scales."""
    lib = _library()
    gpu = _gpu(x, z, w_post, alpha, residual, w_pre, h, y, codes, scales)
    n, xt = cfg.rows * cfg.d, _dtype(cfg.x_dtype)
    _call(gpu, stream, lib.la_gate_norm_fwd, cfg, *_gate_inputs(gpu, cfg, x, z, w_post, alpha),
          _tight(gpu, residual, "residual", n, xt), _tight(gpu, w_pre, "w_pre", cfg.d, _dtype(cfg.w_dtype)),
          _tight(gpu, h, "h", n, xt), _tight(gpu, y, "y", n, _dtype(cfg.out_dtype)),
          _tight(gpu, codes, "codes", n, _code_type(cfg, codes)),
          _tight(gpu, scales, "scales", n // (cfg.group or cfg.d) if cfg.d > 0 else 0, _dtype(_F32)))


def la_gate_norm_bwd_workspace_bytes(cfg: GateNormConfig) -> int:
    return _library().la_gate_norm_bwd_workspace_bytes(cfg)


def la_gate_norm_bwd(cfg: GateNormConfig, x, z, w_post, alpha, h, w_pre, dy, dh, dx, dz, dres, dw_post, dalpha, dw_pre,
                     workspace, ws_bytes: int, stream=None) -> None:
    """Gradients of la_gate_norm_fwd (straight through the codec; dw_post, dalpha and dw_pre float32)."""
    lib = _library()
    gpu = _gpu(x, z, w_post, alpha, h, w_pre, dy, dh, dx, dz, dres, dw_post, dalpha, dw_pre, workspace)
    n, xt, f32 = cfg.rows * cfg.d, _dtype(cfg.x_dtype), _dtype(_F32)
    _call(gpu, stream, lib.la_gate_norm_bwd, cfg, *_gate_inputs(gpu, cfg, x, z, w_post, alpha),
          _tight(gpu, h, "h", n, xt), _tight(gpu, w_pre, "w_pre", cfg.d, _dtype(cfg.w_dtype)),
          _tight(gpu, dy, "dy", n, _dtype(cfg.out_dtype)), _tight(gpu, dh, "dh", n, xt),
          _rows(gpu, dx, "dx", cfg.rows, cfg.d, cfg.ld_x, xt), _rows(gpu, dz, "dz", cfg.rows, cfg.d, cfg.ld_z, xt),
          _tight(gpu, dres, "dres", n, xt), _tight(gpu, dw_post, "dw_post", cfg.head or cfg.d, f32),
          _tight(gpu, dalpha, "dalpha", cfg.d, f32), _tight(gpu, dw_pre, "dw_pre", cfg.d, f32),
          _workspace(gpu, workspace, ws_bytes), int(ws_bytes))
