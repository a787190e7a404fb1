"""Binding of the operators between two recurrences (include/la_proj.h): the matrix product of 8-bit
codes with scales, and the norms around a block with its gate and residual scale.

Arguments are checked and marshalled as in the layer operators' binding.
"""
from __future__ import annotations

import ctypes

from . import layers as _layers
from .layers import _BF16, _F32, _Config, _call, _dtype, _gpu, _library, _rows, _tight, _workspace


class LinearConfig(_Config):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "x_dtype", "out_dtype", "w_dtype", "dw_dtype", "ld_x", "ld_y")]

    def __init__(self, M, N, K, x_dtype=_BF16, out_dtype=_BF16, w_dtype=_F32, dw_dtype=_F32, ld_x=0, ld_y=0):
        super().__init__(M, N, K, x_dtype, out_dtype, w_dtype, dw_dtype, ld_x, ld_y)


def declare(lib) -> None:
    """ctypes signatures of the operators between two recurrences."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    for name, cfg, args in (
            ("la_linear_fwd", LinearConfig, [vp] * 7),
            ("la_linear_bwd", LinearConfig, [vp] * 9 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(cfg)] + args
    for name, cfg in (("la_linear_bwd_workspace_bytes", LinearConfig),):
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
