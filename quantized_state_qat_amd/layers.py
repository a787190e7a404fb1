"""Binding of the layer operators (include/la_layer.h): the short causal convolution, the
selective scan and the RMS norm with the residual's addition.

As in the package's other calls, the functions carry the C ABI's names and only check and
marshal arguments.  Tensors must live on one GPU; the call runs on that GPU's current stream
unless `stream` names another.  Raw integer addresses are passed through unchecked, for a call
on the current device.
"""
from __future__ import annotations

import ctypes

import quantized_state_qat_amd as _la

LA_ACT_NONE, LA_ACT_SILU = 0, 1
_F32, _BF16 = 0, 1


class _Config(ctypes.Structure):
    def __repr__(self):
        return f"{type(self).__name__}({', '.join(f'{n}={getattr(self, n)}' for n, _ in self._fields_)})"


class ConvConfig(_Config):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "width", "act", "x_dtype", "w_dtype", "ld_x", "ld_y")]

    def __init__(self, B, T, C, width, act=LA_ACT_SILU, x_dtype=_BF16, w_dtype=_F32, ld_x=0, ld_y=0):
        super().__init__(B, T, C, width, act, x_dtype, w_dtype, ld_x, ld_y)


class ScanConfig(_Config):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "G", "d_k", "d_v", "softplus", "x_dtype", "dt_dtype",
                                              "out_dtype", "ld_x", "ld_b", "ld_c", "ld_dt")]

    def __init__(self, B, T, H, G, d_k, d_v, softplus=1, x_dtype=_BF16, dt_dtype=_BF16, out_dtype=_BF16, ld_x=0, ld_b=0,
                 ld_c=0, ld_dt=0):
        super().__init__(B, T, H, G, d_k, d_v, softplus, x_dtype, dt_dtype, out_dtype, ld_x, ld_b, ld_c, ld_dt)


class NormConfig(_Config):
    _fields_ = [("rows", ctypes.c_int32), ("d", ctypes.c_int32), ("eps", ctypes.c_float)] + [
        (n, ctypes.c_int32) for n in ("qdq", "group", "x_dtype", "w_dtype", "out_dtype")]

    def __init__(self, rows, d, eps=1e-6, qdq=0, group=0, x_dtype=_BF16, w_dtype=_F32, out_dtype=_BF16):
        super().__init__(rows, d, eps, qdq, group, x_dtype, w_dtype, out_dtype)


def declare(lib) -> None:
    """ctypes signatures of the layer operators."""
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    for name, cfg, args in (
            ("la_conv_fwd", ConvConfig, [vp] * 8),
            ("la_conv_bwd", ConvConfig, [vp] * 12 + [sz, vp]),
            ("la_conv_step", ConvConfig, [vp] * 5 + [i32, vp, vp]),
            ("la_scan_fwd", ScanConfig, [vp] * 12 + [sz, vp]),
            ("la_scan_bwd", ScanConfig, [vp] * 20 + [sz, vp]),
            ("la_scan_step", ScanConfig, [vp] * 9 + [i32, vp, vp]),
            ("la_norm_fwd", NormConfig, [vp] * 8),
            ("la_norm_bwd", NormConfig, [vp] * 7 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(cfg)] + args
    for name, cfg in (("la_conv_bwd_workspace_bytes", ConvConfig), ("la_scan_workspace_bytes", ScanConfig),
                      ("la_scan_bwd_workspace_bytes", ScanConfig), ("la_norm_bwd_workspace_bytes", NormConfig)):
        f = getattr(lib, name)
        f.restype, f.argtypes = sz, [ctypes.POINTER(cfg)]


class _Call:
    """Checks the tensors of one call and makes it on their GPU."""

    def __init__(self, stream):
        import torch
        self.torch, self.stream, self.device = torch, stream, None
        self.types = {_F32: torch.float32, _BF16: torch.bfloat16}

    def _same_gpu(self, t, name):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
        at = t.device.index
        if self.device is None:
            self.device = at
        elif at != self.device:
            raise ValueError(f"{name} is on GPU {at}, an earlier argument on GPU {self.device}")

    def tight(self, t, name, numel, *dtypes):
        """Address of a contiguous tensor of at least `numel` elements."""
        if t is None or isinstance(t, int):
            return t
        self._same_gpu(t, name)
        if t.dtype not in dtypes:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if t.numel() < numel:
            raise ValueError(f"{name} holds {t.numel()} elements, the configuration needs {numel}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def rows(self, t, name, tokens, width, ld, dtype):
        """Address of `tokens` rows of `width` contiguous elements, `ld` (0: width) elements apart."""
        if t is None or isinstance(t, int):
            return t
        self._same_gpu(t, name)
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        ld = ld or width
        if t.numel() < tokens * width:
            raise ValueError(f"{name} holds {t.numel()} elements, the configuration needs {tokens * width}")
        if ld == width and t.is_contiguous():
            return t.data_ptr()
        inner, want = 1, 1  # elements of the row walked so far, the stride the next dimension must have
        for n, step in zip(reversed(t.shape), reversed(t.stride())):
            if n != 1 and step != want:
                raise ValueError(f"{name} has strides {t.stride()}: rows of {width} contiguous elements, {ld} apart, "
                                 "are needed")
            if inner < width:
                inner *= n
                want = ld if inner == width else inner
                if inner > width:
                    raise ValueError(f"{name} has shape {tuple(t.shape)}: its last dimensions must make up a row of {width}")
            else:
                want *= n
        return t.data_ptr()

    def __call__(self, fn, *args):
        torch = self.torch
        if self.device is None or self.device == torch.cuda.current_device():
            status = fn(*args, self._stream())
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, self._stream())
        if status:
            _la._check(status)

    def _stream(self):
        s = self.stream
        if s is None:
            return self.torch.cuda.current_stream(self.device).cuda_stream
        if isinstance(s, int):
            return s
        if self.device is not None and s.device.index != self.device:
            raise ValueError(f"stream is on GPU {s.device.index}, the tensors on GPU {self.device}")
        return s.cuda_stream


def _workspace(call, workspace, ws_bytes):
    if workspace is None or isinstance(workspace, int):
        return workspace
    call._same_gpu(workspace, "workspace")
    if workspace.numel() * workspace.element_size() < int(ws_bytes):
        raise ValueError(f"workspace holds fewer than the {int(ws_bytes)} bytes passed as ws_bytes")
    return _la._ptr(workspace)


def _tokens(cfg, cu_seqlens):
    return cfg.T if cu_seqlens is not None else cfg.B * cfg.T


# ------------------------------------------------------------------ short causal convolution
def la_conv_fwd(cfg: ConvConfig, x, weight, bias, state0, y, state_T=None, cu_seqlens=None, stream=None) -> None:
    """y = act(causal depthwise convolution of state0 ++ x); state_T = its last rows."""
    lib, k = _la.load_library(), _Call(stream)
    xt, wt, n = k.types.get(cfg.x_dtype, k.torch.float32), k.types.get(cfg.w_dtype, k.torch.float32), _tokens(cfg, cu_seqlens)
    st = cfg.B * (cfg.width - 1) * cfg.C
    k(lib.la_conv_fwd, cfg, k.tight(cu_seqlens, "cu_seqlens", cfg.B + 1, k.torch.int32), k.rows(x, "x", n, cfg.C, cfg.ld_x, xt),
      k.tight(weight, "weight", cfg.C * cfg.width, wt), k.tight(bias, "bias", cfg.C, wt), k.tight(state0, "state0", st, xt),
      k.rows(y, "y", n, cfg.C, cfg.ld_y, xt), k.tight(state_T, "state_T", st, xt))


def la_conv_bwd_workspace_bytes(cfg: ConvConfig) -> int:
    return _la.load_library().la_conv_bwd_workspace_bytes(cfg)


def la_conv_bwd(cfg: ConvConfig, x, weight, bias, state0, dy, dstate_T, dx, dweight, dbias, dstate0, workspace,
                ws_bytes: int, cu_seqlens=None, stream=None) -> None:
    """Gradients of la_conv_fwd (dweight and dbias float32)."""
    lib, k = _la.load_library(), _Call(stream)
    xt, wt, n = k.types.get(cfg.x_dtype, k.torch.float32), k.types.get(cfg.w_dtype, k.torch.float32), _tokens(cfg, cu_seqlens)
    st, f32 = cfg.B * (cfg.width - 1) * cfg.C, k.torch.float32
    k(lib.la_conv_bwd, cfg, k.tight(cu_seqlens, "cu_seqlens", cfg.B + 1, k.torch.int32), k.rows(x, "x", n, cfg.C, cfg.ld_x, xt),
      k.tight(weight, "weight", cfg.C * cfg.width, wt), k.tight(bias, "bias", cfg.C, wt), k.tight(state0, "state0", st, xt),
      k.rows(dy, "dy", n, cfg.C, cfg.ld_y, xt), k.tight(dstate_T, "dstate_T", st, xt),
      k.rows(dx, "dx", n, cfg.C, cfg.ld_x, xt), k.tight(dweight, "dweight", cfg.C * cfg.width, f32),
      k.tight(dbias, "dbias", cfg.C, f32), k.tight(dstate0, "dstate0", st, xt), _workspace(k, workspace, ws_bytes),
      int(ws_bytes))


def la_conv_step(cfg: ConvConfig, x, weight, bias, state, y, slots=None, n_slots: int = 0, stream=None) -> None:
    """One token; the state (or its slot of the pool) is shifted in place."""
    lib, k = _la.load_library(), _Call(stream)
    xt, wt = k.types.get(cfg.x_dtype, k.torch.float32), k.types.get(cfg.w_dtype, k.torch.float32)
    units = max(int(n_slots), 0) if slots is not None else cfg.B
    k(lib.la_conv_step, cfg, k.rows(x, "x", cfg.B, cfg.C, cfg.ld_x, xt), k.tight(weight, "weight", cfg.C * cfg.width, wt),
      k.tight(bias, "bias", cfg.C, wt), k.tight(state, "state", units * (cfg.width - 1) * cfg.C, xt),
      k.tight(slots, "slots", cfg.B, k.torch.int32), int(n_slots), k.rows(y, "y", cfg.B, cfg.C, cfg.ld_y, xt))


# ----------------------------------------------------------------------------- selective scan
def _scan_inputs(k, cfg, n, x, dt, A, b, c, D, dt_bias):
    xt, f32 = k.types.get(cfg.x_dtype, k.torch.float32), k.torch.float32
    return (k.rows(x, "x", n, cfg.H * cfg.d_v, cfg.ld_x, xt), k.rows(dt, "dt", n, cfg.H, cfg.ld_dt, k.types.get(cfg.dt_dtype, k.torch.float32)),
            k.tight(A, "A", cfg.H, f32), k.rows(b, "b", n, cfg.G * cfg.d_k, cfg.ld_b, xt),
            k.rows(c, "c", n, cfg.G * cfg.d_k, cfg.ld_c, xt), k.tight(D, "D", cfg.H, f32),
            k.tight(dt_bias, "dt_bias", cfg.H, f32))


def la_scan_workspace_bytes(cfg: ScanConfig) -> int:
    return _la.load_library().la_scan_workspace_bytes(cfg)


def la_scan_fwd(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S0, y, S_T, workspace, ws_bytes: int, cu_seqlens=None,
                stream=None) -> None:
    """S <- exp(Delta A) S + Delta b x^T, y = S^T c + D x over every sequence."""
    lib, k = _la.load_library(), _Call(stream)
    n, st, f32 = _tokens(cfg, cu_seqlens), cfg.B * cfg.H * cfg.d_k * cfg.d_v, k.torch.float32
    k(lib.la_scan_fwd, cfg, k.tight(cu_seqlens, "cu_seqlens", cfg.B + 1, k.torch.int32),
      *_scan_inputs(k, cfg, n, x, dt, A, b, c, D, dt_bias), k.tight(S0, "S0", st, f32),
      k.tight(y, "y", n * cfg.H * cfg.d_v, k.types.get(cfg.out_dtype, k.torch.float32)), k.tight(S_T, "S_T", st, f32),
      _workspace(k, workspace, ws_bytes), int(ws_bytes))


def la_scan_bwd_workspace_bytes(cfg: ScanConfig) -> int:
    return _la.load_library().la_scan_bwd_workspace_bytes(cfg)


def la_scan_bwd(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S0, dy, dS_T, dx, ddt, dA, db, dc, dD, ddt_bias, dS0,
                workspace, ws_bytes: int, cu_seqlens=None, stream=None) -> None:
    """Gradients of la_scan_fwd."""
    lib, k = _la.load_library(), _Call(stream)
    n, st, f32 = _tokens(cfg, cu_seqlens), cfg.B * cfg.H * cfg.d_k * cfg.d_v, k.torch.float32
    xt = k.types.get(cfg.x_dtype, k.torch.float32)
    k(lib.la_scan_bwd, cfg, k.tight(cu_seqlens, "cu_seqlens", cfg.B + 1, k.torch.int32),
      *_scan_inputs(k, cfg, n, x, dt, A, b, c, D, dt_bias), k.tight(S0, "S0", st, f32),
      k.tight(dy, "dy", n * cfg.H * cfg.d_v, k.types.get(cfg.out_dtype, k.torch.float32)), k.tight(dS_T, "dS_T", st, f32),
      k.rows(dx, "dx", n, cfg.H * cfg.d_v, cfg.ld_x, xt), k.rows(ddt, "ddt", n, cfg.H, cfg.ld_dt, k.types.get(cfg.dt_dtype, k.torch.float32)),
      k.tight(dA, "dA", cfg.H, f32), k.rows(db, "db", n, cfg.G * cfg.d_k, cfg.ld_b, xt),
      k.rows(dc, "dc", n, cfg.G * cfg.d_k, cfg.ld_c, xt), k.tight(dD, "dD", cfg.H, f32),
      k.tight(ddt_bias, "ddt_bias", cfg.H, f32), k.tight(dS0, "dS0", st, f32), _workspace(k, workspace, ws_bytes),
      int(ws_bytes))


def la_scan_step(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S, y, slots=None, n_slots: int = 0, stream=None) -> None:
    """One token; the state (or its slot of the pool) is advanced in place."""
    lib, k = _la.load_library(), _Call(stream)
    units = max(int(n_slots), 0) if slots is not None else cfg.B
    k(lib.la_scan_step, cfg, *_scan_inputs(k, cfg, cfg.B, x, dt, A, b, c, D, dt_bias),
      k.tight(S, "S", units * cfg.H * cfg.d_k * cfg.d_v, k.torch.float32), k.tight(slots, "slots", cfg.B, k.torch.int32),
      int(n_slots), k.tight(y, "y", cfg.B * cfg.H * cfg.d_v, k.types.get(cfg.out_dtype, k.torch.float32)))


# -------------------------------------------------- RMS norm with the residual's addition
def la_norm_fwd(cfg: NormConfig, x, residual, weight, res_out, y, codes=None, scales=None, stream=None) -> None:
    """res_out = x + residual, y = its RMS norm, and with a quantizer its codes and scales."""
    lib, k = _la.load_library(), _Call(stream)
    t, n, xt = k.torch, cfg.rows * cfg.d, k.types.get(cfg.x_dtype, k.torch.float32)
    eight = (t.int8, t.uint8, t.float8_e4m3fn)
    k(lib.la_norm_fwd, cfg, k.tight(x, "x", n, xt), k.tight(residual, "residual", n, xt),
      k.tight(weight, "weight", cfg.d, k.types.get(cfg.w_dtype, k.torch.float32)), k.tight(res_out, "res_out", n, xt),
      k.tight(y, "y", n, k.types.get(cfg.out_dtype, k.torch.float32)), k.tight(codes, "codes", n, *eight),
      k.tight(scales, "scales", n // (cfg.group or cfg.d) if cfg.d > 0 else 0, t.float32))


def la_norm_bwd_workspace_bytes(cfg: NormConfig) -> int:
    return _la.load_library().la_norm_bwd_workspace_bytes(cfg)


def la_norm_bwd(cfg: NormConfig, h, weight, dy, dres, dx, dweight, workspace, ws_bytes: int, stream=None) -> None:
    """Gradients of la_norm_fwd from its res_out (straight through the codec)."""
    lib, k = _la.load_library(), _Call(stream)
    n, xt = cfg.rows * cfg.d, k.types.get(cfg.x_dtype, k.torch.float32)
    k(lib.la_norm_bwd, cfg, k.tight(h, "h", n, xt), k.tight(weight, "weight", cfg.d, k.types.get(cfg.w_dtype, k.torch.float32)),
      k.tight(dy, "dy", n, k.types.get(cfg.out_dtype, k.torch.float32)), k.tight(dres, "dres", n, xt), k.tight(dx, "dx", n, xt),
      k.tight(dweight, "dweight", cfg.d, k.torch.float32), _workspace(k, workspace, ws_bytes), int(ws_bytes))
