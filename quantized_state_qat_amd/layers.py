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
                      ("la_scan_bwd_workspace_bytes", ScanConfig), ("la_scan_bwd_varlen_workspace_bytes", ScanConfig),
                      ("la_norm_bwd_workspace_bytes", NormConfig)):
        f = getattr(lib, name)
        f.restype, f.argtypes = sz, [ctypes.POINTER(cfg)]


_torch = None   # set by the first call: the package imports torch with the library
_types = ()     # torch dtypes by la_dtype
_current = None  # GPU index -> its current stream's handle


def _library():
    global _torch, _types, _current
    lib = _la.load_library()
    if _torch is None:
        import torch
        _types = (torch.float32, torch.bfloat16)
        # (a stream object costs a microsecond a call, a fifth of a short one)
        _current = getattr(torch._C, "_cuda_getCurrentRawStream", lambda gpu: torch.cuda.current_stream(gpu).cuda_stream)
        _torch = torch  # (last: another thread's call goes by it)
    return lib


def _dtype(code):
    return _types[code] if code in (_F32, _BF16) else _types[_F32]  # (an unknown code is refused by the library)


def _code_type(cfg, codes):
    """The dtype that a tensor of codes must have: uint8, or the quantizer's own."""
    if codes is None or codes.__class__ is int or codes.dtype is _torch.uint8:
        return _torch.uint8
    return _torch.int8 if cfg.qdq == _la.LA_QDQ_INT8_GROUP else _torch.float8_e4m3fn


def _gpu(*tensors):
    """The GPU of the first tensor among the arguments (all of a call's: any of them may be missing
    or a raw address); None when it is on the host or there is none."""
    for t in tensors:
        if t is not None and t.__class__ is not int:
            return t.get_device() if t.is_cuda else None
    return None


def _elsewhere(t, name, gpu):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
    raise ValueError(f"{name} is on GPU {t.get_device()}, the first tensor on {'the host' if gpu is None else f'GPU {gpu}'}")


def _tight(gpu, t, name, numel, dtype):
    """Address of a contiguous tensor of at least `numel` elements."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != gpu:
        _elsewhere(t, name, gpu)
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the configuration needs {numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(gpu, t, name, tokens, width, ld, dtype):
    """Address of `tokens` rows of `width` contiguous elements, `ld` (0: width) elements apart."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != gpu:
        _elsewhere(t, name, gpu)
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() < tokens * width:
        raise ValueError(f"{name} holds {t.numel()} elements, the configuration needs {tokens * width}")
    if (ld == 0 or ld == width) and t.is_contiguous():
        return t.data_ptr()
    ld = ld or width
    shape, strides = t.shape, t.stride()
    if len(shape) == 3 and strides == (ld, shape[2], 1) and shape[1] * shape[2] == width:  # tokens of heads or groups
        return t.data_ptr()
    inner = want = 1  # elements of the row walked so far, the stride the next dimension must have
    for n, step in zip(shape[::-1], strides[::-1]):
        if step != want and n != 1:
            raise ValueError(f"{name} has strides {strides}: rows of {width} contiguous elements, {ld} apart, are needed")
        if inner < width:
            inner *= n
            if inner > width:
                raise ValueError(f"{name} has shape {tuple(t.shape)}: its last dimensions must make up a row of {width}")
            want = ld if inner == width else inner
        else:
            want *= n
    return t.data_ptr()


def _workspace(gpu, workspace, ws_bytes):
    if workspace is None or workspace.__class__ is int:
        return workspace
    if workspace.get_device() != gpu:
        _elsewhere(workspace, "workspace", gpu)
    if workspace.numel() * workspace.element_size() < ws_bytes:
        raise ValueError(f"workspace holds fewer than the {int(ws_bytes)} bytes passed as ws_bytes")
    return _la._ptr(workspace)


def _call(gpu, stream, fn, *args):
    """The call on its tensors' GPU and that GPU's current stream, or `stream`."""
    cuda = _torch.cuda
    if stream is None:
        stream = _current(cuda.current_device() if gpu is None else gpu)
    elif stream.__class__ is not int:
        if gpu is not None and stream.device.index != gpu:
            raise ValueError(f"stream is on GPU {stream.device.index}, the tensors on GPU {gpu}")
        stream = stream.cuda_stream
    if gpu is None or gpu == cuda.current_device():
        status = fn(*args, stream)
    else:
        with cuda.device(gpu):
            status = fn(*args, stream)
    if status:
        _la._check(status)


def _tokens(cfg, cu_seqlens):
    return cfg.T if cu_seqlens is not None else cfg.B * cfg.T


# ------------------------------------------------------------------ short causal convolution
def la_conv_fwd(cfg: ConvConfig, x, weight, bias, state0, y, state_T=None, cu_seqlens=None, stream=None) -> None:
    """y = act(causal depthwise convolution of state0 ++ x); state_T = its last rows."""
    lib = _library()
    gpu = _gpu(x, weight, y, bias, state0, state_T, cu_seqlens)
    xt, wt, n = _dtype(cfg.x_dtype), _dtype(cfg.w_dtype), _tokens(cfg, cu_seqlens)
    st = cfg.B * (cfg.width - 1) * cfg.C
    _call(gpu, stream, lib.la_conv_fwd, cfg,
          _tight(gpu, cu_seqlens, "cu_seqlens", cfg.B + 1, _torch.int32), _rows(gpu, x, "x", n, cfg.C, cfg.ld_x, xt),
          _tight(gpu, weight, "weight", cfg.C * cfg.width, wt), _tight(gpu, bias, "bias", cfg.C, wt),
          _tight(gpu, state0, "state0", st, xt),
          _rows(gpu, y, "y", n, cfg.C, cfg.ld_y, xt), _tight(gpu, state_T, "state_T", st, xt))


def la_conv_bwd_workspace_bytes(cfg: ConvConfig) -> int:
    return _la.load_library().la_conv_bwd_workspace_bytes(cfg)


def la_conv_bwd(cfg: ConvConfig, x, weight, bias, state0, dy, dstate_T, dx, dweight, dbias, dstate0, workspace,
                ws_bytes: int, cu_seqlens=None, stream=None) -> None:
    """Gradients of la_conv_fwd (dweight and dbias float32)."""
    lib = _library()
    gpu = _gpu(x, weight, dy, dx, bias, state0, dstate_T, dweight, dbias, dstate0, workspace, cu_seqlens)
    xt, wt, n = _dtype(cfg.x_dtype), _dtype(cfg.w_dtype), _tokens(cfg, cu_seqlens)
    st, f32 = cfg.B * (cfg.width - 1) * cfg.C, _torch.float32
    _call(gpu, stream, lib.la_conv_bwd, cfg,
          _tight(gpu, cu_seqlens, "cu_seqlens", cfg.B + 1, _torch.int32), _rows(gpu, x, "x", n, cfg.C, cfg.ld_x, xt),
          _tight(gpu, weight, "weight", cfg.C * cfg.width, wt), _tight(gpu, bias, "bias", cfg.C, wt),
          _tight(gpu, state0, "state0", st, xt),
          _rows(gpu, dy, "dy", n, cfg.C, cfg.ld_y, xt), _tight(gpu, dstate_T, "dstate_T", st, xt),
          _rows(gpu, dx, "dx", n, cfg.C, cfg.ld_x, xt), _tight(gpu, dweight, "dweight", cfg.C * cfg.width, f32),
          _tight(gpu, dbias, "dbias", cfg.C, f32), _tight(gpu, dstate0, "dstate0", st, xt), _workspace(gpu, workspace, ws_bytes),
          int(ws_bytes))


def la_conv_step(cfg: ConvConfig, x, weight, bias, state, y, slots=None, n_slots: int = 0, stream=None) -> None:
    """One token; the state (or its slot of the pool) is shifted in place."""
    lib = _library()
    gpu = _gpu(x, weight, state, y, bias, slots)
    xt, wt = _dtype(cfg.x_dtype), _dtype(cfg.w_dtype)
    units = max(int(n_slots), 0) if slots is not None else cfg.B
    _call(gpu, stream, lib.la_conv_step, cfg,
          _rows(gpu, x, "x", cfg.B, cfg.C, cfg.ld_x, xt), _tight(gpu, weight, "weight", cfg.C * cfg.width, wt),
          _tight(gpu, bias, "bias", cfg.C, wt), _tight(gpu, state, "state", units * (cfg.width - 1) * cfg.C, xt),
          _tight(gpu, slots, "slots", cfg.B, _torch.int32), int(n_slots), _rows(gpu, y, "y", cfg.B, cfg.C, cfg.ld_y, xt))


# ----------------------------------------------------------------------------- selective scan
def _scan_inputs(gpu, cfg, n, x, dt, A, b, c, D, dt_bias):
    xt, f32 = _dtype(cfg.x_dtype), _torch.float32
    return (_rows(gpu, x, "x", n, cfg.H * cfg.d_v, cfg.ld_x, xt), _rows(gpu, dt, "dt", n, cfg.H, cfg.ld_dt, _dtype(cfg.dt_dtype)),
            _tight(gpu, A, "A", cfg.H, f32), _rows(gpu, b, "b", n, cfg.G * cfg.d_k, cfg.ld_b, xt),
            _rows(gpu, c, "c", n, cfg.G * cfg.d_k, cfg.ld_c, xt), _tight(gpu, D, "D", cfg.H, f32),
            _tight(gpu, dt_bias, "dt_bias", cfg.H, f32))


def la_scan_workspace_bytes(cfg: ScanConfig) -> int:
    return _la.load_library().la_scan_workspace_bytes(cfg)


def la_scan_fwd(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S0, y, S_T, workspace, ws_bytes: int, cu_seqlens=None,
                stream=None) -> None:
    """S <- exp(Delta A) S + Delta b x^T, y = S^T c + D x over every sequence."""
    lib = _library()
    gpu = _gpu(x, dt, A, b, c, y, D, dt_bias, S0, S_T, workspace, cu_seqlens)
    n, st, f32 = _tokens(cfg, cu_seqlens), cfg.B * cfg.H * cfg.d_k * cfg.d_v, _torch.float32
    _call(gpu, stream, lib.la_scan_fwd, cfg,
          _tight(gpu, cu_seqlens, "cu_seqlens", cfg.B + 1, _torch.int32),
          *_scan_inputs(gpu, cfg, n, x, dt, A, b, c, D, dt_bias), _tight(gpu, S0, "S0", st, f32),
          _tight(gpu, y, "y", n * cfg.H * cfg.d_v, _dtype(cfg.out_dtype)), _tight(gpu, S_T, "S_T", st, f32),
          _workspace(gpu, workspace, ws_bytes), int(ws_bytes))


def la_scan_bwd_workspace_bytes(cfg: ScanConfig) -> int:
    return _la.load_library().la_scan_bwd_workspace_bytes(cfg)


def la_scan_bwd_varlen_workspace_bytes(cfg: ScanConfig) -> int:
    """What la_scan_bwd needs with cu_seqlens (la_scan_bwd_workspace_bytes is enough too)."""
    return _la.load_library().la_scan_bwd_varlen_workspace_bytes(cfg)


def la_scan_bwd(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S0, dy, dS_T, dx, ddt, dA, db, dc, dD, ddt_bias, dS0,
                workspace, ws_bytes: int, cu_seqlens=None, stream=None) -> None:
    """Gradients of la_scan_fwd."""
    lib = _library()
    gpu = _gpu(x, dt, A, b, c, dy, dx, D, dt_bias, S0, dS_T, ddt, dA, db, dc, dD, ddt_bias, dS0, workspace, cu_seqlens)
    n, st, f32 = _tokens(cfg, cu_seqlens), cfg.B * cfg.H * cfg.d_k * cfg.d_v, _torch.float32
    xt = _dtype(cfg.x_dtype)
    _call(gpu, stream, lib.la_scan_bwd, cfg,
          _tight(gpu, cu_seqlens, "cu_seqlens", cfg.B + 1, _torch.int32),
          *_scan_inputs(gpu, cfg, n, x, dt, A, b, c, D, dt_bias), _tight(gpu, S0, "S0", st, f32),
          _tight(gpu, dy, "dy", n * cfg.H * cfg.d_v, _dtype(cfg.out_dtype)), _tight(gpu, dS_T, "dS_T", st, f32),
          _rows(gpu, dx, "dx", n, cfg.H * cfg.d_v, cfg.ld_x, xt), _rows(gpu, ddt, "ddt", n, cfg.H, cfg.ld_dt, _dtype(cfg.dt_dtype)),
          _tight(gpu, dA, "dA", cfg.H, f32), _rows(gpu, db, "db", n, cfg.G * cfg.d_k, cfg.ld_b, xt),
          _rows(gpu, dc, "dc", n, cfg.G * cfg.d_k, cfg.ld_c, xt), _tight(gpu, dD, "dD", cfg.H, f32),
          _tight(gpu, ddt_bias, "ddt_bias", cfg.H, f32), _tight(gpu, dS0, "dS0", st, f32), _workspace(gpu, workspace, ws_bytes),
          int(ws_bytes))


def la_scan_step(cfg: ScanConfig, x, dt, A, b, c, D, dt_bias, S, y, slots=None, n_slots: int = 0, stream=None) -> None:
    """One token; the state (or its slot of the pool) is advanced in place."""
    lib = _library()
    gpu = _gpu(x, dt, A, b, c, S, y, D, dt_bias, slots)
    units = max(int(n_slots), 0) if slots is not None else cfg.B
    _call(gpu, stream, lib.la_scan_step, cfg,
          *_scan_inputs(gpu, cfg, cfg.B, x, dt, A, b, c, D, dt_bias),
          _tight(gpu, S, "S", units * cfg.H * cfg.d_k * cfg.d_v, _torch.float32), _tight(gpu, slots, "slots", cfg.B, _torch.int32),
          int(n_slots), _tight(gpu, y, "y", cfg.B * cfg.H * cfg.d_v, _dtype(cfg.out_dtype)))


# -------------------------------------------------- RMS norm with the residual's addition
def la_norm_fwd(cfg: NormConfig, x, residual, weight, res_out, y, codes=None, scales=None, stream=None) -> None:
    """res_out = x + residual, y = its RMS norm, and with a quantizer its codes (uint8, or int8 for
    INT8 and float8_e4m3fn for E4M3) and scales."""
    lib = _library()
    gpu = _gpu(x, residual, weight, res_out, y, codes, scales)
    n, xt = cfg.rows * cfg.d, _dtype(cfg.x_dtype)
    _call(gpu, stream, lib.la_norm_fwd, cfg,
          _tight(gpu, x, "x", n, xt), _tight(gpu, residual, "residual", n, xt),
          _tight(gpu, weight, "weight", cfg.d, _dtype(cfg.w_dtype)), _tight(gpu, res_out, "res_out", n, xt),
          _tight(gpu, y, "y", n, _dtype(cfg.out_dtype)), _tight(gpu, codes, "codes", n, _code_type(cfg, codes)),
          _tight(gpu, scales, "scales", n // (cfg.group or cfg.d) if cfg.d > 0 else 0, _torch.float32))


def la_norm_bwd_workspace_bytes(cfg: NormConfig) -> int:
    return _la.load_library().la_norm_bwd_workspace_bytes(cfg)


def la_norm_bwd(cfg: NormConfig, h, weight, dy, dres, dx, dweight, workspace, ws_bytes: int, stream=None) -> None:
    """Gradients of la_norm_fwd from its res_out (straight through the codec)."""
    lib = _library()
    gpu = _gpu(h, weight, dy, dres, dx, dweight, workspace)
    n, xt = cfg.rows * cfg.d, _dtype(cfg.x_dtype)
    _call(gpu, stream, lib.la_norm_bwd, cfg,
          _tight(gpu, h, "h", n, xt), _tight(gpu, weight, "weight", cfg.d, _dtype(cfg.w_dtype)),
          _tight(gpu, dy, "dy", n, _dtype(cfg.out_dtype)), _tight(gpu, dres, "dres", n, xt), _tight(gpu, dx, "dx", n, xt),
          _tight(gpu, dweight, "dweight", cfg.d, _torch.float32), _workspace(gpu, workspace, ws_bytes), int(ws_bytes))
