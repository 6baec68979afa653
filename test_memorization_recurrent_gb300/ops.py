"""Python binding of include/atlas_ops.h: norm, layer norm, short convolution, selective
scan and gated linear recurrence.

Like the binding of the memory update it only marshals: ``make_*_cfg`` fills a C
description, the calls turn torch tensors into device pointers, enqueue on a stream and
raise ``AtlasError`` on a non-zero status.  Tensor arguments are checked before the call:
an element type other than the description's, a tensor that is not on the current CUDA
device, one that ends before the elements the description names, or one that is not
contiguous where the description has no strides of its own for it, raises
``AtlasError(ERR_INVALID)``.  Raw device pointers (ints) are passed on as they are.
"""
from __future__ import annotations

import ctypes

F32, BF16, F16, E4M3 = 0, 1, 2, 3
ACT_NONE, ACT_SILU = 0, 1
NORM_MAX_D, CONV_MAX_W, SCAN_MAX_N = 32768, 8, 128

OPS_EXPORTS = ("atlas_norm_forward", "atlas_norm_backward", "atlas_norm_backward_workspace_bytes",
               "atlas_layernorm_forward", "atlas_layernorm_backward",
               "atlas_layernorm_backward_workspace_bytes",
               "atlas_conv_forward", "atlas_conv_backward", "atlas_conv_backward_workspace_bytes",
               "atlas_scan_forward", "atlas_scan_workspace_bytes", "atlas_scan_backward",
               "atlas_scan_backward_workspace_bytes", "atlas_glr_forward", "atlas_glr_workspace_bytes",
               "atlas_glr_kept_bytes", "atlas_glr_backward", "atlas_glr_backward_workspace_bytes")

_int, _long, _vp, _size = ctypes.c_int, ctypes.c_long, ctypes.c_void_p, ctypes.c_size_t


class _Cfg(ctypes.Structure):
    """A description whose tensors' extents are worked out once, and again after a field that
    they depend on is set."""
    extents = None
    kept_bytes = None
    home = None  # the device of the tensors it was made with

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name not in ("workspace", "workspace_bytes", "held", "extents", "kept_bytes", "home"):
            super().__setattr__("extents", None)
            super().__setattr__("kept_bytes", None)


class AtlasNormCfg(_Cfg):
    """Mirror of ``atlas_norm_cfg`` in include/atlas_ops.h."""
    _fields_ = [("rows", _long), ("d", _int), ("dtype", _int), ("r_dtype", _int),
                ("w_dtype", _int), ("out_dtype", _int), ("group", _int), ("eps", ctypes.c_float),
                ("x_stride", _long), ("r_stride", _long), ("y_stride", _long),
                ("workspace", _vp), ("workspace_bytes", _size)]


class AtlasConvCfg(_Cfg):
    """Mirror of ``atlas_conv_cfg`` in include/atlas_ops.h."""
    _fields_ = [("B", _int), ("L", _int), ("C", _int), ("W", _int), ("act", _int), ("dtype", _int),
                ("w_dtype", _int), ("head_dim", _int), ("x_batch_stride", _long),
                ("x_token_stride", _long), ("y_batch_stride", _long), ("y_token_stride", _long),
                ("y_head_stride", _long), ("seq_start", _vp), ("slot", _vp), ("n_slots", _int),
                ("carry", _vp), ("status_dev", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class AtlasScanCfg(_Cfg):
    """Mirror of ``atlas_scan_cfg`` in include/atlas_ops.h."""
    _fields_ = [("B", _int), ("L", _int), ("D", _int), ("N", _int), ("G", _int), ("dtype", _int),
                ("softplus", _int), ("x_batch_stride", _long), ("x_token_stride", _long),
                ("dt_batch_stride", _long), ("dt_token_stride", _long), ("z_batch_stride", _long),
                ("z_token_stride", _long), ("y_batch_stride", _long), ("y_token_stride", _long),
                ("b_batch_stride", _long), ("b_token_stride", _long), ("c_batch_stride", _long),
                ("c_token_stride", _long), ("seq_start", _vp), ("slot", _vp), ("n_slots", _int),
                ("carry", _vp), ("status_dev", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class AtlasGlrCfg(_Cfg):
    """Mirror of ``atlas_glr_cfg`` in include/atlas_ops.h."""
    _fields_ = [("B", _int), ("L", _int), ("D", _int), ("dtype", _int), ("c", ctypes.c_float),
                ("x_batch_stride", _long), ("x_token_stride", _long), ("r_batch_stride", _long),
                ("r_token_stride", _long), ("i_batch_stride", _long), ("i_token_stride", _long),
                ("z_batch_stride", _long), ("z_token_stride", _long), ("y_batch_stride", _long),
                ("y_token_stride", _long), ("seq_start", _vp), ("slot", _vp), ("n_slots", _int),
                ("carry", _vp), ("status_dev", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


def declare(lib) -> None:
    """Argument types of the operators' entry points in an opened library."""
    norm, conv, scan, glr = (ctypes.POINTER(c) for c in (AtlasNormCfg, AtlasConvCfg, AtlasScanCfg, AtlasGlrCfg))
    lib.atlas_norm_forward.argtypes = [_vp] * 3 + [norm] + [_vp] * 4
    lib.atlas_norm_backward.argtypes = [_vp] * 4 + [norm] + [_vp] * 3
    lib.atlas_layernorm_forward.argtypes = [_vp] * 4 + [norm] + [_vp] * 4
    lib.atlas_layernorm_backward.argtypes = [_vp] * 4 + [norm] + [_vp] * 4
    lib.atlas_conv_forward.argtypes = [_vp] * 3 + [conv] + [_vp] * 4
    lib.atlas_conv_backward.argtypes = [_vp] * 3 + [conv] + [_vp] * 7
    lib.atlas_scan_forward.argtypes = [_vp] * 8 + [scan] + [_vp] * 4
    lib.atlas_scan_backward.argtypes = [_vp] * 8 + [scan] + [_vp] * 12
    lib.atlas_glr_forward.argtypes = [_vp] * 7 + [glr] + [_vp] * 5
    lib.atlas_glr_backward.argtypes = [_vp] * 7 + [glr] + [_vp] * 12
    for name in OPS_EXPORTS:
        getattr(lib, name).restype = _size if name.endswith("_bytes") else _int
    lib.atlas_norm_backward_workspace_bytes.argtypes = [norm]
    lib.atlas_layernorm_backward_workspace_bytes.argtypes = [norm]
    lib.atlas_conv_backward_workspace_bytes.argtypes = [conv]
    lib.atlas_scan_workspace_bytes.argtypes = [scan]
    lib.atlas_scan_backward_workspace_bytes.argtypes = [scan]
    for name in ("atlas_glr_workspace_bytes", "atlas_glr_kept_bytes", "atlas_glr_backward_workspace_bytes"):
        getattr(lib, name).argtypes = [glr]


# ------------------------------------------------------------------ descriptions

def make_norm_cfg(rows, d, dtype=BF16, r_dtype=None, w_dtype=None, out_dtype=None, group=0,
                  eps=1e-6, x_stride=0, r_stride=0, y_stride=0, workspace=None,
                  workspace_bytes=0) -> AtlasNormCfg:
    """rows x d norm; r_dtype, w_dtype and out_dtype default to dtype.  group: channels per
    scale of an E4M3 output (0: one scale a row).  Strides in elements, 0 = d."""
    def or_dtype(t):
        return int(dtype if t is None else t)
    cfg = AtlasNormCfg(int(rows), int(d), int(dtype), or_dtype(r_dtype), or_dtype(w_dtype),
                       or_dtype(out_dtype), int(group), float(eps), int(x_stride), int(r_stride),
                       int(y_stride), _space(workspace, workspace_bytes), int(workspace_bytes))
    cfg.held = workspace
    cfg.home = _home(workspace)
    return cfg


def make_conv_cfg(B, L, C, W, act=ACT_SILU, dtype=BF16, w_dtype=None, head_dim=0,
                  x_strides=(0, 0), y_strides=(0, 0, 0), seq_start=None, slot=None, n_slots=0,
                  carry=None, status_dev=None, workspace=None, workspace_bytes=0) -> AtlasConvCfg:
    """x_strides: (batch, token), y_strides: (batch, token, head) in elements, all 0 =
    contiguous.  seq_start, slot, carry, status_dev: device tensors (int32 [B + 1],
    int32 [B], uint8 [B], int32 [1]), which the description holds on to."""
    xb, xt = x_strides
    yb, yt, yh = tuple(y_strides) + (0,) * (3 - len(y_strides))
    cfg = AtlasConvCfg(int(B), int(L), int(C), int(W), int(act), int(dtype),
                       int(dtype if w_dtype is None else w_dtype), int(head_dim), int(xb), int(xt),
                       int(yb), int(yt), int(yh), *_sequences(B, seq_start, slot, n_slots, carry),
                       _checked(status_dev, "int32", 1, "status_dev"), _space(workspace, workspace_bytes),
                       int(workspace_bytes))
    cfg.held = (seq_start, slot, carry, status_dev, workspace)  # as long as the description
    cfg.home = _home(*cfg.held)
    return cfg


def make_scan_cfg(B, L, D, N, G=1, dtype=BF16, softplus=True, x_strides=(0, 0),
                  dt_strides=(0, 0), z_strides=(0, 0), y_strides=(0, 0), B_strides=(0, 0),
                  C_strides=(0, 0), seq_start=None, slot=None, n_slots=0, carry=None,
                  status_dev=None, workspace=None, workspace_bytes=0) -> AtlasScanCfg:
    """Strides: (batch, token) in elements, (0, 0) = contiguous.  Device tensors as for
    ``make_conv_cfg``."""
    s = [int(v) for p in (x_strides, dt_strides, z_strides, y_strides, B_strides, C_strides)
         for v in p]
    cfg = AtlasScanCfg(int(B), int(L), int(D), int(N), int(G), int(dtype), int(bool(softplus)),
                       *s, *_sequences(B, seq_start, slot, n_slots, carry),
                       _checked(status_dev, "int32", 1, "status_dev"), _space(workspace, workspace_bytes),
                       int(workspace_bytes))
    cfg.held = (seq_start, slot, carry, status_dev, workspace)
    cfg.home = _home(*cfg.held)
    return cfg


def make_glr_cfg(B, L, D, c=8.0, dtype=BF16, x_strides=(0, 0), r_strides=(0, 0), i_strides=(0, 0),
                 z_strides=(0, 0), y_strides=(0, 0), seq_start=None, slot=None, n_slots=0, carry=None,
                 status_dev=None, workspace=None, workspace_bytes=0) -> AtlasGlrCfg:
    """Strides: (batch, token) in elements, (0, 0) = contiguous.  Device tensors as for
    ``make_conv_cfg``."""
    s = [int(v) for p in (x_strides, r_strides, i_strides, z_strides, y_strides) for v in p]
    cfg = AtlasGlrCfg(int(B), int(L), int(D), int(dtype), float(c), *s,
                      *_sequences(B, seq_start, slot, n_slots, carry),
                      _checked(status_dev, "int32", 1, "status_dev"), _space(workspace, workspace_bytes),
                      int(workspace_bytes))
    cfg.held = (seq_start, slot, carry, status_dev, workspace)
    cfg.home = _home(*cfg.held)
    return cfg


# ------------------------------------------------------------------ arguments

def _error(msg):
    from . import ERR_INVALID, AtlasError
    return AtlasError(ERR_INVALID, msg)


def _space(t, nbytes):
    """Address of a workspace tensor that holds nbytes."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise _error(f"workspace must be a contiguous CUDA tensor of at least {nbytes} bytes")
    return t.data_ptr()


def _checked(t, dtype, n, name):
    """Address of a contiguous device tensor of at least n elements of a named type."""
    if t is None or isinstance(t, int):
        return t
    import torch
    if t.dtype != getattr(torch, dtype) or not t.is_cuda or t.numel() < n or not t.is_contiguous():
        raise _error(f"{name} must be a contiguous {dtype} CUDA tensor of at least {n} elements")
    return t.data_ptr()


def _home(*tensors):
    """The device of a description's tensors, which have to agree; None without any."""
    home = {t.get_device() for t in tensors if t is not None and not isinstance(t, int)}
    if len(home) > 1:
        raise _error("the tensors of a description are on different devices")
    return home.pop() if home else None


def _sequences(B, seq_start, slot, n_slots, carry):
    return (_checked(seq_start, "int32", int(B) + 1, "seq_start"),
            _checked(slot, "int32", int(B), "slot"), int(n_slots),
            _checked(carry, "uint8", int(B), "carry"))


_types = _device = _raw_stream = _fn = None


def _setup():
    """What every call needs, looked up once."""
    global _types, _device, _raw_stream, _fn
    import torch

    from . import load_library
    lib = load_library()
    torch.cuda.current_device()  # initialises CUDA
    _types = (torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn)
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _device = torch._C._cuda_getDevice
    _fn = {name: getattr(lib, name) for name in OPS_EXPORTS}


def _begin(cfg):
    """The current device, that of the description's tensors too; before anything else of a call."""
    if _fn is None:
        _setup()
    device = _device()
    if cfg.home is not None and cfg.home != device:
        raise _error(f"the description's tensors are not on the current device (cuda:{device})")
    return device


def _arg(t, code, extent, name, device):
    """Address of one argument (a tensor, an address or None) after its checks.  extent: twice
    the elements from the first to the last one that the description names, plus one where
    they have to be contiguous."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not _types[code]:
        raise _error(f"{name} is {t.dtype}, the description says {_types[code]}")
    if t.get_device() != device:
        raise _error(f"{name} is not on the current device (cuda:{device})")
    if extent & 1:
        if not t.is_contiguous():
            raise _error(f"{name} is not contiguous")
        if t.numel() < extent >> 1:
            raise _error(f"{name} has fewer than the {extent >> 1} elements the description names")
    elif t.numel() < extent >> 1 or not t.is_contiguous():
        # a strided view ends further on than its elements count, an expanded one, whose elements repeat, before
        if t.is_contiguous() or t.untyped_storage().nbytes() // t.element_size() - t.storage_offset() < extent >> 1:
            raise _error(f"{name} ends before the {extent >> 1} elements the description names")
    return t.data_ptr()


def _call(name, args, stream, device):
    if stream is None:
        stream = _raw_stream(device)
    elif type(stream) is not int:
        stream = stream.cuda_stream
    rc = _fn[name](*args, stream)
    if rc != 0:
        from . import AtlasError, atlas_mem_strerror
        raise AtlasError(rc, atlas_mem_strerror(rc))


def _bytes(fn, cfg):
    from . import load_library
    n = int(getattr(load_library(), fn)(ctypes.byref(cfg)))
    if n == 2 ** 64 - 1:
        raise _error("invalid or uncovered description")
    return n


def _known(*codes):
    for code in codes:
        if not 0 <= code <= E4M3:
            raise _error(f"no element type {code}")


def _dense(n):
    return 2 * n + 1


def _tokens(cfg, sb, st, width):
    """Extent of a [B, L, width] tensor (packed: [L, width])."""
    if cfg.L < 1 or cfg.B < 1:
        return 0
    if not sb and not st:
        return _dense((1 if cfg.seq_start else cfg.B) * cfg.L * width)
    return 2 * ((0 if cfg.seq_start else (cfg.B - 1) * sb) + (cfg.L - 1) * st + width)


def _rows(cfg, stride):
    if cfg.rows < 1:
        return 0
    return 2 * ((cfg.rows - 1) * stride + cfg.d) if stride else _dense(cfg.rows * cfg.d)


# ------------------------------------------------------------------ norm

def _norm_extents(c):
    _known(c.dtype, c.r_dtype, c.w_dtype, c.out_dtype)
    groups = 1 if c.group <= 0 or c.group >= c.d else -(-c.d // c.group)
    c.extents = e = (c.dtype, c.r_dtype, c.w_dtype, c.out_dtype, _dense(c.d), _rows(c, c.x_stride), _rows(c, c.r_stride),
                     _rows(c, c.y_stride), _dense(c.rows * groups))
    return e


def atlas_norm_forward(x, residual, weight, cfg: AtlasNormCfg, y, residual_out=None, scale=None,
                       stream=None) -> None:
    """y = norm(x + residual) * weight; residual_out receives x + residual, scale the scales
    of an E4M3 output.  residual, weight and residual_out may be None."""
    dev = _begin(cfg)
    t, r, w, o, d, nx, nr, ny, ns = cfg.extents or _norm_extents(cfg)
    _call("atlas_norm_forward",
          (_arg(x, t, nx, "x", dev), _arg(residual, r, nr, "residual", dev), _arg(weight, w, d, "weight", dev), cfg,
           _arg(y, o, ny, "y", dev), _arg(residual_out, r, nr, "residual_out", dev), _arg(scale, F32, ns, "scale", dev)),
          stream, dev)


def atlas_norm_backward_workspace_bytes(cfg: AtlasNormCfg) -> int:
    return _bytes("atlas_norm_backward_workspace_bytes", cfg)


def atlas_norm_backward(h, weight, dy, dh, cfg: AtlasNormCfg, dx, dw=None, stream=None) -> None:
    """dx = dL/dh and dw = dL/d weight from dy = dL/dy and (or None) dh, the gradient that
    reaches the residual stream from later layers."""
    dev = _begin(cfg)
    t, r, w, _, d, _, nr, ny, _ = cfg.extents or _norm_extents(cfg)
    _call("atlas_norm_backward",
          (_arg(h, r, nr, "h", dev), _arg(weight, w, d, "weight", dev), _arg(dy, t, ny, "dy", dev),
           _arg(dh, r, nr, "dh", dev), cfg, _arg(dx, r, nr, "dx", dev), _arg(dw, F32, d, "dw", dev)), stream, dev)


# ------------------------------------------------------------------ layer norm

def atlas_layernorm_forward(x, residual, weight, bias, cfg: AtlasNormCfg, y, residual_out=None, scale=None,
                            stream=None) -> None:
    """y = layernorm(x + residual) * weight + bias, described as a norm (``make_norm_cfg``, eps > 0);
    residual, weight, bias and residual_out may be None."""
    dev = _begin(cfg)
    t, r, w, o, d, nx, nr, ny, ns = cfg.extents or _norm_extents(cfg)
    _call("atlas_layernorm_forward",
          (_arg(x, t, nx, "x", dev), _arg(residual, r, nr, "residual", dev), _arg(weight, w, d, "weight", dev),
           _arg(bias, w, d, "bias", dev), cfg, _arg(y, o, ny, "y", dev), _arg(residual_out, r, nr, "residual_out", dev),
           _arg(scale, F32, ns, "scale", dev)), stream, dev)


def atlas_layernorm_backward_workspace_bytes(cfg: AtlasNormCfg) -> int:
    return _bytes("atlas_layernorm_backward_workspace_bytes", cfg)


def atlas_layernorm_backward(h, weight, dy, dh, cfg: AtlasNormCfg, dx, dw=None, dbias=None, stream=None) -> None:
    """dx = dL/dh, dw and dbias from dy = dL/dy and (or None) dh, the gradient that reaches the
    residual stream from later layers."""
    dev = _begin(cfg)
    t, r, w, _, d, _, nr, ny, _ = cfg.extents or _norm_extents(cfg)
    _call("atlas_layernorm_backward",
          (_arg(h, r, nr, "h", dev), _arg(weight, w, d, "weight", dev), _arg(dy, t, ny, "dy", dev),
           _arg(dh, r, nr, "dh", dev), cfg, _arg(dx, r, nr, "dx", dev), _arg(dw, F32, d, "dw", dev),
           _arg(dbias, F32, d, "dbias", dev)), stream, dev)


# ------------------------------------------------------------------ conv

def _conv_extents(c):
    _known(c.dtype, c.w_dtype)
    hd, C, n = c.head_dim, c.C, c.n_slots if c.slot else c.B
    if c.L < 1 or c.B < 1:
        ny = 0
    elif not hd:
        ny = _tokens(c, c.y_batch_stride, c.y_token_stride, C)
    elif not (c.y_batch_stride or c.y_token_stride or c.y_head_stride):
        ny = _dense((1 if c.seq_start else c.B) * c.L * C)
    else:
        ny = 2 * ((0 if c.seq_start else (c.B - 1) * c.y_batch_stride) + (C // hd - 1) * c.y_head_stride
                  + (c.L - 1) * c.y_token_stride + hd)
    c.extents = e = (c.dtype, c.w_dtype, _dense(C), _dense(C * c.W), _tokens(c, c.x_batch_stride, c.x_token_stride, C),
                     ny, _dense(n * (c.W - 1) * C), _dense(c.B * (c.W - 1) * C))
    return e


def atlas_conv_forward(x, weight, bias, cfg: AtlasConvCfg, y, state_in=None, state_out=None,
                       stream=None) -> None:
    """Short causal convolution of every channel; L = 1 is the single-token form.  state_in
    and state_out ([B or n_slots, W - 1, C]) may be None or the same tensor."""
    dev = _begin(cfg)
    t, w, C, nw, nx, ny, n, _ = cfg.extents or _conv_extents(cfg)
    _call("atlas_conv_forward",
          (_arg(x, t, nx, "x", dev), _arg(weight, w, nw, "weight", dev), _arg(bias, w, C, "bias", dev), cfg,
           _arg(y, t, ny, "y", dev), _arg(state_in, t, n, "state_in", dev), _arg(state_out, t, n, "state_out", dev)),
          stream, dev)


def atlas_conv_backward_workspace_bytes(cfg: AtlasConvCfg) -> int:
    return _bytes("atlas_conv_backward_workspace_bytes", cfg)


def atlas_conv_backward(x, weight, bias, cfg: AtlasConvCfg, state_in, dy, dstate, dx, dw, dbias,
                        stream=None) -> None:
    """Gradients of the convolution (see include/atlas_ops.h); dstate is dL/d state_out on
    entry and dL/d state_in on return."""
    dev = _begin(cfg)
    t, w, C, nw, nx, ny, _, n = cfg.extents or _conv_extents(cfg)
    _call("atlas_conv_backward",
          (_arg(x, t, nx, "x", dev), _arg(weight, w, nw, "weight", dev), _arg(bias, w, C, "bias", dev), cfg,
           _arg(state_in, t, n, "state_in", dev), _arg(dy, t, ny, "dy", dev), _arg(dstate, F32, n, "dstate", dev),
           _arg(dx, t, nx, "dx", dev), _arg(dw, F32, nw, "dw", dev), _arg(dbias, F32, C, "dbias", dev)), stream, dev)


# ------------------------------------------------------------------ scan

def _scan_extents(c):
    _known(c.dtype)
    D, gn, dn = c.D, c.G * c.N, c.D * c.N
    c.extents = e = (c.dtype, _dense(D), _dense(dn), _tokens(c, c.x_batch_stride, c.x_token_stride, D),
                     _tokens(c, c.dt_batch_stride, c.dt_token_stride, D),
                     _tokens(c, c.b_batch_stride, c.b_token_stride, gn),
                     _tokens(c, c.c_batch_stride, c.c_token_stride, gn),
                     _tokens(c, c.z_batch_stride, c.z_token_stride, D),
                     _tokens(c, c.y_batch_stride, c.y_token_stride, D), _dense((c.n_slots if c.slot else c.B) * dn),
                     _dense(c.B * dn))
    return e


def atlas_scan_workspace_bytes(cfg: AtlasScanCfg) -> int:
    return _bytes("atlas_scan_workspace_bytes", cfg)


def atlas_scan_backward_workspace_bytes(cfg: AtlasScanCfg) -> int:
    return _bytes("atlas_scan_backward_workspace_bytes", cfg)


def atlas_scan_forward(x, dt, A, Bm, Cm, Dskip, z, dt_bias, cfg: AtlasScanCfg, y, h_in=None,
                       h_out=None, stream=None) -> None:
    """Selective scan; L = 1 is the single-token form.  Dskip, z, dt_bias, h_in and h_out
    may be None; h_in and h_out ([B or n_slots, D, N]) may be the same tensor."""
    dev = _begin(cfg)
    t, D, dn, nx, nt, nb, nc, nz, ny, n, _ = cfg.extents or _scan_extents(cfg)
    _call("atlas_scan_forward",
          (_arg(x, t, nx, "x", dev), _arg(dt, t, nt, "dt", dev), _arg(A, F32, dn, "A", dev), _arg(Bm, t, nb, "B", dev),
           _arg(Cm, t, nc, "C", dev), _arg(Dskip, F32, D, "Dskip", dev), _arg(z, t, nz, "z", dev),
           _arg(dt_bias, F32, D, "dt_bias", dev), cfg, _arg(y, t, ny, "y", dev), _arg(h_in, F32, n, "h_in", dev),
           _arg(h_out, F32, n, "h_out", dev)), stream, dev)


def atlas_scan_backward(x, dt, A, Bm, Cm, Dskip, z, dt_bias, cfg: AtlasScanCfg, h_in, dy, dh, dx,
                        ddt, dA, dB, dC, dD, dz, ddt_bias, stream=None) -> None:
    """Gradients of the scan (see include/atlas_ops.h); dh is dL/d h_out on entry and
    dL/d h_in on return."""
    dev = _begin(cfg)
    t, D, dn, nx, nt, nb, nc, nz, ny, _, n = cfg.extents or _scan_extents(cfg)
    _call("atlas_scan_backward",
          (_arg(x, t, nx, "x", dev), _arg(dt, t, nt, "dt", dev), _arg(A, F32, dn, "A", dev), _arg(Bm, t, nb, "B", dev),
           _arg(Cm, t, nc, "C", dev), _arg(Dskip, F32, D, "Dskip", dev), _arg(z, t, nz, "z", dev),
           _arg(dt_bias, F32, D, "dt_bias", dev), cfg, _arg(h_in, F32, n, "h_in", dev), _arg(dy, t, ny, "dy", dev),
           _arg(dh, F32, n, "dh", dev), _arg(dx, t, nx, "dx", dev), _arg(ddt, t, nt, "ddt", dev),
           _arg(dA, F32, dn, "dA", dev), _arg(dB, t, nb, "dB", dev), _arg(dC, t, nc, "dC", dev),
           _arg(dD, F32, D, "dD", dev), _arg(dz, t, nz, "dz", dev), _arg(ddt_bias, F32, D, "ddt_bias", dev)), stream, dev)


# ------------------------------------------------------------------ glr

def _glr_extents(c):
    _known(c.dtype)
    D = c.D
    c.extents = e = (c.dtype, _dense(D), _tokens(c, c.x_batch_stride, c.x_token_stride, D),
                     _tokens(c, c.r_batch_stride, c.r_token_stride, D), _tokens(c, c.i_batch_stride, c.i_token_stride, D),
                     _tokens(c, c.z_batch_stride, c.z_token_stride, D), _tokens(c, c.y_batch_stride, c.y_token_stride, D),
                     _dense((c.n_slots if c.slot else c.B) * D), _dense(c.B * D))
    return e


def _kept(t, cfg, device):
    """Address of the kept states, a tensor of any type."""
    if t is None or type(t) is int:
        return t
    nbytes = cfg.kept_bytes
    if nbytes is None:
        nbytes = cfg.kept_bytes = _bytes("atlas_glr_kept_bytes", cfg)
    if t.get_device() != device or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise _error(f"kept must be a contiguous tensor of at least {nbytes} bytes on the current device (cuda:{device})")
    return t.data_ptr()


def atlas_glr_workspace_bytes(cfg: AtlasGlrCfg) -> int:
    return _bytes("atlas_glr_workspace_bytes", cfg)


def atlas_glr_kept_bytes(cfg: AtlasGlrCfg) -> int:
    return _bytes("atlas_glr_kept_bytes", cfg)


def atlas_glr_backward_workspace_bytes(cfg: AtlasGlrCfg) -> int:
    return _bytes("atlas_glr_backward_workspace_bytes", cfg)


def atlas_glr_forward(x, r, i, z, lam, r_bias, i_bias, cfg: AtlasGlrCfg, y, h_in=None, h_out=None, kept=None,
                      stream=None) -> None:
    """Gated linear recurrence; L = 1 is the single-token form.  i, z, r_bias, i_bias, h_in, h_out and kept may be
    None; h_in and h_out ([B or n_slots, D]) may be the same tensor.  kept (``atlas_glr_kept_bytes``)
    receives what the backward pass starts from."""
    dev = _begin(cfg)
    t, D, nx, nr, ni, nz, ny, n, _ = cfg.extents or _glr_extents(cfg)
    _call("atlas_glr_forward",
          (_arg(x, t, nx, "x", dev), _arg(r, t, nr, "r", dev), _arg(i, t, ni, "i", dev), _arg(z, t, nz, "z", dev),
           _arg(lam, F32, D, "lam", dev), _arg(r_bias, F32, D, "r_bias", dev), _arg(i_bias, F32, D, "i_bias", dev), cfg,
           _arg(y, t, ny, "y", dev), _arg(h_in, F32, n, "h_in", dev), _arg(h_out, F32, n, "h_out", dev),
           _kept(kept, cfg, dev)), stream, dev)


def atlas_glr_backward(x, r, i, z, lam, r_bias, i_bias, cfg: AtlasGlrCfg, h_in, kept, dy, dh, dx, dr, di, dz, dlam,
                       dr_bias, di_bias, stream=None) -> None:
    """Gradients of the recurrence (see include/atlas_ops.h); dh is dL/d h_out on entry and dL/d h_in on return,
    kept what the forward pass kept, or None."""
    dev = _begin(cfg)
    t, D, nx, nr, ni, nz, ny, _, n = cfg.extents or _glr_extents(cfg)
    _call("atlas_glr_backward",
          (_arg(x, t, nx, "x", dev), _arg(r, t, nr, "r", dev), _arg(i, t, ni, "i", dev), _arg(z, t, nz, "z", dev),
           _arg(lam, F32, D, "lam", dev), _arg(r_bias, F32, D, "r_bias", dev), _arg(i_bias, F32, D, "i_bias", dev), cfg,
           _arg(h_in, F32, n, "h_in", dev), _kept(kept, cfg, dev), _arg(dy, t, ny, "dy", dev), _arg(dh, F32, n, "dh", dev),
           _arg(dx, t, nx, "dx", dev), _arg(dr, t, nr, "dr", dev), _arg(di, t, ni, "di", dev), _arg(dz, t, nz, "dz", dev),
           _arg(dlam, F32, D, "dlam", dev), _arg(dr_bias, F32, D, "dr_bias", dev), _arg(di_bias, F32, D, "di_bias", dev)),
          stream, dev)
