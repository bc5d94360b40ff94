"""Python binding of liblores (the LoReS quantized recurrent-state decode step on
MI355X / gfx950).

The functions carry the C ABI's names (include/lores.h) and only marshal
arguments: torch tensors become device pointers, the current torch stream
becomes the hipStream_t, shapes and dtypes are checked so that no raw pointer
is handed over with too few elements.  All computation happens in the HIP
kernels of liblores.so; if the library is missing, calls raise.

PyTorch serves only as the device allocator and stream provider.
"""
import ctypes
import warnings

import numpy as np

from . import _lib
from ._lib import (LORES_BF16, LORES_FP8, LORES_FP32, LORES_INT4, LORES_INT6, LORES_INT8,
                   LORES_MAX_NORM, LORES_MAX_WINDOW, LORES_ROUND_NEAREST, LORES_ROUND_STOCHASTIC, LORES_SCALE_KEY,
                   LORES_SCALE_VALUE, LoresLayout, LoresLibraryMissing)

__all__ = ["LORES_FP32", "LORES_BF16", "LORES_INT8", "LORES_INT4", "LORES_INT6", "LORES_FP8",
           "LORES_ROUND_STOCHASTIC", "LORES_ROUND_NEAREST", "LORES_SCALE_VALUE", "LORES_SCALE_KEY",
           "LoresError", "lores_state_set_rounding",
           "LORES_MAX_WINDOW", "LoresLibraryMissing", "LoresState", "lores_state_alloc",
           "lores_state_alloc_axis", "lores_state_alloc_window",
           "lores_state_layout",
           "lores_state_head_map", "lores_decay_stat", "lores_assign_precision",
           "lores_decode_step", "lores_step_launches", "lores_quant_state", "lores_dequant_state",
           "lores_scan", "lores_scan_workspace", "lores_scan_backward", "lores_rmsnorm", "lores_rmsnorm_backward",
           "LORES_MAX_NORM",
           "lores_last_error", "lores_spec_version"]


class LoresError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{_lib.STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(rc):
    if rc != 0:
        raise LoresError(rc, _lib.lib().lores_last_error().decode())


def _stream_ptr(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dev_ptr(t, name, dtype, numel, device):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the state is on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


def _host_array(x, dtype):
    a = np.ascontiguousarray(np.asarray(x, dtype=dtype))
    return a, a.ctypes.data_as(ctypes.c_void_p)


def lores_spec_version():
    return _lib.lib().lores_spec_version()


def lores_last_error():
    return _lib.lib().lores_last_error().decode()


class LoresState:
    """A quantized recurrent state: the library handle plus its device buffer.

    The buffer is a torch uint8 tensor (caller-owned device memory); the handle
    is freed when this object is garbage-collected.
    """

    def __init__(self, handle, buf, B, H, d_k, d_v, head_prec, scale_axis=LORES_SCALE_VALUE,
                 window=1):
        self._h = handle
        self.buf = buf
        self.device = buf.device
        self.B, self.H, self.d_k, self.d_v = B, H, d_k, d_v
        self.head_prec = list(head_prec)
        self.rounding = LORES_ROUND_STOCHASTIC
        self.scale_axis = scale_axis
        self.window = window

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            try:
                _lib.lib().lores_state_free(h)
            except Exception:
                pass
            self._h = None


def lores_state_alloc(B, H, d_k, d_v, head_prec, device=None, stream=None, buf=None,
                      scale_axis=LORES_SCALE_VALUE, window=1):
    """Plan the packed layout; size query if device and buf are both None.

    Returns the byte size (size query) or a LoresState whose buffer (a new
    torch uint8 tensor on `device`, or the given `buf`) is cleared to S_0 = 0
    on `stream`.  scale_axis: LORES_SCALE_VALUE (one scale per value row,
    lores_state_alloc) or LORES_SCALE_KEY (one per key column,
    lores_state_alloc_axis).  window > 1: requantize the scaled heads once per
    window of that many steps (lores_state_alloc_window).
    """
    L = _lib.lib()
    hp, hp_ptr = _host_array(head_prec, np.uint8)
    if hp.size != H:
        raise ValueError(f"head_prec must have H = {H} entries")
    window = int(window)

    def alloc(ptr, size, stream_ptr, out):
        if window != 1:
            return L.lores_state_alloc_window(B, H, d_k, d_v, hp_ptr, int(scale_axis), window, ptr,
                                              size, stream_ptr, out)
        return L.lores_state_alloc_axis(B, H, d_k, d_v, hp_ptr, int(scale_axis), ptr, size,
                                        stream_ptr, out)
    nbytes = ctypes.c_size_t(0)
    _check(alloc(None, ctypes.byref(nbytes), None, None))
    if device is None and buf is None:
        return nbytes.value
    import torch
    if buf is None:
        buf = torch.empty(nbytes.value, dtype=torch.uint8, device=device)
    device = buf.device
    size = ctypes.c_size_t(buf.numel() * buf.element_size())
    out = ctypes.c_void_p()
    _check(alloc(ctypes.c_void_p(buf.data_ptr()), ctypes.byref(size), _stream_ptr(stream, device),
                 ctypes.byref(out)))
    return LoresState(out.value, buf, B, H, d_k, d_v, hp.tolist(), int(scale_axis), window)


lores_state_alloc_axis = lores_state_alloc
lores_state_alloc_window = lores_state_alloc


def lores_state_layout(state):
    lay = LoresLayout()
    _check(_lib.lib().lores_state_layout(ctypes.c_void_p(state.handle), ctypes.byref(lay)))
    return {"B": lay.B, "H": lay.H, "d_k": lay.d_k, "d_v": lay.d_v, "d_v_pad": lay.d_v_pad,
            "n_class": list(lay.n_class), "codes_offset": list(lay.codes_offset),
            "scales_offset": list(lay.scales_offset),
            "unit_code_bytes": list(lay.unit_code_bytes), "total_bytes": lay.total_bytes,
            "scale_axis": lay.scale_axis, "unit_scales": lay.unit_scales,
            "window": lay.window, "window_fill": lay.window_fill,
            "window_offset": list(lay.window_offset),
            "unit_window_bytes": list(lay.unit_window_bytes)}


def lores_state_head_map(state):
    prec = np.zeros(state.H, np.uint8)
    slot = np.zeros(state.H, np.int32)
    _check(_lib.lib().lores_state_head_map(ctypes.c_void_p(state.handle),
                                           prec.ctypes.data_as(ctypes.c_void_p),
                                           slot.ctypes.data_as(ctypes.c_void_p)))
    return prec, slot


def lores_state_set_rounding(state, mode):
    """LORES_ROUND_STOCHASTIC (default) or LORES_ROUND_NEAREST for later steps."""
    _check(_lib.lib().lores_state_set_rounding(ctypes.c_void_p(state.handle), int(mode)))
    state.rounding = int(mode)


def lores_step_launches(state):
    """Kernel launches one lores_decode_step on `state` enqueues."""
    n = ctypes.c_int32(0)
    _check(_lib.lib().lores_step_launches(ctypes.c_void_p(state.handle), ctypes.byref(n)))
    return n.value


def lores_decay_stat(alpha):
    """Mean log(alpha) per head; alpha host array [n, H] or [n, H, width] (fp32)."""
    a = np.ascontiguousarray(np.asarray(alpha, dtype=np.float32))
    if a.ndim == 2:
        a = a[:, :, None]
    if a.ndim != 3:
        raise ValueError("alpha must be [n, H] or [n, H, width]")
    n, H, W = a.shape
    stat = np.zeros(H, np.float64)
    _check(_lib.lib().lores_decay_stat(a.ctypes.data_as(ctypes.c_void_p), n, H, W,
                                       stat.ctypes.data_as(ctypes.c_void_p)))
    return stat


def lores_assign_precision(stat, tier_frac, tier_prec):
    s, sp = _host_array(stat, np.float64)
    f, fp = _host_array(tier_frac, np.float64)
    p, pp = _host_array(tier_prec, np.uint8)
    if f.size != p.size:
        raise ValueError("tier_frac and tier_prec must have the same length")
    out = np.zeros(s.size, np.uint8)
    _check(_lib.lib().lores_assign_precision(sp, s.size, fp, pp, f.size,
                                             out.ctypes.data_as(ctypes.c_void_p)))
    return out.tolist()


def lores_decode_step(state, q, k, v, alpha, beta, delta, seed, t, o=None, seq_base=0,
                      head_base=0, stream=None):
    """One decode step t for all B x H units; returns o [B, H, d_v] fp32."""
    import torch
    B, H, dk, dv, dev = state.B, state.H, state.d_k, state.d_v, state.device
    in_bf16 = q.dtype == torch.bfloat16
    in_dt = torch.bfloat16 if in_bf16 else torch.float32
    per_channel = alpha.numel() == B * H * dk and dk != 1
    if o is None:
        o = torch.empty((B, H, dv), dtype=torch.float32, device=dev)
    args = (_dev_ptr(q, "q", in_dt, B * H * dk, dev), _dev_ptr(k, "k", in_dt, B * H * dk, dev),
            _dev_ptr(v, "v", in_dt, B * H * dv, dev))
    a_ptr = _dev_ptr(alpha, "alpha", torch.float32, B * H * dk if per_channel else B * H, dev)
    b_ptr = _dev_ptr(beta, "beta", torch.float32, B * H, dev)
    o_ptr = _dev_ptr(o, "o", torch.float32, B * H * dv, dev)
    _check(_lib.lib().lores_decode_step(ctypes.c_void_p(state.handle), *args, int(in_bf16), a_ptr,
                                        int(per_channel), b_ptr, int(delta), int(seed), int(t),
                                        int(seq_base), int(head_base), o_ptr,
                                        _stream_ptr(stream, dev)))
    return o


def lores_quant_state(state, X, seed, seq_base=0, head_base=0, stream=None):
    """fp32 [B, H, d_v, d_k] -> the packed state (requantized, draws keyed at t = 0)."""
    import torch
    shape = (state.B, state.H, state.d_v, state.d_k)
    ptr = _dev_ptr(X, "X", torch.float32, int(np.prod(shape)), state.device)
    _check(_lib.lib().lores_quant_state(ctypes.c_void_p(state.handle), ptr, int(seed),
                                        int(seq_base), int(head_base),
                                        _stream_ptr(stream, state.device)))


def lores_dequant_state(state, out=None, stream=None):
    """Packed state -> fp32 [B, H, d_v, d_k]."""
    import torch
    shape = (state.B, state.H, state.d_v, state.d_k)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=state.device)
    ptr = _dev_ptr(out, "out", torch.float32, int(np.prod(shape)), state.device)
    _check(_lib.lib().lores_dequant_state(ctypes.c_void_p(state.handle), ptr,
                                          _stream_ptr(stream, state.device)))
    return out


# ---------------------------------------------------------------- sequences
#
# The smallest of these calls take a few microseconds on the GPU, so the
# checks below hand plain integers to the library and look nothing up twice;
# outputs come from an input's new_empty and streams by the device's index,
# which cost the host 0.7 and 0.9 us less than torch.empty(device=) and a
# lookup by device.

class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NOTHING = _Nothing()


def _on(stream):
    """Allocations inside belong to `stream`, where the kernels that use them run."""
    import torch
    return _NOTHING if stream is None else torch.cuda.stream(stream)


def _raw_stream(stream, device):
    import torch
    return (torch.cuda.current_stream(device.index) if stream is None else stream).cuda_stream


def _no_graph(what):
    warnings.warn(f"{what} records no autograd graph: no gradient will reach its inputs. Call it and "
                  f"{what}_backward from a torch.autograd.Function, or under torch.no_grad()", stacklevel=3)


def _whole(t, name, dtype, shape, device):
    """The address of a contiguous tensor of this shape (None: NULL)."""
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the inputs are on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _need(t, name, dtype, shape, device):
    if t is None:
        raise TypeError(f"{name} must be a torch tensor")
    return _whole(t, name, dtype, shape, device)


def _rows4(t, name, dtype, shape, device):
    """A [B, T, heads, width] tensor with a contiguous last dimension: its
    address and its other strides."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, q is on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    st = t.stride()
    if st[3] != 1 and shape[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), st[:3]


def _scan_inputs(q, k, v, alpha, beta, delta, S0, lengths):
    import torch
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, T, heads, width], got {list(t.shape)}")
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"q must be on the GPU, got {dev}")
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q must be torch.bfloat16 or torch.float32, got {dt}")
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    d = _lib.LoresScanDims(B, T, H, Hk, dk, dv, int(dt == torch.bfloat16), int(delta))
    qp, d.q_stride[:] = _rows4(q, "q", dt, (B, T, Hk, dk), dev)
    kp, d.k_stride[:] = _rows4(k, "k", dt, (B, T, Hk, dk), dev)
    vp, d.v_stride[:] = _rows4(v, "v", dt, (B, T, H, dv), dev)
    f32 = torch.float32
    args = (qp, kp, vp, _need(alpha, "alpha", f32, (B, T, H), dev),
            _need(beta, "beta", f32, (B, T, H), dev),
            _whole(lengths, "lengths", torch.int32, (B,), dev),
            _whole(S0, "S0", f32, (B, H, dv, dk), dev))
    return d, args, dev, dt


def lores_scan_workspace(q, v, delta, backward=False):
    """Bytes of device workspace a lores_scan (or lores_scan_backward) of these
    shapes needs."""
    import torch
    B, T, Hk, dk = q.shape
    d = _lib.LoresScanDims(B, T, v.shape[2], Hk, dk, v.shape[3], int(q.dtype == torch.bfloat16),
                           int(delta))
    n = ctypes.c_size_t(0)
    _check(_lib.lib().lores_scan_workspace(ctypes.byref(d), int(backward), ctypes.byref(n)))
    return n.value


def _scan_work(d, backward, workspace, dev):
    import torch
    n = ctypes.c_size_t(0)
    _check(_lib.lib().lores_scan_workspace(ctypes.byref(d), backward, ctypes.byref(n)))
    if workspace is None:
        if not n.value:
            return None, None, 0
        workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def lores_scan(q, k, v, alpha, beta, delta, S0=None, lengths=None, o=None, S=None, workspace=None,
               stream=None):
    """The recurrence over whole sequences, unquantized: a prompt, or a
    training step's forward pass.

    q, k [B, T, H_k, d_k] and v [B, T, H, d_v] (bf16 or fp32, any strides with
    a contiguous last dimension; H_k divides H), alpha, beta [B, T, H] fp32,
    S0 [B, H, d_v, d_k] fp32 or None (zero), lengths [B] int32 on the device
    or None.  Returns (o [B, T, H, d_v] of q's type, S [B, H, d_v, d_k] fp32);
    S is what lores_quant_state takes, and may be S0.  workspace: a device
    tensor of at least lores_scan_workspace bytes, or None to allocate it.
    No autograd graph is recorded (lores_scan_backward has the gradients).
    """
    import torch
    d, args, dev, dt = _scan_inputs(q, k, v, alpha, beta, delta, S0, lengths)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or alpha.requires_grad
                                    or beta.requires_grad or S0 is not None and S0.requires_grad):
        _no_graph("lores_scan")
    with _on(stream):
        if o is None:
            o = v.new_empty(v.shape)
        if S is None:
            S = v.new_empty((d.B, d.H, d.d_v, d.d_k), dtype=torch.float32)
        work, wp, wn = _scan_work(d, 0, workspace, dev)
    _check(_lib.lib().lores_scan(
        ctypes.byref(d), *args, _need(o, "o", dt, v.shape, dev),
        _need(S, "S", torch.float32, (d.B, d.H, d.d_v, d.d_k), dev), wp, wn,
        _raw_stream(stream, dev)))
    return o, S


def lores_scan_backward(q, k, v, alpha, beta, delta, do, dS=None, S0=None, lengths=None,
                        workspace=None, stream=None):
    """Gradients of lores_scan's inputs from do (and dS) of its outputs.

    The forward pass is recomputed; do [B, T, H, d_v] has q's type, dS
    [B, H, d_v, d_k] is fp32 or None (zero).  Returns (dq, dk, dv, dalpha,
    dbeta, dS0), each of its input's type and shape, contiguous.
    """
    import torch
    d, args, dev, dt = _scan_inputs(q, k, v, alpha, beta, delta, S0, lengths)
    f32 = torch.float32
    dop = _need(do, "do", dt, v.shape, dev)
    dSp = _whole(dS, "dS", f32, (d.B, d.H, d.d_v, d.d_k), dev)
    with _on(stream):
        dq, dk, dv = q.new_empty(q.shape), q.new_empty(q.shape), v.new_empty(v.shape)
        da = v.new_empty((d.B, d.T, d.H), dtype=f32)
        db = torch.empty_like(da)
        dS0 = v.new_empty((d.B, d.H, d.d_v, d.d_k), dtype=f32)
        work, wp, wn = _scan_work(d, 1, workspace, dev)
    out = (dq, dk, dv, da, db, dS0)
    _check(_lib.lib().lores_scan_backward(
        ctypes.byref(d), *args, dop, dSp, *(t.data_ptr() for t in out), wp, wn,
        _raw_stream(stream, dev)))
    return out


def _norm_rows(t, name, dtype, shape, device):
    """A tensor of rows [..., n]: its address and the elements between rows."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the rows are on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    n = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), n
    if t.dim() != 2 or (t.stride(1) != 1 and n != 1) or t.stride(0) < n:
        raise ValueError(f"{name} must be contiguous, or [rows, n] with contiguous rows")
    return t.data_ptr(), t.stride(0)


def _norm_shape(x, weight):
    import torch
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError("the rows and weight must be torch tensors")
    if x.device.type != "cuda":
        raise ValueError(f"the rows must be on the GPU, got {x.device}")
    bf, f32 = torch.bfloat16, torch.float32
    for t, name in ((x, "the rows"), (weight, "weight")):
        if t.dtype is not bf and t.dtype is not f32:
            raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"rows must be [..., n] with n >= 1, got {list(x.shape)}")
    n = x.shape[-1]
    wp = _need(weight, "weight", weight.dtype, (n,), x.device)
    return x.numel() // n, n, wp, int(weight.dtype is bf), int(x.dtype is bf)


def lores_rmsnorm(x, weight, eps, residual=None, out_prec=None, stream=None):
    """Root-mean-square norm of the rows of x [..., n], of x + residual if given.

    Returns (y, scales, h).  out_prec None, LORES_FP32 or LORES_BF16: y in x's
    type, fp32 or bf16, scales None.  LORES_INT8 / LORES_FP8: y holds int8
    codes / torch.float8_e4m3fn values and scales [...] fp32 one factor per
    row.  h is the sum x + residual in x's type (x itself without a residual).
    No autograd graph is recorded (lores_rmsnorm_backward has the gradients).
    """
    import torch
    rows, n, wp, w_bf16, in_bf16 = _norm_shape(x, weight)
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad
                                    or residual is not None and residual.requires_grad):
        _no_graph("lores_rmsnorm")
    dev, dt = x.device, x.dtype
    xp, xs = _norm_rows(x, "x", dt, x.shape, dev)
    rp, rs = (None, 0) if residual is None else _norm_rows(residual, "residual", dt, x.shape, dev)
    if out_prec is None:
        out_prec = LORES_BF16 if in_bf16 else LORES_FP32
    quant = out_prec == LORES_INT8 or out_prec == LORES_FP8
    if quant:
        yt = torch.int8 if out_prec == LORES_INT8 else torch.float8_e4m3fn
    elif out_prec == LORES_FP32 or out_prec == LORES_BF16:
        yt = torch.float32 if out_prec == LORES_FP32 else torch.bfloat16
    else:
        raise ValueError("out_prec must be LORES_FP32, LORES_BF16, LORES_INT8 or LORES_FP8")
    h, hp, scales, sp = x, None, None, None
    with _on(stream):
        y = x.new_empty(x.shape, dtype=yt)
        if quant:
            scales = x.new_empty(x.shape[:-1], dtype=torch.float32)
            sp = scales.data_ptr()
        if residual is not None:
            h = x.new_empty(x.shape)
            hp = h.data_ptr()
    _check(_lib.lib().lores_rmsnorm(xp, xs, rp, rs, wp, w_bf16, rows, n, in_bf16, eps, out_prec,
                                    y.data_ptr(), sp, hp, _raw_stream(stream, dev)))
    return y, scales, h


def lores_rmsnorm_backward(h, weight, dy, eps, dresidual=None, stream=None):
    """Gradients (dx, dw) of lores_rmsnorm's unquantized output: dx [..., n] of
    h's type, for x and the residual alike, with the gradient dresidual that
    reaches h otherwise added; dw [n] fp32."""
    import torch
    rows, n, wp, w_bf16, in_bf16 = _norm_shape(h, weight)
    dev, dt = h.device, h.dtype
    hp, hs = _norm_rows(h, "h", dt, h.shape, dev)
    dyp = _need(dy, "dy", dt, h.shape, dev)
    drp = _whole(dresidual, "dresidual", dt, h.shape, dev)
    size = ctypes.c_size_t(0)
    _check(_lib.lib().lores_rmsnorm_workspace(rows, n, ctypes.byref(size)))
    with _on(stream):
        dx = h.new_empty(h.shape)
        dw = h.new_empty(n, dtype=torch.float32)
        work = h.new_empty(size.value, dtype=torch.uint8)
    _check(_lib.lib().lores_rmsnorm_backward(hp, hs, wp, w_bf16, dyp, drp, rows, n, in_bf16, eps,
                                             dx.data_ptr(), dw.data_ptr(), work.data_ptr(),
                                             size.value, _raw_stream(stream, dev)))
    return dx, dw
