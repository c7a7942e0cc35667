"""torch-tensor front end of libmssm.

Each function checks tensor metadata, allocates the outputs with torch
(device memory), and passes raw device pointers plus the current HIP stream
to the C ABI.  No arithmetic of the method happens here.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib


class MssmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_status_name(status), message))
        self.status = status


def _status_name(s: int) -> str:
    try:
        return _lib.lib().mssm_status_string(s).decode()
    except OSError:
        return "status %d" % s


def _check(status: int):
    if status != _lib.MSSM_OK:
        msg = _lib.lib().mssm_last_error().decode()
        raise MssmError(status, msg)


def _io_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _lib.MSSM_F32
    if t.dtype == torch.bfloat16:
        return _lib.MSSM_BF16
    raise TypeError("activations must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))


def _need_shape(t, name, shape):
    """Caller-supplied output buffers must have exactly the output's shape:
    the C ABI sees only their addresses, so a smaller buffer would be written
    past its end on the device."""
    if t is not None and t.shape != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _stream_handle(device):
    # the handle alone: a torch.cuda.Stream object of it takes 1.8 us to make
    return torch._C._cuda_getCurrentRawStream(device.index)


_AS_IT_IS = contextlib.nullcontext()


def _on_device(device):
    """torch.cuda.device(device), which takes 1.3 us, only where it changes
    the current device."""
    return _AS_IT_IS if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def version() -> int:
    return int(_lib.lib().mssm_version())


@contextlib.contextmanager
def forced_variant(variant: int):
    """Run the enclosed calls (on this thread) with a fixed kernel variant."""
    L = _lib.lib()
    prev = L.mssm_force_variant(int(variant))
    try:
        yield
    finally:
        L.mssm_force_variant(prev)


def last_variant() -> int:
    return int(_lib.lib().mssm_last_variant())


def device_status(clear: bool = False) -> int:
    """Status bits the library's kernels set on the current device
    (``_lib.DEVICE_LOOKBACK_TIMEOUT``); waits for the device first."""
    import ctypes
    bits = ctypes.c_uint32(0)
    _check(_lib.lib().mssm_device_status(ctypes.byref(bits), 1 if clear else 0))
    return int(bits.value)


def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                       return_last_state=True, out=None, h_out=None, h0=None):
    """Selective-scan forward on the GPU.

    u, delta, z: (batch, dim, L) float32 or bfloat16 (all the same dtype);
    B, C: (batch, N, L) same dtype; A: (dim, N) float32; D, delta_bias:
    (dim,) float32; h0: (batch, dim, N) float32 initial state (None: zero;
    it may be passed as ``h_out`` too, to advance a state in place).
    Returns ``(y, h_last)`` with y like u and h_last (batch, dim, N) float32
    (None if ``return_last_state`` is False).
    """
    L = _lib.lib()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    io = u.dtype
    for name, t in (("u", u), ("delta", delta), ("B", B), ("C", C), ("z", z)):
        _need(t, name, io, dev)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0)):
        _need(t, name, torch.float32, dev)
    batch, dim, seqlen = u.shape
    N = A.shape[1]
    if h0 is not None and tuple(h0.shape) != (batch, dim, N):
        raise ValueError("h0 must be (batch, dim, N)")
    if delta.shape != u.shape or (z is not None and z.shape != u.shape):
        raise ValueError("u, delta, z must share one (batch, dim, L) shape")
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, N)")
    if tuple(B.shape) != (batch, N, seqlen) or tuple(C.shape) != (batch, N, seqlen):
        raise ValueError("B and C must be (batch, N, L)")
    for name, t in (("D", D), ("delta_bias", delta_bias)):
        if t is not None and tuple(t.shape) != (dim,):
            raise ValueError("%s must be (dim,)" % name)
    _need_shape(out, "out", u.shape)
    _need_shape(h_out, "h_out", (batch, dim, N))
    y = out if out is not None else torch.empty_like(u)
    _need(y, "out", io, dev)
    h_last = None
    if return_last_state:
        h_last = h_out if h_out is not None else torch.empty(
            (batch, dim, N), dtype=torch.float32, device=dev)
        _need(h_last, "h_out", torch.float32, dev)
    dims = _lib.ScanDims(batch, seqlen, dim, N)
    dt = _lib.DTypes(_io_dtype(u), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        if h0 is None:
            st = L.mssm_selective_scan_fwd(
                _ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                _ptr(D), _ptr(z), _ptr(y), _ptr(h_last), dims, dt,
                _stream_handle(dev))
        else:
            st = L.mssm_selective_scan_fwd_h0(
                _ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last), dims, dt,
                _stream_handle(dev))
    _check(st)
    return y, h_last


def selective_scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None, h0=None,
                               *, out, h_out):
    """``selective_scan_fwd`` through the entry point that allocates nothing
    on the device (mssm_selective_scan_fwd_h0_noalloc): the caller passes
    the outputs ``out`` (like u) and ``h_out`` ((batch, dim, N) float32,
    or None), and scratch comes from the library's fixed per-device array.
    Calls that overlap on one device race on that array."""
    L = _lib.lib()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    io = u.dtype
    for name, t in (("u", u), ("delta", delta), ("B", B), ("C", C), ("z", z)):
        _need(t, name, io, dev)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0)):
        _need(t, name, torch.float32, dev)
    if out is None:
        raise ValueError("out is required")
    batch, dim, seqlen = u.shape
    N = A.shape[1]
    if delta.shape != u.shape or (z is not None and z.shape != u.shape):
        raise ValueError("u, delta, z must share one (batch, dim, L) shape")
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, N)")
    if tuple(B.shape) != (batch, N, seqlen) or tuple(C.shape) != (batch, N, seqlen):
        raise ValueError("B and C must be (batch, N, L)")
    for name, t in (("D", D), ("delta_bias", delta_bias)):
        if t is not None and tuple(t.shape) != (dim,):
            raise ValueError("%s must be (dim,)" % name)
    for name, t in (("h0", h0), ("h_out", h_out)):
        _need_shape(t, name, (batch, dim, N))
    _need_shape(out, "out", u.shape)
    _need(out, "out", io, dev)
    _need(h_out, "h_out", torch.float32, dev)
    dims = _lib.ScanDims(batch, seqlen, dim, N)
    dtp = _lib.DTypes(_io_dtype(u), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        st = L.mssm_selective_scan_fwd_h0_noalloc(
            _ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(z), _ptr(h0), _ptr(out), _ptr(h_out), dims, dtp, _stream_handle(dev))
    _check(st)
    return out, h_out


def selective_scan_conv_fwd(x, conv_w, delta, A, B, C, D=None, z=None, delta_bias=None,
                            conv_b=None, h0=None, return_last_state=True, out=None, h_out=None):
    """Selective-scan forward fed by its convolution prologue on the GPU:
    the scan of u = silu(conv_b + causal width-4 depthwise conv(x)), with u
    formed on chip.

    x: (batch, dim, L) like the scan's u; conv_w: (dim, 4) float32; conv_b:
    (dim,) float32.  Other arguments and the result as for
    ``selective_scan_fwd``.
    """
    L = _lib.lib()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    _need(conv_w, "conv_w", torch.float32, dev)
    _need(conv_b, "conv_b", torch.float32, dev)
    batch, dim, seqlen = x.shape
    if tuple(conv_w.shape) != (dim, _lib.CONV_WIDTH):
        raise ValueError("conv_w must be (dim, %d)" % _lib.CONV_WIDTH)
    if conv_b is not None and tuple(conv_b.shape) != (dim,):
        raise ValueError("conv_b must be (dim,)")
    io = x.dtype
    for name, t in (("x", x), ("delta", delta), ("B", B), ("C", C), ("z", z)):
        _need(t, name, io, dev)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0)):
        _need(t, name, torch.float32, dev)
    N = A.shape[1]
    if delta.shape != x.shape or (z is not None and z.shape != x.shape):
        raise ValueError("x, delta, z must share one (batch, dim, L) shape")
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, N)")
    if tuple(B.shape) != (batch, N, seqlen) or tuple(C.shape) != (batch, N, seqlen):
        raise ValueError("B and C must be (batch, N, L)")
    if h0 is not None and tuple(h0.shape) != (batch, dim, N):
        raise ValueError("h0 must be (batch, dim, N)")
    for name, t in (("D", D), ("delta_bias", delta_bias)):
        if t is not None and tuple(t.shape) != (dim,):
            raise ValueError("%s must be (dim,)" % name)
    _need_shape(out, "out", x.shape)
    _need_shape(h_out, "h_out", (batch, dim, N))
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", io, dev)
    h_last = None
    if return_last_state:
        h_last = h_out if h_out is not None else torch.empty(
            (batch, dim, N), dtype=torch.float32, device=dev)
        _need(h_last, "h_out", torch.float32, dev)
    dims = _lib.ScanDims(batch, seqlen, dim, N)
    dtp = _lib.DTypes(_io_dtype(x), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        st = L.mssm_selective_scan_fwd_conv(
            _ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(delta), _ptr(delta_bias), _ptr(A),
            _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last), dims, dtp,
            _stream_handle(dev))
    _check(st)
    return y, h_last


def selective_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, h0=None,
                       dh_last=None):
    """Gradients of the selective scan on the GPU for output gradients ``dy``
    (like u) and ``dh_last`` (batch, dim, N) float32 (None: zero).

    Returns a dict of float32 tensors: du, ddelta (batch, dim, L); dA
    (dim, N); dB, dC (batch, N, L); dD, ddelta_bias (dim,); dz (batch, dim,
    L, when z is given); dh0 (batch, dim, N).
    """
    L = _lib.lib()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    io = u.dtype
    for name, t in (("u", u), ("delta", delta), ("B", B), ("C", C), ("z", z), ("dy", dy)):
        _need(t, name, io, dev)
    for name, t in (("A", A), ("D", D), ("delta_bias", delta_bias), ("h0", h0),
                    ("dh_last", dh_last)):
        _need(t, name, torch.float32, dev)
    batch, dim, seqlen = u.shape
    N = A.shape[1]
    if delta.shape != u.shape or dy.shape != u.shape or (z is not None and z.shape != u.shape):
        raise ValueError("u, delta, z, dy must share one (batch, dim, L) shape")
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, N)")
    if tuple(B.shape) != (batch, N, seqlen) or tuple(C.shape) != (batch, N, seqlen):
        raise ValueError("B and C must be (batch, N, L)")
    for name, t in (("h0", h0), ("dh_last", dh_last)):
        if t is not None and tuple(t.shape) != (batch, dim, N):
            raise ValueError("%s must be (batch, dim, N)" % name)
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"du": torch.empty(u.shape, **f32), "ddelta": torch.empty(u.shape, **f32),
         "dA": torch.empty((dim, N), **f32), "dB": torch.empty((batch, N, seqlen), **f32),
         "dC": torch.empty((batch, N, seqlen), **f32), "dD": torch.empty((dim,), **f32),
         "ddelta_bias": torch.empty((dim,), **f32),
         "dz": None if z is None else torch.empty(u.shape, **f32),
         "dh0": torch.empty((batch, dim, N), **f32)}
    dims = _lib.ScanDims(batch, seqlen, dim, N)
    dtp = _lib.DTypes(_io_dtype(u), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        st = L.mssm_selective_scan_bwd(
            _ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(h0), _ptr(dy), _ptr(dh_last), _ptr(g["du"]), _ptr(g["ddelta"]),
            _ptr(g["ddelta_bias"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
            _ptr(g["dz"]), _ptr(g["dh0"]), dims, dtp, _stream_handle(dev))
    _check(st)
    return g


def ssd_scalar_fwd(x, dt, A, B, C, D=None, dt_bias=None, chunk=0,
                   return_last_state=True, out=None, h_out=None, h0=None, z=None):
    """Mamba-2 scalar-decay forward on the GPU.

    x, z: (batch, L, H, P); dt: (batch, L, H); B, C: (batch, L, G, N), all
    in one activation dtype; A, D, dt_bias: (H,) float32; h0: (batch, H, P,
    N) float32 initial state (None: zero; may also be ``h_out``); z gates
    the output with silu(z) (None: no gate).  Returns ``(y, h_last)``: y
    like x, h_last (batch, H, P, N) float32.
    """
    L = _lib.lib()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    io = x.dtype
    for name, t in (("x", x), ("dt", dt), ("B", B), ("C", C), ("z", z)):
        _need(t, name, io, dev)
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias), ("h0", h0)):
        _need(t, name, torch.float32, dev)
    batch, seqlen, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if h0 is not None and tuple(h0.shape) != (batch, H, P, N):
        raise ValueError("h0 must be (batch, H, P, N)")
    if z is not None and z.shape != x.shape:
        raise ValueError("z must be shaped like x")
    if tuple(dt.shape) != (batch, seqlen, H):
        raise ValueError("dt must be (batch, L, H)")
    if tuple(B.shape) != (batch, seqlen, G, N) or tuple(C.shape) != tuple(B.shape):
        raise ValueError("B and C must be (batch, L, G, N)")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        if t is not None and tuple(t.shape) != (H,):
            raise ValueError("%s must be (H,)" % name)
    _need_shape(out, "out", x.shape)
    _need_shape(h_out, "h_out", (batch, H, P, N))
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", io, dev)
    h_last = None
    if return_last_state:
        h_last = h_out if h_out is not None else torch.empty(
            (batch, H, P, N), dtype=torch.float32, device=dev)
        _need(h_last, "h_out", torch.float32, dev)
    dims = _lib.SSDDims(batch, seqlen, H, P, N, G, int(chunk))
    dtp = _lib.DTypes(_io_dtype(x), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        if z is not None:
            st = L.mssm_ssd_scalar_fwd_gated(
                _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last), dims, dtp,
                _stream_handle(dev))
        elif h0 is None:
            st = L.mssm_ssd_scalar_fwd(
                _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                _ptr(D), _ptr(y), _ptr(h_last), dims, dtp, _stream_handle(dev))
        else:
            st = L.mssm_ssd_scalar_fwd_h0(
                _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                _ptr(D), _ptr(h0), _ptr(y), _ptr(h_last), dims, dtp,
                _stream_handle(dev))
    _check(st)
    return y, h_last


def selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None,
                           out=None):
    """One decode step on the GPU, advancing ``state`` in place.

    state: (batch, dim, N) float32; x, dt, z: (batch, dim) float32 or
    bfloat16 (one dtype); B, C: (batch, N) same dtype; A: (dim, N) float32;
    D, dt_bias: (dim,) float32.  Returns y (batch, dim) like x.
    """
    L = _lib.lib()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    io = x.dtype
    for name, t in (("x", x), ("dt", dt), ("B", B), ("C", C), ("z", z)):
        _need(t, name, io, dev)
    for name, t in (("state", state), ("A", A), ("D", D), ("dt_bias", dt_bias)):
        _need(t, name, torch.float32, dev)
    if x.dim() != 2:
        raise ValueError("x must be (batch, dim)")
    batch, dim = x.shape
    N = A.shape[1]
    if tuple(state.shape) != (batch, dim, N):
        raise ValueError("state must be (batch, dim, N)")
    if tuple(dt.shape) != (batch, dim) or (z is not None and tuple(z.shape) != (batch, dim)):
        raise ValueError("dt and z must be (batch, dim)")
    if tuple(A.shape) != (dim, N):
        raise ValueError("A must be (dim, N)")
    if tuple(B.shape) != (batch, N) or tuple(C.shape) != (batch, N):
        raise ValueError("B and C must be (batch, N)")
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None and tuple(t.shape) != (dim,):
            raise ValueError("%s must be (dim,)" % name)
    _need_shape(out, "out", x.shape)
    y = out if out is not None else torch.empty_like(x)
    _need(y, "out", io, dev)
    dims = _lib.StepDims(batch, dim, N)
    dtp = _lib.DTypes(_io_dtype(x), _lib.MSSM_F32)
    with torch.cuda.device(dev):
        st = L.mssm_selective_state_update(
            _ptr(state), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
            _ptr(D), _ptr(z), _ptr(y), dims, dtp, _stream_handle(dev))
    _check(st)
    return y


def _on_gpu(t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor, got %s" % type(t).__name__)
    if t.device.type != "cuda":
        raise ValueError("tensors must live on a GPU device")
    return t.device


def _workspace(nbytes, dev):
    """Scratch of a call from torch's allocator, whose blocks are 512-byte
    aligned and stay with the stream (and the graph capture) they are
    allocated on.  Returns (tensor or None, address or None, bytes)."""
    if nbytes <= 0:     # none needed, or sizes that the call refuses, with the reason
        return None, None, 0
    t = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    return t, t.data_ptr(), nbytes


def _output(out, x):
    """The caller's output like x, or a new one."""
    if out is None:
        return torch.empty_like(x)
    _need_shape(out, "out", x.shape)
    _need(out, "out", x.dtype, x.device)
    return out


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None):
    """Layer norm over the last dimension on the GPU.

    x: (..., dim) float32 or bfloat16; weight, bias: (dim,) float32 (None: 1
    and 0).  Returns ``(y, mean, rstd)``: y like x, mean and rstd (...)
    float32, which the backward takes (NaN where dim is 0).
    """
    L = _lib.lib()
    dev = _on_gpu(x)
    _need(x, "x")
    io = _io_dtype(x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    for name, t in (("weight", weight), ("bias", bias)):
        _need(t, name, torch.float32, dev)
        if t is not None and t.shape != (dim,):
            raise ValueError("%s must be (dim,)" % name)
    y = _output(out, x)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    if dim == 0:    # of no values, and the library has nothing to do
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    with _on_device(dev):
        st = L.mssm_layer_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), float(eps), _ptr(y),
                                   _ptr(mean), _ptr(rstd), _lib.NormDims(rows, dim),
                                   _lib.DTypes(io, _lib.MSSM_F32), _stream_handle(dev))
    _check(st)
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None):
    """Gradients of the layer norm for the output gradient ``dy`` (like x);
    mean and rstd are the forward's.  Returns a dict: dx like x, dweight and
    dbias (dim,) float32."""
    L = _lib.lib()
    dev = _on_gpu(x)
    io = _io_dtype(x)
    _need(x, "x")
    _need(dy, "dy", x.dtype, dev)
    if dy is None or dy.shape != x.shape or x.dim() < 1:
        raise ValueError("x and dy must share one (..., dim) shape")
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            raise ValueError("%s is required" % name)
        _need(t, name, torch.float32, dev)
        _need_shape(t, name, x.shape[:-1])
    _need(weight, "weight", torch.float32, dev)
    _need_shape(weight, "weight", (dim,))
    g = {"dx": torch.empty_like(x),
         "dweight": x.new_empty((dim,), dtype=torch.float32),
         "dbias": x.new_empty((dim,), dtype=torch.float32)}
    dims, dt = _lib.NormDims(rows, dim), _lib.DTypes(io, _lib.MSSM_F32)
    with _on_device(dev):
        ws, at, nbytes = _workspace(L.mssm_layer_norm_bwd_workspace(dims, dt), dev)
        st = L.mssm_layer_norm_bwd(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight),
                                   _ptr(g["dx"]), _ptr(g["dweight"]), _ptr(g["dbias"]), at, nbytes,
                                   dims, dt, _stream_handle(dev))
    _check(st)
    return g


def _recurrence_args(x, r, i, lam, ndim):
    """Shared checks of the gated recurrence; returns (device, dim)."""
    dev = _on_gpu(x)
    _io_dtype(x)
    _need(x, "x")
    if x.dim() != ndim:
        raise ValueError("x must be (batch, L, dim)" if ndim == 3 else "x must be (batch, dim)")
    for name, t in (("r", r), ("i", i)):
        if t is None:
            raise ValueError("%s is required" % name)
        _need(t, name, x.dtype, dev)
        _need_shape(t, name, x.shape)
    if lam is None:
        raise ValueError("lam is required")
    _need(lam, "lam", torch.float32, dev)
    _need_shape(lam, "lam", (x.shape[-1],))
    return dev, x.shape[-1]


def gated_recurrence_fwd(x, r, i, lam, scale=8.0, h0=None, return_last_state=True, out=None,
                         h_out=None):
    """Gated linear recurrence on the GPU:
    log a_t = -scale softplus(lam) sigmoid(r_t),
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y_t = h_t.

    x, r, i: (batch, L, dim) float32 or bfloat16 (one dtype); lam: (dim,)
    float32; h0: (batch, dim) float32 initial state (None: zero; it may be
    passed as ``h_out`` too, to advance a state in place).  Returns
    ``(y, h_last)``: y like x, h_last (batch, dim) float32 (None if
    ``return_last_state`` is False).
    """
    L = _lib.lib()
    dev, dim = _recurrence_args(x, r, i, lam, 3)
    batch, seqlen = x.shape[:2]
    for name, t in (("h0", h0), ("h_out", h_out)):
        _need(t, name, torch.float32, dev)
        _need_shape(t, name, (batch, dim))
    y = _output(out, x)
    h_last = None
    if return_last_state:
        h_last = h_out if h_out is not None else torch.empty(
            (batch, dim), dtype=torch.float32, device=dev)
    dims, dt = _lib.RecurrenceDims(batch, seqlen, dim), _lib.DTypes(_io_dtype(x), _lib.MSSM_F32)
    with _on_device(dev):
        ws, at, nbytes = _workspace(L.mssm_gated_recurrence_workspace(dims, dt, 0), dev)
        st = L.mssm_gated_recurrence_fwd(
            _ptr(x), _ptr(r), _ptr(i), _ptr(lam), float(scale), _ptr(h0), _ptr(y), _ptr(h_last),
            at, nbytes, dims, dt, _stream_handle(dev))
    _check(st)
    return y, h_last


def gated_recurrence_bwd(x, r, i, lam, y, dy, scale=8.0, h0=None, dh_last=None):
    """Gradients of the gated linear recurrence for output gradients ``dy``
    (like x) and ``dh_last`` ((batch, dim) float32, None: zero); y is the
    forward's output.  Returns a dict: dx, dr, di like x; dlam (dim,) and dh0
    (batch, dim) float32."""
    L = _lib.lib()
    dev, dim = _recurrence_args(x, r, i, lam, 3)
    batch, seqlen = x.shape[:2]
    for name, t in (("y", y), ("dy", dy)):
        if t is None:
            raise ValueError("%s is required" % name)
        _need(t, name, x.dtype, dev)
        _need_shape(t, name, x.shape)
    for name, t in (("h0", h0), ("dh_last", dh_last)):
        _need(t, name, torch.float32, dev)
        _need_shape(t, name, (batch, dim))
    g = {"dx": torch.empty_like(x), "dr": torch.empty_like(x), "di": torch.empty_like(x),
         "dlam": torch.empty((dim,), dtype=torch.float32, device=dev),
         "dh0": torch.empty((batch, dim), dtype=torch.float32, device=dev)}
    dims, dt = _lib.RecurrenceDims(batch, seqlen, dim), _lib.DTypes(_io_dtype(x), _lib.MSSM_F32)
    with _on_device(dev):
        ws, at, nbytes = _workspace(L.mssm_gated_recurrence_workspace(dims, dt, 1), dev)
        st = L.mssm_gated_recurrence_bwd(
            _ptr(x), _ptr(r), _ptr(i), _ptr(lam), float(scale), _ptr(h0), _ptr(y), _ptr(dy),
            _ptr(dh_last), _ptr(g["dx"]), _ptr(g["dr"]), _ptr(g["di"]), _ptr(g["dlam"]),
            _ptr(g["dh0"]), at, nbytes, dims, dt, _stream_handle(dev))
    _check(st)
    return g


def gated_recurrence_update(state, x, r, i, lam, scale=8.0, out=None):
    """One decode step of the gated linear recurrence, advancing ``state``
    ((batch, dim) float32) in place; x, r, i: (batch, dim).  Returns y like
    x."""
    L = _lib.lib()
    dev, dim = _recurrence_args(x, r, i, lam, 2)
    if state is None:
        raise ValueError("state is required")
    _need(state, "state", torch.float32, dev)
    _need_shape(state, "state", x.shape)
    y = _output(out, x)
    with _on_device(dev):
        st = L.mssm_gated_recurrence_update(
            _ptr(state), _ptr(x), _ptr(r), _ptr(i), _ptr(lam), float(scale), _ptr(y),
            _lib.RecurrenceDims(x.shape[0], 1, dim), _lib.DTypes(_io_dtype(x), _lib.MSSM_F32),
            _stream_handle(dev))
    _check(st)
    return y


def _loss_args(hidden, weight, targets):
    """Shared checks of the projected cross entropy; returns (device, dims,
    dtypes, whether both matrices start on 16-byte boundaries)."""
    dev = _on_gpu(hidden)
    io = _io_dtype(hidden)
    _need(hidden, "hidden")
    for name, t in (("weight", weight), ("targets", targets)):
        if t is None:
            raise ValueError("%s is required" % name)
    _need(weight, "weight", hidden.dtype, dev)
    _need(targets, "targets", torch.int64, dev)
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden must be (tokens, dim) and weight (vocab, dim)")
    _need_shape(targets, "targets", (hidden.shape[0],))
    return (dev, _lib.LossDims(hidden.shape[0], hidden.shape[1], weight.shape[0]),
            _lib.DTypes(io, _lib.MSSM_F32),
            int((hidden.data_ptr() | weight.data_ptr()) % 16 == 0))


def linear_cross_entropy_fwd(hidden, weight, targets, ignore_index=-100):
    """Softmax cross entropy of the logits ``hidden @ weight.T`` on the GPU,
    without storing them.

    hidden: (tokens, dim), weight: (vocab, dim), float32 or bfloat16 (one
    dtype); targets: (tokens,) int64.  Returns ``(loss, lse)``, both (tokens,)
    float32: the loss is 0 where the target is ``ignore_index`` and NaN where
    it is out of range; lse is the logits' log sum exp, which the backward
    takes.
    """
    L = _lib.lib()
    dev, dims, dt, on16 = _loss_args(hidden, weight, targets)
    loss = hidden.new_empty((hidden.shape[0],), dtype=torch.float32)
    lse = torch.empty_like(loss)
    with _on_device(dev):
        ws, at, nbytes = _workspace(L.mssm_linear_cross_entropy_workspace(dims, dt, 0, on16), dev)
        st = L.mssm_linear_cross_entropy_fwd(_ptr(hidden), _ptr(weight), _ptr(targets),
                                             int(ignore_index), _ptr(loss), _ptr(lse), at, nbytes,
                                             dims, dt, _stream_handle(dev))
    _check(st)
    return loss, lse


def linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss, ignore_index=-100):
    """Gradients of the projected cross entropy for the gradients ``dloss``
    ((tokens,) float32) of the tokens' losses; lse is the forward's.  Returns
    a dict: dhidden like hidden, dweight like weight."""
    L = _lib.lib()
    dev, dims, dt, on16 = _loss_args(hidden, weight, targets)
    for name, t in (("lse", lse), ("dloss", dloss)):
        if t is None:
            raise ValueError("%s is required" % name)
        _need(t, name, torch.float32, dev)
        _need_shape(t, name, (hidden.shape[0],))
    g = {"dhidden": torch.empty_like(hidden), "dweight": torch.empty_like(weight)}
    with _on_device(dev):
        ws, at, nbytes = _workspace(L.mssm_linear_cross_entropy_workspace(dims, dt, 1, on16), dev)
        st = L.mssm_linear_cross_entropy_bwd(_ptr(hidden), _ptr(weight), _ptr(targets),
                                             int(ignore_index), _ptr(lse), _ptr(dloss),
                                             _ptr(g["dhidden"]), _ptr(g["dweight"]), at, nbytes,
                                             dims, dt, _stream_handle(dev))
    _check(st)
    return g


def probe_copy(src, dst):
    """Launch the streaming copy probe (mssm_probe_copy) from ``src`` to
    ``dst`` (contiguous device tensors of the same byte size) on the current
    stream."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst must hold the same number of bytes")
    _need(src, "src")
    _need(dst, "dst")
    with torch.cuda.device(src.device):
        _check(_lib.lib().mssm_probe_copy(_ptr(src), _ptr(dst), nbytes,
                                          _stream_handle(src.device)))


def probe_valu(op: int, iters: int, out):
    """Launch the ALU issue-rate probe (mssm_probe_valu) for operation ``op``
    (``_lib.PROBE_*``); ``out`` is a float32 device tensor of at least
    ``_lib.PROBE_VALU_THREADS`` elements.  Returns the lane-operations the
    launch performs."""
    _need(out, "out", torch.float32)
    if out.numel() < _lib.PROBE_VALU_THREADS:
        raise ValueError("out needs %d elements" % _lib.PROBE_VALU_THREADS)
    with torch.cuda.device(out.device):
        _check(_lib.lib().mssm_probe_valu(int(op), int(iters), _ptr(out),
                                          _stream_handle(out.device)))
    return _lib.PROBE_VALU_THREADS * int(iters) * _lib.PROBE_VALU_OPS_PER_ITER
