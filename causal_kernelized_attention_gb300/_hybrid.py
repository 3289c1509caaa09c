"""Hybrid-layer operators: rotary positions, the gated recurrence, window attention with sinks.

Marshalling only, as in ``_binding``: each function checks shapes and types, allocates the
outputs that were not given and calls the C entry point of the same name on the tensors'
device (on ``stream``, or that device's current stream).
"""
from __future__ import annotations

import ctypes
import math

from ._binding import LA_BF16, LA_F32, RotarySpec, _check, load_library

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "ramp": 3}


_entry = {}  # C entry points by name
torch = None  # imported by the first call (the package itself imports without it)


def _start():
    global torch
    import torch as module
    torch = module


def _place(*ts):
    """Checks that the tensors given are contiguous and on one CUDA device; returns its index."""
    dev = -1
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError("tensors must be on a CUDA device")
        if dev >= 0 and i != dev:
            raise ValueError("tensors must be on one device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        dev = i
    return dev


def _call(name, dev, stream, *args):
    """The C entry point with device `dev` current, on `stream` or the device's current stream."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(load_library(), name)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError("stream must be on the tensors' device")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st:
        _check(name, st)


def _like(t, stream):
    """A new tensor like t, of `stream`'s memory when one is given (it is written there)."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _new(shape, dtype, device, stream, make="empty"):
    if stream is None:
        return getattr(torch, make)(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return getattr(torch, make)(shape, dtype=dtype, device=device)


def _dtype_code(first, *others):
    """The element type that all the tensors share, as the library counts it."""
    d = first.dtype
    for t in others:
        if t is not None and t.dtype is not d:
            raise TypeError("tensors must share one dtype")
    if d is torch.bfloat16:
        return LA_BF16
    if d is torch.float32:
        return LA_F32
    raise TypeError("tensors must be float32 or bfloat16, got %s" % d)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _shaped(what, t, shape, dtype=None):
    if t is not None and (t.shape != shape or (dtype is not None and t.dtype is not dtype)):
        raise ValueError("%s must be %s%s" % (what, "" if dtype is None else "%s " % dtype, list(shape)))


def _fit(sizes):
    """Checks the bits of all sizes, which the library takes as 32-bit numbers."""
    if sizes >> 31:
        raise ValueError("sizes must fit 32 bits")


def _out(what, t, shape, dtype, dev):
    """Checks an output that the caller supplied."""
    if _place(t) != dev:
        raise ValueError("tensors must be on one device")
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    _shaped(what, t, shape)
    return t


def _whole(what, v):
    try:
        i = int(v)
    except (TypeError, ValueError, OverflowError):
        i = None
    if i is None or i != v:
        raise TypeError("%s must be a whole number, got %r" % (what, v))
    return i


def _int(what, v):
    if type(v) is not int:
        v = _whole(what, v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError("%s must fit 32 bits" % what)
    return v


# ---------------------------------------------------------------- rotary positions
def _rotary(name, q, k, oq, ok, positions, offset, rot, layout, base, scaling, factor, original, ramp, amplitude, stream):
    if torch is None:
        _start()
    if q.dim() not in (3, 4) or (k is not None and k.dim() != q.dim()):
        raise ValueError("q and k must be [B, H, N, d], or [B, H, d] for one token")
    if k is None and ok is not None:
        raise ValueError("an output for k without k")
    B, Hq, N, d = q.shape if q.dim() == 4 else (q.shape[0], q.shape[1], 1, q.shape[2])
    Hk = 0 if k is None else k.shape[1]
    _fit(B | Hq | Hk | N | d)
    if type(offset) is not int:
        offset = _whole("offset", offset)
    if not -2 ** 63 <= offset < 2 ** 63:
        raise ValueError("offset must fit 64 bits")
    original, rot = _int("original", original), d if rot is None else _int("rot", rot)
    dev = _place(q, k, positions)
    code = _dtype_code(q, k)
    if k is not None:
        _shaped("k", k, (B, Hk, N, d) if q.dim() == 4 else (B, Hk, d))
        ok = _like(k, stream) if ok is None else _out("the output for k", ok, k.shape, k.dtype, dev)
    oq = _like(q, stream) if oq is None else _out("the output for q", oq, q.shape, q.dtype, dev)
    if positions is not None and (positions.dtype is not torch.int32 or positions.shape != (B, N)
                                  and not (q.dim() == 3 and positions.shape == (B,))):
        raise ValueError("positions must be int32 [B, N]")
    if layout not in _LAYOUTS or scaling not in _SCALINGS:
        raise ValueError("layout is one of %s, scaling one of %s" % (sorted(_LAYOUTS), sorted(_SCALINGS)))
    spec = RotarySpec(rot, _LAYOUTS[layout], _SCALINGS[scaling], original, base, factor, ramp[0], ramp[1], amplitude)
    _call(name, dev, stream, q.data_ptr(), _ptr(k), oq.data_ptr(), _ptr(ok), _ptr(positions), offset,
          ctypes.byref(spec), B, Hq, Hk, N, d, code)
    return oq if k is None else (oq, ok)


def la_rotary_forward(q, k=None, oq=None, ok=None, positions=None, offset: int = 0, rot: int = None, layout="half",
                      base: float = 10000.0, scaling="none", factor: float = 1.0, original: int = 0,
                      ramp=(1.0, 32.0), amplitude: float = 1.0, stream=None):
    """Turns q [B,Hq,N,d] and k [B,Hk,N,d] (or [B,H,d], one token) by their positions: int32 [B,N],
    or offset + n.  The first `rot` features (all by default) turn in pairs, layout "half" or
    "interleaved", at base^(-2i/rot), scaled "none", "linear", "ntk" or "ramp" by `factor`
    (ramp: by parts between `ramp` turns over `original` tokens).  oq = q and ok = k turn in
    place.  Returns (oq, ok), or oq when k is None."""
    return _rotary("la_rotary_forward", q, k, oq, ok, positions, offset, rot, layout, base, scaling, factor, original,
                   ramp, amplitude, stream)


def la_rotary_backward(doq, dok=None, dq=None, dk=None, positions=None, offset: int = 0, rot: int = None, layout="half",
                       base: float = 10000.0, scaling="none", factor: float = 1.0, original: int = 0,
                       ramp=(1.0, 32.0), amplitude: float = 1.0, stream=None):
    """Gradients (dq, dk) of la_rotary_forward from its outputs' (same options)."""
    return _rotary("la_rotary_backward", doq, dok, dq, dk, positions, offset, rot, layout, base, scaling, factor,
                   original, ramp, amplitude, stream)


# ---------------------------------------------------------------- gated recurrence
def la_recurrence_forward(x, alpha, h0=None, h=None, hN=None, stream=None):
    """h_t = alpha_t h_{t-1} + x_t per channel; x [B,N,D], alpha fp32 [B,N,D], h0 fp32 [B,D] (None: zeros).
    Returns (h in the dtype of x, the last state hN fp32 [B,D])."""
    if torch is None:
        _start()
    if x.dim() != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = x.shape
    _fit(B | N | D)
    dev = _place(x, alpha, h0)
    code = _dtype_code(x)
    _shaped("alpha", alpha, x.shape, torch.float32)
    _shaped("h0", h0, (B, D), torch.float32)
    h = _like(x, stream) if h is None else _out("h", h, x.shape, x.dtype, dev)
    hN = _new((B, D), torch.float32, x.device, stream) if hN is None else _out("hN", hN, (B, D), torch.float32, dev)
    _call("la_recurrence_forward", dev, stream, x.data_ptr(), alpha.data_ptr(), _ptr(h0), h.data_ptr(), hN.data_ptr(),
          B, N, D, code)
    return h, hN


def la_recurrence_backward(alpha, h, dh, h0=None, dhN=None, dx=None, dalpha=None, dh0=None, stream=None):
    """Gradients of la_recurrence_forward from its output h, dh and dhN (None: zeros).  Returns
    (dx, dalpha fp32, dh0 fp32 -- None when neither h0 nor dh0 was given)."""
    if torch is None:
        _start()
    if h.dim() != 3:
        raise ValueError("h must be [B, N, D]")
    B, N, D = h.shape
    _fit(B | N | D)
    dev = _place(alpha, h, dh, h0, dhN)
    code = _dtype_code(h, dh)
    _shaped("alpha", alpha, h.shape, torch.float32)
    _shaped("dh", dh, h.shape)
    _shaped("h0", h0, (B, D), torch.float32)
    _shaped("dhN", dhN, (B, D), torch.float32)
    dx = _like(h, stream) if dx is None else _out("dx", dx, h.shape, h.dtype, dev)
    dalpha = _like(alpha, stream) if dalpha is None else _out("dalpha", dalpha, h.shape, torch.float32, dev)
    if dh0 is not None:
        _out("dh0", dh0, (B, D), torch.float32, dev)
    elif h0 is not None:
        dh0 = _like(h0, stream)
    _call("la_recurrence_backward", dev, stream, alpha.data_ptr(), h.data_ptr(), dh.data_ptr(), _ptr(h0), _ptr(dhN),
          dx.data_ptr(), dalpha.data_ptr(), _ptr(dh0), B, N, D, code)
    return dx, dalpha, dh0


def la_recurrence_step(state, x, alpha, h=None, stream=None):
    """One token of la_recurrence_forward: state fp32 [B,D] in place, x, alpha [B,D]; returns h [B,D]."""
    if torch is None:
        _start()
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    shape = x.shape
    _fit(shape[0] | shape[1])
    dev = _place(state, x, alpha)
    code = _dtype_code(x)
    _shaped("alpha", alpha, shape, torch.float32)
    _shaped("state", state, shape, torch.float32)
    h = _like(x, stream) if h is None else _out("h", h, shape, x.dtype, dev)
    _call("la_recurrence_step", dev, stream, state.data_ptr(), x.data_ptr(), alpha.data_ptr(), h.data_ptr(),
          shape[0], shape[1], code)
    return h


# ---------------------------------------------------------------- window attention
def _window_shapes(q, k, v, lens):
    if torch is None:
        _start()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Hq, Nq, d], k and v [B, Hk, Nk, d]")
    B, Hq, Nq, d = q.shape
    Hk, Nk = k.shape[1:3]
    _fit(B | Hq | Hk | Nq | Nk | d)
    _shaped("k", k, (B, Hk, Nk, d))
    _shaped("v", v, k.shape)
    _shaped("lens", lens, (B,), torch.int32)
    return B, Hq, Hk, Nq, Nk, d


def _scale(scale, d):
    return 1.0 / math.sqrt(max(d, 1)) if scale is None else float(scale)


def la_window_forward(q, k, v, window: int, sinks: int = 0, lens=None, scale: float = None, o=None, lse=None,
                      stream=None):
    """Causal softmax attention over the last `window` keys and the first `sinks`; q [B,Hq,Nq,d] (the
    last Nq tokens), k, v [B,Hk,Nk,d], lens int32 [B] valid tokens per entry (None: all), scale
    1/sqrt(d) by default.  Returns (o, lse fp32 [B,Hq,Nq]); padding rows give 0 and -inf."""
    if torch is None:
        _start()
    B, Hq, Hk, Nq, Nk, d = _window_shapes(q, k, v, lens)
    window, sinks = _int("window", window), _int("sinks", sinks)
    dev = _place(q, k, v, lens)
    code = _dtype_code(q, k, v)
    o = _like(q, stream) if o is None else _out("o", o, q.shape, q.dtype, dev)
    lse = (_new((B, Hq, Nq), torch.float32, q.device, stream) if lse is None
           else _out("lse", lse, (B, Hq, Nq), torch.float32, dev))
    _call("la_window_forward", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          _ptr(lens), B, Hq, Hk, Nq, Nk, d, window, sinks, _scale(scale, d), code)
    return o, lse


def la_window_backward(q, k, v, o, lse, dout, window: int, sinks: int = 0, lens=None, scale: float = None, dq=None,
                       dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * o) for la_window_forward, from its o and lse."""
    if torch is None:
        _start()
    B, Hq, Hk, Nq, Nk, d = _window_shapes(q, k, v, lens)
    window, sinks = _int("window", window), _int("sinks", sinks)
    dev = _place(q, k, v, o, lse, dout, lens)
    code = _dtype_code(q, k, v, o, dout)
    _shaped("o", o, q.shape)
    _shaped("dout", dout, q.shape)
    _shaped("lse", lse, (B, Hq, Nq), torch.float32)
    dq = _like(q, stream) if dq is None else _out("dq", dq, q.shape, q.dtype, dev)
    dk = _like(k, stream) if dk is None else _out("dk", dk, k.shape, k.dtype, dev)
    dv = _like(v, stream) if dv is None else _out("dv", dv, v.shape, v.dtype, dev)
    _call("la_window_backward", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(lens), B, Hq, Hk, Nq, Nk, d, window, sinks,
          _scale(scale, d), code)
    return dq, dk, dv


def la_window_cache(k, v, window: int, sinks: int = 0, lens=None, kc=None, vc=None, stream=None):
    """Ring caches (kc, vc) [B,Hk,sinks+window,d] of a prefill k, v [B,Hk,N,d]: token j in slot j while
    j < sinks, else in sinks + (j - sinks) % window.  Slots without a token are left as they
    were (zeros in caches made here)."""
    if torch is None:
        _start()
    if k.dim() != 4:
        raise ValueError("k and v must be [B, Hk, N, d]")
    B, Hk, N, d = k.shape
    _fit(B | Hk | N | d)
    window, sinks = _int("window", window), _int("sinks", sinks)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1, sinks at least 0")
    shape = (B, Hk, sinks + window, d)
    dev = _place(k, v, lens)
    code = _dtype_code(k, v)
    _shaped("v", v, k.shape)
    _shaped("lens", lens, (B,), torch.int32)
    kc = _new(shape, k.dtype, k.device, stream, "zeros") if kc is None else _out("kc", kc, shape, k.dtype, dev)
    vc = _new(shape, k.dtype, k.device, stream, "zeros") if vc is None else _out("vc", vc, shape, k.dtype, dev)
    _call("la_window_cache", dev, stream, k.data_ptr(), v.data_ptr(), kc.data_ptr(), vc.data_ptr(), _ptr(lens), B, Hk,
          N, d, window, sinks, code)
    return kc, vc


def la_window_decode_step(kc, vc, q, k, v, pos, window: int, sinks: int = 0, scale: float = None, o=None, stream=None):
    """One decode step on ring caches kc, vc [B,Hk,sinks+window,d] (updated in place): q [B,Hq,d], k, v
    [B,Hk,d], pos int32 [B] the new token's position per entry (negative: idle).  Returns o [B,Hq,d]."""
    if torch is None:
        _start()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [B, Hq, d], k and v [B, Hk, d]")
    B, Hq, d = q.shape
    Hk = k.shape[1]
    _fit(B | Hq | Hk | d)
    window, sinks = _int("window", window), _int("sinks", sinks)
    dev = _place(kc, vc, q, k, v, pos)
    code = _dtype_code(q, k, v, kc, vc)
    _shaped("k", k, (B, Hk, d))
    _shaped("v", v, (B, Hk, d))
    shape = (B, Hk, sinks + window, d)
    _shaped("kc", kc, shape)
    _shaped("vc", vc, shape)
    _shaped("pos", pos, (B,), torch.int32)
    o = _like(q, stream) if o is None else _out("o", o, q.shape, q.dtype, dev)
    _call("la_window_decode_step", dev, stream, kc.data_ptr(), vc.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          o.data_ptr(), pos.data_ptr(), B, Hq, Hk, d, window, sinks, _scale(scale, d), code)
    return o
