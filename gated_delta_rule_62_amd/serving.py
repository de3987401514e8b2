"""Bindings of the serving operators: the single-token recurrences on pooled states.

Like the package's other bindings they check dtypes, shapes, devices and strides, pass raw
pointers, sizes and torch's current stream to the C ABI declared in ``include/kda.h``, and
turn status codes into exceptions; every computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes

_VP, _I64, _F32, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int

_STEP = [_VP] * 5 + [_F32] + [_VP] * 3 + [_F32, _VP, _I32, _I64, _VP, _VP] + [_I64] * 3
_LA_STEP = ([_VP, _I64] * 3 + [_VP, _VP, _F32, _VP, _VP, _I32, _I64, _VP, _VP] + [_I64] * 4)


def declare(lib) -> None:
    """Sets the argument types of the serving operators' C functions."""
    for name, args in (("kda_step", _STEP), ("kda_la_step", _LA_STEP)):
        getattr(lib, name).argtypes = args + [_VP]
        getattr(lib, name).restype = _I32
        getattr(lib, name + "_check").argtypes = args
        getattr(lib, name + "_check").restype = _I32


def _lib():
    from . import load_library
    return load_library()


def _raise(status: int) -> None:
    from . import KdaError
    raise KdaError(status)


def _tensor(name, t, dtype, shape, dev):
    """A contiguous tensor of this dtype, shape and device; its address."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError("%s must be %s %s, got %s %s" % (name, dtype, list(shape), t.dtype,
                                                          list(t.shape)))
    if t.device != dev:
        raise ValueError("every tensor must live on the same GPU")
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _optional(name, t, dtype, shape, dev):
    return None if t is None else _tensor(name, t, dtype, shape, dev)


def _rows(name, t, shape, dev):
    """A bf16 tensor [..., heads, D] whose tokens lie one fixed row stride apart: its
    address and that stride in elements."""
    import torch
    if t.dtype != torch.bfloat16 or tuple(t.shape) != shape:
        raise ValueError("%s must be bfloat16 %s, got %s %s" % (name, list(shape), t.dtype,
                                                                list(t.shape)))
    if t.device != dev:
        raise ValueError("every tensor must live on the same GPU")
    heads, D = shape[-2:]
    if t.is_contiguous():
        return t.data_ptr(), heads * D
    st = t.stride()
    if (st[-1] == 1 or D == 1) and (st[-2] == D or heads == 1):
        if len(shape) == 3:
            return t.data_ptr(), st[0] if shape[0] > 1 else heads * D
        B, T = shape[:2]
        row = st[1] if T > 1 else st[0] if B > 1 else heads * D
        if B == 1 or T == 1 or st[0] == T * row:
            return t.data_ptr(), row
    raise ValueError("%s must have contiguous heads, its tokens one row stride apart" % name)


def _device(q):
    if q.device.type != "cuda":
        raise ValueError("every tensor must live on the same GPU")
    return q.device


def _stream_ptr(stream, dev):
    import torch
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _launch(fn, dev, args) -> None:
    """Calls a C operator with dev current (the library launches on the current device)."""
    import torch
    if torch.cuda.current_device() == dev.index:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != 0:
        _raise(st)


def _pool(state, slot_in, slot_out, N, H, D, dev):
    import torch
    from . import _state_dtype_code
    if state.dim() != 4:
        raise ValueError("state must be [slots,H,D,D]")
    slots = state.shape[0]
    return (_tensor("state", state, state.dtype, (slots, H, D, D), dev), _state_dtype_code(state),
            slots, _optional("slot_in", slot_in, torch.int64, (N,), dev),
            _optional("slot_out", slot_out, torch.int64, (N,), dev))


def kda_step(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, state, slot_in=None,
             slot_out=None, stream=None) -> None:
    """One token of each request through the recurrence of ``kda_fwd`` (asynchronous on
    ``stream``).

    q, k, v, g, out: bf16 ``[N,H,D]``; beta bf16 ``[N,H]``; A_log fp32 ``[H]``; dt_bias fp32
    ``[H,D]``; state: the pool, bf16 or fp32 ``[slots,H,D,D]`` in the layout of ``kda_fwd``'s
    states, updated in place.  Request n reads slot ``slot_in[n]`` (int64 ``[N]``; None: n)
    and writes slot ``slot_out[n]`` (None: slot_in); an index outside the pool reads zeros
    or writes nothing.  A slot that one request writes must not be named by another.
    """
    import torch
    if q.dim() != 3:
        raise ValueError("q must be [N,H,D]")
    N, H, D = shape = tuple(q.shape)
    dev = _device(q)
    args = (_tensor("q", q, torch.bfloat16, shape, dev), _tensor("k", k, torch.bfloat16, shape, dev),
            _tensor("v", v, torch.bfloat16, shape, dev), _tensor("g", g, torch.bfloat16, shape, dev),
            _tensor("beta", beta, torch.bfloat16, (N, H), dev), float(scale),
            _tensor("out", out, torch.bfloat16, shape, dev), _tensor("A_log", A_log, torch.float32, (H,), dev),
            _tensor("dt_bias", dt_bias, torch.float32, (H, D), dev), float(lower_bound),
            *_pool(state, slot_in, slot_out, N, H, D, dev), N, H, D, _stream_ptr(stream, dev))
    _launch(_lib().kda_step, dev, args)


def kda_la_step(q, k, v, g, scale, out, state, decay=None, slot_in=None, slot_out=None,
                stream=None) -> None:
    """One token of each request through linear attention with one decay per head:
    ``S = exp(g + decay) S + v k^T``, ``out = scale S q``.

    q, k: bf16 ``[N,Hk,D]``, v, out: bf16 ``[N,H,D]`` with H a multiple of Hk (q, k, v may be
    views with a row stride); g: fp32 ``[N,H]`` log decays or None; decay: fp32 ``[H]`` log
    decays or None; state and slots as for ``kda_step``.
    """
    import torch
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must be [N,heads,D]")
    N, H, D = v.shape
    Hk = q.shape[1]
    dev = _device(q)
    args = (*_rows("q", q, (N, Hk, D), dev), *_rows("k", k, (N, Hk, D), dev),
            *_rows("v", v, (N, H, D), dev), _optional("g", g, torch.float32, (N, H), dev),
            _optional("decay", decay, torch.float32, (H,), dev), float(scale),
            _tensor("out", out, torch.bfloat16, (N, H, D), dev),
            *_pool(state, slot_in, slot_out, N, H, D, dev), N, H, Hk, D,
            _stream_ptr(stream, dev))
    _launch(_lib().kda_la_step, dev, args)
