"""Bindings of the serving operators: the single-token recurrences on pooled states, linear
attention with one decay per head, and causal softmax attention with grouped heads.

Like the package's other bindings they check dtypes, shapes, devices and strides, pass raw
pointers, sizes and torch's current stream to the C ABI declared in ``include/kda.h``, and
turn status codes into exceptions; every computation runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import KdaError, load_library

try:
    from ._tensor_args import optional as _optional, rows as _rows, tensor as _tensor
except ImportError as e:
    raise ImportError("the bindings' argument checks (_tensor_args.so) are not built; run "
                      "gated_delta_rule_62_amd.build() (or __graft_entry__.build())") from e

# dtype codes of _tensor_args (the first two are the C ABI's state dtypes)
bf16, fp32, int64 = 0, 1, 2


def _device(q) -> int:
    if not q.is_cuda:
        raise ValueError("every tensor must live on the same GPU")
    return q.get_device()


def _stream_ptr(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _launch(fn, dev, args) -> None:
    """Calls a C operator with dev current (the library launches on the current device)."""
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != 0:
        raise KdaError(st)


def _dtype_code(t):
    if t.dtype is torch.bfloat16:
        return bf16
    if t.dtype is torch.float32:
        return fp32
    raise TypeError("state tensors must be bfloat16 or float32, got %s" % t.dtype)


def _pool(state, slot_in, slot_out, N, H, D, dev):
    if state.dim() != 4:
        raise ValueError("state must be [slots,H,D,D]")
    slots = state.shape[0]
    code = _dtype_code(state)
    return (_tensor("state", state, code, (slots, H, D, D), dev), code, slots,
            _optional("slot_in", slot_in, int64, (N,), dev),
            _optional("slot_out", slot_out, int64, (N,), dev))


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
    if q.dim() != 3:
        raise ValueError("q must be [N,H,D]")
    N, H, D = shape = tuple(q.shape)
    dev = _device(q)
    args = (_tensor("q", q, bf16, shape, dev), _tensor("k", k, bf16, shape, dev),
            _tensor("v", v, bf16, shape, dev), _tensor("g", g, bf16, shape, dev),
            _tensor("beta", beta, bf16, (N, H), dev), float(scale),
            _tensor("out", out, bf16, shape, dev), _tensor("A_log", A_log, fp32, (H,), dev),
            _tensor("dt_bias", dt_bias, fp32, (H, D), dev), float(lower_bound),
            *_pool(state, slot_in, slot_out, N, H, D, dev), N, H, D, _stream_ptr(stream, dev))
    _launch(load_library().kda_step, dev, args)


def kda_la_step(q, k, v, g, scale, out, state, decay=None, slot_in=None, slot_out=None,
                stream=None) -> None:
    """One token of each request through linear attention with one decay per head:
    ``S = exp(g + decay) S + v k^T``, ``out = scale S q``.

    q, k: bf16 ``[N,Hk,D]``, v, out: bf16 ``[N,H,D]`` with H a multiple of Hk (q, k, v may be
    views with a row stride); g: fp32 ``[N,H]`` log decays or None; decay: fp32 ``[H]`` log
    decays or None; state and slots as for ``kda_step``.
    """
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must be [N,heads,D]")
    N, H, D = v.shape
    Hk = q.shape[1]
    dev = _device(q)
    args = (*_rows("q", q, bf16, (N, Hk, D), dev), *_rows("k", k, bf16, (N, Hk, D), dev),
            *_rows("v", v, bf16, (N, H, D), dev), _optional("g", g, fp32, (N, H), dev),
            _optional("decay", decay, fp32, (H,), dev), float(scale),
            _tensor("out", out, bf16, (N, H, D), dev),
            *_pool(state, slot_in, slot_out, N, H, D, dev), N, H, Hk, D,
            _stream_ptr(stream, dev))
    _launch(load_library().kda_la_step, dev, args)


def _state(name, t, N, H, D, dev):
    """Address and dtype code of a prompt's initial or final states, or nothing."""
    if t is None:
        return None, 0
    code = _dtype_code(t)
    return _tensor(name, t, code, (N, H, D, D), dev), code


def _workspace(workspace, need, dev, stream):
    """Address, size and owner of the caller's workspace, or of one from torch's allocator
    for this call (taken for the stream it runs on, so that nothing else uses it meanwhile)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device="cuda:%d" % dev)
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream, dev)
            with torch.cuda.stream(s):
                workspace = torch.empty(need, dtype=torch.uint8, device="cuda:%d" % dev)
    elif workspace.dtype != torch.uint8 or workspace.dim() != 1:
        raise ValueError("workspace must be a 1-d uint8 tensor")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and live on the same GPU")
    return workspace.data_ptr(), workspace.numel(), workspace


def kda_la_workspace_bytes(T_total: int, num_seqs: int, H: int, D: int, segment: int = 0) -> int:
    """Bytes of the workspace of ``kda_la_fwd`` (0: this call needs none)."""
    n = load_library().kda_la_workspace_bytes(int(T_total), int(num_seqs), int(H), int(D), int(segment))
    if n < 0:
        raise KdaError(int(n))
    return int(n)


def kda_la_fwd(q, k, v, g, scale, out, decay=None, initial_state=None, final_state=None,
               cu_seqlens=None, segment: int = 0, workspace=None, stream=None) -> None:
    """Prompts through linear attention with one decay per head (asynchronous on ``stream``):
    ``S = exp(g_t + decay) S + v_t k_t^T``, ``out_t = scale S q_t``.

    q, k: bf16 ``[B,T,Hk,D]``, v: bf16 ``[B,T,H,D]`` with H a multiple of Hk (views with one
    row stride are taken as they are); out: bf16 ``[B,T,H,D]``; g: fp32 ``[B,T,H]`` log decays
    or None; decay: fp32 ``[H]`` log decays or None; states ``[N,H,D,D]`` bf16 or fp32 or
    None, and ``cu_seqlens``, as for ``kda_fwd``.  ``segment``: 0 (automatic) or tokens per
    segment (a multiple of 64).  ``workspace``: a uint8 tensor of at least
    ``kda_la_workspace_bytes(B*T, N, H, D, segment)`` bytes for this call alone; None takes
    one from torch's allocator where the call needs it.
    """
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must be [B,T,heads,D]")
    B, T, H, D = v.shape
    Hk = q.shape[2]
    dev = _device(q)
    if torch._C._cuda_getDevice() != dev:  # schedules go by the current device
        with torch.cuda.device(dev):
            return kda_la_fwd(q, k, v, g, scale, out, decay, initial_state, final_state,
                              cu_seqlens, segment, workspace, stream)
    cu, N = None, B
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        cu = _tensor("cu_seqlens", cu_seqlens, int64, (N + 1,), dev)
    lib = load_library()
    need = lib.kda_la_workspace_bytes(B * T, N, H, D, int(segment))
    ws, ws_bytes, _keep = _workspace(workspace, max(need, 0), dev, stream)
    args = (*_rows("q", q, bf16, (B, T, Hk, D), dev), *_rows("k", k, bf16, (B, T, Hk, D), dev),
            *_rows("v", v, bf16, (B, T, H, D), dev), _optional("g", g, fp32, (B, T, H), dev),
            _optional("decay", decay, fp32, (H,), dev), float(scale),
            _tensor("out", out, bf16, (B, T, H, D), dev),
            *_state("initial_state", initial_state, N, H, D, dev),
            *_state("final_state", final_state, N, H, D, dev), cu, N, B, T, H, Hk, D,
            int(segment), ws, ws_bytes, _stream_ptr(stream, dev))
    _launch(lib.kda_la_fwd, dev, args)


def kda_attn_workspace_bytes(num_seqs: int, Bq: int, Tq: int, Bk: int, Tk: int, Hq: int, Hk: int,
                             D: int, splits: int = 0) -> int:
    """Bytes of the workspace of ``kda_attn_fwd`` (0: this call needs none)."""
    n = load_library().kda_attn_workspace_bytes(int(num_seqs), int(Bq), int(Tq), int(Bk), int(Tk), int(Hq),
                                        int(Hk), int(D), int(splits))
    if n < 0:
        raise KdaError(int(n))
    return int(n)


def kda_attn_fwd(q, k, v, scale, out, lse=None, cu_seqlens_q=None, cu_seqlens_k=None, k_lens=None,
                 splits: int = 0, workspace=None, stream=None) -> None:
    """Causal softmax attention with grouped heads (asynchronous on ``stream``).  Query i of a
    sequence of Lq queries and Lk keys sees keys ``j <= i + Lk - Lq``; one that sees none
    gets out 0 and lse minus infinity.

    q: bf16 ``[Bq,Tq,Hq,D]``, k, v: bf16 ``[Bk,Tk,Hk,D]`` with Hq a multiple of Hk (views with
    one row stride are taken as they are); out: bf16 ``[Bq,Tq,Hq,D]``; lse: fp32
    ``[Bq,Tq,Hq]`` or None.  Queries are packed (``cu_seqlens_q`` int64 ``[N+1]``, Bq == 1) or
    batch rows; keys are packed (``cu_seqlens_k``, Bk == 1) or batch rows of a cache of which
    the first ``k_lens[n]`` (int64 ``[N]``; None: all) are in use.  ``splits``: 0 (automatic)
    or parts of each row's keys; ``workspace``: a uint8 tensor of at least
    ``kda_attn_workspace_bytes(...)`` bytes for this call alone; None takes one from torch's
    allocator where the call needs it.
    """
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B,T,heads,D]")
    Bq, Tq, Hq, D = q.shape
    Bk, Tk, Hk, _ = k.shape
    dev = _device(q)
    if torch._C._cuda_getDevice() != dev:  # schedules go by the current device
        with torch.cuda.device(dev):
            return kda_attn_fwd(q, k, v, scale, out, lse, cu_seqlens_q, cu_seqlens_k, k_lens,
                                splits, workspace, stream)
    N = cu_seqlens_q.numel() - 1 if cu_seqlens_q is not None else Bq
    lib = load_library()
    need = lib.kda_attn_workspace_bytes(N, Bq, Tq, Bk, Tk, Hq, Hk, D, int(splits))
    ws, ws_bytes, _keep = _workspace(workspace, max(need, 0), dev, stream)
    args = (*_rows("q", q, bf16, (Bq, Tq, Hq, D), dev), *_rows("k", k, bf16, (Bk, Tk, Hk, D), dev),
            *_rows("v", v, bf16, (Bk, Tk, Hk, D), dev), float(scale),
            _tensor("out", out, bf16, (Bq, Tq, Hq, D), dev),
            _optional("lse", lse, fp32, (Bq, Tq, Hq), dev),
            _optional("cu_seqlens_q", cu_seqlens_q, int64, (N + 1,), dev),
            _optional("cu_seqlens_k", cu_seqlens_k, int64, (N + 1,), dev),
            _optional("k_lens", k_lens, int64, (N,), dev), N, Bq, Tq, Bk, Tk, Hq, Hk, D,
            int(splits), ws, ws_bytes, _stream_ptr(stream, dev))
    _launch(lib.kda_attn_fwd, dev, args)
