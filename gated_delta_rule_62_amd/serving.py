"""Bindings of the serving operators: the single-token recurrences on pooled states, linear
attention with one decay per head, and causal softmax attention with grouped heads.

Like the package's other bindings they check dtypes, shapes, devices and strides, pass raw
pointers, sizes and torch's current stream to the C ABI declared in ``include/kda.h`` (both
in a compiled module, ``csrc/serving_calls.cpp``), and turn status codes into exceptions;
every computation runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import KdaError, load_library

try:
    from . import _serving_calls as _calls
except ImportError as e:
    raise ImportError("the serving operators' calls (_serving_calls.so) are not built; run "
                      "gated_delta_rule_62_amd.build() (or __graft_entry__.build())") from e


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
    st = _calls.step(load_library().kda_step_at, q, k, v, g, beta, scale, out, A_log, dt_bias,
                     lower_bound, state, slot_in, slot_out, stream)
    if st != 0:
        raise KdaError(st)


def kda_la_step(q, k, v, g, scale, out, state, decay=None, slot_in=None, slot_out=None,
                stream=None) -> None:
    """One token of each request through linear attention with one decay per head:
    ``S = exp(g + decay) S + v k^T``, ``out = scale S q``.

    q, k: bf16 ``[N,Hk,D]``, v, out: bf16 ``[N,H,D]`` with H a multiple of Hk (q, k, v may be
    views with a row stride); g: fp32 ``[N,H]`` log decays or None; decay: fp32 ``[H]`` log
    decays or None; state and slots as for ``kda_step``.
    """
    st = _calls.la_step(load_library().kda_la_step_at, q, k, v, g, scale, out, state, decay,
                        slot_in, slot_out, stream)
    if st != 0:
        raise KdaError(st)


def _workspace(need, q, stream):
    """A workspace from torch's allocator for one call, taken for the stream it runs on, so
    that nothing else uses it meanwhile."""
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=q.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, q.device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=q.device)


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
    lib = load_library()
    args = (lib.kda_la_fwd_at, lib.kda_la_workspace_bytes_at, q, k, v, g, scale, out, decay,
            initial_state, final_state, cu_seqlens, segment)
    st = _calls.la_fwd(*args, workspace, stream)
    if st > 0:  # the bytes it wants
        st = _calls.la_fwd(*args, _workspace(st, q, stream), stream)
    if st != 0:
        raise KdaError(st)


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
    lib = load_library()
    args = (lib.kda_attn_fwd_at, lib.kda_attn_workspace_bytes_at, q, k, v, scale, out, lse,
            cu_seqlens_q, cu_seqlens_k, k_lens, splits)
    st = _calls.attn_fwd(*args, workspace, stream)
    if st > 0:  # the bytes it wants
        st = _calls.attn_fwd(*args, _workspace(st, q, stream), stream)
    if st != 0:
        raise KdaError(st)
