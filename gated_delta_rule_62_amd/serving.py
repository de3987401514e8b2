"""Bindings of the serving operators: the single-token recurrences on pooled states, linear
attention with one decay per head, causal softmax attention with grouped heads, and what layers
call around them: norms with gate and residual, rotary positions, caches in 4 bits.

Like the package's other bindings they check dtypes, shapes, devices and strides, pass raw
pointers, sizes and torch's current stream to the C ABI declared in ``include/kda.h`` (both
in a compiled module, ``csrc/serving_calls.cpp``), and turn status codes into exceptions;
every computation runs in the library's kernels.
"""
from __future__ import annotations

import math

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


def kda_norm(x, out=None, weight=None, eps: float = 1e-6, post_weight=None, gate=None,
             gate_fn: str = "sigmoid", residual=None, residual_out=None,
             residual_scale: float = 1.0, stream=None) -> None:
    """The norms before and after a block, with its gate and the residual sum, in one pass over
    the rows (asynchronous on ``stream``); every part is optional:
    ``u = rms_norm(x, groups) post_weight``, ``u = u act(gate)``,
    ``h = residual + residual_scale u`` (written to residual_out),
    ``out = rms_norm(h) weight``; without ``weight`` out is h.

    x, gate: bf16 ``[..,W]`` (views whose rows lie one stride apart are taken as they are);
    post_weight: ``[G]``, norms over groups of G channels (G: W, or 32, 64, 128, 256 or 512);
    weight: ``[W]``; both bf16 or both fp32; gate_fn: "sigmoid" or "silu"; residual and
    residual_out: bf16 or fp32 ``[..,W]``, possibly the same tensor; out: bf16 ``[..,W]``, which
    may be left out with a residual and without a weight.
    """
    st = _calls.norm(load_library().kda_norm_at, x, out, weight, eps, post_weight, gate, gate_fn,
                     residual, residual_out, residual_scale, stream)
    if st != 0:
        raise KdaError(st)


def kda_rope_freqs(rot: int, base: float = 10000.0, method: str = "", factor: float = 1.0,
                   original: int = 4096, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """Frequencies for ``kda_rope``, fp64 ``[rot/2]``, and its amplitude.

    method "": powers of the base.  "linear": positions interpolated, every frequency divided by
    factor.  "yarn": a pair that turns at most ``slow`` times over the ``original`` context is
    interpolated, one that turns ``fast`` times or more is kept, and the amplitude is
    ``0.1 ln(factor) + 1`` (1 for a factor of at most 1).  Between the two the blend is linear in
    the number of turns; a model whose program blends linearly in the pair's index has other
    frequencies there and passes its own to ``kda_rope``.
    """
    if rot < 2 or rot % 2 or not base > 0 or not factor > 0 or not fast > slow:
        raise ValueError("rot must be even and positive, base and factor positive, fast above slow")
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    amplitude = 1.0
    if method == "linear":
        f = f / factor
    elif method == "yarn":
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif method:
        raise ValueError("method must be '', 'linear' or 'yarn'")
    return f.to(device), amplitude


def kda_rope(q, k, freqs, q_out, k_out, positions=None, offsets=None, cu_seqlens=None,
             interleaved: bool = False, amplitude: float = 1.0, inverse: bool = False,
             stream=None) -> None:
    """Rotary positions of queries and keys (asynchronous on ``stream``): pairs of a head's first
    ``2 len(freqs)`` channels are turned by position times frequency, the rest is copied.

    q, q_out: bf16 ``[B,T,Hq,D]``, k, k_out: bf16 ``[B,T,Hk,D]`` or both None; views with one row
    stride are taken as they are, and an output may be its input.  freqs: fp64 ``[rot/2]`` radians
    per position (``kda_rope_freqs``).  Positions: int64 ``[B,T]``, or ``offsets[n] + t`` for
    token t of sequence n (int64 ``[N]``; None: 0), sequences packed (``cu_seqlens`` int64
    ``[N+1]``, B == 1) or batch rows.  ``interleaved``: pairs ``(2i, 2i+1)`` instead of
    ``(i, i + rot/2)``; ``amplitude`` multiplies the turned channels; ``inverse`` turns back.
    """
    st = _calls.rope(load_library().kda_rope_at, q, k, freqs, q_out, k_out, positions, offsets,
                     cu_seqlens, interleaved, amplitude, inverse, stream)
    if st != 0:
        raise KdaError(st)


def kda_cache4_empty(slots: int, heads: int, capacity: int, D: int, device="cuda"):
    """An empty cache in 4 bits for ``kda_cache4_put`` and ``kda_attn4_fwd``: the tensors k4, ks,
    v4, vs (uint8; ``include/kda.h`` says what is where) for ``slots`` requests of up to
    ``capacity`` positions (a multiple of 32)."""
    if capacity % 32 or D not in (64, 128):
        raise ValueError("capacity must be a multiple of 32 and D 64 or 128")
    tiles = capacity // 32
    shapes = ((slots, heads, capacity, D // 2), (slots, heads, tiles, D // 32, 32),
              (slots, heads, tiles, 16 * D), (slots, heads, tiles, D // 32, 32))
    return tuple(torch.zeros(s, dtype=torch.uint8, device=device) for s in shapes)


def kda_cache4_put(k, v, k4, ks, v4, vs, offsets=None, cu_seqlens=None, slots=None, k_out=None,
                   v_out=None, stream=None) -> None:
    """New keys and values into caches in 4 bits (asynchronous on ``stream``): token t of sequence
    n goes to position ``offsets[n] + t`` of slot ``slots[n]``.

    k, v: bf16 ``[B,T,Hk,D]`` (views with one row stride are taken as they are); k4, ks, v4, vs: as
    ``kda_cache4_empty`` makes them, updated in place; offsets: int64 ``[N]`` (None: 0); slots:
    int64 ``[N]`` (None: n); cu_seqlens as for ``kda_fwd``.  k_out, v_out: bf16 ``[B,T,Hk,D]`` for
    the values that the cache then stands for, or both None.  Positions outside the capacity and
    slots outside the cache are not stored.
    """
    st = _calls.put4(load_library().kda_cache4_put_at, k, v, k4, ks, v4, vs, offsets, cu_seqlens,
                     slots, k_out, v_out, stream)
    if st != 0:
        raise KdaError(st)


def kda_attn4_workspace_bytes(num_seqs: int, Bq: int, Tq: int, capacity: int, Hq: int, Hk: int,
                              D: int, part: int = 0) -> int:
    """Bytes of the workspace of ``kda_attn4_fwd`` (0: this call needs none)."""
    n = load_library().kda_attn4_workspace_bytes(int(num_seqs), int(Bq), int(Tq), int(capacity),
                                                 int(Hq), int(Hk), int(D), int(part))
    if n < 0:
        raise KdaError(int(n))
    return int(n)


def kda_attn4_fwd(q, k4, ks, v4, vs, scale, out, lse=None, k_lens=None, cu_seqlens_q=None,
                  slots=None, part: int = 0, workspace=None, stream=None) -> None:
    """``kda_attn_fwd`` over caches in 4 bits (asynchronous on ``stream``): sequence n's keys are
    the first ``k_lens[n]`` positions (int64 ``[N]``; None: all) of slot ``slots[n]`` (int64
    ``[N]``; None: n), its queries the last of them.

    q, scale, out, lse, cu_seqlens_q: as for ``kda_attn_fwd``; k4, ks, v4, vs: as for
    ``kda_cache4_put``, D 64 or 128.  ``part``: 0 (automatic) or keys per part, a multiple of 32;
    ``workspace``: a uint8 tensor of at least ``kda_attn4_workspace_bytes(...)`` bytes for this
    call alone; None takes one from torch's allocator where the call needs it (prompts: up to
    8 GiB for the caches in bf16, by their capacity); an empty one: no workspace, one part, which
    is also what a call with ``part`` 0 falls back to where the allocator has no memory left
    (slower for prompts, and rounded as such a call).
    """
    lib = load_library()
    args = (lib.kda_attn4_fwd_at, lib.kda_attn4_workspace_bytes_at, q, k4, ks, v4, vs, scale, out,
            lse, k_lens, cu_seqlens_q, slots, part)
    st = _calls.attn4_fwd(*args, workspace, stream)
    if st > 0:  # the bytes it wants
        try:
            workspace = _workspace(st, q, stream)
        except torch.OutOfMemoryError:
            if part:  # parts are written there
                raise
            workspace = torch.empty(0, dtype=torch.uint8, device=q.device)
        st = _calls.attn4_fwd(*args, workspace, stream)
    if st != 0:
        raise KdaError(st)
