"""The single-token recurrences (kda_step, kda_la_step) against their 64-bit definitions.

Bounds.  The state update is a chain of fp32 operations: with u = 2^-24, the decay factor
carries the error of its exponent (a few roundings of an argument of at most |lb| or |lam|)
plus a few roundings, kh and qh a few each, a row sum of D terms at most log2(64) + D / 16
levels of a tree.  C counts them generously; every term is relative to the sum of absolute
values.  A bf16 output adds half a bf16 step of the value.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.serving_forms as forms
from tests.serving_forms import U16, U32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _c(lam):
    """Roundings of one state element and of one output: 24 in the decay's argument (each
    relative to |lam|), 40 in everything else."""
    return 40 + 24 * lam


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _step_inputs(g, N, H, D):
    return dict(q=_normal(g, N, H, D), k=_normal(g, N, H, D), v=_normal(g, N, H, D),
                g=_normal(g, N, H, D), beta=_normal(g, N, H),
                A_log=torch.rand((H,), generator=g, device=DEV),
                dt_bias=torch.rand((H, D), generator=g, device=DEV))


def _run_step(x, scale, lb, pool, **slots):
    out = torch.full_like(x["q"], float("nan"))
    kda.kda_step(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, out, x["A_log"], x["dt_bias"],
                 lb, pool, **slots)
    return out


def _want_step(x, scale, lb, S):
    d = {n: t.double() for n, t in x.items()}
    return forms.step(d["q"], d["k"], d["v"], d["g"], d["beta"], scale, d["A_log"], d["dt_bias"],
                      lb, S.double())


def _pool(g, slots, H, D, dtype):
    return torch.randn((slots, H, D, D), generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,H,D,lb", [
    (1, 1, 32, -5.0), (3, 5, 32, -0.5), (1, 2, 64, -5.0), (7, 3, 64, -30.0), (1, 1, 128, -5.0),
    (5, 7, 128, -5.0), (33, 8, 128, -5.0), (70, 16, 128, -1e30), (9, 130, 64, -5.0),
    (40, 70, 32, -5.0), (11, 96, 128, -5.0)])
def test_step(N, H, D, lb, dtype):
    print("kda_step", N, H, D, lb, dtype, flush=True)
    g = _gen(N * 1000 + H)
    x = _step_inputs(g, N, H, D)
    slots = 2 * N + 3
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(1)).to(DEV)
    src, dst = order[:N].contiguous(), order[N:2 * N].contiguous()
    pool = _pool(g, slots, H, D, dtype)
    before = pool.clone()
    scale = D ** -0.5
    out = _run_step(x, scale, lb, pool, slot_in=src, slot_out=dst)
    o, S, o_mag, S_mag = _want_step(x, scale, lb, before[src])
    c = _c(min(-lb, 100.0))  # beyond that the factor is zero to fp32
    forms.check(out, o, U16 * o.abs() + c * U32 * o_mag + forms.TINY, "out")
    half = U16 * S.abs() if dtype == torch.bfloat16 else 0 * S
    forms.check(pool[dst], S, half + c * U32 * S_mag + forms.TINY, "state")
    rest = torch.ones(slots, dtype=torch.bool, device=DEV)
    rest[dst] = False
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,H,Hk,D,gate", [
    (1, 1, 1, 32, "both"), (3, 6, 2, 32, "none"), (2, 8, 8, 64, "token"), (9, 12, 3, 64, "head"),
    (1, 3, 1, 128, "token"), (20, 32, 8, 128, "both"), (65, 16, 16, 128, "head"),
    (130, 40, 8, 64, "token")])
def test_la_step(N, H, Hk, D, gate, dtype):
    print("kda_la_step", N, H, Hk, D, gate, dtype, flush=True)
    g = _gen(N * 77 + H)
    q, k, v = torch.split(_normal(g, N, 2 * Hk + H, D), [Hk, Hk, H], dim=1)  # row-strided views
    gt = -4 * torch.rand((N, H), generator=g, device=DEV) if gate in ("token", "both") else None
    dec = -torch.rand((H,), generator=g, device=DEV) if gate in ("head", "both") else None
    if gt is not None:
        gt[0, 0] = -float("inf")  # a reset: the old state is dropped
        gt[-1, -1] = 0.5  # above zero: no decay from the gate and the head together
    pool = _pool(g, N + 2, H, D, dtype)
    before = pool.clone()
    scale = -0.3
    out = torch.full((N, H, D), float("nan"), device=DEV, dtype=torch.bfloat16)
    kda.kda_la_step(q, k, v, gt, scale, out, pool, decay=dec)
    lam = torch.zeros((N, H), device=DEV, dtype=torch.float64)
    lam = lam + (gt.double() if gt is not None else 0) + (dec.double() if dec is not None else 0)
    lam = lam.clamp(max=0.0)
    rep = H // Hk
    o, S, o_mag, S_mag = forms.la_step(q.double().repeat_interleave(rep, 1),
                                       k.double().repeat_interleave(rep, 1), v.double(), lam,
                                       scale, before[:N].double())
    c = _c(5.0)
    forms.check(out, o, U16 * o.abs() + c * U32 * o_mag + forms.TINY, "out")
    half = U16 * S.abs() if dtype == torch.bfloat16 else 0 * S
    forms.check(pool[:N], S, half + c * U32 * S_mag + forms.TINY, "state")
    assert torch.equal(pool[N:], before[N:])


@pytest.mark.parametrize("D", [32, 128])
def test_slots_outside_the_pool(D):
    """An index outside the pool reads zeros or stores nothing; a forked slot is read twice."""
    g = _gen(5)
    N, H, slots = 6, 4, 5
    x = _step_inputs(g, N, H, D)
    pool = _pool(g, slots, H, D, torch.float32)
    before = pool.clone()
    src = torch.tensor([-1, 2, 5, 2, 1 << 40, 4], device=DEV)
    dst = torch.tensor([0, 1, -7, 3, 5, -(1 << 62)], device=DEV)
    out = _run_step(x, 0.25, -2.0, pool, slot_in=src, slot_out=dst)
    S0 = torch.zeros((N, H, D, D), device=DEV)
    for n, s in enumerate(src.tolist()):
        if 0 <= s < slots:
            S0[n] = before[s]
    o, S, o_mag, S_mag = _want_step(x, 0.25, -2.0, S0)
    c = _c(2.0)
    forms.check(out, o, U16 * o.abs() + c * U32 * o_mag + forms.TINY, "out")
    for n, s in enumerate(dst.tolist()):
        if 0 <= s < slots:
            forms.check(pool[s], S[n], c * U32 * S_mag[n] + forms.TINY, "slot %d" % s)
    assert torch.equal(pool[[2, 4]], before[[2, 4]])


def test_nan_and_infinity_stay_in_their_rows():
    """A NaN in one value component reaches that value row only; a NaN gate its whole head."""
    g = _gen(6)
    N, H, D = 2, 3, 64
    q, k, v = (_normal(g, N, H, D) for _ in range(3))
    v[0, 1, 7] = float("nan")
    v[1, 2, 9] = float("inf")
    gt = -torch.rand((N, H), generator=g, device=DEV)
    gt[0, 0] = float("nan")
    pool = _pool(g, N, H, D, torch.float32)
    out = torch.empty((N, H, D), device=DEV, dtype=torch.bfloat16)
    kda.kda_la_step(q, k, v, gt, 1.0, out, pool)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 1, 7] = want[1, 2, 9] = True
    want[0, 0] = True
    assert torch.equal(bad, want)


def test_steps_continue_a_prefill():
    """The states of kda_fwd are slots of the pool: prompt plus single tokens equals one
    longer prompt (within kda_fwd's own error, out rel-L2 5e-3)."""
    g = _gen(7)
    N, H, D, T, more = 3, 4, 128, 70, 5
    x = _step_inputs(g, N * (T + more), H, D)
    x = {n: (t.view(N, T + more, *t.shape[1:]) if n not in ("A_log", "dt_bias") else t)
         for n, t in x.items()}
    scale, lb = D ** -0.5, -5.0

    def prefill(upto, state):
        c = {n: (t[:, :upto].contiguous() if n not in ("A_log", "dt_bias") else t)
             for n, t in x.items()}
        out = torch.empty_like(c["q"])
        kda.kda_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], scale, out, c["A_log"],
                    c["dt_bias"], lb, final_state=state)
        return out

    pool = torch.zeros((N, H, D, D), device=DEV)
    whole = torch.empty_like(pool)
    out_all = prefill(T + more, whole)
    prefill(T, pool)
    for t in range(T, T + more):
        tok = {n: (y[:, t].contiguous() if n not in ("A_log", "dt_bias") else y)
               for n, y in x.items()}
        o = _run_step(tok, scale, lb, pool)
        ref = out_all[:, t].double()
        assert float((o.double() - ref).norm() / ref.norm()) <= 1e-2  # twice kda_fwd's bound
    assert float((pool - whole).norm() / whole.norm()) <= 1e-2


def test_capture_and_streams():
    """Captured and replayed, on another stream, and beside another call: the eager results."""
    g = _gen(8)
    N, H, D = 4, 8, 128
    x, y = _step_inputs(g, N, H, D), _step_inputs(g, N, H, D)
    pool = _pool(g, N, H, D, torch.float32)
    start = pool.clone()
    want = []
    for _ in range(4):
        want.append((_run_step(x, 1.0, -5.0, pool), pool.clone()))
    pool.copy_(start)
    out = torch.empty_like(x["q"])
    call = lambda s=None: kda.kda_step(x["q"], x["k"], x["v"], x["g"], x["beta"], 1.0, out,
                                       x["A_log"], x["dt_bias"], -5.0, pool, stream=s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    pool.copy_(start)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(pool, want[i][1]), i
        out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _pool(g, N, H, D, torch.bfloat16)
    call(side)
    _run_step(y, 1.0, -5.0, other)  # the current stream, at the same time
    torch.cuda.synchronize()
    assert torch.equal(out, want[3][0]) and torch.equal(pool, want[3][1])
