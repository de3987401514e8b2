"""Linear attention with one decay per head over prompts (kda_la_fwd) against its 64-bit
definition, token by token.

Bounds.  out: the scores and the state operand are rounded to bf16 once each, every term of
the sum by at most half a bf16 step of itself, so U16 times the sum of absolute values
(scores and state share the terms), plus half a bf16 step of the result.  Everything else
is fp32: per chunk the state is scaled and added to (6 roundings), and a weight carries the
error of its exponent, a sum of at most 16 terms in four levels times log2(e): 8 roundings
of the largest sum of a 16-token tile in base 2.  The last bits of the matrix products'
sums, 64 more.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.serving_forms as forms
from tests.serving_forms import U16, U32

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOG2E = 1.4426950408889634


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _inputs(seed, lens, H, Hk, D, gate="both", state="fp32", packed=True, strong=0.3):
    """Packed sequences, or equal ones as batch rows; q, k, v views of one tensor's rows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    q, k, v = torch.split(_normal(g, B, T, 2 * Hk + H, D), [Hk, Hk, H], dim=2)
    x = dict(q=q, k=k, v=v, g=None, decay=None, cu=None, initial=None, lens=lens)
    if gate in ("token", "both"):
        x["g"] = -strong * torch.rand((B, T, H), generator=g, device=DEV)
    if gate in ("head", "both"):
        x["decay"] = -0.2 * torch.rand((H,), generator=g, device=DEV)
    if packed:
        x["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(DEV)
    if state:
        x["initial"] = torch.randn((len(lens), H, D, D), generator=g, device=DEV).to(
            torch.float32 if state == "fp32" else torch.bfloat16)
    return x


def _run(x, scale, out_state=torch.float32, **more):
    B, T, H, D = x["v"].shape
    out = torch.full((B, T, H, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    final = torch.full((len(x["lens"]), H, D, D), float("nan"), dtype=out_state, device=DEV)
    kda.kda_la_fwd(x["q"], x["k"], x["v"], x["g"], scale, out, decay=x["decay"],
                   initial_state=x["initial"], final_state=final, cu_seqlens=x["cu"], **more)
    return out, final


def _compare(x, scale, out, final):
    B, T, H, D = x["v"].shape
    rep = H // x["q"].shape[2]
    flat = lambda t: t.reshape(B * T, *t.shape[2:]).double()
    q, k, v = flat(x["q"]).repeat_interleave(rep, 1), flat(x["k"]).repeat_interleave(rep, 1), \
        flat(x["v"])
    lam = torch.zeros((B * T, H), dtype=torch.float64, device=DEV)
    if x["g"] is not None:
        lam = lam + flat(x["g"])
    if x["decay"] is not None:
        lam = lam + x["decay"].double()
    lam = lam.clamp(max=0.0)
    at = 0
    for n, length in enumerate(x["lens"]):
        span = slice(at, at + length)
        S = torch.zeros((H, D, D), dtype=torch.float64, device=DEV)
        if x["initial"] is not None:
            S = x["initial"][n].double()
        o, S, o_mag, S_mag = forms.la_prompt(q[span], k[span], v[span], lam[span], scale, S)
        tile = float(-lam[span].clamp(min=-87.4).min()) * 16 * LOG2E if length else 0.0
        c = (64 + 6 * (length // 64 + 1) + 8 * tile) * U32
        what = "sequence %d of %d tokens" % (n, length)
        forms.check(flat(out)[span], o, U16 * o.abs() + (U16 + c) * o_mag + 1e-30, what + ", out")
        half = U16 * S.abs() if final.dtype == torch.bfloat16 else 0 * S
        forms.check(final[n], S, half + c * S_mag + 1e-30, what + ", state")
        at += length


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens,H,Hk,segment", [
    ([1], 1, 1, 0), ([64], 2, 1, 0), ([63, 1, 65], 3, 3, 0), ([0, 17, 0, 129, 0], 4, 2, 0),
    ([300, 700, 1024], 6, 2, 0), ([33] * 20, 9, 3, 0), ([200, 64, 0, 1, 513], 4, 4, 64),
    ([128, 128, 127, 129], 6, 1, 128), ([1000], 5, 5, 192)])
def test_packed(lens, H, Hk, segment, D):
    print("kda_la_fwd packed", lens, H, Hk, segment, D, flush=True)
    x = _inputs(H * 100 + D, lens, H, Hk, D)
    out, final = _run(x, D ** -0.5, segment=segment)
    _compare(x, D ** -0.5, out, final)


@pytest.mark.parametrize("gate,state,out_state", [
    ("token", "bf16", torch.bfloat16), ("head", None, torch.float32),
    ("none", "fp32", torch.bfloat16), ("both", "bf16", torch.float32)])
@pytest.mark.parametrize("B,T,segment", [(1, 5, 0), (3, 100, 0), (2, 400, 128)])
def test_batched(B, T, segment, gate, state, out_state):
    print("kda_la_fwd batched", B, T, segment, gate, state, out_state, flush=True)
    x = _inputs(B * T, [T] * B, 4, 2, 64, gate=gate, state=state, packed=False)
    out, final = _run(x, -0.7, out_state, segment=segment)
    _compare(x, -0.7, out, final)


def test_automatic_segments():
    """A long sequence of few heads is split by the library's own rule."""
    x = _inputs(3, [4000], 2, 2, 64)
    assert kda.kda_la_workspace_bytes(4000, 1, 2, 64) > 0
    out, final = _run(x, 0.125)
    _compare(x, 0.125, out, final)


@pytest.mark.parametrize("segment", [0, 64])
def test_strong_decays_and_resets(segment):
    """Resets (a log decay of minus infinity) drop the past, here inside one tile and at tile
    and chunk borders; strong decays underflow; decays above zero count as none."""
    x = _inputs(11, [260], 3, 3, 64, gate="token", strong=30.0)
    x["g"][:, :, 0] = -0.01
    for t in (5, 9, 16, 63, 64, 128, 200):
        x["g"][0, t, 0] = -float("inf")
    x["g"][0, 70:90, 0] = 3.0
    out, final = _run(x, 0.3, segment=segment)
    _compare(x, 0.3, out, final)


@pytest.mark.parametrize("segment", [0, 64])
def test_state_in_place(segment):
    """final_state may be initial_state: also in segments, where other workgroups read it."""
    x = _inputs(12, [400, 0, 30, 129], 4, 2, 128)
    out, final = _run(x, 1.0, segment=segment)
    state = x["initial"].clone()
    again = torch.empty_like(out)
    kda.kda_la_fwd(x["q"], x["k"], x["v"], x["g"], 1.0, again, decay=x["decay"],
                   initial_state=state, final_state=state, cu_seqlens=x["cu"], segment=segment)
    assert torch.equal(again, out) and torch.equal(state, final)
    _compare(x, 1.0, out, final)


def test_prompt_then_steps():
    """A prompt's final states are the pool of kda_la_step: prompt plus single tokens equals
    one longer prompt."""
    T, more, H, Hk, D = 150, 4, 6, 2, 128
    x = _inputs(13, [T + more] * 2, H, Hk, D, packed=False)
    out, final = _run(x, 0.1)
    head = {n: (t[:, :T].contiguous() if n in "qkvg" else t) for n, t in x.items()}
    head["lens"] = [T, T]
    _, pool = _run(head, 0.1)
    for t in range(T, T + more):
        o = torch.empty((2, H, D), dtype=torch.bfloat16, device=DEV)
        kda.kda_la_step(x["q"][:, t], x["k"][:, t], x["v"][:, t], x["g"][:, t].contiguous(), 0.1,
                        o, pool, decay=x["decay"])
        # the prompt's out carries two bf16 roundings of sums, the step's one
        err = float((o.double() - out[:, t].double()).norm() / out[:, t].double().norm())
        assert err <= 3 * U16, err
    err = float((pool.double() - final.double()).norm() / final.double().norm())
    assert err <= 1e-6, err


def test_nan_gate_reaches_its_head_only():
    x = _inputs(14, [100, 80], 3, 1, 32)
    x["g"][0, 70, 1] = float("nan")
    out, final = _run(x, 1.0)
    bad = torch.isnan(out[0]).any(-1)
    assert bad[70:100, 1].all() and not bad[:64].any() and not bad[100:].any()
    assert not bad[:, 0].any() and not bad[:, 2].any()
    assert torch.isnan(final[0, 1]).all() and not torch.isnan(final[1]).any()


@pytest.mark.parametrize("lens,H,Hk,D,segment", [([150, 90], 4, 2, 32, 0), ([150, 90], 4, 2, 64, 0),
                                                 ([150, 90], 4, 2, 128, 0), ([700], 6, 3, 128, 0),
                                                 ([700], 6, 3, 128, 128)])
def test_infinities_and_nan_reach_later_tokens_only(lens, H, Hk, D, segment):
    """Those of v: later outputs and the state in their value; of q: its token; of k: later
    tokens of its heads.  Everything else is bit for bit what it is without them."""
    print("kda_la_fwd odd", lens, H, Hk, D, segment, flush=True)
    x = _inputs(21, lens, H, Hk, D)
    want, want_final = _run(x, 0.5, segment=segment)
    got = torch.zeros(want.shape, dtype=torch.bool, device=DEV)  # where one is seen
    state = torch.zeros(want_final.shape, dtype=torch.bool, device=DEV)
    y = dict(x, **{n: x[n].clone() for n in "qkv"})
    for t, d, value in [(3, 5, float("inf")), (70, 0, float("nan")), (75, D - 1, -float("inf")),
                        (lens[0] - 1, 17, float("nan"))]:
        y["v"][0, t, 1, d] = value
        got[0, t:lens[0], 1, d] = True
        state[0, 1, d] = True
    y["q"][0, 66, 0, 2] = float("nan")
    got[0, 66, :H // Hk] = True
    y["k"][0, 90, Hk - 1, 4] = float("nan")
    got[0, 90:lens[0], H - H // Hk:] = True
    state[0, H - H // Hk:, :, 4] = True
    out, final = _run(y, 0.5, segment=segment)
    assert torch.equal(out.isfinite(), ~got) and torch.equal(out[~got], want[~got])
    # k reaches its column of the state, and what the products take along with it
    rest = ~state
    rest[0, H - H // Hk:] = False
    assert not final[state].isfinite().any() and torch.equal(final[rest], want_final[rest])


def test_capture_and_streams():
    """Captured and replayed beside eager work, on another stream, workspaces of their own."""
    x = _inputs(15, [700], 4, 4, 64)
    y = _inputs(16, [300, 650], 4, 4, 64)
    want = [_run(z, 0.5, segment=128) for z in (x, y)]
    ws = torch.empty(kda.kda_la_workspace_bytes(700, 1, 4, 64, 128), dtype=torch.uint8, device=DEV)
    out, final = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    call = lambda s=None, w=ws: kda.kda_la_fwd(
        x["q"], x["k"], x["v"], x["g"], 0.5, out, decay=x["decay"], initial_state=x["initial"],
        final_state=final, cu_seqlens=x["cu"], segment=128, workspace=w, stream=s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_(), final.zero_()
        graph.replay()
        other = _run(y, 0.5, segment=128)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0][0]) and torch.equal(final, want[0][1])
        assert torch.equal(other[0], want[1][0]) and torch.equal(other[1], want[1][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_(), final.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side, None)
    other = _run(y, 0.5, segment=128)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(final, want[0][1])
    assert torch.equal(other[0], want[1][0]) and torch.equal(other[1], want[1][1])
