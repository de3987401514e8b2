"""Infinities and NaN in segmented linear attention (kda_la_fwd): under decays that end the
state-only pass long before a segment's first token, they must reach the later segments all
the same, and nothing else.

No tolerance: what is not finite has to be where the recurrence has it, a NaN gate's in every
value of its head, k's in every value too (and in its column of the state), v's in its value;
everything else equals the same call without them bit for bit.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
from tests.test_gpu_la import _inputs, _run

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def _plain(x, scale, out_state=torch.float32):
    """The same call without segments: a workspace of no bytes leaves none to it."""
    return _run(x, scale, out_state, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))


def _decaying(seed, lens, H, Hk, D, packed=True):
    """Head 0 decays slowly, the others by e^-1.7 a token and more."""
    x = _inputs(seed, lens, H, Hk, D, gate="token", packed=packed)
    x["g"] = x["g"] - 1.7
    x["g"][..., 0] += 1.69
    return x


def _spoil(x, plant):
    """A copy of x with (tensor, token, head, element, value) planted; where `out` and the
    final state stop being finite, by the recurrence."""
    y = dict(x, **{n: x[n].clone() for n in "qkvg"})
    B, T, H, D = x["v"].shape
    group = H // x["q"].shape[2]
    rows = torch.zeros((B * T, H, D), dtype=torch.bool, device=DEV)
    state = torch.zeros((len(x["lens"]), H, D, D), dtype=torch.bool, device=DEV)
    start = [0]
    for n in x["lens"]:
        start.append(start[-1] + n)
    for name, t, h, e, value in plant:
        n = max(i for i in range(len(x["lens"])) if start[i] <= t and x["lens"][i])
        later = slice(t, start[n + 1])
        if name == "g":
            y["g"].view(B * T, H)[t, h] = value
            rows[later, h] = state[n, h] = True
            continue
        at = y[name].reshape(B * T, -1, D)
        at[t, h, e] = value
        y[name] = at.view(y[name].shape)
        if name == "v":
            rows[later, h, e] = state[n, h, e] = True
        else:
            heads = slice(h * group, (h + 1) * group)
            rows[later, heads] = state[n, heads, :, e] = True
    return y, rows.view(B, T, H, D), state


PLANTS = {"gate": [("g", 3, 1, 0, NAN)], "v": [("v", 10, 2, 5, INF), ("v", 77, 1, 0, NAN)],
          "k": [("k", 20, 1, 7, NAN)], "k-inf": [("k", 1, 1, 30, -INF)],
          "slow": [("g", 70, 0, 0, NAN), ("v", 100, 0, 2, -INF)]}


@pytest.mark.parametrize("plant", sorted(PLANTS))
@pytest.mark.parametrize("lens,H,Hk,D,segment", [
    ([700], 4, 2, 32, 128), ([700], 4, 2, 64, 192), ([450], 4, 2, 128, 128),
    ([900], 4, 2, 128, 256), ([300, 0, 513, 40], 4, 2, 64, 64)])
def test_reach_every_later_segment(lens, H, Hk, D, segment, plant):
    print("kda_la_fwd segments", plant, lens, H, Hk, D, segment, flush=True)
    x = _decaying(31, lens, H, Hk, D)
    y, rows, state = _spoil(x, PLANTS[plant])
    for out_state in (torch.float32, torch.bfloat16):
        want, want_state = _run(x, 0.5, out_state, segment=segment)
        assert want.isfinite().all() and want_state.isfinite().all()
        out, final = _run(y, 0.5, out_state, segment=segment)
        assert torch.equal(out.isfinite(), ~rows) and torch.equal(out[~rows], want[~rows])
        assert torch.equal(final.isfinite(), ~state)
        assert torch.equal(final[~state], want_state[~state])
        one, one_state = _plain(y, 0.5, out_state)
        assert torch.equal(one.isfinite(), ~rows) and torch.equal(one_state.isfinite(), ~state)


@pytest.mark.parametrize("segment", [64, 128])
def test_several_sequences_and_segments(segment):
    """Planted in middle and last segments, in the second of three sequences of a batch; the
    last token of a segment; the states in place."""
    x = _decaying(32, [500, 500, 500], 4, 4, 64, packed=False)
    y, rows, state = _spoil(x, [("v", 500 + 127, 1, 9, NAN), ("g", 500 + 260, 2, 0, NAN),
                                ("k", 500 + 499, 3, 0, INF), ("v", 1000, 3, 63, INF)])
    want, want_state = _run(x, 0.5, segment=segment)
    out = torch.empty_like(want)
    kept = y["initial"].clone()
    kda.kda_la_fwd(y["q"], y["k"], y["v"], y["g"], 0.5, out, initial_state=kept, final_state=kept,
                   segment=segment)
    assert torch.equal(out.isfinite(), ~rows) and torch.equal(out[~rows], want[~rows])
    assert torch.equal(kept.isfinite(), ~state) and torch.equal(kept[~state], want_state[~state])


def test_in_the_automatic_schedule():
    """A long prompt that the library splits by itself, a NaN among its first tokens; without
    a final state too, and replayed from a graph beside a clean call."""
    x = _inputs(33, [4000], 2, 2, 64, gate="token", strong=3.0)
    assert kda.kda_la_workspace_bytes(4000, 1, 2, 64) > 0
    y, rows, state = _spoil(x, [("g", 100, 1, 0, NAN)])
    want, _ = _run(x, 0.125)
    out, final = _run(y, 0.125)
    assert torch.equal(out.isfinite(), ~rows) and torch.equal(final.isfinite(), ~state)
    assert torch.equal(out[~rows], want[~rows])
    call = lambda z, o: kda.kda_la_fwd(z["q"], z["k"], z["v"], z["g"], 0.125, o,
                                       initial_state=z["initial"], cu_seqlens=z["cu"])
    again, clean = torch.empty_like(out), torch.empty_like(out)
    call(x, clean)  # without a final state the sums have another number of parts
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(y, again)
    for _ in range(3):
        again.zero_()
        graph.replay()
        other = torch.empty_like(out)
        call(x, other)
        torch.cuda.synchronize()
        assert torch.equal(other, clean)
        assert torch.equal(again.isfinite(), ~rows) and torch.equal(again[~rows], clean[~rows])
