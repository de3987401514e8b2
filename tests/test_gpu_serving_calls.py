"""The serving operators' compiled calls from Python: what they refuse before anything is
launched, the kinds of stream they take, and calls from several threads at once."""
from __future__ import annotations

import threading

import pytest
import torch

import gated_delta_rule_62_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _calls():
    """One good call of each operator: name -> (function, its arguments by name)."""
    g = torch.Generator(device=DEV).manual_seed(31)
    r = lambda *shape, dtype=torch.bfloat16: _rand(g, *shape, dtype=dtype)
    N, H, Hk, D, T = 3, 4, 2, 64, 200
    f32 = torch.float32
    step = dict(q=r(N, H, D), k=r(N, H, D), v=r(N, H, D), g=r(N, H, D), beta=r(N, H), scale=0.1,
                out=r(N, H, D), A_log=r(H, dtype=f32), dt_bias=r(H, D, dtype=f32),
                lower_bound=-5.0, state=r(5, H, D, D, dtype=f32),
                slot_in=torch.tensor([0, 2, 4], device=DEV),
                slot_out=torch.tensor([0, 2, 4], device=DEV))
    la_step = dict(q=r(N, Hk, D), k=r(N, Hk, D), v=r(N, H, D), g=-r(N, H, dtype=f32).abs(),
                   scale=0.1, out=r(N, H, D), state=r(5, H, D, D), decay=None, slot_in=None,
                   slot_out=None)
    la = dict(q=r(1, T, Hk, D), k=r(1, T, Hk, D), v=r(1, T, H, D),
              g=-r(1, T, H, dtype=f32).abs(), scale=0.1, out=r(1, T, H, D), decay=None,
              initial_state=None, final_state=r(2, H, D, D, dtype=f32),
              cu_seqlens=torch.tensor([0, 90, T], device=DEV), segment=64)
    attn = dict(q=r(1, T, H, D), k=r(1, T, Hk, D), v=r(1, T, Hk, D), scale=0.1,
                out=r(1, T, H, D), lse=r(1, T, H, dtype=f32),
                cu_seqlens_q=torch.tensor([0, 90, T], device=DEV),
                cu_seqlens_k=torch.tensor([0, 90, T], device=DEV), k_lens=None, splits=2)
    return {"step": (kda.kda_step, step), "la_step": (kda.kda_la_step, la_step),
            "la": (kda.kda_la_fwd, la), "attn": (kda.kda_attn_fwd, attn)}


@pytest.mark.parametrize("name", ["step", "la_step", "la", "attn"])
def test_refusals(name):
    """Every tensor argument: no tensor, on the CPU, of another dtype, shape or stride."""
    print("refusals", name, flush=True)
    fn, good = _calls()[name]
    fn(**good)
    torch.cuda.synchronize()
    before = {k: v.clone() for k, v in good.items() if isinstance(v, torch.Tensor)}
    nullable = {"g", "decay", "slot_in", "slot_out", "initial_state", "final_state", "cu_seqlens",
                "lse", "cu_seqlens_q", "cu_seqlens_k", "k_lens"}
    for key, t in before.items():
        bads = [(TypeError, 3), (ValueError, t.cpu()), (ValueError, t[None]),
                ((ValueError, TypeError), t.to(torch.float64))]
        if t.dim() > 1:
            wide = torch.empty(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=DEV)
            bads.append((ValueError, wide[..., ::2]))
        if key not in nullable or (name == "step" and key == "g"):
            bads.append((TypeError, None))
        for error, bad in bads:
            with pytest.raises(error):
                fn(**dict(good, **{key: bad}))
    with pytest.raises(TypeError):
        fn(**dict(good, scale="one"))
    with pytest.raises(TypeError):
        fn(**dict(good, stream="other"))
    with pytest.raises(kda.KdaError):
        fn(**dict(good, scale=float("nan")))
    if name in ("la", "attn"):
        for bad in (torch.empty(64, device=DEV), torch.empty((8, 8), dtype=torch.uint8, device=DEV),
                    torch.empty(64, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                fn(**dict(good, workspace=bad))
        with pytest.raises(kda.KdaError):  # too small
            fn(**dict(good, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)))
        with pytest.raises(kda.KdaError):
            fn(**dict(good, **{"segment" if name == "la" else "splits": -64}))
    torch.cuda.synchronize()
    for key, t in before.items():
        assert torch.equal(t, good[key]), key


def test_streams_of_every_kind():
    """None, a torch stream and a raw stream's address run on that stream."""
    _, good = _calls()["attn"]
    kda.kda_attn_fwd(**good)
    torch.cuda.synchronize()
    want = good["out"].clone()
    side = torch.cuda.Stream()
    main = torch.cuda.default_stream()
    for stream, runs_on in ((None, main), (side, side), (side.cuda_stream, side), (main, main)):
        good["out"].zero_()
        torch.cuda.synchronize()
        kda.kda_attn_fwd(**good, stream=stream)
        runs_on.synchronize()
        assert torch.equal(good["out"], want)
    good["out"].zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        kda.kda_attn_fwd(**good)
    side.synchronize()
    assert torch.equal(good["out"], want)


def test_threads():
    """Calls from four threads, each on a stream of its own, give what they give alone."""
    calls = [_calls() for _ in range(4)]
    _, alone = _calls()["la"]
    kda.kda_la_fwd(**alone)
    torch.cuda.synchronize()
    failures = []

    def work(c):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    fn, good = c["la"]
                    good["out"].zero_()
                    fn(**good)
                    s.synchronize()
                    assert torch.equal(good["out"], alone["out"])
                    assert torch.equal(good["final_state"], alone["final_state"])
        except BaseException as e:  # reported by the main thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
