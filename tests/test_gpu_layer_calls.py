"""The compiled calls of the norms, rotary positions and 4-bit caches: what they refuse before
anything is launched, the kinds of stream they take, calls from several threads at once."""
from __future__ import annotations

import threading

import pytest
import torch

import gated_delta_rule_62_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _calls():
    """One good call of each operator: name -> (function, its arguments by name)."""
    g = torch.Generator(device=DEV).manual_seed(41)
    r = lambda *shape, dtype=BF16: torch.randn(shape, generator=g, device=DEV).to(dtype)
    ints = lambda *x: torch.tensor(x, dtype=torch.int64, device=DEV)
    B, T, Hq, Hk, D, W = 1, 70, 4, 2, 64, 256
    norm = dict(x=r(B, T, W), out=r(B, T, W), weight=r(W, dtype=F32), eps=1e-5,
                post_weight=r(64, dtype=F32), gate=r(B, T, W), gate_fn="silu",
                residual=r(B, T, W, dtype=F32), residual_out=r(B, T, W, dtype=F32),
                residual_scale=0.5)
    cu = ints(0, 30, T)
    rope = dict(q=r(B, T, Hq, D), k=r(B, T, Hk, D), freqs=kda.kda_rope_freqs(D)[0],
                q_out=r(B, T, Hq, D), k_out=r(B, T, Hk, D), positions=None, offsets=ints(3, 9),
                cu_seqlens=cu, amplitude=1.0)
    k4, ks, v4, vs = kda.kda_cache4_empty(3, Hk, 128, D)
    put = dict(k=r(B, T, Hk, D), v=r(B, T, Hk, D), k4=k4, ks=ks, v4=v4, vs=vs, offsets=ints(0, 50),
               cu_seqlens=cu, slots=ints(2, 0), k_out=r(B, T, Hk, D), v_out=r(B, T, Hk, D))
    cache = kda.kda_cache4_empty(3, Hk, 128, D)
    kda.kda_cache4_put(put["k"], put["v"], *cache, cu_seqlens=cu)
    attn4 = dict(q=r(B, T, Hq, D), k4=cache[0], ks=cache[1], v4=cache[2], vs=cache[3], scale=0.1,
                 out=r(B, T, Hq, D), lse=r(B, T, Hq, dtype=F32), k_lens=ints(30, 40),
                 cu_seqlens_q=cu, slots=ints(0, 1), part=64)
    return {"norm": (kda.kda_norm, norm), "rope": (kda.kda_rope, rope),
            "put": (kda.kda_cache4_put, put), "attn4": (kda.kda_attn4_fwd, attn4)}


# arguments that may be None by themselves
NULLABLE = {"weight", "post_weight", "gate", "offsets", "cu_seqlens", "slots", "lse", "k_lens",
            "cu_seqlens_q", "positions"}


@pytest.mark.parametrize("name", ["norm", "rope", "put", "attn4"])
def test_refusals(name):
    """Every tensor argument: no tensor, on the CPU, of another dtype, shape or stride."""
    print("refusals", name, flush=True)
    fn, good = _calls()[name]
    fn(**good)
    torch.cuda.synchronize()
    before = {k: v.clone() for k, v in good.items() if isinstance(v, torch.Tensor)}
    for key, t in before.items():
        bads = [(TypeError, 3), (ValueError, t.cpu()), (ValueError, t[None]),
                ((ValueError, TypeError), t.to(torch.float16))]
        if t.dim() > 1:
            wide = torch.empty(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=DEV)
            bads.append((ValueError, wide[..., ::2]))
        if key not in NULLABLE:
            bads.append(((TypeError, ValueError, kda.KdaError), None))
        for error, bad in bads:
            with pytest.raises(error):
                fn(**dict(good, **{key: bad}))
    for key, bad, error in (("stream", "other", TypeError), ("eps", "one", TypeError),
                            ("eps", -1.0, kda.KdaError), ("residual_scale", None, TypeError),
                            ("gate_fn", "relu", ValueError), ("gate_fn", 1, ValueError),
                            ("amplitude", float("nan"), kda.KdaError), ("amplitude", "x", TypeError),
                            ("scale", float("nan"), kda.KdaError), ("part", -64, kda.KdaError),
                            ("part", 1.5, TypeError)):
        if key in good or key == "stream":
            with pytest.raises(error):
                fn(**dict(good, **{key: bad}))
    if name == "attn4":
        for bad in (torch.empty(64, device=DEV), torch.empty((8, 8), dtype=torch.uint8, device=DEV),
                    torch.empty(64, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                fn(**dict(good, workspace=bad))
        with pytest.raises(kda.KdaError):  # too small
            fn(**dict(good, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)))
    if name == "norm":
        with pytest.raises(ValueError):  # weights of two dtypes
            fn(**dict(good, weight=good["weight"].to(BF16)))
        with pytest.raises(ValueError):  # residuals of two dtypes
            fn(**dict(good, residual=good["residual"].to(BF16)))
        with pytest.raises(kda.KdaError):  # an output that is an input
            fn(**dict(good, out=good["x"]))
    if name == "rope":
        with pytest.raises(kda.KdaError):  # a part of its input's rows
            fn(**dict(good, q_out=good["q"].flatten()[:-256 * 8].view(1, 62, 4, 64),
                      q=good["q"][:, 8:], k=None, k_out=None,
                      cu_seqlens=torch.tensor([0, 30, 62], device=DEV)))
    torch.cuda.synchronize()
    for key, t in before.items():
        assert torch.equal(t, good[key]), key


@pytest.mark.parametrize("name", ["norm", "rope", "put", "attn4"])
def test_streams_of_every_kind(name):
    """None, a torch stream and a raw stream's address run on that stream."""
    fn, good = _calls()[name]
    outs = [k for k in ("out", "residual_out", "q_out", "k_out", "v_out", "lse", "k4", "vs")
            if k in good and not (name == "attn4" and k in ("k4", "vs"))]
    fn(**good)
    torch.cuda.synchronize()
    want = {k: good[k].clone() for k in outs}
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    for stream, runs_on in ((None, main), (side, side), (side.cuda_stream, side), (main, main)):
        for k in outs:
            good[k].zero_()
        torch.cuda.synchronize()
        fn(**good, stream=stream)
        runs_on.synchronize()
        assert all(torch.equal(good[k], want[k]) for k in outs)
    for k in outs:
        good[k].zero_()
    with torch.cuda.stream(side):
        side.wait_stream(main)
        fn(**good)
    side.synchronize()
    assert all(torch.equal(good[k], want[k]) for k in outs)


def test_threads():
    """Calls of all four from four threads, each on a stream of its own, give what they give
    alone."""
    alone = _calls()
    for fn, good in alone.values():
        fn(**good)
    torch.cuda.synchronize()
    mine = [_calls() for _ in range(4)]
    torch.cuda.synchronize()
    failures = []

    def work(calls):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    for name, (fn, good) in calls.items():
                        fn(**good)
                    s.synchronize()
                    for name, (_, good) in calls.items():
                        for k, v in good.items():
                            if isinstance(v, torch.Tensor):
                                assert torch.equal(v, alone[name][1][k]), (name, k)
        except BaseException as e:  # reported by the main thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in mine]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
