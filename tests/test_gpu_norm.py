"""The norms before and after a block with gate and residual (kda_norm) against the formulas in 64
bits; bounds in tests/layer_forms.py."""
from __future__ import annotations

import itertools

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms
from tests.serving_forms import U16, U32, check

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _run(g, R, W, group=0, gate="", res=None, pre=True, wt=F32, alpha=0.5, strided=False,
         in_place=False, eps=1e-6):
    wide = _normal(g, R, 2 * W + 8)
    x = wide[:, :W] if strided else wide[:, :W].contiguous()
    z = wide[:, W + 8:] if strided else wide[:, W + 8:].contiguous()
    kw = dict(eps=eps, residual_scale=alpha, gate_fn=gate or "sigmoid")
    kw["gate"] = z if gate else None
    kw["post_weight"] = _normal(g, group, dtype=wt) if group else None
    kw["weight"] = _normal(g, W, dtype=wt) if pre else None
    r = _normal(g, R, W, dtype=res) if res is not None else None
    h, hb, y, yb = forms.norm(x, kw["weight"], eps, kw["post_weight"], kw["gate"], kw["gate_fn"], r,
                              alpha, res_u=U16 if res is BF16 else U32)
    h_out = None
    if r is not None:
        h_out = r if in_place else torch.full_like(r, 7.0)
    out = torch.full((R, W), 7.0, dtype=BF16, device=DEV)
    kda.kda_norm(x, out, residual=r, residual_out=h_out, **kw)
    check(out, y, yb, "out")
    if r is not None:
        check(h_out, h, hb, "residual_out")
    return x, out, h_out


WIDTHS = [8, 40, 512, 520, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 12288, 16384]


@pytest.mark.parametrize("W", WIDTHS)
def test_widths(W):
    """Every kernel size and its edges, all parts at once and each alone; odd numbers of rows."""
    print("kda_norm", W, flush=True)
    g = _gen(W)
    _run(g, 5, W, group=W, gate="silu", res=F32, wt=BF16)
    _run(g, 3, W)
    _run(g, 1, W, group=W, pre=False)
    _run(g, 7, W, gate="sigmoid", pre=False)
    _run(g, 2, W, res=BF16, pre=False, alpha=-1.25)


@pytest.mark.parametrize("group,heads", itertools.product([32, 64, 128, 256, 512], [1, 3, 16, 32]))
def test_groups(group, heads):
    """Norms of heads, gated, with and without what couples a row's heads."""
    print("kda_norm groups", group, heads, flush=True)
    g, W = _gen(group + heads), group * heads
    _run(g, 9, W, group=group, gate="sigmoid", pre=False, strided=True)
    _run(g, 9, W, group=group, gate="silu", res=BF16, wt=BF16, strided=True)
    _run(g, 130, W, group=group, res=F32, pre=False)


@pytest.mark.parametrize("R", [1, 4, 63, 64, 65, 1000])
def test_rows_strides_and_in_place(R):
    g = _gen(R)
    for W in (64, 1024, 4096):
        _run(g, R, W, group=64, gate="silu", res=F32, strided=True, in_place=True)
        _run(g, R, W, res=BF16, wt=BF16, strided=True, in_place=True)


def test_leading_dimensions():
    """[B,T,H D] rows as one tensor, also as a view of wider rows; out may be left out."""
    g = _gen(1)
    x, w = _normal(g, 2, 5, 3 * 128), _normal(g, 128, dtype=F32)
    r = _normal(g, 2, 5, 3 * 128, dtype=F32)
    wide = _normal(g, 2, 5, 1024)
    z = wide[..., 256:640]
    h = torch.empty_like(r)
    kda.kda_norm(x, post_weight=w, gate=z, residual=r, residual_out=h)
    want, bound, _, _ = forms.norm(x, post_weight=w, gate=z, residual=r, res_u=U32)
    check(h, want, bound, "residual_out")
    one = torch.empty((256,), dtype=BF16, device=DEV)  # a single row without other dimensions
    kda.kda_norm(wide[0, 0, :256], one, weight=_normal(g, 256).fill_(1))
    _, _, want, bound = forms.norm(wide[0, 0, :256], torch.ones(256, device=DEV))
    check(one, want, bound, "out")
    kda.kda_norm(x[:, :0], torch.empty_like(x[:, :0]), weight=_normal(g, 384))  # no rows


def test_odd_values_stay_in_their_rows():
    """Zero rows, infinities and NaN: as the formulas, in their own rows (and groups) only."""
    g = _gen(2)
    for W in (256, 4096):
        x, w = _normal(g, 6, W), _normal(g, W)
        x[1] = 0
        x[2, 3], x[3, 5], x[4, 70] = float("inf"), float("nan"), float("-inf")
        out = torch.empty_like(x)
        kda.kda_norm(x, out, weight=w)
        _, _, y, yb = forms.norm(x, w)
        check(out, y, yb, "out")
        kda.kda_norm(x, out, post_weight=w[:64].contiguous())
        _, _, y, yb = forms.norm(x, post_weight=w[:64])
        check(out, y, yb, "groups")
        assert torch.isfinite(out[2, 64:]).all() and torch.isfinite(out[4, :64]).all()


def test_gates_far_from_zero():
    g = _gen(3)
    W = 1024
    x = _normal(g, 4, W)
    z = torch.linspace(-120, 120, 4 * W, device=DEV).to(BF16).view(4, W)
    for fn in ("sigmoid", "silu"):
        out = torch.empty_like(x)
        kda.kda_norm(x, out, gate=z, gate_fn=fn)
        _, _, y, yb = forms.norm(x, gate=z, gate_fn=fn)
        check(out, y, yb, fn)


def test_largest_gates():
    """Gates at the ends of bf16's range, and beyond: closed ones give zero however large the row."""
    g = _gen(8)
    W, inf = 64, float("inf")
    x = _normal(g, 5, W)
    z = torch.empty_like(x)
    z[0], z[1], z[2], z[3] = -3e38, -1e30, 300.0, -300.0
    x[0], x[1, ::2] = 1e10, -1e20
    z[4] = torch.tensor([-inf, inf, float("nan"), 3e38] * (W // 4), device=DEV)
    x[4, 3::4] = 0.5
    for fn in ("sigmoid", "silu"):
        out = torch.empty_like(x)
        kda.kda_norm(x, out, gate=z, gate_fn=fn)
        _, _, y, yb = forms.norm(x, gate=z, gate_fn=fn)
        assert (y[:2] == 0).all()
        check(out[:2], y[:2], torch.full_like(y[:2], 1e-37), fn + " closed")
        check(out[2:], y[2:], yb[2:], fn)


def test_many_rows_of_one_head():
    """More rows than a launch of one workgroup each would like."""
    _run(_gen(4), 300001, 128, group=128, gate="sigmoid", pre=False)


def test_repeats_itself_and_replays():
    g = _gen(5)
    R, W = 33, 8192
    x, z, w = _normal(g, R, W), _normal(g, R, W), _normal(g, W)
    r = _normal(g, R, W, dtype=F32)
    h, out = torch.empty_like(r), torch.empty_like(x)
    call = lambda s=None: kda.kda_norm(x, out, weight=w, post_weight=w, gate=z, residual=r,
                                       residual_out=h, stream=s)
    call()
    torch.cuda.synchronize()
    want = h.clone(), out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for _ in range(3):
        h.zero_(), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(out, want[1])
        h.zero_(), out.zero_()
        torch.cuda.synchronize()
        call(side)
        side.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(out, want[1])
