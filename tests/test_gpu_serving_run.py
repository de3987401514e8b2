"""The serving operators together, as a server runs them: a packed batch of prompts through a
stack of a KDA layer, a linear-attention layer and a softmax-attention layer, then single
tokens of the same requests over the states and caches that the prompts left.

Every layer's output is checked against its 64-bit definition on the very inputs that the
kernels had, prompts and single tokens alike, and the tokens' rows against those of one longer
prompt.  Bounds: the operators' own, in relative L2 norm: three bf16 roundings for linear and
softmax attention (two inside, one of the result), kda_fwd's published 5e-3 for the KDA
prompt, two roundings for the KDA step.  Between the two ways of computing one row the layers
before it differ too; three layers of at most 2e-2 each.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.serving_forms as forms
from tests.serving_forms import U16
from tests.test_gpu_attn import _want as attn_form

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, HK, D, WIDE = 8, 2, 64, 256
SCALE, LB = D ** -0.5, -5.0


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


class Stack:
    def __init__(self, g):
        def weight(n):
            return (torch.randn((WIDE, n), generator=g, device=DEV) * WIDE ** -0.5).bfloat16()
        self.kda_in, self.kda_out = weight((4 * D + 1) * H), weight(H * D).t().contiguous()
        self.la_in, self.la_out = weight((2 * HK + H) * D + H), weight(H * D).t().contiguous()
        self.at_in, self.at_out = weight((2 * HK + H) * D), weight(H * D).t().contiguous()
        self.A_log = torch.rand((H,), generator=g, device=DEV)
        self.dt_bias = torch.rand((H, D), generator=g, device=DEV)
        self.decay = -torch.exp2(-torch.arange(1, H + 1, device=DEV).float())

    def project_kda(self, x):
        y = (x @ self.kda_in).view(*x.shape[:-1], H, 4 * D + 1)
        q, k, v, g = (t.contiguous() for t in torch.split(y[..., :4 * D], D, dim=-1))
        return q, k, v, g, y[..., 4 * D].contiguous()

    def project_la(self, x):
        y = x @ self.la_in
        q, k, v = torch.split(y[..., :(2 * HK + H) * D].unflatten(-1, (2 * HK + H, D)),
                              [HK, HK, H], dim=-2)
        return (q.contiguous(), k.contiguous(), v.contiguous(),
                -torch.nn.functional.softplus(y[..., (2 * HK + H) * D:].float()))

    def project_at(self, x):  # views of the projection's rows
        return torch.split((x @ self.at_in).unflatten(-1, (2 * HK + H, D)), [H, HK, HK], dim=-2)

    def prompts(self, x, lens, states):
        """x [1, T, WIDE]; fills the states; returns the last layer's hidden rows."""
        cu = torch.tensor([0] + lens).cumsum(0).to(DEV)
        q, k, v, g, b = self.project_kda(x)
        out = torch.empty_like(q)
        kda.kda_fwd(q, k, v, g, b, SCALE, out, self.A_log, self.dt_bias, LB,
                    final_state=states["kda"], cu_seqlens=cu)
        x = x + out.flatten(-2) @ self.kda_out

        q, k, v, gt = self.project_la(x)
        out = torch.empty_like(v)
        kda.kda_la_fwd(q, k, v, gt, SCALE, out, decay=self.decay, final_state=states["la"],
                       cu_seqlens=cu)
        lam = gt.double() + self.decay.double()
        at = 0
        for n, length in enumerate(lens):
            s = slice(at, at + length)
            rep = lambda t: t[0, s].double().repeat_interleave(H // HK, 1)
            o, S, _, _ = forms.la_prompt(rep(q), rep(k), v[0, s].double(), lam[0, s], SCALE,
                                         torch.zeros((H, D, D), dtype=torch.float64, device=DEV))
            assert _rel(out[0, s], o) <= 3 * U16 and _rel(states["la"][n], S) <= 1e-6
            at += length
        x = x + out.flatten(-2) @ self.la_out

        q, k, v = self.project_at(x)
        out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
        kda.kda_attn_fwd(q, k, v, SCALE, out, cu_seqlens_q=cu, cu_seqlens_k=cu)
        at = 0
        for n, length in enumerate(lens):
            s = slice(at, at + length)
            assert _rel(out[0, s], attn_form(q[0, s], k[0, s], v[0, s], SCALE)[0]) <= 3 * U16
            states["k"][n, :length], states["v"][n, :length] = k[0, s], v[0, s]
            at += length
        return x + out.flatten(-2) @ self.at_out

    def tokens(self, x, lens, slots, states):
        """x [N, WIDE]: one token of each request, whose states sit in `slots`."""
        before = states["kda"][slots].double()
        q, k, v, g, b = self.project_kda(x)
        out = torch.empty_like(q)
        kda.kda_step(q, k, v, g, b, SCALE, out, self.A_log, self.dt_bias, LB, states["kda"],
                     slot_in=slots)
        o = forms.step(*(t.double() for t in (q, k, v, g, b)), SCALE, self.A_log.double(),
                       self.dt_bias.double(), LB, before)[0]
        assert _rel(out, o) <= 2 * U16
        x = x + out.flatten(-2) @ self.kda_out

        before = states["la"][slots].double()
        q, k, v, gt = self.project_la(x)
        out = torch.empty_like(v)
        kda.kda_la_step(q, k, v, gt, SCALE, out, states["la"], decay=self.decay, slot_in=slots)
        rep = lambda t: t.double().repeat_interleave(H // HK, 1)
        o = forms.la_step(rep(q), rep(k), v.double(), gt.double() + self.decay.double(), SCALE,
                          before)[0]
        assert _rel(out, o) <= 2 * U16
        x = x + out.flatten(-2) @ self.la_out

        q, k, v = (t.unsqueeze(1) for t in self.project_at(x))
        for n, length in enumerate(lens):
            states["k"][n, length], states["v"][n, length] = k[n, 0], v[n, 0]
        lens = [length + 1 for length in lens]
        out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
        kda.kda_attn_fwd(q, states["k"], states["v"], SCALE, out,
                         k_lens=torch.tensor(lens, device=DEV))
        for n, length in enumerate(lens):
            want = attn_form(q[n], states["k"][n, :length], states["v"][n, :length], SCALE)[0]
            assert _rel(out[n], want) <= 3 * U16
        return x + out[:, 0].flatten(-2) @ self.at_out, lens


def _states(N, cap):
    return dict(kda=torch.zeros((N, H, D, D), device=DEV),
                la=torch.zeros((N, H, D, D), device=DEV),
                k=torch.full((N, cap, HK, D), float("nan"), dtype=torch.bfloat16, device=DEV),
                v=torch.full((N, cap, HK, D), float("nan"), dtype=torch.bfloat16, device=DEV))


def test_prompts_then_tokens():
    g = torch.Generator(device=DEV).manual_seed(21)
    stack, more, lens = Stack(g), 3, [70, 1, 200, 33]
    N, cap = len(lens), 256
    rows = [torch.randn((n + more, WIDE), generator=g, device=DEV).bfloat16() for n in lens]
    whole = stack.prompts(torch.cat(rows)[None], [n + more for n in lens], _states(N, cap))[0]
    states = _states(N, cap)
    stack.prompts(torch.cat([r[:n] for r, n in zip(rows, lens)])[None], lens, states)
    slots, now = torch.arange(N, device=DEV), list(lens)
    for i in range(more):
        x, now = stack.tokens(torch.stack([r[n + i] for r, n in zip(rows, lens)]), now, slots,
                              states)
        at = 0
        for n, length in enumerate(lens):
            assert _rel(x[n], whole[at + length + i].double()) <= 6e-2
            at += length + more
