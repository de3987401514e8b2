"""The operators together, as a server runs them: a packed batch of prompts through a softmax layer
with rotary positions and a 4-bit cache and a KDA layer with gated head norms, between pre-norms of
an fp32 residual stream; then single tokens and a few drafted ones of the same requests over what
the prompts left.

Every call is checked against its 64-bit definition on the very inputs that it had, within the
bounds of the operators' own tests (the KDA layer in relative L2 norm, kda_fwd's published 5e-3).
Projections are torch's.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms
from tests.serving_forms import U16, U32, check
from tests.test_gpu_attn import _want as attn_form

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
HQ, HK, D, WIDE, CAP = 8, 2, 64, 256, 160
SCALE, LB, ALPHA = D ** -0.5, -5.0, 0.5


class Layers:
    def __init__(self, g, slots):
        def weight(a, b):
            return (torch.randn((a, b), generator=g, device=DEV) * a ** -0.5).to(BF16)
        self.qkv, self.o = weight(WIDE, (HQ + 2 * HK) * D), weight(HQ * D, WIDE)
        self.kda_in, self.kda_o = weight(WIDE, (5 * D + 1) * HQ), weight(HQ * D, WIDE)
        self.n1, self.n2, self.n3, self.post = (
            1 + 0.1 * torch.randn(WIDE, generator=g, device=DEV) for _ in range(4))
        self.head = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
        self.A_log = torch.rand(HQ, generator=g, device=DEV)
        self.dt_bias = torch.rand((HQ, D), generator=g, device=DEV)
        self.freqs, self.amp = kda.kda_rope_freqs(D, method="yarn", factor=4.0, original=64)
        self.cache = kda.kda_cache4_empty(slots, HK, CAP, D)
        self.state = torch.zeros((slots, HQ, D, D), device=DEV)

    def run(self, h, lens, start, slots):
        """One pass of rows h [1, T, WIDE] (fp32 stream): sequence n's lens[n] tokens from position
        start[n] on, its caches and states in slots[n]."""
        N, T = len(lens), h.shape[1]
        cu = torch.tensor([0] + lens).cumsum(0).to(DEV)
        off, slot = (torch.tensor(x, device=DEV) for x in (start, slots))
        pos = torch.cat([s + torch.arange(n) for n, s in zip(lens, start)]).to(DEV)[None]
        seqs = [(sum(lens[:n]), x) for n, x in enumerate(lens)]

        # ---- softmax layer: norm, projection, positions, cache, attention
        x = torch.empty((1, T, WIDE), dtype=BF16, device=DEV)
        none = torch.zeros_like(x)  # the stream's own norm: nothing is added to it
        kda.kda_norm(none, x, weight=self.n1, residual=h, residual_out=h)
        _, _, y, yb = forms.norm(none, self.n1, residual=h)
        check(x, y, yb, "first norm")
        rows = (x @ self.qkv).unflatten(-1, (HQ + 2 * HK, D))
        q, k, v = torch.split(rows, [HQ, HK, HK], dim=2)
        want_q, want_k = (forms.rope(t, pos, self.freqs, self.amp) for t in (q, k))
        kda.kda_rope(q, k, self.freqs, q, k, offsets=off, cu_seqlens=cu, amplitude=self.amp)
        check(q, *want_q, "q")
        check(k, *want_k, "k")
        kda.kda_cache4_put(k, v, *self.cache, offsets=off, cu_seqlens=cu, slots=slot)
        out = torch.empty((1, T, HQ, D), dtype=BF16, device=DEV)
        kda.kda_attn4_fwd(q, *self.cache, SCALE, out, k_lens=off + cu.diff(), cu_seqlens_q=cu,
                          slots=slot)
        kc = forms.values(*forms.unpack(self.cache[0], self.cache[1], D, False)).transpose(1, 2)
        vc = forms.values(*forms.unpack(self.cache[2], self.cache[3], D, True)).transpose(1, 2)
        for n, (at, length) in enumerate(seqs):
            L = start[n] + length
            o, _, ob, _ = attn_form(q[0, at:at + length], kc[slots[n], :L], vc[slots[n], :L], SCALE)
            check(out[0, at:at + length], o, ob, "attention %d" % n)
            # the new positions hold their own keys' and values' codes
            want = forms.values(*forms.quantise(k[0, at:at + length]))
            assert torch.equal(kc[slots[n], start[n]:L], want)
            want = forms.values(*forms.quantise(v[0, at:at + length]))
            assert torch.equal(vc[slots[n], start[n]:L], want)

        # ---- between the layers: the block's norm, the scaled sum, the next norm
        block = out.flatten(-2) @ self.o
        new, x = torch.empty_like(h), torch.empty_like(x)
        kda.kda_norm(block, x, weight=self.n2, post_weight=self.post, residual=h,
                     residual_out=new, residual_scale=ALPHA)
        hw, hb, y, yb = forms.norm(block, self.n2, post_weight=self.post, residual=h, alpha=ALPHA,
                                   res_u=U32)
        check(new, hw, hb, "stream")
        check(x, y, yb, "second norm")
        h = new

        # ---- KDA layer and its gated head norm
        y = (x @ self.kda_in).unflatten(-1, (HQ, 5 * D + 1))
        q, k, v, g, z = (t.contiguous() for t in torch.split(y[..., :5 * D], D, dim=-1))
        beta = y[..., 5 * D].contiguous()
        if max(lens) == 1:
            out = torch.empty((N, HQ, D), dtype=BF16, device=DEV)
            kda.kda_step(*(t[0] for t in (q, k, v, g, beta)), SCALE, out, self.A_log, self.dt_bias,
                         LB, self.state, slot_in=slot)
            out = out[None]
        else:
            out = torch.empty_like(q)
            before, after = self.state[slot], torch.empty((N, HQ, D, D), device=DEV)
            kda.kda_fwd(q, k, v, g, beta, SCALE, out, self.A_log, self.dt_bias, LB,
                        initial_state=before, final_state=after, cu_seqlens=cu)
            self.state[slot] = after
        o = torch.empty((1, T, HQ * D), dtype=BF16, device=DEV)
        kda.kda_norm(out.flatten(-2), o, post_weight=self.head, gate=z.flatten(-2))
        _, _, y, yb = forms.norm(out.flatten(-2), post_weight=self.head, gate=z.flatten(-2))
        check(o, y, yb, "head norm")

        # ---- the last sum and norm, the stream in place
        block = o @ self.kda_o
        hw, hb, y, yb = forms.norm(block, self.n3, residual=h, res_u=U32)
        kda.kda_norm(block, x, weight=self.n3, residual=h, residual_out=h)
        check(h, hw, hb, "stream in place")
        check(x, y, yb, "last norm")
        return h, x


def test_prompts_then_tokens_then_drafts():
    g = torch.Generator(device=DEV).manual_seed(3)
    layers = Layers(g, 5)
    lens, slots, at = [70, 1, 33], [4, 0, 2], [0, 0, 0]
    rows = lambda n: torch.randn((1, n, WIDE), generator=g, device=DEV)
    h, x = layers.run(rows(sum(lens)), lens, at, slots)
    assert torch.isfinite(x).all()
    at = lens
    for step in ([1, 1, 1], [1, 1, 1], [3, 1, 2], [1, 1, 1], [5, 5, 5]):
        h, x = layers.run(rows(sum(step)), step, at, slots)
        assert torch.isfinite(x).all()
        at = [a + s for a, s in zip(at, step)]


@pytest.mark.parametrize("cut", [1, 32, 37, 99])
def test_a_prompt_in_two_chunks_is_the_prompt(cut):
    """Chunked prefill: turned and stored in two calls, the cache holds the same bytes, and the
    second chunk's attention is the prompt's rows, within the formula's bounds."""
    g = torch.Generator(device=DEV).manual_seed(cut)
    T = 100
    rows = torch.randn((1, T, HQ + 2 * HK, D), generator=g, device=DEV).to(BF16)
    freqs, _ = kda.kda_rope_freqs(D)
    caches, outs = [], []
    for chunks in ([(0, T)], [(0, cut), (cut, T)]):
        cache = kda.kda_cache4_empty(1, HK, CAP, D)
        for a, b in chunks:
            q, k, v = torch.split(rows[:, a:b], [HQ, HK, HK], dim=2)
            off = torch.tensor([a], device=DEV)
            qo, ko = torch.empty_like(q), torch.empty_like(k)
            kda.kda_rope(q, k, freqs, qo, ko, offsets=off)
            kda.kda_cache4_put(ko, v, *cache, offsets=off)
            out = torch.empty((1, b - a, HQ, D), dtype=BF16, device=DEV)
            kda.kda_attn4_fwd(qo, *cache, SCALE, out, k_lens=off + (b - a))
        caches.append(cache)
        outs.append((qo, out))
    assert all(torch.equal(a, b) for a, b in zip(*caches))
    kc, vc = (forms.values(*forms.unpack(caches[0][i], caches[0][i + 1], D, i > 0)).transpose(1, 2)
              for i in (0, 2))
    want, _, bound, _ = attn_form(outs[0][0][0], kc[0, :T], vc[0, :T], SCALE)
    check(outs[0][1][0], want, bound, "the prompt")
    check(outs[1][1][0], want[cut:], bound[cut:], "the second chunk")


def test_a_step_in_a_graph():
    """One decode step of norm, positions, cache and attention in a captured graph: every replay
    takes the positions, lengths and inputs its tensors hold by then, and gives what eager calls
    give."""
    g = torch.Generator(device=DEV).manual_seed(5)
    N = 3
    w = torch.ones(WIDE, device=DEV)
    proj = (torch.randn((WIDE, (HQ + 2 * HK) * D), generator=g, device=DEV) / 16).to(BF16)
    freqs, _ = kda.kda_rope_freqs(D)
    h = torch.randn((N, 1, WIDE), generator=g, device=DEV).to(BF16)
    x = torch.empty_like(h)
    qkv = torch.empty((N, 1, (HQ + 2 * HK) * D), dtype=BF16, device=DEV)
    out = torch.empty((N, 1, HQ, D), dtype=BF16, device=DEV)
    off, lens = torch.tensor([0, 40, 90], device=DEV), torch.empty(N, dtype=torch.int64, device=DEV)
    cache = [torch.randint(0, 120, t.shape, generator=g, device=DEV, dtype=torch.uint8)
             for t in kda.kda_cache4_empty(N, HK, CAP, D)]
    ws = torch.empty(max(1, kda.kda_attn4_workspace_bytes(N, N, 1, CAP, HQ, HK, D, 64)),
                     dtype=torch.uint8, device=DEV)

    def step():
        kda.kda_norm(h, x, weight=w)
        torch.matmul(x, proj, out=qkv)
        q, k, v = torch.split(qkv.unflatten(-1, (HQ + 2 * HK, D)), [HQ, HK, HK], dim=2)
        kda.kda_rope(q, k, freqs, q, k, offsets=off)
        kda.kda_cache4_put(k, v, *cache, offsets=off)
        torch.add(off, 1, out=lens)
        kda.kda_attn4_fwd(q, *cache, SCALE, out, k_lens=lens, part=64, workspace=ws)
        off.add_(1)

    start = [t.clone() for t in (off, h, *cache)]
    inputs = [torch.randn((N, 1, WIDE), generator=g, device=DEV).to(BF16) for _ in range(4)]
    want = []
    for i in inputs:
        h.copy_(i)
        step()
        want.append(out.clone())
    after = [t.clone() for t in (off, *cache)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((off, h, *cache), start):
        t.copy_(s)
    for i, o in zip(inputs, want):
        h.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o)
    for t, s in zip((off, *cache), after):
        assert torch.equal(t, s)
