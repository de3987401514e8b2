"""Attention over caches in 4 bits (kda_attn4_fwd) against its 64-bit definition on the values that
the caches stand for.

Bounds: those of kda_attn_fwd's tests (tests/test_gpu_attn.py), which allow one bf16 rounding of
the probabilities for their product with v.
"""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms
from tests.serving_forms import check
from tests.test_gpu_attn import _want

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(BF16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _cache(g, S, Hk, cap, D, lens=None, slots=None):
    """A cache of normal values, and what it stands for: k, v [S, cap, Hk, D].  Behind each
    length codes and scales of any kind, NaN among them."""
    cache, seen = [], []
    for is_v in (False, True):
        code, byte = forms.quantise(torch.randn((S, Hk, cap, D), generator=g, device=DEV))
        seen.append(forms.values(code, byte).transpose(1, 2))
        if lens is not None:
            for n, length in enumerate(lens):
                s = slots[n] if slots else n
                if 0 <= s < S:
                    byte[s, :, length:] = 255
                    byte[s, :, length + 1::3] = 254
                    code[s, :, length:] = 15
        cache += forms.pack(code, byte, D, is_v)
    return cache, seen[0], seen[1]


def _check_seq(out, lse, q, k, v, scale, what):
    o, z, ob, zb = _want(q, k, v, scale)
    check(out, o, ob, what + ", out")
    if lse is not None:
        check(lse, z, zb, what + ", lse")


def _run(seed, ql, kl, Hq, Hk, D, cap, S=None, slots=None, packed=True, behind=0, scale=None,
         **more):
    g = _gen(seed)
    N = len(ql)
    S = N if S is None else S
    scale = D ** -0.5 if scale is None else scale
    cache, k, v = _cache(g, S, Hk, cap, D, kl, slots)
    B, T = (1, sum(ql) + behind) if packed else (N, ql[0])
    q, _ = torch.split(_normal(g, B, T, Hq + 3, D), [Hq, 3], dim=2)
    out = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    kda.kda_attn4_fwd(q, *cache, scale, out, lse=lse, k_lens=_ints(kl),
                      cu_seqlens_q=_ints([0] + ql).cumsum(0) if packed else None,
                      slots=None if slots is None else _ints(slots), **more)
    at = 0
    for n, (lq, lk) in enumerate(zip(ql, kl)):
        row, a = (0, at) if packed else (n, 0)
        s = slots[n] if slots else n
        lk = lk if 0 <= s < S else 0
        s = min(max(s, 0), S - 1)
        _check_seq(out[row, a:a + lq], lse[row, a:a + lq], q[row, a:a + lq], k[s, :lk], v[s, :lk],
                   scale, "sequence %d (%d, %d)" % (n, lq, lk))
        at += lq
    if packed:
        assert (out[0, at:] == 7.0).all() and (lse[0, at:] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,Hq,Hk,cap", [
    ([1], [1], 1, 1, 32), ([1, 1, 1, 1], [0, 31, 32, 33], 3, 1, 64), ([1] * 3, [200, 1, 77], 16, 4, 256),
    ([5, 5], [5, 190], 6, 2, 192), ([2, 0, 9], [100, 7, 9], 12, 1, 128), ([33], [33], 4, 4, 64),
    ([65, 1, 200], [65, 0, 300], 6, 2, 320), ([100, 64, 20], [0, 10, 20], 8, 2, 32),
    ([1], [700], 32, 1, 704), ([300, 33], [500, 33], 12, 1, 512)])
def test_packed(ql, kl, Hq, Hk, cap, D):
    print("kda_attn4_fwd packed", ql, kl, Hq, Hk, cap, D, flush=True)
    _run(len(ql) * 31 + Hq, ql, kl, Hq, Hk, D, cap, behind=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,Hq,Hk,cap,part", [
    ([1, 1], [700, 3], 8, 2, 704, 64), ([2, 0, 3], [64, 5, 1000], 12, 4, 1024, 32),
    ([40, 9], [500, 9], 2, 1, 512, 96), ([1], [0], 2, 2, 64, 32), ([7], [640], 3, 1, 640, 128),
    ([200, 70], [10, 333], 2, 2, 352, 160)])
def test_parts(ql, kl, Hq, Hk, cap, part, D):
    """Parts of the keys, empty ones among them; rows behind the last sequence stay."""
    print("kda_attn4_fwd parts", ql, kl, Hq, Hk, cap, part, D, flush=True)
    _run(part, ql, kl, Hq, Hk, D, cap, behind=3, part=part)


@pytest.mark.parametrize("Tq,Hq,Hk,D", [(1, 8, 2, 128), (1, 3, 3, 64), (1, 32, 1, 128),
                                        (4, 12, 2, 64), (5, 24, 2, 128), (30, 4, 1, 128)])
def test_batch_rows_and_slots(Tq, Hq, Hk, D):
    """Batch rows over slots in another order, two over one slot, some outside the cache."""
    print("kda_attn4_fwd rows", Tq, Hq, Hk, D, flush=True)
    lens = [1, 0, 31, 32, 33, 200, 511, 700]
    _run(Tq * Hq, [Tq] * 8, lens, Hq, Hk, D, 704, packed=False)
    _run(Tq, [Tq] * 8, lens, Hq, Hk, D, 704, S=11, slots=[9, 3, 0, 10, 1, 2, 8, 5], packed=False)
    _run(Tq, [Tq] * 4, [50, 60, 70, 80], Hq, Hk, D, 96, S=3, slots=[2, -1, 0, 3], packed=False)
    g = _gen(Tq + 7)
    cache, k, v = _cache(g, 2, Hk, 64, D)
    q = _normal(g, 3, Tq, Hq, D)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.2, out, lse=lse, k_lens=_ints([60, 64, 35]),
                      slots=_ints([1, 0, 1]))
    for n, (s, lk) in enumerate(((1, 60), (0, 64), (1, 35))):
        _check_seq(out[n], lse[n], q[n], k[s, :lk], v[s, :lk], 0.2, "row %d" % n)
    # lengths outside the cache are clamped into it; without lengths all of it
    kda.kda_attn4_fwd(q[:2], *cache, 0.0, out[:2], lse=lse[:2], k_lens=_ints([-5, 1 << 40]))
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    _check_seq(out[1], lse[1], q[1], k[1], v[1], 0.0, "clamped row")
    kda.kda_attn4_fwd(q[:2], *cache, 0.2, out[:2])
    _check_seq(out[0], None, q[0], k[0], v[0], 0.2, "all positions")


def test_long_caches_in_the_automatic_parts():
    assert kda.kda_attn4_workspace_bytes(1, 1, 3, 20032, 6, 2, 128) > 0
    _run(61, [3], [20001], 6, 2, 128, 20032)
    _run(62, [1, 1], [5003, 12000], 4, 1, 64, 12000)
    _run(63, [150], [5003], 4, 1, 64, 5024)


PROMPTS = [([700, 500], [700, 900], 16, 2, 128, 928), ([650, 1, 900], [2000, 40, 900], 8, 1, 128, 2016),
           ([600, 0, 700], [600, 33, 701], 32, 4, 64, 704), ([1500], [1400], 12, 1, 128, 1408)]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D,cap", PROMPTS)
def test_prompts_expand_the_caches(ql, kl, Hq, Hk, D, cap):
    """Enough rows for the automatic choice to expand the caches; slots in another order, one
    outside, rows behind the last sequence; and the same call without a workspace."""
    print("kda_attn4_fwd prompts", ql, kl, Hq, Hk, D, cap, flush=True)
    N = len(ql)
    need = kda.kda_attn4_workspace_bytes(N, 1, sum(ql) + 3, cap, Hq, Hk, D)
    assert need >= N * cap * Hk * D * 4
    _run(71, ql, kl, Hq, Hk, D, cap, behind=3)
    _run(72, ql, kl, Hq, Hk, D, cap, S=N + 2, slots=[N + 1 - n for n in range(N)], behind=3)
    _run(73, ql, kl, Hq, Hk, D, cap, S=N, slots=[-1] + list(range(1, N)), behind=3)
    _run(74, ql, kl, Hq, Hk, D, cap, behind=3,
         workspace=torch.empty(0, dtype=torch.uint8, device=DEV))


def test_prompts_as_batch_rows():
    assert kda.kda_attn4_workspace_bytes(3, 3, 400, 448, 16, 2, 128) >= 3 * 448 * 2 * 128 * 4
    _run(75, [400] * 3, [448, 400, 12], 16, 2, 128, 448, packed=False)


def test_large_and_growing_scores():
    """Scores of a few hundred, growing along the keys, and falling."""
    g = _gen(5)
    L, H, D = 640, 2, 128
    for sign in (1, -1):
        q = _normal(g, 1, 40, H, D)
        q[..., 0] = 30.0
        x = torch.randn((1, H, L, D), generator=g, device=DEV)
        x[..., 0] = sign * torch.linspace(-100, 100, L, device=DEV)
        code, byte = forms.quantise(x)
        k = forms.values(code, byte).transpose(1, 2)
        vc, vb = forms.quantise(torch.randn((1, H, L, D), generator=g, device=DEV))
        v = forms.values(vc, vb).transpose(1, 2)
        cache = forms.pack(code, byte, D, False) + forms.pack(vc, vb, D, True)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse)
        _check_seq(out[0], lse[0], q[0], k[0], v[0], 0.1, "sign %d" % sign)


def test_scales_of_every_size():
    """Values from 2^-127 to 2^60: scale bytes from 0 on, in one cache."""
    g = _gen(6)
    L, H, D = 96, 1, 64
    q = _normal(g, 1, 3, H, D)
    code = torch.randint(0, 16, (1, H, L, D), generator=g, device=DEV)
    kb = torch.randint(100, 130, (1, H, L, 2), generator=g, device=DEV)
    vb = torch.randint(0, 187, (1, H, L, 2), generator=g, device=DEV)
    cache = forms.pack(code, kb, D, False) + forms.pack(code, vb, D, True)
    k, v = forms.values(code, kb).transpose(1, 2), forms.values(code, vb).transpose(1, 2)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.05, out, lse=lse)
    _check_seq(out[0], lse[0], q[0], k[0], v[0], 0.05, "scales")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Lk,Hq,Hk,part", [
    (1, 700, 8, 2, 0), (4, 100, 8, 2, 0), (4, 100, 8, 2, 32), (40, 500, 2, 1, 512),
    (200, 200, 2, 2, 0), (300, 333, 4, 2, 128), (150, 130, 12, 1, 0), (1200, 1250, 24, 2, 0),
    (600, 640, 16, 4, 1280), (500, 900, 8, 2, 320)])
def test_infinities_and_nan_behind_the_last_visible_key(Lq, Lk, Hq, Hk, part, D):
    """Blocks of NaN and values beyond bf16's range, in k and v, reach the queries that see them,
    and nothing else."""
    print("kda_attn4_fwd odd v", Lq, Lk, Hq, Hk, part, D, flush=True)
    g = _gen(Lk + D)
    cap, inf, off, G = -(-Lk // 32) * 32, float("inf"), Lk - Lq, Hq // Hk
    q = _normal(g, 1, Lq, Hq, D)
    kc, kb = forms.quantise(torch.randn((1, Hk, cap, D), generator=g, device=DEV))
    vc, vb = forms.quantise(torch.randn((1, Hk, cap, D), generator=g, device=DEV))
    k, v = (forms.values(*x).transpose(1, 2)[0, :Lk] for x in ((kc, kb), (vc, vb)))
    # a block of v of the first channels: codes of nothing but one infinity each
    want, lse_w, bound, lse_b = None, None, None, None
    odd = [(0, 1, 7), (1, 1, 15), (2, 2, 7), (17, 3, 15), (Lq // 2, D - 1, 7), (Lq - 1, D - 1, None)]
    clean = v.clone()
    marks = []
    for i, d, c in odd:  # as seen by query i and those behind it, in the last key/value head
        j = i + off
        if 0 <= j < Lk and i < Lq:
            b = d // 32
            vc[0, Hk - 1, j, 32 * b:32 * b + 32] = 0
            clean[j, Hk - 1, 32 * b:32 * b + 32] = 0
            if c is None:
                vb[0, Hk - 1, j, b] = 255
                marks.append((i, slice(32 * b, 32 * b + 32), float("nan")))
            else:
                vb[0, Hk - 1, j, b] = 254
                vc[0, Hk - 1, j, d] = c
                marks.append((i, d, inf if c == 7 else -inf))
    if Lk > Lq:  # a key that every query sees
        vb[0, 0, 0, 0], vc[0, 0, 0, :32], clean[0, 0, :32] = 254, 0, 0
        vc[0, 0, 0, 7] = 7
        marks.append((None, 7, inf))
    want, lse_w, bound, lse_b = _want(q[0], k, clean, 0.1)
    for i, d, x in marks:
        if i is None:
            want[:, :G, d] += x
        else:
            want[i:, Hq - G:, d] += x
    if off >= 0 and Lq > 20:  # a key nobody before its query sees
        kb[0, 0, 19 + off, 0] = 255
        want[19:, :G], lse_w[19:, :G] = float("nan"), float("nan")
    cache = forms.pack(kc, kb, D, False) + forms.pack(vc, vb, D, True)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse, k_lens=_ints([Lk]), part=part)
    check(out[0], want, bound, "out")
    check(lse[0], lse_w, lse_b, "lse")


def test_beyond_32_bit_offsets():
    g = _gen(7)
    S, Hk, cap, D, L = 3, 16, 1 << 22, 128, 70
    cache = kda.kda_cache4_empty(S, Hk, cap, D)
    k, v = _normal(g, S, L, Hk, D), _normal(g, S, L, Hk, D)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kda.kda_cache4_put(k, v, *cache, k_out=ko, v_out=vo)
    q = _normal(g, S, 1, Hk, D)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse, k_lens=_ints([L] * S))
    for n in range(S):
        _check_seq(out[n], lse[n], q[n], ko[n], vo[n], 0.1, "slot %d" % n)


def test_as_the_bf16_cache_of_the_same_values():
    """The two attentions over what is the same cache."""
    g = _gen(8)
    for Lq, D in ((1, 128), (9, 64), (140, 128)):
        Lk, Hq, Hk = 300, 8, 2
        k, v = _normal(g, 1, Lk, Hk, D), _normal(g, 1, Lk, Hk, D)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        cache = kda.kda_cache4_empty(1, Hk, 320, D)
        kda.kda_cache4_put(k, v, *cache, k_out=ko, v_out=vo)
        q = _normal(g, 1, Lq, Hq, D)
        a, b = torch.empty_like(q), torch.empty_like(q)
        kda.kda_attn4_fwd(q, *cache, 0.1, a, k_lens=_ints([Lk]))
        kda.kda_attn_fwd(q, ko, vo, 0.1, b)
        _check_seq(a[0], None, q[0], ko[0], vo[0], 0.1, "4 bits")
        _check_seq(b[0], None, q[0], ko[0], vo[0], 0.1, "bf16")


def test_capture_workspaces_and_streams():
    g = _gen(9)
    N, cap, Hq, Hk, D = 3, 928, 8, 2, 128
    x = []
    for lens in ([900, 3, 411], [1, 899, 0]):
        cache, _, _ = _cache(g, N, Hk, cap, D)
        x.append((_normal(g, N, 1, Hq, D), cache, _ints(lens)))
    want = []
    for q, c, n in x:
        out = torch.empty_like(q)
        kda.kda_attn4_fwd(q, *c, 0.1, out, k_lens=n, part=256)
        want.append(out)
    q, c, n = x[0]
    ws = torch.empty(kda.kda_attn4_workspace_bytes(N, N, 1, cap, Hq, Hk, D, 256),
                     dtype=torch.uint8, device=DEV)
    out, other = torch.empty_like(q), torch.empty_like(q)
    call = lambda s=None, w=ws: kda.kda_attn4_fwd(q, *c, 0.1, out, k_lens=n, part=256, workspace=w,
                                                  stream=s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        kda.kda_attn4_fwd(x[1][0], *x[1][1], 0.1, other, k_lens=x[1][2], part=256)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(other, want[1])
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side, None)
    kda.kda_attn4_fwd(x[1][0], *x[1][1], 0.1, other, k_lens=x[1][2], part=256)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(other, want[1])
