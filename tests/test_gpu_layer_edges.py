"""Calls of the operators over 4-bit caches that their documentation allows at its edges: tokens in
front of the first sequence, one slot filled by two sequences, an expanding call in a graph whose
lengths change between replays, and expanded caches beyond 32-bit offsets.  Bounds as in
tests/test_gpu_attn4.py.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms
from tests.test_gpu_attn4 import BF16, DEV, _cache, _check_seq, _gen, _ints, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ql,kl,Hq,Hk,D,cap,part", [
    ([1, 5], [40, 300], 8, 2, 128, 320, 0), ([3, 0, 2], [200, 9, 64], 12, 4, 64, 224, 64),
    ([700, 500], [700, 900], 16, 2, 128, 928, 0)])
def test_tokens_in_front_of_the_first_sequence(ql, kl, Hq, Hk, D, cap, part):
    print("kda_attn4_fwd front", ql, kl, Hq, Hk, D, cap, part, flush=True)
    front, behind, N = 37, 3, len(ql)
    g = _gen(cap + part)
    cache, k, v = _cache(g, N, Hk, cap, D, kl)
    q = _normal(g, 1, front + sum(ql) + behind, Hq, D)
    out = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse, k_lens=_ints(kl),
                      cu_seqlens_q=_ints([front] + ql).cumsum(0), part=part)
    at = front
    for n, (lq, lk) in enumerate(zip(ql, kl)):
        _check_seq(out[0, at:at + lq], lse[0, at:at + lq], q[0, at:at + lq], k[n, :lk], v[n, :lk],
                   0.1, "sequence %d" % n)
        at += lq
    for x in (out, lse):
        assert (x[0, :front] == 7.0).all() and (x[0, at:] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_two_sequences_fill_one_slot(D):
    """Their positions lie in the same tiles but do not meet: it is the cache of both in one."""
    print("kda_cache4_put two sequences, one slot", D, flush=True)
    g = _gen(D)
    Hk, cap, cut, L = 3, 96, 37, 71
    k, v = _normal(g, 1, L, Hk, D), _normal(g, 1, L, Hk, D)
    one, two = kda.kda_cache4_empty(2, Hk, cap, D), kda.kda_cache4_empty(2, Hk, cap, D)
    kda.kda_cache4_put(k, v, *one, cu_seqlens=_ints([0, L]), slots=_ints([1]))
    kda.kda_cache4_put(k, v, *two, offsets=_ints([0, cut]), cu_seqlens=_ints([0, cut, L]),
                       slots=_ints([1, 1]))
    for a, b in zip(one, two):
        assert torch.equal(a, b)


def test_an_expanding_call_replayed_with_other_lengths():
    print("kda_attn4_fwd expanding replays", flush=True)
    g = _gen(12)
    ql, Hq, Hk, D, cap = [700, 500], 16, 2, 128, 928
    cache, k, v = _cache(g, 2, Hk, cap, D)
    q = _normal(g, 1, sum(ql), Hq, D)
    lens, cu = _ints([700, 900]), _ints([0] + ql).cumsum(0)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    need = kda.kda_attn4_workspace_bytes(2, 1, sum(ql), cap, Hq, Hk, D)
    assert need >= 2 * cap * Hk * D * 4
    call = lambda: kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse, k_lens=lens, cu_seqlens_q=cu)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for kl in ([700, 900], [928, 1], [0, 928], [450, 450]):
        lens.copy_(_ints(kl))
        out.zero_()
        graph.replay()
        at = 0
        for n, (lq, lk) in enumerate(zip(ql, kl)):
            _check_seq(out[0, at:at + lq], lse[0, at:at + lq], q[0, at:at + lq], k[n, :lk],
                       v[n, :lk], 0.1, "lengths %s, sequence %d" % (kl, n))
            at += lq
        replayed = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)


def test_expanded_caches_beyond_32_bit_offsets():
    """4 GiB of keys and of values in bf16; the second sequence's lie behind 2 GiB of both."""
    print("kda_attn4_fwd 8 GiB expanded", flush=True)
    g = _gen(13)
    N, Tq, H, D, cap, L = 2, 1600, 8, 128, 1 << 20, 400
    assert kda.kda_attn4_workspace_bytes(N, N, Tq, cap, H, H, D) >= 8 << 30
    cache = kda.kda_cache4_empty(N, H, cap, D)
    ends = [cap, cap - 33]
    k, v = _normal(g, N, L, H, D), _normal(g, N, L, H, D)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kda.kda_cache4_put(k, v, *cache, offsets=_ints([e - L for e in ends]), k_out=ko, v_out=vo)
    # what lies in front scores minus a large number: its keys are -8 times the query's direction
    q = _normal(g, N, Tq, H, D)
    q[..., 0] = 20.0
    code = torch.zeros((1, 1, 32, D), dtype=torch.int64, device=DEV)
    code[..., 0] = 15
    byte = torch.full((1, 1, 32, D // 32), 130, dtype=torch.int64, device=DEV)
    far, far_s = forms.pack(code, byte, D, False)
    for n, e in enumerate(ends):
        tiles = (e - L) // 32
        cache[0][n, :, :32 * tiles] = far[0].repeat(1, tiles, 1)
        cache[1][n, :, :tiles] = far_s[0]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn4_fwd(q, *cache, 0.1, out, lse=lse, k_lens=_ints(ends))
    for n, e in enumerate(ends):
        front = (e - L) // 32 * 32
        edge = e - L - front  # positions of the mixed tile that hold zeros
        keys = torch.cat((torch.zeros((edge, H, D), dtype=BF16, device=DEV), ko[n]))
        vals = torch.cat((torch.zeros((edge, H, D), dtype=BF16, device=DEV), vo[n]))
        # queries that see all of the last L keys but the diagonal's: the last L of them
        some = slice(Tq - L // 2, Tq)
        _check_seq(out[n, some], lse[n, some], q[n, some], keys, vals, 0.1, "sequence %d" % n)
