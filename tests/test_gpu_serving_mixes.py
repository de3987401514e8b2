"""The serving operators on the batches a server packs: many sequences, prompts beside single
tokens, and one sequence alone and among others, where the schedule and with it the roundings
are others.  Bounds: those of tests/test_gpu_attn.py and tests/test_gpu_la.py, which hold for
every schedule.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
from tests.serving_forms import U16
from tests.test_gpu_attn import _check_seq, _gen, _normal, _packed
from tests.test_gpu_la import _compare, _inputs, _run
from tests.test_gpu_la import test_infinities_and_nan_reach_later_tokens_only as odd_values

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _lengths(n, most, seed):
    """n lengths from 0 to most, of the kinds that end tiles in different places."""
    g = torch.Generator().manual_seed(seed)
    kinds = [0, 1, 63, 64, 65, 127, 128, 129, most]
    return [kinds[i] if i < len(kinds) else int(torch.randint(0, most + 1, (1,), generator=g))
            for i in torch.randperm(n, generator=g).tolist()]


@pytest.mark.parametrize("n,Hq,Hk,D,splits", [(17, 4, 2, 128, 0), (40, 6, 2, 64, 0),
                                              (17, 3, 3, 64, 3), (40, 4, 1, 128, 2)])
def test_many_packed_prompts(n, Hq, Hk, D, splits):
    """More sequences than are ranked by length, over keys of their own and earlier ones, fewer
    keys than queries among them."""
    print("kda_attn_fwd many", n, Hq, Hk, D, splits, flush=True)
    ql = _lengths(n, 210, n)
    more = _lengths(n, 260, n + 1)
    kl = [max(0, q + m - 90) if i % 3 == 0 else q + m if i % 3 == 1 else q
          for i, (q, m) in enumerate(zip(ql, more))]
    assert sum(ql) * (Hq // Hk) > 64 * n  # tiles of rows, not the kernel for few
    assert any(k < q for q, k in zip(ql, kl)) and 0 in ql
    _packed(n, ql, kl, Hq, Hk, D, behind=5, splits=splits)


@pytest.mark.parametrize("ql,Hq,Hk,D", [
    ([2000] + [1] * 63, 8, 2, 128), ([1] * 30 + [900] + [1] * 30, 4, 4, 64),
    ([1] * 100 + [1000] + [1] * 156, 8, 2, 64), ([4] * 20 + [300] + [1] * 90, 4, 1, 128)])
def test_prompts_beside_single_tokens(ql, Hq, Hk, D):
    """The mean decides the kernel: single tokens in the prompts' one, a prompt in theirs."""
    print("kda_attn_fwd mixed", len(ql), Hq, Hk, D, flush=True)
    g = torch.Generator().manual_seed(len(ql))
    kl = [q + int(torch.randint(0, 300, (1,), generator=g)) if q < 10 else q for q in ql]
    _packed(len(ql), ql, kl, Hq, Hk, D)


@pytest.mark.parametrize("ql,Hq,Hk,D,splits", [
    ([1, 5, 0, 2], 8, 2, 128, 0), ([70, 1, 0, 200, 129], 4, 2, 64, 0),
    ([1] * 9 + [30] * 11, 6, 1, 64, 3), ([90] * 18, 2, 2, 128, 2)])
def test_packed_queries_over_caches(ql, Hq, Hk, D, splits):
    """Packed queries, keys in rows of a cache filled to different lengths; NaN behind them."""
    print("kda_attn_fwd packed over caches", ql, Hq, Hk, D, splits, flush=True)
    g, N, cap = _gen(len(ql) + D), len(ql), 333
    lens = [(q + 61 * n) % (cap + 1) for n, q in enumerate(ql)]
    q = _normal(g, 1, sum(ql) + 2, Hq, D)
    k, v = torch.split(_normal(g, N, cap, 2 * Hk, D), [Hk, Hk], dim=2)
    for n, length in enumerate(lens):
        k[n, length:], v[n, length:] = float("nan"), float("nan")
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, splits=splits,
                     k_lens=torch.tensor(lens, device=DEV),
                     cu_seqlens_q=torch.tensor([0] + ql).cumsum(0).to(DEV))
    at = 0
    for n, (length, lk) in enumerate(zip(ql, lens)):
        s = slice(at, at + length)
        _check_seq(out[0, s], lse[0, s], q[0, s], k[n, :lk], v[n, :lk], 0.1, "sequence %d" % n)
        at += length
    assert (out[0, at:] == 7.0).all() and (lse[0, at:] == 7.0).all()


@pytest.mark.parametrize("Tq,kl,Hq,Hk,D", [(1, [5, 0, 400, 33], 8, 2, 64),
                                           (150, [150, 20, 700], 4, 4, 128)])
def test_rows_of_queries_over_packed_keys(Tq, kl, Hq, Hk, D):
    """Queries as batch rows, keys packed."""
    print("kda_attn_fwd rows over packed keys", Tq, kl, Hq, Hk, D, flush=True)
    g, N = _gen(Tq), len(kl)
    q = _normal(g, N, Tq, Hq, D)
    k, v = _normal(g, 1, sum(kl), Hk, D), _normal(g, 1, sum(kl), Hk, D)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse,
                     cu_seqlens_k=torch.tensor([0] + kl).cumsum(0).to(DEV))
    at = 0
    for n, lk in enumerate(kl):
        s = slice(at, at + lk)
        _check_seq(out[n], lse[n], q[n], k[0, s], v[0, s], 0.1, "sequence %d" % n)
        at += lk


@pytest.mark.parametrize("segment", [0, 64])
def test_no_tokens(segment):
    """A packed batch without a token passes its states through, in segments too."""
    H, D = 3, 32
    x = _inputs(54, [0, 0], H, H, D)
    out, final = _run(x, 1.0, segment=segment)
    assert out.numel() == 0 and torch.equal(final, x["initial"])


@pytest.mark.parametrize("D", [32, 64, 128])
def test_one_prompt_alone_and_packed(D):
    """Few tokens carry second bf16 parts, more do not; a final state's type, or having none,
    decides the parts of its update.  Each is within the bound, and the two of one prompt
    within both."""
    lens, H, Hk, scale = [300, 400, 65, 130], 4, 2, D ** -0.5
    x = _inputs(51, lens, H, Hk, D)
    out, final = _run(x, scale)
    _compare(x, scale, out, final)
    at = 0
    for n, length in enumerate(lens):
        one = {k: t[:, at:at + length] for k, t in x.items() if k in "qkv"}
        one.update(g=x["g"][:, at:at + length].contiguous(), decay=x["decay"],
                   initial=x["initial"][n:n + 1], lens=[length],
                   cu=torch.tensor([0, length], device=DEV))
        for out_state in (torch.float32, torch.bfloat16):
            alone, state = _run(one, scale, out_state)
            _compare(one, scale, alone, state)
            got, ref = alone[0].double(), out[0, at:at + length].double()
            # three roundings to bf16 on either side at most: scores, state operand, result
            assert float((got - ref).norm() / ref.norm()) <= 6 * U16
        at += length


@pytest.mark.parametrize("D", [32, 64])
def test_odd_values_without_second_parts(D):
    assert 700 * 6 > 2048
    odd_values([700], 6, 3, D, 0)


def test_bounds_hold_where_values_cancel():
    """The roundings inside are relative to the sum of the terms' absolute values, not to the
    result: values of alternating sign whose weighted sum is far below them."""
    x = _inputs(53, [900], 4, 4, 64, gate="head")
    x["v"] = x["v"].abs()
    x["v"][:, 1::2] *= -1
    out, final = _run(x, 0.125)
    _compare(x, 0.125, out, final)
