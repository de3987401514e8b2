"""The serving operators on the batches a server packs: many sequences, prompts beside single
tokens, and one sequence alone and among others, where the schedule and with it the roundings
are others.  Bounds: those of tests/test_gpu_attn.py and tests/test_gpu_la.py, which hold for
every schedule.
"""
from __future__ import annotations

import pytest
import torch

from tests.serving_forms import U16
from tests.test_gpu_attn import _packed
from tests.test_gpu_la import _compare, _inputs, _run
from tests.test_gpu_la import test_infinities_and_nan_reach_later_tokens_only as odd_values

pytestmark = pytest.mark.gpu


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
                   cu=torch.tensor([0, length], device="cuda"))
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
