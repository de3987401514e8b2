"""kda_attn_fwd at scale zero and at scales far below one, with scores that are large before
them: the scaled scores are ordinary numbers.

Bounds: those of tests/test_gpu_attn.py.  Beyond them a scale whose product with log2(e) is
below the fp32 normal range is rounded to a step of 2^-149, and zero is taken as one step: a
finite score (below 2^128) moves by at most ln 2 2^-21 for that, 3.3e-7 or six fp32
roundings of a weight, of which the bounds count 64 and more.
"""
from __future__ import annotations

import struct

import pytest
import torch

import gated_delta_rule_62_amd as kda
from tests.test_gpu_attn import _check_seq, _gen, _normal

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Lq,Lk,Hq,Hk,D,splits", [(1, 300, 4, 2, 64, 1), (3, 500, 8, 2, 128, 4),
                                                  (200, 260, 4, 2, 128, 1), (150, 150, 2, 2, 64, 2)])
@pytest.mark.parametrize("scale,power", [(0.0, 17), (0.0, 0), (1e-34, 17), (1e-31, 15), (3e-36, 18),
                                         (1e-40, 18)])
def test_large_scores_small_scales(scale, power, Lq, Lk, Hq, Hk, D, splits):
    print("kda_attn_fwd scale", scale, power, Lq, Lk, Hq, Hk, D, splits, flush=True)
    scale = struct.unpack("f", struct.pack("f", scale))[0]
    g = _gen(40 + Lk)
    # one product of q and k dominates: scores of about 10^(2 power)
    q, k, v = _normal(g, 1, Lq, Hq, D), _normal(g, 1, Lk, Hk, D), _normal(g, 1, Lk, Hk, D)
    q[..., 5] = (q[..., 5].float() * 10.0 ** power).bfloat16()
    k[..., 5] = (k[..., 5].float() * 10.0 ** power).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, k, v, scale, out, lse=lse, splits=splits)
    _check_seq(out[0], lse[0], q[0], k[0], v[0], scale, "scale %g" % scale)
