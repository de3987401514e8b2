"""Joins of kda_attn_fwd's splits, bit for bit: the digests are those of the first version of the
join, on inputs of integer arithmetic.

A row's normaliser is the sum over the lanes of a wave, each lane's first addition fused with its
own product, so that lanes may differ in its last bit: the order of the additions is part of the
result.
"""
from __future__ import annotations

import hashlib

import pytest
import torch

import gated_delta_rule_62_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"

# Hq, Hk, D, sequences, queries and keys of each, splits, packed queries -> out, lse
CASES = [
    ((8, 2, 64, 3, 40, 1500, 33, True), "267eb15d9a6be959", "5fdef0fcf73e6ef4"),
    ((12, 1, 64, 3, 40, 1500, 64, False), "181a987cc83635e7", "6abd117195624fea"),
    ((3, 3, 64, 3, 5, 1500, 7, True), "e2ee39844a25eada", "e0a84a74bd16f769"),
    ((8, 2, 128, 3, 40, 1500, 33, False), "96efc581e2c4ff52", "d3cde0d5c31fc942"),
    ((12, 1, 128, 1, 40, 1500, 64, True), "424e782b287e67f7", "e51a024ade86fdc8"),
    ((32, 8, 128, 1, 256, 4096, 0, False), "6a99a159bc495861", "b18f9e03c3feba90"),
]


def inputs(case):
    Hq, Hk, D, N, Tq, Tk, splits, packed = case

    def values(seed, *shape):
        n = torch.Size(shape).numel()
        i = (torch.arange(n, dtype=torch.int64) + seed) * 1103515245 % (1 << 31)
        i = (i ^ i >> 11) * 12345679 % (1 << 31)
        return ((i >> 9) % 4001 - 2000).float().div(800).to(torch.bfloat16).view(shape).to(DEV)

    q = values(1, *((1, N * Tq) if packed else (N, Tq)), Hq, D)
    k, v = values(7, N, Tk, Hk, D), values(13, N, Tk, Hk, D)
    lens = torch.tensor([Tk - 37 * n for n in range(N)], dtype=torch.int64, device=DEV)
    cu = torch.arange(N + 1, dtype=torch.int64, device=DEV) * Tq if packed else None
    return q, k, v, lens, cu


def digest(t):
    raw = t.contiguous().view(torch.uint8).cpu().numpy().tobytes()
    return hashlib.sha256(raw).hexdigest()[:16]


@pytest.mark.parametrize("case,out_digest,lse_digest", CASES)
def test_the_joins_bits(case, out_digest, lse_digest):
    print("kda_attn_fwd joins", case, flush=True)
    q, k, v, lens, cu = inputs(case)
    splits = case[6]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    if splits == 0:
        N, Tq, Tk, Hq, Hk, D = case[3], case[4], case[5], case[0], case[1], case[2]
        assert kda.kda_attn_workspace_bytes(N, N, Tq, N, Tk, Hq, Hk, D) > 0
    kda.kda_attn_fwd(q, k, v, 0.08, out, lse=lse, cu_seqlens_q=cu, k_lens=lens, splits=splits)
    assert (digest(out), digest(lse)) == (out_digest, lse_digest)
