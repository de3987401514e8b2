"""Causal softmax attention with grouped heads (kda_attn_fwd) against its 64-bit definition.

Bounds.  A score is a sum of D products in fp32, off by at most (D + 8) U32 of the sum of
their absolute values (scaling and the subtraction of the maximum included); that, and four
roundings of the exponential, is the relative error of its probability.  Probabilities are
rounded to bf16 for the product with v (U16 of each term), the sums over L keys are off by at
most L U32 of the sums of absolute values, and out is rounded to bf16.  lse: the scores'
error, the sum's, and a few roundings of the result.
"""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.serving_forms as forms
from tests.serving_forms import U16, U32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _want(q, k, v, scale):
    """One sequence: q [Lq, Hq, D], k, v [Lk, Hk, D].  out, lse and their bounds."""
    Lq, Hq, D = q.shape
    Lk, Hk = k.shape[:2]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    k, v = k.repeat_interleave(Hq // Hk, 0), v.repeat_interleave(Hq // Hk, 0)
    x = scale * (q @ k.transpose(1, 2))
    x_mag = scale * (q.abs() @ k.abs().transpose(1, 2))
    seen = (torch.arange(Lk, device=DEV)[None, :]
            <= torch.arange(Lq, device=DEV)[:, None] + (Lk - Lq))
    x = x.masked_fill(~seen, -math.inf)
    if Lk == 0:
        zero = torch.zeros((Lq, Hq, D), dtype=torch.float64, device=DEV)
        none = torch.full((Lq, Hq), -math.inf, dtype=torch.float64, device=DEV)
        return zero, none, zero, torch.zeros_like(none)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    d = ((D + 8) * U32 * x_mag.masked_fill(~seen, 0.0)).amax(-1) + 4 * U32
    out = p @ v
    bound = (U16 + 2 * d + (Lk + 64) * U32)[..., None] * (p @ v.abs()) + U16 * out.abs() + 1e-30
    lse_bound = d + (Lk + 8) * U32 + 8 * U32 * torch.where(lse == -math.inf, 0.0, lse.abs())
    return (out.transpose(0, 1), lse.transpose(0, 1), bound.transpose(0, 1),
            lse_bound.transpose(0, 1))


def _check_seq(out, lse, q, k, v, scale, what):
    o, z, ob, zb = _want(q, k, v, scale)
    forms.check(out, o, ob, what + ", out")
    forms.check(lse, z, zb, what + ", lse")


def _packed(seed, ql, kl, Hq, Hk, D, scale=None, behind=0, **more):
    """Packed queries and keys, views of wider rows; `behind` query rows after the last."""
    g = _gen(seed)
    scale = D ** -0.5 if scale is None else scale
    q, _ = torch.split(_normal(g, 1, sum(ql) + behind, Hq + Hk, D), [Hq, Hk], dim=2)
    k, v = torch.split(_normal(g, 1, sum(kl), 2 * Hk, D), [Hk, Hk], dim=2)
    cu = [torch.tensor([0] + x, dtype=torch.int64).cumsum(0).to(DEV) for x in (ql, kl)]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    kda.kda_attn_fwd(q, k, v, scale, out, lse=lse, cu_seqlens_q=cu[0], cu_seqlens_k=cu[1], **more)
    a = b = 0
    for n, (lq, lk) in enumerate(zip(ql, kl)):
        _check_seq(out[0, a:a + lq], lse[0, a:a + lq], q[0, a:a + lq], k[0, b:b + lk],
                   v[0, b:b + lk], scale, "sequence %d (%d, %d)" % (n, lq, lk))
        a, b = a + lq, b + lk
    assert (out[0, a:] == 7.0).all() and (lse[0, a:] == 7.0).all()
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,Hq,Hk", [
    ([1], [1], 1, 1), ([5], [5], 3, 1), ([128], [128], 4, 4), ([65, 0, 1, 200], [65, 0, 1, 200], 6, 2),
    ([300, 33], [700, 33], 12, 1), ([100, 64, 20], [0, 10, 20], 8, 2), ([129], [2000], 2, 2),
    ([1, 1, 1], [5, 0, 900], 24, 2), ([9, 2, 17], [1000, 64, 17], 4, 4), ([700], [701], 5, 5)])
def test_packed(ql, kl, Hq, Hk, D):
    print("kda_attn_fwd packed", ql, kl, Hq, Hk, D, flush=True)
    _packed(len(ql) * 31 + Hq, ql, kl, Hq, Hk, D)


@pytest.mark.parametrize("ql,kl,Hq,Hk,splits", [
    ([1, 1], [700, 3], 8, 2, 3), ([2, 0, 3], [64, 5, 1000], 12, 4, 64), ([40, 9], [500, 9], 2, 1, 5),
    ([300], [1500], 4, 2, 4), ([200, 70], [10, 333], 2, 2, 2), ([1], [0], 2, 2, 2)])
def test_splits(ql, kl, Hq, Hk, splits):
    """Parts of the keys, empty ones among them; rows behind the last sequence stay."""
    print("kda_attn_fwd splits", ql, kl, Hq, Hk, splits, flush=True)
    _packed(splits, ql, kl, Hq, Hk, 128, behind=3, splits=splits)
    _packed(splits, ql, kl, Hq, Hk, 64, behind=70, splits=splits)


@pytest.mark.parametrize("Tq,Hq,Hk,D", [(1, 8, 2, 128), (1, 3, 3, 64), (1, 32, 1, 128),
                                        (4, 12, 2, 64), (5, 24, 2, 128), (30, 4, 1, 128)])
def test_caches(Tq, Hq, Hk, D):
    """Rows of a cache filled to different lengths; what lies behind them is never used."""
    print("kda_attn_fwd caches", Tq, Hq, Hk, D, flush=True)
    g = _gen(Tq * Hq)
    lens = [1, 0, 31, 32, 33, 200, 511, 700]
    N, cap = len(lens), 700
    q = _normal(g, N, Tq, Hq, D)
    k, v = _normal(g, N, cap, Hk, D), _normal(g, N, cap, Hk, D)
    for n, length in enumerate(lens):
        k[n, length:] = float("nan")
        v[n, length:] = float("inf")
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.2, out, lse=lse, k_lens=torch.tensor(lens, device=DEV))
    for n, length in enumerate(lens):
        _check_seq(out[n], lse[n], q[n], k[n, :length], v[n, :length], 0.2, "row %d" % n)
    # lengths outside the cache are clamped into it
    out2 = torch.empty_like(out)
    wild = torch.tensor([-5, 1 << 40] * (N // 2), device=DEV)
    k2, v2 = k.nan_to_num(0.0, 0.0, 0.0), v.nan_to_num(0.0, 0.0, 0.0)
    kda.kda_attn_fwd(q, k2, v2, 0.2, out2, k_lens=wild)
    assert (out2[0] == 0).all()
    o, _, ob, _ = _want(q[1], k2[1], v2[1], 0.2)
    forms.check(out2[1], o, ob, "clamped row")


def test_batched_prompts_and_all_keys():
    g = _gen(4)
    q, k, v = _normal(g, 2, 150, 6, 64), _normal(g, 2, 170, 3, 64), _normal(g, 2, 170, 3, 64)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.0, out, lse=lse)  # scale zero: the mean of the visible keys
    for n in range(2):
        _check_seq(out[n], lse[n], q[n], k[n], v[n], 0.0, "row %d" % n)


def test_large_and_growing_scores():
    """Scores of a few hundred, growing along the keys, so the running maximum is raised
    often; and scores that fall, so it never is again."""
    g = _gen(5)
    L, H, D = 600, 2, 128
    for sign in (1, -1):
        q, k, v = _normal(g, 1, L, H, D), _normal(g, 1, L, H, D), _normal(g, 1, L, H, D)
        q[..., 0] = 30.0
        k[0, :, :, 0] = (sign * torch.linspace(-100, 100, L, device=DEV)).to(torch.bfloat16)[:, None]
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse)
        _check_seq(out[0], lse[0], q[0], k[0], v[0], 0.1, "sign %d" % sign)


def test_caches_beyond_32_bit_offsets():
    """Cache rows more than 2^32 bytes apart."""
    g = _gen(6)
    N, cap, Hk, D, L = 3, 1 << 19, 16, 128, 100
    k = torch.empty((N, cap, Hk, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    q = _normal(g, N, 1, Hk, D)
    k[:, :L], v[:, :L] = _normal(g, N, L, Hk, D), _normal(g, N, L, Hk, D)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse, k_lens=torch.full((N,), L, device=DEV))
    for n in range(N):
        _check_seq(out[n], lse[n], q[n], k[n, :L], v[n, :L], 0.1, "row %d" % n)


def test_long_caches_in_the_automatic_parts():
    """Lengths that the library splits by itself, odd ones, packed and as cache rows."""
    assert kda.kda_attn_workspace_bytes(1, 1, 3, 1, 20001, 6, 2, 128) > 0
    _packed(61, [3], [20001], 6, 2, 128)
    _packed(62, [150], [5003], 4, 1, 64)


def test_nan_stays_in_its_head():
    g = _gen(7)
    q, k, v = (_normal(g, 1, 90, 4, 64) for _ in range(3))
    q[0, 40, 1, 3] = float("nan")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, k, v, 0.1, out, lse=lse)
    want = torch.zeros((90, 4), dtype=torch.bool, device=DEV)
    want[40, 1] = True
    assert torch.equal(torch.isnan(lse[0]), want)
    assert torch.equal(torch.isnan(out[0]).all(-1), want)
    assert torch.equal(torch.isnan(out[0]).any(-1), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Lk,Hq,Hk,splits", [
    (1, 700, 8, 2, 0), (4, 100, 8, 2, 0), (4, 100, 8, 2, 3), (40, 500, 2, 1, 1), (200, 200, 2, 2, 0),
    (300, 333, 4, 2, 3), (150, 130, 12, 1, 0)])
def test_infinities_and_nan_behind_the_last_visible_key(Lq, Lk, Hq, Hk, splits, D):
    """Infinities and NaN in k and v reach the queries that see them, and nothing else."""
    print("kda_attn_fwd odd v", Lq, Lk, Hq, Hk, splits, D, flush=True)
    g = _gen(Lk + D)
    q, k, v = _normal(g, 1, Lq, Hq, D), _normal(g, 1, Lk, Hk, D), _normal(g, 1, Lk, Hk, D)
    inf, off = float("inf"), Lk - Lq
    want, lse_w, bound, lse_b = _want(q[0], k[0], v[0], 0.1)
    odd, bad = [(0, 1, inf), (1, 1, -inf), (2, 2, inf), (17, 3, -inf), (Lq // 2, D - 1, inf),
                (Lq - 1, 40, float("nan")), (Lq - 1, 41, -inf)], v.clone()
    for i, d, x in odd:  # as seen by query i and those behind it, in the last key/value head
        if 0 <= i + off < Lk and i < Lq:
            bad[0, i + off, Hk - 1, d] = x
            want[i:, Hq - Hq // Hk:, d] += x
    if Lk > Lq:
        bad[0, 0, 0, 7] = inf  # a key that every query sees
        want[:, :Hq // Hk, 7] += inf
    kq, G = k.clone(), Hq // Hk
    if off >= 0 and Lq > 20:  # a key nobody before its query sees
        kq[0, 19 + off, 0] = float("nan")
        want[19:, :G], lse_w[19:, :G] = float("nan"), float("nan")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kda.kda_attn_fwd(q, kq, bad, 0.1, out, lse=lse, splits=splits)
    forms.check(out[0], want, bound, "out")
    forms.check(lse[0], lse_w, lse_b, "lse")


def test_prompt_then_tokens():
    """A prompt's attention, then tokens over the cache it filled: rows of one longer prompt."""
    g = _gen(8)
    T, more, Hq, Hk, D = 140, 3, 8, 2, 128
    q, k, v = _normal(g, 1, T + more, Hq, D), _normal(g, 1, T + more, Hk, D), \
        _normal(g, 1, T + more, Hk, D)
    out = torch.empty_like(q)
    kda.kda_attn_fwd(q, k, v, 0.1, out)
    for t in range(T, T + more):
        one = torch.empty((1, 1, Hq, D), dtype=torch.bfloat16, device=DEV)
        kda.kda_attn_fwd(q[:, t:t + 1], k, v, 0.1, one,
                         k_lens=torch.tensor([t + 1], device=DEV))
        err = float((one[0, 0].double() - out[0, t].double()).norm() / out[0, t].double().norm())
        assert err <= 4 * U16, err  # two roundings on each side


def test_capture_and_streams():
    g = _gen(9)
    N, cap, Hq, Hk, D = 3, 900, 8, 2, 128
    x = [(_normal(g, N, 1, Hq, D), _normal(g, N, cap, Hk, D), _normal(g, N, cap, Hk, D),
          torch.tensor(lens, device=DEV)) for lens in ([900, 3, 411], [1, 899, 0])]
    want = []
    for q, k, v, n in x:
        out = torch.empty_like(q)
        kda.kda_attn_fwd(q, k, v, 0.1, out, k_lens=n, splits=4)
        want.append(out)
    q, k, v, n = x[0]
    ws = torch.empty(kda.kda_attn_workspace_bytes(N, N, 1, N, cap, Hq, Hk, D, 4),
                     dtype=torch.uint8, device=DEV)
    out, other = torch.empty_like(q), torch.empty_like(q)
    call = lambda s=None, w=ws: kda.kda_attn_fwd(q, k, v, 0.1, out, k_lens=n, splits=4,
                                                 workspace=w, stream=s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        kda.kda_attn_fwd(x[1][0], x[1][1], x[1][2], 0.1, other, k_lens=x[1][3], splits=4)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(other, want[1])
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side, None)
    kda.kda_attn_fwd(x[1][0], x[1][1], x[1][2], 0.1, other, k_lens=x[1][3], splits=4)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(other, want[1])
