"""64-bit definitions of the serving operators for the tests, with error bounds.

Each form returns, beside its value, a magnitude: the same sum with every term's absolute
value, which fp32 rounding errors are relative to.  U32 and U16 are the largest relative
errors of one rounding to fp32 and bf16.
"""
from __future__ import annotations

import torch

U32 = torch.finfo(torch.float32).eps / 2
U16 = torch.finfo(torch.bfloat16).eps / 2
TINY = 1e-37  # absolute: products below the fp32 normal range


def step(q, k, v, g, beta, scale, A_log, dt_bias, lb, S):
    """One KDA token: q, k, v, g [.., H, D], beta [.., H], S [.., H, V, K]; all fp64.
    Returns out, S', |out|, |S'|."""
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    lam = lb / (1 + torch.exp(-torch.exp(A_log)[:, None] * (g + dt_bias)))
    S = S * torch.exp(lam)[..., None, :]
    b = 1 / (1 + torch.exp(-beta))[..., None]
    p = (S * k[..., None, :]).sum(-1)
    p_abs = (S * k[..., None, :]).abs().sum(-1)
    new = S + (b * (v - p))[..., :, None] * k[..., None, :]
    mag = S.abs() + (b * (v.abs() + p_abs))[..., :, None] * k.abs()[..., None, :]
    out = scale * (new * q[..., None, :]).sum(-1)
    return out, new, abs(scale) * (mag * q.abs()[..., None, :]).sum(-1), mag


def la_step(q, k, v, lam, scale, S):
    """One token of linear attention: q, k [.., H, D] (already one per head), lam [.., H]."""
    S = S * torch.exp(lam)[..., None, None]
    add = v[..., :, None] * k[..., None, :]
    new, mag = S + add, S.abs() + add.abs()
    out = scale * (new * q[..., None, :]).sum(-1)
    return out, new, abs(scale) * (mag * q.abs()[..., None, :]).sum(-1), mag


def la_prompt(q, k, v, lam, scale, S):
    """A prompt token by token: q, k [T, H, D] (one per head), v [T, H, D], lam [T, H], S
    [H, V, K].  Returns out, S', |out|, |S'|."""
    out, mag = torch.zeros_like(v), torch.zeros_like(v)
    S, S_mag = S.clone(), S.abs()
    a = torch.exp(lam)
    for t in range(v.shape[0]):
        add = v[t][:, :, None] * k[t][:, None, :]
        S = S * a[t][:, None, None] + add
        S_mag = S_mag * a[t][:, None, None] + add.abs()
        out[t] = scale * (S @ q[t][:, :, None])[..., 0]
        mag[t] = abs(scale) * (S_mag @ q[t].abs()[:, :, None])[..., 0]
    return out, S, mag, S_mag


def check(got, want, bound, what):
    """Every element within its bound; NaN and infinities where they are wanted."""
    got, want = got.to(torch.float64), want.to(torch.float64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN elsewhere"
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), what
    err = (got - want).abs()[~odd]
    lim = bound.expand_as(want)[~odd]
    over = err > lim
    if over.any():
        worst = (err / lim.clamp(min=1e-300)).max()
        raise AssertionError("%s: %d of %d elements beyond the bound, the worst %.2f times"
                             % (what, int(over.sum()), err.numel(), float(worst)))
