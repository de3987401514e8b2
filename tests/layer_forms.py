"""64-bit definitions of the norms, rotary positions and 4-bit caches for the tests, with error
bounds beside the values where results are rounded.
"""
from __future__ import annotations

import torch

from tests.serving_forms import U16, U32

CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def norm(x, weight=None, eps=1e-6, post_weight=None, gate=None, gate_fn="sigmoid", residual=None,
         alpha=1.0, out_dtype_u=U16, res_u=0.0):
    """h, its bound, out, its bound; tensors of any dtype, computed in fp64.

    Bounds.  A sum of squares is a sum of positive terms over at most 46 additions in sequence
    (32 of a thread, 6 over a wave, 8 over waves) and one rounding each for square, division and
    the sum with eps, halved by the root, whose result is off by two more roundings: 27 U32 of
    the factor; two products follow: 29.  The gate: the exponent's product is off by 2 U32 of
    its size, |z| U32 after the exponential, which with sum and quotient adds 8; its product 2.
    The residual's multiply-add rounds once.  The second norm's factor moves by the first
    part's errors, at most by their L2 norm relative to the row's.
    """
    u = x.double()
    rel = torch.zeros_like(u)
    if post_weight is not None:
        t = u.unflatten(-1, (-1, post_weight.numel()))
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * post_weight.double()
        u = t.flatten(-2)
        rel = rel + 29 * U32
    if gate is not None:
        z = gate.double()
        s = 1 / (1 + torch.exp(-z))
        u = u * s * (z if gate_fn == "silu" else 1.0)
        rel = rel + (2 * z.abs() + 10) * U32
    err = rel * u.abs()
    h = u
    if residual is not None:
        h = residual.double() + alpha * u
        err = abs(alpha) * err + U32 * h.abs()
    out, out_err = h, err
    if weight is not None:
        f = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
        w = weight.double()
        out = h * f * w
        moved = err.norm(dim=-1, keepdim=True) / h.norm(dim=-1, keepdim=True).clamp(min=1e-300)
        out_err = (w * f).abs() * (err + h.abs() * (moved + 29 * U32))
    tiny = 1e-37
    return (h, err + res_u * (h.abs() + err) + tiny, out,
            out_err + out_dtype_u * (out.abs() + out_err) + tiny)


def rope(x, pos, freqs, amplitude=1.0, interleaved=False, inverse=False):
    """x [.., T, H, D] with pos [.., T]: the turned rows and their bound.

    The angle is a fraction of a turn in 64 bits, rounded to fp32 in half turns (at most 1: pi
    U32 / 2), cosine and sine are off by 4 U32 and the amplitude's product by one, each of the
    two products and their sum by one: 10 U32 of |a| + |b| in all, and the result's rounding.
    """
    half = freqs.numel()
    y = x.double()
    angle = pos.double()[..., None, None] * freqs * (-1 if inverse else 1)
    c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
    else:
        a, b = y[..., :half], y[..., half:2 * half]
    turned = (a * c - b * s, a * s + b * c)
    mag = abs(amplitude) * (a.abs() + b.abs())
    if interleaved:
        head, mag = torch.stack(turned, -1).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)
    else:
        head, mag = torch.cat(turned, -1), torch.cat((mag, mag), -1)
    bound = 10 * U32 * mag + U16 * (head.abs() + 10 * U32 * mag) + 1e-37
    rest = y[..., 2 * half:]
    return torch.cat((head, rest), -1), torch.cat((bound, torch.zeros_like(rest)), -1)


def quantise(x):
    """Blocks of 32 of x [.., D]: codes [.., D] (0 .. 15) and scale bytes [.., D / 32], int64, from
    the definition: the least power of two 2^e, e from -127, with max |x| <= 6 2^e; the nearest
    code, of two the even one; byte 255 and codes 0 for a block with infinities or NaN."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    odd = ~torch.isfinite(b).all(-1)
    top = torch.where(odd, 0.0, top)
    byte = torch.zeros(top.shape, dtype=torch.int64, device=x.device)
    for e in range(-127, 128):
        byte += top > 6 * 2.0 ** e
    y = b.abs() / torch.exp2(byte.double() - 127)[..., None]
    table = torch.tensor(CODES, dtype=torch.float64, device=x.device)
    code = torch.zeros(b.shape, dtype=torch.int64, device=x.device)
    for c in range(1, 8):  # the middle between two codes belongs to the even one
        mid = (table[c - 1] + table[c]) / 2
        code += (y >= mid) if c % 2 == 0 else (y > mid)
    code += 8 * torch.signbit(b)
    code = torch.where(odd[..., None], 0, code)
    return code.flatten(-2), torch.where(odd, 255, byte)


def values(code, byte):
    """What codes and scale bytes stand for, fp64; beyond bf16's range infinity."""
    table = torch.tensor(CODES + [-c for c in CODES], dtype=torch.float64, device=code.device)
    e = byte.double().repeat_interleave(32, -1)
    x = table[code.long()] * torch.exp2(e - 127)
    x = torch.where(x.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(x, torch.inf), x), x)
    return torch.where(e == 255, torch.nan, x)


def place(x):
    """Where position x of a tile of 32 keeps its scales."""
    return 8 * (x % 4) + 2 * (x // 4 % 4) + x // 16


def v_byte(x, pair, D):
    """The byte of position x, channels 2 pair and 2 pair + 1, in a tile of the values' codes."""
    j, i, g, d = x // 16, x // 4 % 4, x % 4, 2 * pair
    if D == 128:
        return 1024 * j + 256 * g + 16 * (d // 8) + 4 * i + d % 8 // 2
    return 256 * g + 16 * (d // 4) + 8 * j + 2 * i + d % 4 // 2


def pack(code, byte, D, v):
    """Codes [.., cap, D] and bytes [.., cap, D / 32] as a cache's two tensors (v: the values')."""
    cap = code.shape[-2]
    two = code[..., 0::2] + 16 * code[..., 1::2]
    x = torch.arange(32, device=code.device)
    b = byte.unflatten(-2, (cap // 32, 32)).transpose(-1, -2)  # tile, block, position
    scales = torch.empty_like(b)
    scales[..., place(x)] = b
    if v:
        t = two.unflatten(-2, (cap // 32, 32))
        at = v_byte(x[:, None], torch.arange(D // 2, device=code.device), D).flatten()
        two = torch.empty(t.shape[:-2] + (16 * D,), dtype=t.dtype, device=t.device)
        two[..., at] = t.flatten(-2)
    return two.to(torch.uint8).contiguous(), scales.to(torch.uint8).contiguous()


def unpack(codes, scales, D, v):
    """The way back: codes [.., cap, D], bytes [.., cap, D / 32]."""
    x = torch.arange(32, device=codes.device)
    byte = scales[..., place(x)].transpose(-1, -2).flatten(-3, -2)
    if v:
        at = v_byte(x[:, None], torch.arange(D // 2, device=codes.device), D).flatten()
        codes = codes[..., at].unflatten(-1, (32, D // 2)).flatten(-3, -2)
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long(), byte.long()
