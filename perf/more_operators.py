"""The operators around the serving operators' attention and states, as cases that can be timed
and compared.

Four operators that a layer of the same hybrid model calls beside its projections:

  norm   kda_norm: the norms before and after a block, with its output gate, the residual sum and
         its scale, in one pass over the rows
  rope   kda_rope: rotary positions of queries and keys
  put    kda_cache4_put: new keys and values into caches held in 4 bits (blocks of 32 values that
         share a power of two)
  attn4  kda_attn4_fwd: causal softmax attention with grouped heads over such caches

``run`` computes them with elementary torch operations in 32 bits (angles in 64), or where ``own``
is true calls the library.  ``exact`` evaluates the definitions in 64 bits.

A cache: slots of Hk heads of `cap` positions, a multiple of 32.  The codes are the sixteen values
0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives; position p sits in tile p // 32 at place x = p % 32 =
16 j + 4 i + g, and value d in block d // 32.
  scales  uint8 [slots, Hk, cap / 32, D / 32, 32]   the power's exponent + 127, at 8 g + 2 i + j
                                                    (255: the block stands for NaN)
  keys    uint8 [slots, Hk, cap, D / 2]             two codes a byte, the even value's low
  values  uint8 [slots, Hk, cap / 32, 16 D]         D 128: [j][g][d // 8][i][d % 8 / 2]
                                                    D  64: [g][d // 4][j][i][d % 4 / 2]
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # four requests' single tokens between two blocks: residual sum and the next norm, latency
        dict(name="norm-token", op="norm", R=4, W=4096, post=0, gate="", res="bf16", alpha=1.0,
             pre=True, wtype="bf16", fused=False),
        # a KDA layer's output in the benchmark's batched prefill, 96 heads: each head normalised
        # and gated, the gate a part of wider projection rows
        dict(name="norm-heads", op="norm", R=2048, W=12288, post=128, gate="sigmoid", res="",
             alpha=1.0, pre=False, wtype="fp32", fused=True),
        # between two blocks of a long document: the norm behind the block, its gate, the residual
        # stream in fp32 with a scaled sum, the norm before the next block
        dict(name="norm-block", op="norm", R=8192, W=4096, post=4096, gate="silu", res="fp32",
             alpha=0.5, pre=True, wtype="bf16", fused=False),
        # one token of two chat requests
        dict(name="rope-token", op="rope", N=2, T=1, lens="", start="200,77", Hq=16, Hk=4, D=64,
             rot=64, interleaved=False, method="", factor=1.0, inverse=False, fused=False),
        # the packed batch [300, 700, 1024] behind earlier tokens, views of projections' rows
        dict(name="rope-packed", op="rope", N=3, T=0, lens="300,700,1024", start="0,1500,77",
             Hq=96, Hk=8, D=128, rot=128, interleaved=False, method="", factor=1.0, inverse=False,
             fused=True),
        # a part of a document far behind its start: half of each head turned, pairs side by side,
        # frequencies scaled for long contexts
        dict(name="rope-far", op="rope", N=1, T=8192, lens="", start="1040000", Hq=32, Hk=8,
             D=128, rot=64, interleaved=True, method="yarn", factor=32.0, inverse=False,
             fused=False),
        # a serving batch's new keys and values
        dict(name="put-tokens", op="put", N=32, lens="", T=1, start="spread", slots=32, cap=8192,
             Hk=8, D=128, values=False, shuffle=False, fused=False),
        # prompts [300, 700, 1024], two of them behind earlier positions, with the values that the
        # cache then stands for
        dict(name="put-prompts", op="put", N=3, lens="300,700,1024", T=0, start="0,1500,77",
             slots=4, cap=4096, Hk=8, D=128, values=True, shuffle=True, fused=True),
        # two chat requests a few words into their answers: one call's latency
        dict(name="attn4-token-short", op="attn4", N=2, q="1,1", k="200,77", slots=2, cap=256,
             Hq=16, Hk=4, D=64, packed=False, shuffle=False, lse=False),
        # a serving batch of single tokens over long caches of different lengths
        dict(name="attn4-token-caches", op="attn4", N=32, q="ones", k="spread", slots=32, cap=8192,
             Hq=32, Hk=8, D=128, packed=False, shuffle=False, lse=False),
        # five drafted tokens of each of sixteen requests, checked at once
        dict(name="attn4-drafts", op="attn4", N=16, q="fives", k="spread", slots=20, cap=4096,
             Hq=32, Hk=4, D=64, packed=True, shuffle=True, lse=True),
        # the packed batch [300, 700, 1024]: a whole prompt and two that continue earlier keys
        dict(name="attn4-prompts", op="attn4", N=3, q="300,700,1024", k="300,2200,1101", slots=4,
             cap=2208, Hq=96, Hk=8, D=128, packed=True, shuffle=True, lse=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(numbers):
    return ",".join(str(x) for x in numbers)


def draw(rng):
    op = rng.choice(["norm", "rope", "put", "attn4", "attn4"])
    if op == "norm":
        post = rng.choice([0, 0, 32, 64, 128, 256, -1])
        if post > 0:
            W = post * _log_int(rng, 1, 12288 // post)
        else:
            W = 8 * _log_int(rng, 1, 2048)
        res = rng.choice(["", "bf16", "fp32"])
        pre = rng.random() < 0.5
        if not (post or pre or res):
            pre = True
        return dict(op=op, R=_log_int(rng, 1, min(65536, (1 << 25) // W)), W=W,
                    post=W if post < 0 else post, gate=rng.choice(["", "sigmoid", "silu"]),
                    res=res, alpha=rng.choice([1.0, 0.5, -1.25]), pre=pre,
                    wtype=rng.choice(["bf16", "fp32"]), fused=rng.random() < 0.3)
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8, 12])
    if op == "rope":
        D = rng.choice([32, 64, 80, 128, 256])
        N = _log_int(rng, 1, 32)
        packed = rng.random() < 0.5
        T = _log_int(rng, 1, max(1, (1 << 18) // (N * (Hq + Hk))))
        lens = [rng.randint(0, T) for _ in range(N)] if packed else []
        return dict(op=op, N=N, T=0 if packed else T,
                    lens=_text(lens[:-1] + [lens[-1] + 1]) if packed else "",
                    start=_text(_log_int(rng, 1, 1 << 20) - 1 for _ in range(N)), Hq=Hq,
                    Hk=rng.choice([0, Hk, Hk]), D=D,
                    rot=rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]),
                    interleaved=rng.random() < 0.5, method=rng.choice(["", "linear", "yarn"]),
                    factor=rng.choice([1.0, 4.0, 32.0]), inverse=rng.random() < 0.3,
                    fused=rng.random() < 0.3)
    N = _log_int(rng, 1, 32)
    cap = 32 * _log_int(rng, 1, 256)
    slots = N + rng.randint(0, 4)
    shuffle = rng.random() < 0.5
    if op == "put":
        T = _log_int(rng, 1, max(1, 4096 // N))
        packed = rng.random() < 0.6
        lens = [rng.randint(0, T) for _ in range(N)] if packed else []
        return dict(op=op, N=N, lens=_text(lens[:-1] + [lens[-1] + 1]) if packed else "",
                    T=0 if packed else T, start=_text(rng.randint(0, cap) for _ in range(N)),
                    slots=slots, cap=cap, Hk=Hk, D=D, values=rng.random() < 0.5, shuffle=shuffle,
                    fused=rng.random() < 0.4)
    lse = rng.random() < 0.5
    if rng.random() < 0.6:  # single tokens, or a few drafted ones
        n_q = rng.choice([1, 1, 1, 2, 5])
        q = [n_q] * N
        k = [rng.randint(0, cap) for _ in range(N)]
        packed = rng.random() < 0.3
    else:
        N = min(N, 8)
        q = [_log_int(rng, 1, max(2, 1600 // N)) for _ in range(N)]
        cap = 32 * _log_int(rng, 2, 96)
        k = [min(cap, x + rng.choice([0, 0, rng.randint(0, 2048)])) for x in q]
        packed = True
    return dict(op=op, N=N, q=_text(q), k=_text(k), slots=slots, cap=cap, Hq=Hq, Hk=Hk, D=D,
                packed=packed, shuffle=shuffle, lse=lse)


# --------------------------------------------------------------------------- inputs

def _numbers(text):
    return [int(x) for x in text.split(",")]


def _spread(n, cap):
    """Lengths from an eighth of a cache to all of it."""
    return [min(cap, cap // 8 + (cap - cap // 8) * ((7 * i) % n) // max(1, n - 1))
            for i in range(n)]


def _lens(case):
    """Tokens of each sequence, and their first positions (rope, put) or key counts (attn4)."""
    N = case["N"]
    if case["op"] == "attn4":
        q = [1] * N if case["q"] == "ones" else [5] * N if case["q"] == "fives" else _numbers(
            case["q"])
        return q, _spread(N, case["cap"]) if case["k"] == "spread" else _numbers(case["k"])
    lens = _numbers(case["lens"]) if case["lens"] else [case["T"]] * N
    if case["start"] == "spread":
        return lens, [x - 1 for x in _spread(N, case["cap"])]
    return lens, _numbers(case["start"])


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(DEV)


def _ints(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _normal(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _views(g, B, T, heads, D):
    """Tensors [B, T, h, D] that are views of one projection's rows [B, T, sum(heads) * D]."""
    return torch.split(_normal(g, B, T, sum(heads), D), heads, dim=2)


def _frequencies(rot, method, factor, base=10000.0, original=4096):
    """Angle per position of each pair, in 64 bits, and the factor of the turned values: plain,
    positions interpolated ("linear"), or interpolated where a pair turns less than once over the
    original context, kept where it turns 32 times and more, and blended between ("yarn")."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if method == "linear":
        return (f / factor).to(DEV), 1.0
    if method == "yarn":
        keep = ((original * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return (f * keep + f / factor * (1 - keep)).to(DEV), 0.1 * math.log(factor) + 1.0
    return f.to(DEV), 1.0


def _cache(g, slots, Hk, cap, D):
    """Empty caches with arbitrary contents."""
    def byte(*shape):
        return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    return dict(k4=byte(slots, Hk, cap, D // 2), v4=byte(slots, Hk, cap // 32, 16 * D),
                ks=byte(slots, Hk, cap // 32, D // 32, 32) % 128 + 64,
                vs=byte(slots, Hk, cap // 32, D // 32, 32) % 128 + 64)


def _slots(case, seed):
    if not case["shuffle"]:
        return None
    order = torch.randperm(case["slots"], generator=torch.Generator().manual_seed(seed))
    return order[:case["N"]].to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        R, W = case["R"], case["W"]
        wt = BF16 if case["wtype"] == "bf16" else torch.float32
        wide = _normal(g, R, 2 * W) if case["fused"] else None
        s["x"] = wide[:, :W] if case["fused"] else _normal(g, R, W)
        s["gate"] = s["post"] = s["res"] = s["pre"] = s["h"] = s["out"] = None
        if case["gate"]:
            s["gate"] = wide[:, W:] if case["fused"] else _normal(g, R, W)
        if case["post"]:
            s["post"] = (1 + 0.2 * _normal(g, case["post"], dtype=torch.float32)).to(wt)
        if case["res"]:
            rt = BF16 if case["res"] == "bf16" else torch.float32
            s["res"] = (3 * _normal(g, R, W, dtype=torch.float32)).to(rt)
            s["h"] = torch.empty_like(s["res"])
        if case["pre"]:
            s["pre"] = (1 + 0.2 * _normal(g, W, dtype=torch.float32)).to(wt)
        if case["pre"] or not case["res"]:
            s["out"] = torch.empty((R, W), dtype=BF16, device=DEV)
        return s
    N, D = case["N"], case["D"]
    lens, start = _lens(case)
    s.update(lens=lens, start=start)
    packed = case["packed"] if op == "attn4" else case["lens"] != ""
    B, T = (1, sum(lens)) if packed else (N, lens[0])
    s["cu"] = _cu(lens) if packed else None
    if op == "rope":
        Hq, Hk = case["Hq"], case["Hk"]
        s["offsets"] = _ints(start)
        s["freqs"], s["amplitude"] = _frequencies(case["rot"], case["method"], case["factor"])
        heads = [Hq, Hk] if Hk else [Hq]
        if case["fused"]:
            xs = _views(g, B, T, heads, D)
        else:
            xs = [_normal(g, B, T, h, D) for h in heads]
        s["q"], s["k"] = xs[0], xs[1] if Hk else None
        s["q_out"] = torch.empty((B, T, Hq, D), dtype=BF16, device=DEV)
        s["k_out"] = torch.empty((B, T, Hk, D), dtype=BF16, device=DEV) if Hk else None
        return s
    Hk, cap = case["Hk"], case["cap"]
    s["slots"] = _slots(case, seed)
    if op == "put":
        s["offsets"] = _ints(start)
        s.update(_cache(g, case["slots"], Hk, cap, D))
        s["k"], s["v"] = (_views(g, B, T, [Hk, Hk], D) if case["fused"]
                          else [_normal(g, B, T, Hk, D) for _ in "kv"])
        s["k_out"] = torch.empty((B, T, Hk, D), dtype=BF16, device=DEV) if case["values"] else None
        s["v_out"] = torch.empty_like(s["k_out"]) if case["values"] else None
        return s
    s["scale"] = 1.0 / math.sqrt(D)
    s["k_lens"] = _ints(start)
    s["q"] = _normal(g, B, T, case["Hq"], D)
    kc, ks = _quantise(_normal(g, case["slots"], Hk, cap, D, dtype=torch.float32))
    s["k4"], s["ks"] = _pack(kc), _tiled_scales(ks)
    vc, vs = _quantise(_normal(g, case["slots"], Hk, cap, D, dtype=torch.float32))
    s["v4"], s["vs"] = _tiled_values(_pack(vc)), _tiled_scales(vs)
    s["out"] = torch.empty((B, T, case["Hq"], D), dtype=BF16, device=DEV)
    s["lse"] = (torch.empty((B, T, case["Hq"]), dtype=torch.float32, device=DEV) if case["lse"]
                else None)
    return s


# ----------------------------------------------------------------------- 4-bit blocks

def _quantise(x):
    """Codes (uint8, one a value) and scales (exponent + 127) of x [.., D] in fp32: the smallest
    power of two that brings a block within 6, values to the nearest code, ties to the even one.
    Every step is exact: divisions by powers of two and comparisons."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1): within 6 = 0.75 2^3 for e - 3, or e - 2
    e = torch.where(top == 0, -127, torch.where(m > 0.75, e - 2, e - 3).clamp(min=-127))
    odd = ~torch.isfinite(top)
    e = torch.where(odd, 128, e)
    y = torch.ldexp(torch.ldexp(b, -(e // 2)[..., None]), -(e - e // 2)[..., None])
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(b).to(torch.uint8)
    code = torch.where(odd[..., None], torch.zeros_like(code), code)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _codes_as(dtype):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=dtype, device=DEV)


def _values(code, scale):
    """What codes [.., D] and scales [.., D / 32] stand for, in fp32."""
    x = _codes_as(torch.float32)[code.int()].unflatten(-1, (-1, 32))
    e = scale.int()[..., None] - 127
    x = torch.ldexp(torch.ldexp(x, e // 2), e - e // 2)
    return torch.where(e == 128, math.nan, x).flatten(-2)


def _pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def _unpack(byte):
    return torch.stack([byte & 15, byte >> 4], -1).flatten(-2)


def _tiled_scales(s):
    """[.., cap, D / 32] -> [.., cap / 32, D / 32, 32]"""
    t = s.unflatten(-2, (-1, 2, 4, 4))  # tile, j, i, g, block
    n = t.dim() - 5
    return t.permute(*range(n + 1), n + 4, n + 3, n + 2, n + 1).flatten(-3).contiguous()


def _tiled_values(b):
    """[.., cap, D / 2] -> [.., cap / 32, 16 D]"""
    half = b.shape[-1]
    t = b.unflatten(-2, (-1, 2, 4, 4)).unflatten(-1, (16, half // 16))  # tile, j, i, g, c, bytes
    n = t.dim() - 6
    order = (1, 3, 4, 2, 5) if half == 64 else (3, 4, 1, 2, 5)
    return t.permute(*range(n + 1), *(n + o for o in order)).flatten(-5).contiguous()


def _rows_of_scales(t):
    """The way back: [.., tiles, D / 32, 32] -> [.., cap, D / 32]"""
    x = t.unflatten(-1, (4, 4, 2))  # tile, block, g, i, j
    n = x.dim() - 5
    return x.permute(*range(n + 1), n + 4, n + 3, n + 2, n + 1).flatten(-5, -2)


def _rows_of_values(t):
    if t.shape[-1] == 2048:  # j, g, c, i, bytes
        x, order = t.unflatten(-1, (2, 4, 16, 4, 4)), (1, 4, 2, 3, 5)
    else:  # g, c, j, i, bytes
        x, order = t.unflatten(-1, (4, 16, 2, 4, 2)), (3, 4, 1, 2, 5)
    n = x.dim() - 6
    return x.permute(*range(n + 1), *(n + o for o in order)).flatten(-2).flatten(-5, -2)


def _value_at(x, D):
    """Place in a tile of the bytes of position x (0 .. 31), [.., D / 2]"""
    byte = torch.arange(D // 2, device=DEV)
    j, i, g = (x // 16)[..., None], (x // 4 % 4)[..., None], (x % 4)[..., None]
    if D == 128:
        return j * 1024 + (g * 16 + byte // 4) * 16 + i * 4 + byte % 4
    return (g * 16 + byte // 2) * 16 + (j * 4 + i) * 2 + byte % 2


# ------------------------------------------------------------------------- plain form

def _act(x, kind):
    y = 1 / (1 + torch.exp(-x))
    return x * y if kind == "silu" else y


def _plain_norm(s):
    case = s["case"]
    u = s["x"].float()
    if case["post"]:
        t = u.view(case["R"], -1, case["post"])
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * s["post"].float()
        u = t.view(case["R"], case["W"])
    if case["gate"]:
        u = u * _act(s["gate"].float(), case["gate"])
    if case["res"]:
        u = s["res"].float() + case["alpha"] * u
        s["h"].copy_(u)
    if case["pre"]:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * s["pre"].float()
    if s["out"] is not None:
        s["out"].copy_(u)


def _sequence_of(cu, n_tokens):
    return torch.searchsorted(cu, torch.arange(n_tokens, device=DEV), right=True) - 1


def _positions(s, B, T):
    """Sequence and position of every token, [B * T]."""
    if s["cu"] is None:
        n = torch.arange(B, device=DEV).repeat_interleave(T)
        return n, s["offsets"][n] + torch.arange(T, device=DEV).repeat(B)
    n = _sequence_of(s["cu"], T)
    return n, s["offsets"][n] + torch.arange(T, device=DEV) - s["cu"][n]


def _plain_rope(s):
    case = s["case"]
    B, T = s["q"].shape[:2]
    rot, half = case["rot"], case["rot"] // 2
    _, at = _positions(s, B, T)
    angle = at.double()[:, None] * s["freqs"]
    c = (torch.cos(angle) * s["amplitude"]).float().view(B, T, 1, half)
    z = (torch.sin(angle) * s["amplitude"]).float().view(B, T, 1, half)
    z = -z if case["inverse"] else z

    def turn(x, out):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            y = torch.cat([torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2),
                           y[..., rot:]], -1)
        else:
            a, b = y[..., :half], y[..., half:rot]
            y = torch.cat([a * c - b * z, a * z + b * c, y[..., rot:]], -1)
        out.copy_(y)

    turn(s["q"], s["q_out"])
    if s["k"] is not None:
        turn(s["k"], s["k_out"])


def _plain_put(s):
    case = s["case"]
    Hk, D, cap = case["Hk"], case["D"], case["cap"]
    B, T = s["k"].shape[:2]
    n, at = _positions(s, B, T)
    slot = s["slots"][n] if s["slots"] is not None else n
    there = at < cap
    slot, at = slot[there], at[there]
    tile, x = at // 32, at % 32
    heads, blocks = torch.arange(Hk, device=DEV), torch.arange(D // 32, device=DEV)
    place = 8 * (x % 4) + 2 * (x // 4 % 4) + x // 16

    def half(x_in, x_out, scales, write):
        code, scale = _quantise(x_in.float().reshape(B * T, Hk, D))
        write(_pack(code)[there])
        scales[slot[:, None, None], heads[:, None], tile[:, None, None], blocks,
               place[:, None, None]] = scale[there]
        if x_out is not None:
            x_out.copy_(_values(code, scale).view(B, T, Hk, D))

    def keys(b):
        s["k4"][slot[:, None], heads, at[:, None]] = b

    def values(b):
        s["v4"][slot[:, None, None], heads[:, None], tile[:, None, None],
                _value_at(x, D)[:, None]] = b

    half(s["k"], s["k_out"], s["ks"], keys)
    half(s["v"], s["v_out"], s["vs"], values)


def _plain_attn4(s):
    case = s["case"]
    N, Hq, Hk, D = case["N"], case["Hq"], case["Hk"], case["D"]
    G = Hq // Hk
    Tk = -(-max(1, max(s["start"])) // 32) * 32
    pick = s["slots"] if s["slots"] is not None else torch.arange(N, device=DEV)
    k = _values(_unpack(s["k4"][pick, :, :Tk]), _rows_of_scales(s["ks"][pick, :, :Tk // 32]))
    v = _values(_unpack(_rows_of_values(s["v4"][pick, :, :Tk // 32])),
                _rows_of_scales(s["vs"][pick, :, :Tk // 32]))
    Lk = s["k_lens"]
    if s["cu"] is None:
        q = s["q"].float()
        Lq = torch.full_like(Lk, q.shape[1])
    else:
        Lq = s["cu"].diff()
        at = s["cu"][:-1, None] + torch.arange(max(s["lens"]), device=DEV)
        in_q = at < s["cu"][1:, None]
        q = s["q"][0][torch.where(in_q, at, 0)].float()
    Tq = q.shape[1]
    q = q.view(N, Tq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * Tq, D)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(N, Hk, G, Tq, Tk).mul_(s["scale"])
    last = torch.arange(Tq, device=DEV) + (Lk - Lq)[:, None]
    seen = torch.arange(Tk, device=DEV) <= torch.minimum(last, Lk[:, None] - 1)[..., None]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(N, Hk, G * Tq, Tk), v).view(N, Hk, G, Tq, D)
    out = torch.where(total == 0, 0.0, out / total).permute(0, 3, 1, 2, 4).reshape(N, Tq, Hq, D)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(N, Tq, Hq)
    if s["cu"] is None:
        s["out"].copy_(out)
        if case["lse"]:
            s["lse"].copy_(lse)
        return
    s["out"][0] = out[in_q].to(BF16)
    if case["lse"]:
        s["lse"][0] = lse[in_q]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_62_amd as kda
        if op == "norm":
            kda.kda_norm(s["x"], s["out"], weight=s["pre"], eps=1e-6, post_weight=s["post"],
                         gate=s["gate"], gate_fn=case["gate"] or "sigmoid", residual=s["res"],
                         residual_out=s["h"], residual_scale=case["alpha"])
        elif op == "rope":
            kda.kda_rope(s["q"], s["k"], s["freqs"], s["q_out"], s["k_out"],
                         offsets=s["offsets"], cu_seqlens=s["cu"],
                         interleaved=case["interleaved"], amplitude=s["amplitude"],
                         inverse=case["inverse"])
        elif op == "put":
            kda.kda_cache4_put(s["k"], s["v"], s["k4"], s["ks"], s["v4"], s["vs"],
                               offsets=s["offsets"], cu_seqlens=s["cu"], slots=s["slots"],
                               k_out=s["k_out"], v_out=s["v_out"])
        else:
            kda.kda_attn4_fwd(s["q"], s["k4"], s["ks"], s["v4"], s["vs"], s["scale"], s["out"],
                              lse=s["lse"], k_lens=s["k_lens"], cu_seqlens_q=s["cu"],
                              slots=s["slots"])
    else:
        {"norm": _plain_norm, "rope": _plain_rope, "put": _plain_put,
         "attn4": _plain_attn4}[op](s)
    names = {"norm": ("h", "out"), "rope": ("q_out", "k_out"),
             "put": ("k4", "ks", "v4", "vs", "k_out", "v_out"), "attn4": ("out", "lse")}[op]
    return {x: s[x] for x in names if s[x] is not None}


# ------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "norm":
        R, W = case["R"], case["W"]
        size = {"": 0, "bf16": 2, "fp32": 4}
        per = 2 + (2 if case["gate"] else 0) + 2 * size[case["res"]]
        per += 2 if case["pre"] or not case["res"] else 0
        weights = size[case["wtype"]] * (case["post"] + (W if case["pre"] else 0))
        flops = (4 if case["post"] else 0) + (6 if case["gate"] else 0) + (
            2 if case["res"] else 0) + (4 if case["pre"] else 0)
        return {"bytes": R * W * per + weights, "flops": R * W * flops}
    lens, start = _lens(case)
    tok, D, Hk = sum(lens), case["D"], case["Hk"]
    if op == "rope":
        heads = case["Hq"] + Hk
        return {"bytes": 4 * tok * heads * D + 4 * case["rot"],
                "flops": 3 * tok * heads * case["rot"]}
    if op == "put":
        kept = sum(max(0, min(n, case["cap"] - at)) for n, at in zip(lens, start))
        read = tok if case["values"] else kept
        b = 4 * read * Hk * D + 2 * kept * Hk * (D // 2 + D // 32)
        return {"bytes": b + (4 * tok * Hk * D if case["values"] else 0),
                "flops": 6 * read * Hk * D}
    Hq = case["Hq"]
    pairs = sum(max(0, lk) * lq - min(lq, lk) * (min(lq, lk) - 1) // 2 if lk >= lq
                else lk * (lk + 1) // 2 for lq, lk in zip(lens, start))
    b = 4 * tok * Hq * D + sum(start) * Hk * 2 * (D // 2 + D // 32)
    return {"bytes": b + (4 * tok * Hq if case["lse"] else 0), "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------------------- exact

def _exact_values(code, byte):
    """Values of single codes [.., D] and scale bytes [.., D / 32] in 64 bits."""
    scale = torch.exp2(byte.double() - 127).repeat_interleave(32, -1)
    x = _codes_as(torch.float64)[code.long()] * scale
    return torch.where(byte.repeat_interleave(32, -1) == 255, math.nan, x)


def _exact_norm(case, s):
    x = s["x"].double()
    if case["post"]:
        parts = torch.stack(x.split(case["post"], -1), 1)
        rms = torch.sqrt(parts.square().sum(-1, keepdim=True) / case["post"] + 1e-6)
        x = (parts / rms * s["post"].double()).reshape(case["R"], case["W"])
    if case["gate"]:
        t = s["gate"].double()
        x = x * torch.sigmoid(t) * (t if case["gate"] == "silu" else 1.0)
    found = {}
    if case["res"]:
        x = found["h"] = s["res"].double() + case["alpha"] * x
    if case["pre"]:
        x = x * s["pre"].double() / torch.sqrt(
            x.square().sum(-1, keepdim=True) / case["W"] + 1e-6)
    if s["out"] is not None:
        found["out"] = x
    return found


def _exact_rope(case, s):
    B, T = s["q"].shape[:2]
    rot = case["rot"]
    at = [a + i for n, a in zip(s["lens"], s["start"]) for i in range(n)]
    angle = _ints(at).double()[:, None] * s["freqs"] * (-1 if case["inverse"] else 1)
    unit = torch.polar(torch.full_like(angle, s["amplitude"]), angle).view(B, T, 1, rot // 2)

    def turn(x):
        y = x.double()
        z = y[..., :rot]
        if case["interleaved"]:
            z = torch.view_as_complex(z.unflatten(-1, (rot // 2, 2)).contiguous()) * unit
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:].contiguous()) * unit
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, y[..., rot:]], -1)

    found = {"q_out": turn(s["q"])}
    if s["k"] is not None:
        found["k_out"] = turn(s["k"])
    return found


def _exact_put(case, s):
    """Position by position, on the host."""
    Hk, D, cap = case["Hk"], case["D"], case["cap"]
    tok = sum(s["lens"])
    table = _codes_as(torch.float64)[:8]
    found = {x: s[x].clone() for x in ("k4", "ks", "v4", "vs")}
    done = []
    for name in "kv":
        x = s[name].double().reshape(tok, Hk, D // 32, 32)
        top = x.abs().amax(-1, keepdim=True)
        powers = torch.arange(254, device=DEV)
        fits = top <= 6 * torch.exp2(powers.double() - 127)  # the first that holds the block
        byte = torch.where(torch.isfinite(top), fits.int().argmax(-1, keepdim=True), 255)
        y = x / torch.exp2(byte.double() - 127)
        near = (y.abs()[..., None] - table).abs()
        best = near.amin(-1, keepdim=True)
        # of two equally near codes the even one
        code = torch.where(near == best, torch.arange(8, device=DEV) % 2 * 8
                           + torch.arange(8, device=DEV), 99).amin(-1) % 8
        code = code + 8 * torch.signbit(x)
        code = torch.where(byte == 255, 0, code).reshape(tok, Hk, D)
        done.append((code, byte.reshape(tok, Hk, D // 32)))
        if s[name + "_out"] is not None:
            found[name + "_out"] = _exact_values(code, byte.reshape(tok, Hk, D // 32)).reshape(
                s[name + "_out"].shape)
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["N"]))
    first = 0
    for n, (length, at) in enumerate(zip(s["lens"], s["start"])):
        for t in range(max(0, min(length, cap - at))):
            p, row = at + t, first + t
            j, i, g = p % 32 // 16, p % 16 // 4, p % 4
            for (code, byte), codes, scales in zip(done, ("k4", "v4"), ("ks", "vs")):
                two = (code[row, :, 0::2] + 16 * code[row, :, 1::2]).to(torch.uint8)
                found[scales][slots[n], :, p // 32, :, 8 * g + 2 * i + j] = byte[row].to(
                    torch.uint8)
                if codes == "k4":
                    found[codes][slots[n], :, p] = two
                elif D == 128:
                    tile = found[codes][slots[n], :, p // 32].view(Hk, 2, 4, 16, 4, 4)
                    tile[:, j, g, :, i] = two.view(Hk, 16, 4)
                else:
                    tile = found[codes][slots[n], :, p // 32].view(Hk, 4, 16, 2, 4, 2)
                    tile[:, g, :, j, i] = two.view(Hk, 16, 2)
        first += length
    return found


def _exact_attn4(case, s):
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    G = Hq // Hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["N"]))
    x = torch.arange(32, device=DEV)
    place = 8 * (x % 4) + 2 * (x // 4 % 4) + x // 16
    in_tile = _value_at(x, D)
    first = 0
    for n, (lq, lk) in enumerate(zip(s["lens"], s["start"])):
        row = 0 if s["cu"] is not None else n
        at = first if s["cu"] is not None else 0
        first += lq
        if lk == 0 or lq == 0:
            continue
        tiles = -(-lk // 32)

        def scales(t):
            return t[slots[n], :, :tiles][..., place].transpose(-1, -2).reshape(Hk, -1, D // 32)

        def nibbles(b):
            return torch.stack([b % 16, b // 16], -1).flatten(-2)

        k = _exact_values(nibbles(s["k4"][slots[n], :, :32 * tiles]), scales(s["ks"]))[:, :lk]
        v4 = s["v4"][slots[n], :, :tiles][..., in_tile].reshape(Hk, -1, D // 2)
        v = _exact_values(nibbles(v4), scales(s["vs"]))[:, :lk]
        hide = (torch.arange(lk, device=DEV)[None, :]
                > torch.arange(lq, device=DEV)[:, None] + (lk - lq))
        for h in range(Hq):
            q = s["q"][row, at:at + lq, h].double()
            score = (s["scale"] * (q @ k[h // G].t())).masked_fill(hide, -math.inf)
            z = torch.logsumexp(score, -1)
            lse[row, at:at + lq, h] = z
            prob = torch.exp(score - torch.where(z == -math.inf, 0.0, z)[:, None])
            out[row, at:at + lq, h] = prob @ v[h // G]
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "put": _exact_put,
            "attn4": _exact_attn4}[case["op"]](case, s)
