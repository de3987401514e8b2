"""The serving operators beside the KDA prefill, as cases that can be timed and compared.

Four operators of one hybrid model that keeps recurrent states and key/value caches:

  attn     kda_attn_fwd: causal softmax attention with grouped heads, over whole prompts, over
           prompts that continue earlier keys, and for single tokens over key/value caches
  la       kda_la_fwd: linear attention with one decay per head, over prompts
  la_step  kda_la_step: its recurrence for one token of each request, states in a pool
  step     kda_step: the KDA recurrence for one token of each request, states in a pool

``run`` computes them with elementary torch operations in 32 bits, or where ``own`` is true
calls the library.  ``exact`` evaluates the definitions token by token in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
CHUNK = 128  # tokens per chunk of the plain linear attention


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # two chat requests a few words into their answers: one call's latency
        dict(name="attn-token-short", op="attn", N=2, q="1,1", k="200,77", slab=256, Hq=16, Hk=4,
             D=64, fused=False, lse=False),
        # a serving batch of single tokens over long key/value caches of different lengths
        dict(name="attn-token-caches", op="attn", N=32, q="ones", k="spread", slab=8192, Hq=32,
             Hk=8, D=128, fused=False, lse=False),
        # the packed batch [300, 700, 1024]: a whole prompt and two that continue earlier keys,
        # q, k and v as views of projections' rows, 96 heads in groups of twelve
        dict(name="attn-packed", op="attn", N=3, q="300,700,1024", k="300,2200,1101", slab=0,
             Hq=96, Hk=8, D=128, fused=True, lse=True),
        # one long document
        dict(name="attn-prompt-long", op="attn", N=1, q="8192", k="8192", slab=0, Hq=32, Hk=8,
             D=128, fused=False, lse=False),
        # the smallest workload of the benchmark: one short prompt, two heads
        dict(name="la-small", op="la", N=1, T=128, lens="", H=2, Hk=2, D=32, state="zero",
             out_state="bf16", gate="token", fused=False),
        # the benchmark's batched prefill
        dict(name="la-batched", op="la", N=2, T=1024, lens="", H=96, Hk=96, D=128, state="bf16",
             out_state="bf16", gate="token", fused=False),
        # many short packed prompts, fixed decays, fp32 states, grouped query/key heads
        dict(name="la-many", op="la", N=64, T=0, lens="short", H=32, Hk=16, D=128, state="fp32",
             out_state="fp32", gate="head", fused=True),
        # one long document: few heads, a long axis
        dict(name="la-long", op="la", N=1, T=32768, lens="", H=32, Hk=32, D=128, state="zero",
             out_state="fp32", gate="token", fused=False),
        # one token of two requests: latency
        dict(name="la-step-few", op="la_step", N=2, slots=8, H=8, Hk=8, D=64, state="fp32",
             gate="token"),
        # a serving batch, states kept in bf16
        dict(name="la-step-batch", op="la_step", N=256, slots=544, H=32, Hk=32, D=128,
             state="bf16", gate="head"),
        # one token of a few requests through a 96-head layer
        dict(name="step-few", op="step", N=4, slots=16, H=96, D=128, state="fp32", lb=-5.0),
        # a serving batch through the same layer
        dict(name="step-batch", op="step", N=96, slots=224, H=96, D=128, state="fp32", lb=-5.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "la", "la", "la_step", "step"])
    if op == "attn":
        D = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 3, 4, 8, 12])
        lse = rng.random() < 0.5
        if rng.random() < 0.4:  # single tokens, or a few drafted ones, over caches
            N = _log_int(rng, 1, 48)
            slab = _log_int(rng, 16, 8192)
            n_q = rng.choice([1, 1, 1, 2, 5])
            return dict(op=op, N=N, q=",".join([str(n_q)] * N),
                        k=",".join(str(rng.randint(0, slab)) for _ in range(N)), slab=slab, Hq=Hq,
                        Hk=Hk, D=D, fused=False, lse=lse)
        N = _log_int(rng, 1, 12)
        q = [_log_int(rng, 1, max(2, 2800 // N)) for _ in range(N)]
        k = [x + (rng.randint(0, 2048) if rng.random() < 0.4 else 0) for x in q]
        return dict(op=op, N=N, q=",".join(map(str, q)), k=",".join(map(str, k)), slab=0, Hq=Hq,
                    Hk=Hk, D=D, fused=rng.random() < 0.5, lse=lse)
    H = _log_int(rng, 1, 96)
    D = rng.choice([32, 64, 128])
    state = rng.choice(["bf16", "fp32"])
    gate = rng.choice(["token", "head", "both"])
    Hk = rng.choice([h for h in (H, H, H // 2, H // 4) if h and H % h == 0])
    if op == "la":
        common = dict(op=op, H=H, Hk=Hk, D=D, state=rng.choice(["none", "bf16", "fp32"]),
                      out_state=state, gate=gate, fused=rng.random() < 0.3)
        if rng.random() < 0.5:
            N = _log_int(rng, 1, 8)
            return dict(N=N, T=_log_int(rng, 1, 8192 // N), lens="", **common)
        N = _log_int(rng, 1, 64)
        return dict(N=N, T=0, lens=",".join(str(rng.choice([0, 1, _log_int(rng, 1, 1024)]))
                                            if rng.random() < 0.2 else str(_log_int(rng, 1, 700))
                                            for _ in range(N)), **common)
    N = _log_int(rng, 1, 128)
    case = dict(op=op, N=N, slots=2 * N + rng.randint(0, 9), H=H, D=D, state=state)
    if op == "la_step":
        return dict(case, Hk=Hk, gate=gate)
    return dict(case, lb=rng.choice([-0.5, -5.0, -20.0]))


# --------------------------------------------------------------------------- inputs

def _lens(case):
    """Query and key lengths (attn) or token counts (la) of the case's sequences."""
    if case["op"] == "la":
        if case["lens"] == "":
            return [case["T"]] * case["N"]
        if case["lens"] == "short":  # 1 .. 512
            return torch.randint(1, 513, (case["N"],),
                                 generator=torch.Generator().manual_seed(5)).tolist()
        return [int(x) for x in case["lens"].split(",")]
    N, slab = case["N"], case["slab"]
    q = [1] * N if case["q"] == "ones" else [int(x) for x in case["q"].split(",")]
    if case["k"] == "spread":  # from an eighth of the cache to all of it
        k = [slab // 8 + (slab - slab // 8) * ((7 * i) % N) // max(1, N - 1) for i in range(N)]
        k = [min(slab, x) for x in k]
    else:
        k = [int(x) for x in case["k"].split(",")]
    return q, k


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(DEV)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _views(g, B, T, heads, D):
    """Tensors [B, T, h, D] that are views of one projection's rows [B, T, sum(heads) * D]."""
    rows = _normal(g, B, T, sum(heads), D)
    return torch.split(rows, heads, dim=2)


def prepare(case, seed):
    g = _gen(seed)
    op, N, D = case["op"], case["N"], case["D"]
    s = dict(case=case, scale=1.0 / math.sqrt(D))
    if op == "attn":
        ql, kl = _lens(case)
        Hq, Hk = case["Hq"], case["Hk"]
        s.update(ql=ql, kl=kl)
        if case["slab"]:  # the caches: rows of equal capacity, each filled to its own length
            s["q"] = _normal(g, N, ql[0], Hq, D)
            s["k"] = _normal(g, N, case["slab"], Hk, D)
            s["v"] = _normal(g, N, case["slab"], Hk, D)
            s["k_lens"] = torch.tensor(kl, dtype=torch.int64, device=DEV)
        else:
            s["cu_q"], s["cu_k"] = _cu(ql), _cu(kl)
            if case["fused"] and ql == kl:
                s["q"], s["k"], s["v"] = _views(g, 1, sum(ql), [Hq, Hk, Hk], D)
            elif case["fused"]:
                s["q"], _ = _views(g, 1, sum(ql), [Hq, Hk], D)
                s["k"], s["v"] = _views(g, 1, sum(kl), [Hk, Hk], D)
            else:
                s["q"] = _normal(g, 1, sum(ql), Hq, D)
                s["k"] = _normal(g, 1, sum(kl), Hk, D)
                s["v"] = _normal(g, 1, sum(kl), Hk, D)
        s["out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
        if case["lse"]:
            s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device=DEV)
        return s
    H = case["H"]
    dtype = torch.float32 if case.get("out_state", case["state"]) == "fp32" else torch.bfloat16
    if op == "la":
        lens, Hk = _lens(case), case["Hk"]
        packed = case["lens"] != ""
        B, T = (1, sum(lens)) if packed else (N, case["T"])
        s.update(lens=lens, cu=_cu(lens) if packed else None)
        if case["fused"]:
            s["q"], s["k"], s["v"] = _views(g, B, T, [Hk, Hk, H], D)
        else:
            s["q"], s["k"], s["v"] = (_normal(g, B, T, h, D) for h in (Hk, Hk, H))
        _decays(s, g, case["gate"], (B, T, H), H)
        s["out"] = torch.empty((B, T, H, D), dtype=torch.bfloat16, device=DEV)
        s["final"] = torch.empty((N, H, D, D), dtype=dtype, device=DEV)
        s["initial"] = None
        if case["state"] == "zero":
            s["initial"] = torch.zeros((N, H, D, D), dtype=torch.bfloat16, device=DEV)
        elif case["state"] != "none":
            s["initial"] = _normal(g, N, H, D, D, dtype=torch.float32 if case["state"] == "fp32"
                                   else torch.bfloat16)
        return s
    # steps: each request reads one slot of the pool and writes another
    slots = case["slots"]
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))
    s["src"], s["dst"] = order[:N].to(DEV), order[N:2 * N].to(DEV)
    s["pool"] = _normal(g, slots, H, D, D, dtype=dtype)
    s["out"] = torch.empty((N, H, D), dtype=torch.bfloat16, device=DEV)
    if op == "la_step":
        s["q"], s["k"], s["v"] = (_normal(g, N, h, D) for h in (case["Hk"], case["Hk"], H))
        _decays(s, g, case["gate"], (N, H), H)
        return s
    s["q"], s["k"], s["v"], s["g"] = (_normal(g, N, H, D) for _ in range(4))
    s["beta"] = _normal(g, N, H)
    s["A_log"] = torch.rand((H,), generator=g, device=DEV)
    s["dt_bias"] = torch.rand((H, D), generator=g, device=DEV)
    return s


def _decays(s, g, gate, shape, H):
    """Log decays: for each token and head (a softplus gate), for each head, or both."""
    s["g"] = s["decay"] = None
    if gate != "head":
        rate = torch.rand((H,), generator=g, device=DEV) * 0.5 + 0.01
        s["g"] = -rate * torch.nn.functional.softplus(_normal(g, *shape, dtype=torch.float32))
    if gate != "token":
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)


# ------------------------------------------------------------------------- plain form

def _rows(cu, n_seq, width):
    """Token index [n_seq, width] of each sequence's padded rows, and which of them exist."""
    at = cu[:-1, None] + torch.arange(width, device=DEV)
    there = at < cu[1:, None]
    return torch.where(there, at, 0), there


def _plain_attn(s):
    case = s["case"]
    N, Hq, Hk, D = case["N"], case["Hq"], case["Hk"], case["D"]
    G = Hq // Hk
    if case["slab"]:
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
        Lk = s["k_lens"]
        Lq = torch.full_like(Lk, q.shape[1])
    else:
        if sum(s["kl"]) == 0:
            s["out"].zero_()
            return
        iq, in_q = _rows(s["cu_q"], N, max(s["ql"]))
        ik, _ = _rows(s["cu_k"], N, max(s["kl"]))
        q, k, v = s["q"][0][iq].float(), s["k"][0][ik].float(), s["v"][0][ik].float()
        Lq, Lk = s["cu_q"].diff(), s["cu_k"].diff()
    Tq, Tk = q.shape[1], k.shape[1]
    q = q.view(N, Tq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * Tq, D)
    k = k.permute(0, 2, 3, 1).contiguous()
    v = v.permute(0, 2, 1, 3).contiguous()
    p = torch.matmul(q, k).view(N, Hk, G, Tq, Tk).mul_(s["scale"])
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
    if case["slab"]:
        s["out"].copy_(out)
        if case["lse"]:
            s["lse"].copy_(lse)
        return
    s["out"][0] = out[in_q].to(torch.bfloat16)
    if case["lse"]:
        s["lse"][0] = lse[in_q]


def _plain_la(s):
    case = s["case"]
    N, H, Hk, D = case["N"], case["H"], case["Hk"], case["D"]
    lens = s["lens"]
    T_all = sum(lens)
    cu = s["cu"] if s["cu"] is not None else torch.arange(N + 1, device=DEV) * case["T"]
    init = (torch.zeros((N, H, D, D), device=DEV) if s["initial"] is None
            else s["initial"].float())
    # chunks of each sequence, one after another; an empty sequence keeps one empty chunk
    counts = [max(1, -(-n // CHUNK)) for n in lens]
    n_chunks = sum(counts)
    per = torch.clamp((cu.diff() + CHUNK - 1) // CHUNK, min=1)
    first = torch.cumsum(per, 0) - per
    seq = torch.repeat_interleave(torch.arange(N, device=DEV), per, output_size=n_chunks)
    nth = torch.arange(n_chunks, device=DEV) - first[seq]
    at = (cu[seq] + nth * CHUNK)[:, None] + torch.arange(CHUNK, device=DEV)
    there = at < cu[seq + 1][:, None]
    at = torch.where(there, at, 0)

    def chunks(x, heads):  # [n_chunks, heads, CHUNK, D]
        if T_all == 0:
            return torch.zeros((n_chunks, heads, CHUNK, D), device=DEV)
        x = x.reshape(T_all, heads, D)[at].float()
        return torch.where(there[..., None, None], x, 0.0).transpose(1, 2).contiguous()

    q, k, v = chunks(s["q"], Hk), chunks(s["k"], Hk), chunks(s["v"], H)
    q, k = (x.repeat_interleave(H // Hk, 1) if H != Hk else x for x in (q, k))
    lam = torch.zeros((n_chunks, CHUNK, H), device=DEV, dtype=torch.float64)
    if s["g"] is not None and T_all:
        lam = lam + s["g"].reshape(T_all, H)[at]
    if s["decay"] is not None:
        lam = lam + s["decay"]
    lam = torch.where(there[..., None], lam, 0.0).transpose(1, 2)
    G = lam.cumsum(-1)  # [n_chunks, H, CHUNK], in 64 bits: differences of long sums
    below = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=DEV).tril()
    w = torch.where(below, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    out = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * w, v)
    left = (G[..., -1:] - G).float().exp()
    add = torch.matmul(v.transpose(-1, -2).contiguous(), k * left[..., None])  # [nc, H, D(v), D(k)]
    # the state before chunk c: every earlier chunk of its sequence, decayed, and the initial state
    end = G[..., -1].t().contiguous().cumsum(-1)  # [H, n_chunks]
    before = end - G[..., -1].t()
    c = torch.arange(n_chunks, device=DEV)
    earlier = (seq[:, None] == seq[None, :]) & (c[None, :] < c[:, None])
    reach = torch.where(earlier, before[:, :, None] - end[:, None, :], -math.inf).float().exp()
    S = torch.matmul(reach, add.transpose(0, 1).reshape(H, n_chunks, D * D))
    S = S.view(H, n_chunks, D, D).transpose(0, 1)
    since = (before - before[:, first[seq]]).float().exp().t()[..., None, None]
    S = S + since * init[seq]
    out = out + torch.matmul(q, S.transpose(-1, -2).contiguous()) * G.float().exp()[..., None]
    last = first + per - 1
    s["final"].copy_(S[last] * G[last][..., -1].float().exp()[..., None, None] + add[last])
    if T_all:
        out = (out * s["scale"]).transpose(1, 2)[there]
        s["out"].view(T_all, H, D).copy_(out)


def _plain_la_step(s):
    case = s["case"]
    H, Hk = case["H"], case["Hk"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q, k = (x.repeat_interleave(H // Hk, 1) if H != Hk else x for x in (q, k))
    lam = torch.zeros(v.shape[:2], device=DEV)
    if s["g"] is not None:
        lam = lam + s["g"]
    if s["decay"] is not None:
        lam = lam + s["decay"]
    S = s["pool"][s["src"]].float()
    S = S * lam.exp()[..., None, None] + v[..., :, None] * k[..., None, :]
    s["pool"][s["dst"]] = S.to(s["pool"].dtype)
    s["out"].copy_(torch.matmul(S, q[..., None])[..., 0] * s["scale"])


def _plain_step(s):
    q, k, v, g = (s[x].float() for x in "qkvg")
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    lam = s["case"]["lb"] * torch.sigmoid(s["A_log"].exp()[:, None] * (g + s["dt_bias"]))
    S = s["pool"][s["src"]].float() * lam.exp()[..., None, :]
    u = torch.sigmoid(s["beta"].float())[..., None] * (v - torch.matmul(S, k[..., None])[..., 0])
    S = S + u[..., :, None] * k[..., None, :]
    s["pool"][s["dst"]] = S.to(s["pool"].dtype)
    s["out"].copy_(torch.matmul(S, q[..., None])[..., 0] * s["scale"])


def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_62_amd as kda
        if op == "attn":
            kda.kda_attn_fwd(s["q"], s["k"], s["v"], s["scale"], s["out"], lse=s.get("lse"),
                             cu_seqlens_q=s.get("cu_q"), cu_seqlens_k=s.get("cu_k"),
                             k_lens=s.get("k_lens"))
        elif op == "la":
            kda.kda_la_fwd(s["q"], s["k"], s["v"], s["g"], s["scale"], s["out"],
                           decay=s["decay"], initial_state=s["initial"], final_state=s["final"],
                           cu_seqlens=s["cu"])
        elif op == "la_step":
            kda.kda_la_step(s["q"], s["k"], s["v"], s["g"], s["scale"], s["out"], s["pool"],
                            decay=s["decay"], slot_in=s["src"], slot_out=s["dst"])
        else:
            kda.kda_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["out"],
                         s["A_log"], s["dt_bias"], s["case"]["lb"], s["pool"],
                         slot_in=s["src"], slot_out=s["dst"])
    else:
        {"attn": _plain_attn, "la": _plain_la, "la_step": _plain_la_step,
         "step": _plain_step}[op](s)
    return {x: s[x] for x in ("out", "lse", "final", "pool") if s.get(x) is not None}


# ------------------------------------------------------------------------------ work

def work(case):
    op, N, D = case["op"], case["N"], case["D"]
    if op == "attn":
        ql, kl = _lens(case)
        Hq, Hk = case["Hq"], case["Hk"]
        # keys that some query sees, and the pairs: query i of Lq sees i + 1 + Lk - Lq keys, if any
        pairs = sum(max(0, lk) * lq - min(lq, lk) * (min(lq, lk) - 1) // 2 if lk >= lq
                    else lk * (lk + 1) // 2 for lq, lk in zip(ql, kl))
        b = 2 * D * (2 * sum(ql) * Hq + 2 * sum(kl) * Hk)
        b += 4 * sum(ql) * Hq if case["lse"] else 0
        return {"bytes": b, "flops": 4 * D * Hq * pairs}
    H = case["H"]
    Hk = case.get("Hk", H)
    size = {"fp32": 4, "bf16": 2, "zero": 2, "none": 0}
    if op == "la":
        T = sum(_lens(case))
        b = T * (2 * D * (2 * Hk + 2 * H) + (0 if case["gate"] == "head" else 4 * H))
        b += N * H * D * D * (size[case["state"]] + size[case["out_state"]])
        return {"bytes": b, "flops": 4 * T * H * D * D}
    b = N * H * D * D * 2 * size[case["state"]]
    if op == "la_step":
        b += N * (2 * D * (2 * Hk + 2 * H) + (0 if case["gate"] == "head" else 4 * H))
        return {"bytes": b, "flops": 4 * N * H * D * D}
    return {"bytes": b + N * H * (10 * D + 2) + 4 * H * (D + 1), "flops": 7 * N * H * D * D}


# ----------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    op, N, D = case["op"], case["N"], case["D"]
    scale = s["scale"]
    if op == "attn":
        Hq, G = case["Hq"], case["Hq"] // case["Hk"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
        at_q = at_k = 0
        for n, (lq, lk) in enumerate(zip(s["ql"], s["kl"])):
            row, key = (n, n) if case["slab"] else (0, 0)
            if case["slab"]:
                at_q = at_k = 0
            hide = (torch.arange(lk, device=DEV)[None, :]
                    > torch.arange(lq, device=DEV)[:, None] + (lk - lq))
            for h in range(Hq if lk else 0):
                q = s["q"][row, at_q:at_q + lq, h].double()
                k = s["k"][key, at_k:at_k + lk, h // G].double()
                v = s["v"][key, at_k:at_k + lk, h // G].double()
                x = (scale * (q @ k.t())).masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[row, at_q:at_q + lq, h] = z
                prob = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
                out[row, at_q:at_q + lq, h] = prob @ v
            at_q, at_k = at_q + lq, at_k + lk
        return {"out": out, "lse": lse} if case["lse"] else {"out": out}
    H = case["H"]
    group = H // case.get("Hk", H)

    def lam(*index):
        x = torch.zeros(H, dtype=torch.float64, device=DEV)
        if s["g"] is not None:
            x = x + s["g"][index].double()
        return x if s["decay"] is None else x + s["decay"].double()

    if op == "la":
        B, T = s["q"].shape[:2]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        S = (torch.zeros((N, H, D, D), dtype=torch.float64, device=DEV) if s["initial"] is None
             else s["initial"].double())
        lens = s["lens"]
        order = sorted(range(N), key=lambda n: -lens[n])  # the longest first: the rest ends earlier
        start = [0] * (N + 1)
        for n in range(N):
            start[n + 1] = start[n] + lens[n]
        rows = torch.tensor([start[n] for n in order], device=DEV)
        S = S[order]
        q, k, v = (x.reshape(B * T, x.shape[2], D) for x in (s["q"], s["k"], s["v"]))
        g = s["g"].reshape(B * T, H) if s["g"] is not None else None
        flat = out.view(B * T, H, D)
        live = N
        for t in range(max(lens)):
            while lens[order[live - 1]] <= t:
                live -= 1
            r = rows[:live] + t
            x = torch.zeros((live, H), dtype=torch.float64, device=DEV)
            if g is not None:
                x = x + g[r].double()
            if s["decay"] is not None:
                x = x + s["decay"].double()
            kt, qt = k[r].double(), q[r].double()
            if group > 1:
                kt, qt = kt.repeat_interleave(group, 1), qt.repeat_interleave(group, 1)
            now = S[:live]
            now.mul_(x.exp()[..., None, None])
            now.addcmul_(v[r].double()[..., :, None], kt[..., None, :])
            flat[r] = scale * (now @ qt[..., None])[..., 0]
        final = torch.empty_like(S)
        final[order] = S
        return {"out": out, "final": final}
    pool = s["pool"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    src, dst = s["src"].tolist(), s["dst"].tolist()
    for n in range(N):
        S = pool[src[n]].clone()
        q, k, v = (s[x][n].double() for x in "qkv")
        if op == "la_step":
            k, q = k.repeat_interleave(group, 0), q.repeat_interleave(group, 0)
            S = lam(n).exp()[:, None, None] * S + v[:, :, None] * k[:, None, :]
        else:
            q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)
            k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
            x = s["A_log"].double().exp()[:, None] * (s["g"][n].double() + s["dt_bias"].double())
            S = S * torch.exp(case["lb"] / (1 + torch.exp(-x)))[:, None, :]
            b = 1 / (1 + torch.exp(-s["beta"][n].double()))
            u = b[:, None] * (v - (S * k[:, None, :]).sum(-1))
            S = S + u[:, :, None] * k[:, None, :]
        pool[dst[n]] = S
        out[n] = scale * (S * q[:, None, :]).sum(-1)
    return {"out": out, "pool": pool}
