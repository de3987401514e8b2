"""Refusals of the norms, rotary positions and 4-bit caches, on the CPU: their *_check functions
compare pointer values and sizes only, and the bindings refuse tensors before anything is
launched.  The forms the GPU tests compare with are checked here against each other."""
from __future__ import annotations

import math
import os

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms

GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.library_path()):
        kda.build()
    return kda.load_library()


def _call(fn, order, base, **over):
    unknown = set(over) - set(base)
    assert not unknown, unknown
    return fn(*[dict(base, **over)[n] for n in order])


NORM = ("x x_row gate gate_row gate_fn post group w w_dtype eps res res_out res_dtype alpha out R "
        "W").split()
NORM_BASE = dict(x=1 * GB, x_row=1024, gate=2 * GB, gate_row=1024, gate_fn=0, post=3 * GB,
                 group=128, w=4 * GB, w_dtype=0, eps=1e-6, res=5 * GB, res_out=6 * GB, res_dtype=1,
                 alpha=1.0, out=7 * GB, R=16, W=1024)


def test_norm_refusals(lib):
    st = lambda **o: _call(lib.kda_norm_check, NORM, NORM_BASE, **o)
    assert st() == st(gate=None) == st(post=None, group=77) == st(w=None) == kda.KDA_OK
    assert st(res=None, res_out=None) == st(w=None, out=None) == kda.KDA_OK
    assert st(group=1024) == st(group=512) == st(group=32) == st(x_row=1032) == kda.KDA_OK
    assert st(R=0, x=None, out=None) == st(res_out=5 * GB) == kda.KDA_OK
    assert st(gate=None, gate_fn=9, gate_row=0) == kda.KDA_OK
    for bad in (dict(x=None), dict(out=None), dict(res=None), dict(res_out=None),
                dict(res=None, res_out=None, w=None, out=None),
                dict(post=None, gate=None, w=None, res=None, res_out=None)):
        assert st(**bad) == kda.KDA_ERR_NULL_ARG, bad
    for bad in (dict(R=-1), dict(W=0), dict(W=1028), dict(W=16392), dict(group=16), dict(group=96),
                dict(group=0), dict(group=-128), dict(group=1023), dict(R=1 << 30),
                dict(W=1024 + 64, x_row=2048, gate_row=2048), dict(x_row=1 << 61)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(gate_fn=2), dict(w_dtype=2), dict(res_dtype=-1)):
        assert st(**bad) == kda.KDA_ERR_BAD_DTYPE, bad
    for bad in (dict(eps=-1e-6), dict(eps=math.nan), dict(alpha=math.inf)):
        assert st(**bad) == kda.KDA_ERR_BAD_SCALE, bad
    for bad in (dict(x_row=1016), dict(gate_row=1025), dict(x=GB + 8), dict(gate=2 * GB + 2),
                dict(post=3 * GB + 4), dict(w=4 * GB + 8), dict(res=5 * GB + 4),
                dict(res_out=6 * GB + 8), dict(out=7 * GB + 2)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    for bad in (dict(out=1 * GB), dict(out=2 * GB), dict(out=6 * GB), dict(out=5 * GB),
                dict(res_out=5 * GB + 16), dict(res_out=1 * GB), dict(out=3 * GB),
                dict(res_out=4 * GB)):
        assert st(**bad) == kda.KDA_ERR_BAD_ALIAS, bad


ROPE = ("q q_row q_out q_out_row k k_row k_out k_out_row freqs rot amp inter inverse pos offsets "
        "cu N B T Hq Hk D").split()
ROPE_BASE = dict(q=1 * GB, q_row=1024, q_out=2 * GB, q_out_row=1024, k=3 * GB, k_row=256,
                 k_out=4 * GB, k_out_row=256, freqs=5 * GB, rot=128, amp=1.0, inter=0, inverse=0,
                 pos=None, offsets=6 * GB, cu=None, N=3, B=3, T=20, Hq=8, Hk=2, D=128)


def test_rope_refusals(lib):
    st = lambda **o: _call(lib.kda_rope_check, ROPE, ROPE_BASE, **o)
    packed = dict(cu=7 * GB, B=1, N=5)
    assert st() == st(**packed) == st(offsets=None) == st(pos=8 * GB, offsets=None) == kda.KDA_OK
    assert st(Hk=0, k=None, k_out=None) == st(rot=2) == st(rot=34) == kda.KDA_OK
    assert st(**packed, T=0, q=None, k=None, q_out=None, k_out=None) == kda.KDA_OK
    for name in ("q", "k", "q_out", "k_out", "freqs"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(rot=0), dict(rot=3), dict(rot=130), dict(D=100), dict(D=0), dict(D=2048),
                dict(Hq=0), dict(Hk=-1), dict(T=0), dict(B=0), dict(T=1 << 24), dict(Hq=1 << 30),
                dict(q_row=1 << 61)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(N=4), dict(cu=7 * GB), dict(pos=8 * GB),
                dict(packed, pos=8 * GB, offsets=None)):
        assert st(**bad) == kda.KDA_ERR_BAD_VARLEN, bad
    assert st(amp=math.inf) == st(amp=math.nan) == kda.KDA_ERR_BAD_SCALE
    for bad in (dict(q_row=1016), dict(k_row=257), dict(q_out_row=8), dict(q=GB + 8),
                dict(k_out=4 * GB + 2)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    # in place, also as columns of one projection's rows; nothing else may be shared
    wide = dict(q_row=2048, k_row=2048, k=GB + 2048)
    assert st(q_out=1 * GB, k_out=3 * GB) == st(**wide) == kda.KDA_OK
    assert st(**wide, q_out=GB, q_out_row=2048, k_out=GB + 2048, k_out_row=2048) == kda.KDA_OK
    for bad in (dict(q_out=GB + 16), dict(q_out=GB, q_out_row=1032), dict(q_out=3 * GB),
                dict(k_out=1 * GB), dict(k_out=2 * GB), dict(q_out=5 * GB), dict(k_out=6 * GB),
                dict(wide, k_out=GB + 1024, k_out_row=2048),
                dict(wide, k_out=GB + 3840, k_out_row=2048)):
        assert st(**bad) == kda.KDA_ERR_BAD_ALIAS, bad
    assert st(**wide, k_out=GB + 3584, k_out_row=2048) == kda.KDA_OK


PUT = ("k k_row v v_row k4 ks v4 vs slots cap k_out v_out offsets slot cu N B T Hk D").split()
PUT_BASE = dict(k=1 * GB, k_row=256, v=2 * GB, v_row=512, k4=10 * GB, ks=20 * GB, v4=30 * GB,
                vs=40 * GB, slots=4, cap=1024, k_out=3 * GB, v_out=4 * GB, offsets=5 * GB,
                slot=6 * GB, cu=None, N=3, B=3, T=20, Hk=2, D=128)


def test_put_refusals(lib):
    st = lambda **o: _call(lib.kda_cache4_put_check, PUT, PUT_BASE, **o)
    packed = dict(cu=7 * GB, B=1, N=9)
    assert st() == st(**packed) == st(offsets=None, slot=None) == kda.KDA_OK
    assert st(k_out=None, v_out=None) == st(D=64) == st(cap=32) == kda.KDA_OK
    assert st(**packed, T=0, k=None, v=None) == kda.KDA_OK
    for bad in [{name: None} for name in ("k", "v", "k4", "ks", "v4", "vs", "k_out", "v_out")]:
        assert st(**bad) == kda.KDA_ERR_NULL_ARG, bad
    for bad in (dict(D=32), dict(D=96), dict(cap=0), dict(cap=1000), dict(cap=1 << 31),
                dict(slots=0), dict(Hk=0), dict(Hk=1 << 24), dict(T=0), dict(B=0), dict(T=-1),
                dict(packed, slot=None), dict(slots=1 << 60), dict(T=1 << 38),
                dict(k_row=1 << 61)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(N=2), dict(cu=7 * GB), dict(packed, N=0)):
        assert st(**bad) == kda.KDA_ERR_BAD_VARLEN, bad
    for bad in (dict(k_row=248), dict(v_row=260), dict(k=GB + 8), dict(k4=10 * GB + 8),
                dict(vs=40 * GB + 4), dict(v_out=4 * GB + 2)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    end = 10 * GB + 4 * 2 * 1024 * 64
    for name in ("k", "v", "ks", "v4", "vs", "k_out", "v_out", "offsets", "slot"):
        assert st(**{name: end - 16}) == kda.KDA_ERR_BAD_ALIAS, name
        assert st(**{name: end}) == kda.KDA_OK, name
    assert st(k_out=1 * GB) == st(v_out=3 * GB) == kda.KDA_ERR_BAD_ALIAS


ATTN4 = ("q q_row k4 ks v4 vs slots cap scale out lse cu k_lens slot N Bq Tq Hq Hk D part ws "
         "ws_bytes").split()
ATTN4_BASE = dict(q=1 * GB, q_row=1024, k4=10 * GB, ks=20 * GB, v4=30 * GB, vs=40 * GB, slots=4,
                  cap=1024, scale=0.1, out=2 * GB, lse=3 * GB, cu=None, k_lens=4 * GB,
                  slot=5 * GB, N=3, Bq=3, Tq=20, Hq=8, Hk=2, D=128, part=0, ws=None, ws_bytes=0)


def test_attn4_refusals(lib):
    st = lambda **o: _call(lib.kda_attn4_fwd_check, ATTN4, ATTN4_BASE, **o)
    packed = dict(cu=6 * GB, Bq=1, N=9)
    assert st() == st(**packed) == st(lse=None, k_lens=None, slot=None) == kda.KDA_OK
    assert st(D=64) == st(Tq=0, q=None, out=None) == st(cap=32) == st(scale=0.0) == kda.KDA_OK
    for name in ("q", "out", "k4", "ks", "v4", "vs"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(D=32), dict(D=96), dict(Hk=3), dict(Hk=0), dict(Hq=0), dict(N=0), dict(Tq=-1),
                dict(cap=0), dict(cap=1000), dict(cap=1 << 31), dict(slots=0),
                dict(Tq=(1 << 28) + 1), dict(q_row=1 << 24), dict(N=5, Bq=5, slot=None),
                dict(packed, slot=None), dict(Hq=1 << 30)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(N=4), dict(Bq=2), dict(cu=6 * GB), dict(Bq=1)):
        assert st(**bad) == kda.KDA_ERR_BAD_VARLEN, bad
    for s in (math.inf, math.nan, -0.1):
        assert st(scale=s) == kda.KDA_ERR_BAD_SCALE
    for bad in (dict(q_row=1016), dict(q=GB + 8), dict(out=2 * GB + 8), dict(k4=10 * GB + 8),
                dict(ks=20 * GB + 1), dict(ws=50 * GB + 8)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    for part in (-32, 1, 100):
        assert st(part=part) == kda.KDA_ERR_BAD_SCHEDULE, part
    assert st(part=32, cap=4096) == kda.KDA_ERR_BAD_SCHEDULE
    for bad in (dict(out=1 * GB), dict(out=10 * GB), dict(lse=2 * GB), dict(lse=20 * GB),
                dict(out=4 * GB), dict(out=5 * GB)):
        assert st(**bad) == kda.KDA_ERR_BAD_ALIAS, bad
    sizes = (3, 3, 20, 1024, 8, 2, 128)
    need = lib.kda_attn4_workspace_bytes(*sizes, 256)
    assert need == 4 * 60 * 8 * 130 * 4
    assert st(part=256) == kda.KDA_ERR_NULL_ARG
    assert st(part=256, ws=50 * GB, ws_bytes=need - 1) == kda.KDA_ERR_BAD_WORKSPACE
    assert st(part=256, ws=50 * GB, ws_bytes=need) == kda.KDA_OK
    for at in (1 * GB, 2 * GB, 3 * GB, 40 * GB):
        assert st(part=256, ws=at, ws_bytes=need) == kda.KDA_ERR_BAD_ALIAS, at
    assert lib.kda_attn4_workspace_bytes(*sizes, 1024) == 0
    assert lib.kda_attn4_workspace_bytes(*sizes, 1 << 20) == 0
    assert lib.kda_attn4_workspace_bytes(1, 1, 1, 32768, 32, 8, 128, 0) > 0
    # prompts: the caches in bf16 and their lengths, but 8 GiB at most; without a workspace none
    prompt = (3, 1, 2024, 2208, 96, 8, 128)
    assert lib.kda_attn4_workspace_bytes(*prompt, 0) == 3 * 2208 * 8 * 128 * 4 + 32
    assert lib.kda_attn4_workspace_bytes(*prompt, 2208) == 0
    assert lib.kda_attn4_workspace_bytes(64, 64, 1024, 1 << 17, 32, 8, 128, 0) == 0
    big = dict(cu=6 * GB, N=3, Bq=1, Tq=2024, cap=2208, Hq=96, Hk=8, q_row=96 * 128)
    assert st(**big) == kda.KDA_OK
    assert st(**big, ws=50 * GB, ws_bytes=1 << 20) == kda.KDA_ERR_BAD_WORKSPACE
    assert st(**big, ws=50 * GB, ws_bytes=GB) == kda.KDA_OK
    assert st(**big, ws=40 * GB, ws_bytes=GB) == kda.KDA_ERR_BAD_ALIAS
    for bad in ((0,) + sizes[1:], sizes[:6] + (80,)):
        assert lib.kda_attn4_workspace_bytes(*bad, 0) == kda.KDA_ERR_BAD_SHAPE


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    c = kda.kda_cache4_empty(1, 4, 64, 64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_norm(x, x, weight=torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_rope(x, None, torch.ones(8, dtype=torch.float64), x, None)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_cache4_put(x, x, *c)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_attn4_fwd(x, *c, 1.0, x)
    with pytest.raises(TypeError, match="x must be a tensor"):
        kda.kda_norm(None, x)
    with pytest.raises(ValueError, match="capacity"):
        kda.kda_cache4_empty(1, 4, 65, 64, device="cpu")


def test_frequencies():
    f, a = kda.kda_rope_freqs(64, base=500000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and a == 1.0
    assert f[0] == 1 and math.isclose(float(f[31]), 500000.0 ** (-62 / 64), rel_tol=1e-14)
    g, a = kda.kda_rope_freqs(64, base=500000.0, method="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4) and a == 1.0
    y, a = kda.kda_rope_freqs(64, base=500000.0, method="yarn", factor=4.0, original=8192,
                              device="cpu")
    turns = 8192 * f / (2 * math.pi)
    assert math.isclose(a, 0.1 * math.log(4.0) + 1, rel_tol=1e-14)
    assert torch.equal(y[turns >= 32], f[turns >= 32])
    assert torch.equal(y[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (y[mid] < f[mid]).all() and (y[mid] > f[mid] / 4).all()
    for bad in (dict(rot=0), dict(rot=7), dict(rot=8, base=0.0), dict(rot=8, factor=-1.0),
                dict(rot=8, method="other"), dict(rot=8, slow=2.0, fast=1.0)):
        with pytest.raises(ValueError):
            kda.kda_rope_freqs(**dict(dict(device="cpu"), **bad))


def test_quantiser_form():
    """The form itself: every bf16 magnitude alone in its block keeps within half a code's step,
    known blocks have known codes, packing is undone by unpacking."""
    bits = torch.arange(0x7f80, dtype=torch.int32)
    x = (bits << 16).view(torch.float32).double()
    block = torch.zeros((len(bits), 32), dtype=torch.float64)
    block[:, 5] = x
    block[:, 7] = -x / 3
    code, byte = forms.quantise(block)
    scale = torch.exp2(byte[:, 0].double() - 127)
    assert (x <= 6 * scale).all() and ((x > 3 * scale) | (byte[:, 0] == 0)).all()
    got = forms.values(code, byte)
    fits = x < 1.75 * 2.0 ** 127  # above, the code stands for 2^128
    assert ((got[:, 5] - x).abs()[fits] <= scale[fits]).all()
    assert torch.isinf(got[~fits, 5]).all()
    known = torch.tensor([0, .25, .26, .75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5, 5.01, 6, -0.0, -.5,
                          -5] + [0.0] * 16)
    code, byte = forms.quantise(known)
    assert byte.tolist() == [127]
    assert code[:16].tolist() == [0, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 8, 9, 14]
    for odd in (math.inf, math.nan):
        block = torch.ones(64)
        block[40] = odd
        code, byte = forms.quantise(block)
        assert byte.tolist() == [125, 255] and not code[32:].any()
        assert torch.isnan(forms.values(code, byte)[32:]).all()
    for D in (64, 128):
        code = torch.randint(0, 16, (2, 3, 64, D))
        byte = torch.randint(0, 256, (2, 3, 64, D // 32))
        for v in (False, True):
            back = forms.unpack(*forms.pack(code, byte, D, v), D, v)
            assert torch.equal(back[0], code) and torch.equal(back[1], byte)
