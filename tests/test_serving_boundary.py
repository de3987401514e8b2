"""Refusals of the serving operators, on the CPU: their *_check functions compare pointer
values and sizes only, and the bindings refuse tensors before anything is launched."""
from __future__ import annotations

import os

import pytest
import torch

import gated_delta_rule_62_amd as kda

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


STEP = ("q k v g beta scale out A_log dt_bias lb state dtype slots slot_in slot_out N H D").split()
STEP_BASE = dict(q=1 * GB, k=2 * GB, v=3 * GB, g=4 * GB, beta=5 * GB, scale=0.1, out=6 * GB,
                 A_log=7 * GB, dt_bias=8 * GB, lb=-5.0, state=100 * GB, dtype=1, slots=16,
                 slot_in=None, slot_out=None, N=8, H=4, D=128)


def test_step_refusals(lib):
    st = lambda **o: _call(lib.kda_step_check, STEP, STEP_BASE, **o)
    assert st() == kda.KDA_OK
    assert st(slot_in=9 * GB, slot_out=10 * GB, N=64) == kda.KDA_OK
    assert st(N=0, q=None, k=None, v=None, g=None, beta=None, out=None) == kda.KDA_OK
    for name in ("q", "k", "v", "g", "beta", "out", "A_log", "dt_bias", "state"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(N=-1), dict(H=0), dict(D=96), dict(D=0), dict(slots=0), dict(N=17),
                dict(H=1 << 24), dict(N=1 << 40, slot_in=9 * GB), dict(H=1 << 62),
                dict(N=1 << 22, slot_in=9 * GB), dict(slots=1 << 50)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    assert st(dtype=2) == kda.KDA_ERR_BAD_DTYPE
    for s in (float("inf"), float("nan")):
        assert st(scale=s) == kda.KDA_ERR_BAD_SCALE
    for lb in (0.0, 1.0, float("nan"), float("-inf")):
        assert st(lb=lb) == kda.KDA_ERR_BAD_LOWER_BOUND
    for name in ("q", "k", "v", "g", "out", "state"):
        assert st(**{name: STEP_BASE[name] + 8}) == kda.KDA_ERR_BAD_LAYOUT, name
    pool_end = 100 * GB + 16 * 4 * 128 * 128 * 4
    for name in ("q", "k", "v", "g", "beta", "out", "A_log", "dt_bias"):
        assert st(**{name: pool_end - 16}) == kda.KDA_ERR_BAD_ALIAS, name
        assert st(**{name: pool_end}) == kda.KDA_OK, name
    assert st(out=1 * GB) == kda.KDA_ERR_BAD_ALIAS
    assert st(slot_in=6 * GB + 16, out=6 * GB) == kda.KDA_ERR_BAD_ALIAS


LA_STEP = ("q q_row k k_row v v_row g decay scale out state dtype slots slot_in slot_out N H Hk "
           "D").split()
LA_STEP_BASE = dict(q=1 * GB, q_row=256, k=2 * GB, k_row=256, v=3 * GB, v_row=512, g=4 * GB,
                    decay=5 * GB, scale=0.1, out=6 * GB, state=100 * GB, dtype=0, slots=16,
                    slot_in=None, slot_out=None, N=8, H=4, Hk=2, D=128)


def test_la_step_refusals(lib):
    st = lambda **o: _call(lib.kda_la_step_check, LA_STEP, LA_STEP_BASE, **o)
    assert st() == kda.KDA_OK
    assert st(g=None, decay=None) == kda.KDA_OK
    assert st(q_row=264, k_row=1 << 20, v_row=520) == kda.KDA_OK
    assert st(N=0, q=None, k=None, v=None, g=None, out=None) == kda.KDA_OK
    for name in ("q", "k", "v", "out", "state"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(Hk=3), dict(Hk=0), dict(Hk=8), dict(D=48), dict(N=17), dict(q_row=1 << 61)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(q_row=248), dict(k_row=257), dict(v_row=0), dict(v_row=-512), dict(q=GB + 2),
                dict(out=6 * GB + 4)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    # views of one projection's rows interleave: inputs may, outputs may not lie between them
    assert st(q_row=1024, k=GB + 512, k_row=1024, v=GB + 1024, v_row=1024) == kda.KDA_OK
    assert st(q_row=1024, out=GB + 1024) == kda.KDA_ERR_BAD_ALIAS
    for name in ("g", "decay", "slot_in", "slot_out"):
        assert st(**{name: 6 * GB + 64}) == kda.KDA_ERR_BAD_ALIAS, name


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros((2, 4, 32), dtype=torch.bfloat16)
    b = torch.zeros((2, 4), dtype=torch.bfloat16)
    pool = torch.zeros((2, 4, 32, 32))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_step(x, x, x, x, b, 1.0, x, torch.zeros(4), torch.zeros(4, 32), -1.0, pool)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_la_step(x, x, x, None, 1.0, x, pool)
    y, cu = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16), torch.tensor([0, 2])
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_la_fwd(y, y, y, None, 1.0, y, cu_seqlens=cu)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_attn_fwd(y, y, y, 1.0, y)
    with pytest.raises(TypeError, match="q must be a tensor"):
        kda.kda_attn_fwd(None, y, y, 1.0, y)
    with pytest.raises(ValueError, match="q and v"):
        kda.kda_la_fwd(x, x, x, None, 1.0, x)


LA = ("q q_row k k_row v v_row g decay scale out s_in in_dtype s_out out_dtype cu N B T H Hk D "
      "segment ws ws_bytes").split()
LA_BASE = dict(q=1 * GB, q_row=256, k=2 * GB, k_row=256, v=3 * GB, v_row=512, g=4 * GB,
               decay=5 * GB, scale=0.1, out=6 * GB, s_in=7 * GB, in_dtype=1, s_out=8 * GB,
               out_dtype=0, cu=None, N=2, B=2, T=100, H=4, Hk=2, D=128, segment=0, ws=None,
               ws_bytes=0)


def test_la_fwd_refusals(lib):
    st = lambda **o: _call(lib.kda_la_fwd_check, LA, LA_BASE, **o)
    packed = dict(cu=9 * GB, B=1, N=5)
    assert st() == kda.KDA_OK and st(**packed) == kda.KDA_OK
    assert st(g=None, decay=None, s_in=None, s_out=None) == kda.KDA_OK
    assert st(**packed, T=0, q=None, k=None, v=None, out=None, g=None) == kda.KDA_OK
    for name in ("q", "k", "v", "out"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(Hk=3), dict(Hk=0), dict(D=96), dict(B=0), dict(T=0), dict(T=-1),
                dict(q_row=1 << 24), dict(v_row=1 << 40), dict(H=1 << 17), dict(T=1 << 41),
                dict(H=1 << 62), dict(N=1 << 30, B=1 << 30)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(N=3), dict(cu=9 * GB), dict(cu=9 * GB, B=1, N=0)):
        assert st(**bad) == kda.KDA_ERR_BAD_VARLEN, bad
    assert st(in_dtype=2) == st(out_dtype=-1) == kda.KDA_ERR_BAD_DTYPE
    assert st(scale=float("nan")) == kda.KDA_ERR_BAD_SCALE
    for bad in (dict(q_row=248), dict(k_row=260), dict(v_row=504), dict(s_in=7 * GB + 4),
                dict(s_out=8 * GB + 8), dict(out=6 * GB + 2), dict(ws=20 * GB + 8)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    for seg in (-64, 1, 63, 100, 1 << 21):
        assert st(segment=seg) == kda.KDA_ERR_BAD_SCHEDULE, seg
    # the exact state alias only
    assert st(s_out=7 * GB, out_dtype=1) == kda.KDA_OK
    assert st(s_out=7 * GB, out_dtype=0) == kda.KDA_ERR_BAD_ALIAS
    assert st(s_out=7 * GB + 64, out_dtype=1) == kda.KDA_ERR_BAD_ALIAS
    for over in (dict(out=1 * GB), dict(out=7 * GB), dict(s_out=3 * GB), dict(s_out=6 * GB),
                 dict(out=4 * GB + 64)):
        assert st(**over) == kda.KDA_ERR_BAD_ALIAS, over
    # segments need their workspace
    need = lib.kda_la_workspace_bytes(200, 2, 4, 128, 64)
    assert need == (200 // 64 + 3) * 4 * (128 * 128 + 1) * 4
    assert st(segment=64) == kda.KDA_ERR_NULL_ARG
    assert st(segment=64, ws=20 * GB, ws_bytes=need - 1) == kda.KDA_ERR_BAD_WORKSPACE
    assert st(segment=64, ws=20 * GB, ws_bytes=need) == kda.KDA_OK
    for at in (6 * GB, 8 * GB, 7 * GB, 1 * GB):
        assert st(segment=64, ws=at, ws_bytes=need) == kda.KDA_ERR_BAD_ALIAS, at
    assert lib.kda_la_workspace_bytes(200, 2, 4, 128, 0) == 0
    assert lib.kda_la_workspace_bytes(1 << 15, 1, 32, 128, 0) > 0
    for bad in ((-1, 1, 4, 128, 0), (1, 0, 4, 128, 0), (1, 1, 0, 128, 0), (1, 1, 4, 100, 0),
                (1 << 40, 1, 1 << 10, 128, 64), (1 << 62, 1, 4, 128, 0)):
        assert lib.kda_la_workspace_bytes(*bad) == kda.KDA_ERR_BAD_SHAPE, bad


ATTN = ("q q_row k k_row v v_row scale out lse cu_q cu_k k_lens N Bq Tq Bk Tk Hq Hk D splits ws "
        "ws_bytes").split()
ATTN_BASE = dict(q=1 * GB, q_row=1024, k=2 * GB, k_row=256, v=3 * GB, v_row=256, scale=0.1,
                 out=4 * GB, lse=5 * GB, cu_q=None, cu_k=None, k_lens=None, N=3, Bq=3, Tq=20, Bk=3,
                 Tk=50, Hq=8, Hk=2, D=128, splits=0, ws=None, ws_bytes=0)


def test_attn_refusals(lib):
    st = lambda **o: _call(lib.kda_attn_fwd_check, ATTN, ATTN_BASE, **o)
    packed = dict(cu_q=6 * GB, cu_k=7 * GB, Bq=1, Bk=1)
    assert st() == st(**packed) == st(lse=None) == kda.KDA_OK
    assert st(k_lens=8 * GB) == kda.KDA_OK
    assert st(cu_q=6 * GB, Bq=1, k_lens=8 * GB) == kda.KDA_OK  # packed queries, cache rows
    assert st(cu_k=7 * GB, Bk=1) == kda.KDA_OK
    assert st(Tq=0, q=None, out=None, lse=None) == kda.KDA_OK
    assert st(Tk=0, k=None, v=None) == kda.KDA_OK
    for name in ("q", "k", "v", "out"):
        assert st(**{name: None}) == kda.KDA_ERR_NULL_ARG, name
    for bad in (dict(D=32), dict(D=96), dict(Hk=3), dict(Hk=0), dict(Hq=0), dict(N=0), dict(Tq=-1),
                dict(Tk=(1 << 30) + 1), dict(Tq=(1 << 28) + 1), dict(q_row=1 << 24),
                dict(k_row=1 << 33), dict(Hq=1 << 30), dict(N=1 << 40, Bq=1 << 40, Bk=1 << 40),
                dict(Tq=1 << 28, N=1 << 20, Bq=1 << 20, Bk=1 << 20)):
        assert st(**bad) == kda.KDA_ERR_BAD_SHAPE, bad
    for bad in (dict(N=4), dict(Bq=2), dict(Bk=2), dict(cu_q=6 * GB), dict(cu_k=7 * GB),
                dict(Bq=1), dict(Bk=1), dict(packed, k_lens=8 * GB)):
        assert st(**bad) == kda.KDA_ERR_BAD_VARLEN, bad
    for s in (float("inf"), float("nan"), -0.1):
        assert st(scale=s) == kda.KDA_ERR_BAD_SCALE
    for bad in (dict(q_row=1016), dict(k_row=255), dict(v_row=260), dict(k=2 * GB + 2),
                dict(out=4 * GB + 8), dict(ws=9 * GB + 4)):
        assert st(**bad) == kda.KDA_ERR_BAD_LAYOUT, bad
    for bad in (-1, 65):
        assert st(splits=bad) == kda.KDA_ERR_BAD_SCHEDULE
    for bad in (dict(out=1 * GB), dict(lse=4 * GB), dict(out=3 * GB - 16), dict(lse=2 * GB),
                dict(k_lens=4 * GB)):
        assert st(**bad) == kda.KDA_ERR_BAD_ALIAS, bad
    sizes = (3, 3, 20, 3, 50, 8, 2, 128)
    need = lib.kda_attn_workspace_bytes(*sizes, 4)
    assert need == 4 * 60 * 8 * 130 * 4
    assert st(splits=4) == kda.KDA_ERR_NULL_ARG
    assert st(splits=4, ws=9 * GB, ws_bytes=need - 1) == kda.KDA_ERR_BAD_WORKSPACE
    assert st(splits=4, ws=9 * GB, ws_bytes=need) == kda.KDA_OK
    for at in (1 * GB, 4 * GB, 5 * GB):
        assert st(splits=4, ws=at, ws_bytes=need) == kda.KDA_ERR_BAD_ALIAS
    assert lib.kda_attn_workspace_bytes(*sizes, 1) == 0
    assert lib.kda_attn_workspace_bytes(1, 1, 1, 1, 8192, 32, 8, 128, 0) > 0
    assert lib.kda_attn_workspace_bytes(1, 1, 8192, 1, 8192, 32, 8, 128, 0) == 0
    # a million query tokens of 96 heads is one launch; parts of them would be too many rows
    big = dict(N=1, Bq=1, Bk=1, Tq=1 << 20, Tk=1 << 20, Hq=96, Hk=8, q_row=96 * 128, k_row=8 * 128,
               v_row=8 * 128, q=100 * GB, k=200 * GB, v=300 * GB, out=400 * GB, lse=500 * GB)
    assert st(**big) == kda.KDA_OK
    assert st(**big, splits=2, ws=600 * GB, ws_bytes=1 << 50) == kda.KDA_ERR_BAD_SHAPE
    for bad in ((0,) + sizes[1:], sizes[:7] + (80,)):
        assert lib.kda_attn_workspace_bytes(*bad, 0) == kda.KDA_ERR_BAD_SHAPE
