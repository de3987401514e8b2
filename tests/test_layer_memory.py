"""kda_attn4_fwd where memory is short: a workspace that torch cannot allocate is done without, as
with an empty one, unless the caller asked for parts, which need it."""
from __future__ import annotations

import types

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms


def _full(need, q, stream):
    raise torch.OutOfMemoryError("no %d bytes" % need)


def _serving():
    kda.kda_attn4_fwd  # loads the bindings
    from gated_delta_rule_62_amd import serving
    return serving


def test_the_second_call_has_an_empty_workspace(monkeypatch):
    serving = _serving()
    seen = []

    def call(fn, ws_fn, q, *rest):
        workspace = rest[-2]
        seen.append(workspace)
        return 1 << 33 if workspace is None else 0

    monkeypatch.setattr(serving, "_calls", types.SimpleNamespace(attn4_fwd=call))
    monkeypatch.setattr(serving, "_workspace", _full)
    q = torch.zeros(1, 1, 1, 64)
    serving.kda_attn4_fwd(q, q, q, q, q, 1.0, q)
    assert seen[0] is None and seen[1].dtype == torch.uint8 and seen[1].numel() == 0
    with pytest.raises(torch.OutOfMemoryError):
        serving.kda_attn4_fwd(q, q, q, q, q, 1.0, q, part=64)


@pytest.mark.gpu
def test_a_prompt_without_the_memory_to_expand_its_cache(monkeypatch):
    print("kda_attn4_fwd without memory", flush=True)
    serving = _serving()
    g = torch.Generator(device="cuda").manual_seed(3)
    L, Hq, Hk, D, cap = 900, 16, 2, 128, 928
    cache = []
    for is_v in (False, True):
        cache += forms.pack(*forms.quantise(torch.randn((1, Hk, cap, D), generator=g,
                                                        device="cuda")), D, is_v)
    q = torch.randn((1, L, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([L], device="cuda")
    assert kda.kda_attn4_workspace_bytes(1, 1, L, cap, Hq, Hk, D) > 0
    want, out = torch.empty_like(q), torch.empty_like(q)
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    kda.kda_attn4_fwd(q, *cache, 0.1, want, k_lens=lens, workspace=empty)
    monkeypatch.setattr(serving, "_workspace", _full)
    kda.kda_attn4_fwd(q, *cache, 0.1, out, k_lens=lens)
    assert torch.equal(out, want)
    with pytest.raises(torch.OutOfMemoryError):
        kda.kda_attn4_fwd(q, *cache, 0.1, out, k_lens=lens, part=64)
