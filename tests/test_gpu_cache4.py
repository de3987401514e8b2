"""New keys and values into caches in 4 bits (kda_cache4_put): codes and scales are exactly those of
the definition in tests/layer_forms.py, and everything else stays as it was."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_62_amd as kda
import tests.layer_forms as forms

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(BF16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _dirty(g, slots, Hk, cap, D):
    c = kda.kda_cache4_empty(slots, Hk, cap, D)
    for t in c:
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


def _check(cache, before, k, v, places, D):
    """places: (token row of k and v, slot, position); the rest of the cache as before."""
    rows = [p[0] for p in places]
    for (codes, scales), (codes0, scales0), x, is_v in (
            (cache[:2], before[:2], k, False), (cache[2:], before[2:], v, True)):
        code, byte = forms.unpack(codes0, scales0, D, is_v)
        if places:
            c, b = forms.quantise(x[rows])
            slot, pos = _ints([p[1] for p in places]), _ints([p[2] for p in places])
            code[slot, :, pos], byte[slot, :, pos] = c, b
        want = forms.pack(code, byte, D, is_v)
        assert torch.equal(scales, want[1]), "scales, values %s" % is_v
        assert torch.equal(codes, want[0]), "codes, values %s" % is_v


def _put(g, lens, start, slots, S, Hk, cap, D, behind=0, packed=True, values=True, strided=True):
    B, T = (1, sum(lens) + behind) if packed else (len(lens), lens[0])
    both = _normal(g, B, T, 2 * Hk, D)
    k, v = torch.split(both, [Hk, Hk], dim=2)
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    cache = _dirty(g, S, Hk, cap, D)
    before = [t.clone() for t in cache]
    ko = torch.full((B, T, Hk, D), 7.0, dtype=BF16, device=DEV) if values else None
    vo = ko.clone() if values else None
    kda.kda_cache4_put(k, v, *cache, offsets=None if start is None else _ints(start),
                       cu_seqlens=_ints([0] + lens).cumsum(0) if packed else None,
                       slots=None if slots is None else _ints(slots), k_out=ko, v_out=vo)
    places, row = [], 0
    for n, length in enumerate(lens):
        at, s = start[n] if start else 0, slots[n] if slots else n
        places += [(row + t, s, at + t) for t in range(length)
                   if 0 <= at + t < cap and 0 <= s < S]
        row += length
    flat = lambda x: x.reshape(B * T, Hk, D)
    _check(cache, before, flat(k), flat(v), places, D)
    if values:
        for x, y in ((k, ko), (v, vo)):
            want = forms.values(*forms.quantise(flat(x)[:row])).reshape(-1, Hk, D)
            assert torch.equal(flat(y)[:row].double(), want)
            assert (flat(y)[row:] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,start,slots,S,Hk,cap", [
    ([1], [0], None, 1, 1, 32), ([1, 1, 1], [31, 32, 95], None, 3, 2, 96),
    ([5, 0, 40], [30, 3, 7], [2, 0, 4], 5, 3, 128), ([300, 33], [1, 100], [1, 0], 2, 2, 320),
    ([64, 31, 32, 33], [0, 0, 0, 0], None, 4, 1, 64), ([2], [31], [0], 1, 8, 64)])
def test_packed(lens, start, slots, S, Hk, cap, D):
    """Prompts and single tokens that begin and end inside tiles, slots in any order."""
    print("kda_cache4_put", lens, start, slots, S, Hk, cap, D, flush=True)
    g = _gen(sum(lens) + D)
    _put(g, lens, start, slots, S, Hk, cap, D)
    _put(g, lens, start, slots, S, Hk, cap, D, behind=3, values=False, strided=False)


@pytest.mark.parametrize("T,start", [(1, [5, 0, 63]), (5, [30, 31, 59]), (64, [0, 0, 0]), (33, None)])
def test_batch_rows(T, start):
    g = _gen(T)
    for D in (64, 128):
        _put(g, [T] * 3, start, None, 4, 2, 64, D, packed=False)


def test_outside():
    """Positions and slots outside the cache are left out, their values still given."""
    g = _gen(6)
    far = (1 << 63) - 3
    for D in (64, 128):
        for start, slots in (([60, 64, 1000], [0, 1, 2]), ([-3, -40, 10], [2, 1, 0]),
                             ([0, 0, 0], [-1, 3, 1 << 40]), ([far, -far, 0], [0, 1, 2])):
            _put(g, [9, 50, 2], start, slots, 3, 2, 64, D)
            _put(g, [9, 50, 2], start, slots, 3, 2, 64, D, values=False)


def test_every_magnitude():
    """Every bf16, each beside every other of its block: signed zeros, the smallest and largest,
    ties, infinities and NaN."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF16)
    order = torch.randperm(65536, generator=torch.Generator().manual_seed(1)).to(DEV)
    near = torch.sort(bits.float().nan_to_num(0.0, 0.0, 0.0).abs())[0].to(BF16)  # alike together
    for x in (bits, bits[order], near, -near, torch.full_like(bits, -0.0)):
        k = x.view(1, -1, 2, 128).contiguous()
        T = k.shape[1]
        v = k.flip(1).contiguous()
        cache = kda.kda_cache4_empty(1, 2, T, 128)
        before = [t.clone() for t in cache]
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        kda.kda_cache4_put(k, v, *cache, k_out=ko, v_out=vo)
        _check(cache, before, k[0], v[0], [(t, 0, t) for t in range(T)], 128)
        want = forms.values(*forms.quantise(k[0]))
        got = ko[0].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(1.0, 2.0, 3.0), want.nan_to_num(1.0, 2.0, 3.0))


def test_beyond_32_bit_offsets():
    """Slots more than 2^32 bytes apart."""
    g = _gen(8)
    S, Hk, cap, D = 3, 16, 1 << 22, 128
    cache = kda.kda_cache4_empty(S, Hk, cap, D)
    k, v = _normal(g, 1, 4, Hk, D), _normal(g, 1, 4, Hk, D)
    kda.kda_cache4_put(k, v, *cache, offsets=_ints([cap - 4]), slots=_ints([2]),
                       cu_seqlens=_ints([0, 4]))
    last = [t[2:, :, -32 * t.shape[2] // cap:].contiguous() for t in cache]
    _check(last, [torch.zeros_like(t) for t in last], k[0], v[0],
           [(t, 0, 28 + t) for t in range(4)], D)
    assert not any(t[:2].any() for t in cache)


def test_token_by_token_is_the_prompt():
    g = _gen(9)
    T, Hk, D = 70, 2, 64
    k, v = _normal(g, 1, T, Hk, D), _normal(g, 1, T, Hk, D)
    whole, steps = kda.kda_cache4_empty(1, Hk, 96, D), kda.kda_cache4_empty(1, Hk, 96, D)
    kda.kda_cache4_put(k, v, *whole)
    for t in range(T):
        kda.kda_cache4_put(k[:, t:t + 1], v[:, t:t + 1], *steps, offsets=_ints([t]))
    assert all(torch.equal(a, b) for a, b in zip(whole, steps))


def test_replays():
    g = _gen(10)
    k, v = _normal(g, 3, 1, 4, 128), _normal(g, 3, 1, 4, 128)
    cache = kda.kda_cache4_empty(3, 4, 64, 128)
    off = _ints([0, 5, 40])
    graph = torch.cuda.CUDAGraph()
    kda.kda_cache4_put(k, v, *cache, offsets=off)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kda.kda_cache4_put(k, v, *cache, offsets=off)
    for step in range(3):  # the replay takes the positions that the tensor holds by then
        for t in cache:
            t.zero_()
        off.add_(3)
        graph.replay()
        torch.cuda.synchronize()
        _check(cache, [torch.zeros_like(t) for t in cache], k[:, 0], v[:, 0],
               [(n, n, int(p)) for n, p in enumerate(off.tolist())], 128)
