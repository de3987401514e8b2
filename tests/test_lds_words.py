"""CPU guard on the single words that attention over 4-bit caches loads from memory to LDS
(load_lds_word, inline assembly), beside the wider loads of tests/test_lds_loads.py: what the
compiler knows of them, from the gfx950 assembly of small kernels around them.  Nothing runs."""
from __future__ import annotations

import re
import subprocess

import pytest

from gated_delta_rule_62_amd import _build
from tests.test_lds_loads import _kernel

SOURCE = """
#include "attn4_kernel.hip"
namespace kda {
__global__ void probe_word_m0(const uint8_t* src, unsigned* out, int which) {
  __shared__ alignas(1024) unsigned a[2][64];
  const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(src, 2048);
  auto to = (__attribute__((address_space(3))) void*)&a[which][0];
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, threadIdx.x * 4, 0, 0, 0);
  load_lds_word<ONCE>(src + 4 * threadIdx.x, (const uint8_t*)&a[1 - which][0]);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, threadIdx.x * 4 + 256, 0, 0, 0);
  lds_barrier();
  out[threadIdx.x] = a[which][threadIdx.x];
}
__global__ void probe_word_waits(const uint8_t* src, int* out) {
  __shared__ alignas(1024) int a[64];
  load_lds_word<ONCE>(src + 4 * threadIdx.x, (const uint8_t*)a);
  const int before = a[threadIdx.x];
  wait_loads();
  const int after = a[threadIdx.x];
  wait_lds();
  load_lds_word<ONCE>(src + 4 * threadIdx.x, (const uint8_t*)a);
  out[threadIdx.x] = before + 3 * after;
}
}
"""


@pytest.fixture(scope="module", params=["true", "false"])
def asm(request, tmp_path_factory):
    folder = tmp_path_factory.mktemp("lds_words")
    src, out = folder / "probe.hip", folder / "probe.s"
    src.write_text(SOURCE.replace("ONCE", request.param))
    subprocess.run([_build.hipcc()] + _build.HIP_FLAGS +
                   ["-I" + _build.CSRC, "--cuda-device-only", "-S", "-x", "hip", str(src), "-o",
                    str(out)], check=True, capture_output=True)
    text = out.read_text()
    words = [line for line in text.splitlines() if "global_load_lds_dword " in line]
    assert words and any(line.rstrip().endswith(" nt") for line in words)
    return text


def test_the_address_register_is_known_to_change(asm):
    """A load to LDS by the compiler's own means, on both sides of a word's to another place: the
    second has its address register written again."""
    loads, written = [], False
    for line in _kernel(asm, "probe_word_m0"):
        written |= line.startswith("s_mov_b32 m0")
        if line.startswith("global_load_lds") or line.startswith("buffer_load") and "lds" in line:
            loads.append((line.split("_")[0], written))
            written = False
    assert loads == [("buffer", True), ("global", True), ("buffer", True)], loads


def test_no_access_moves_over_a_wait(asm):
    """LDS is read before and after the wait for the word, and no load starts before the wait for
    the reads."""
    order = [op for line in _kernel(asm, "probe_word_waits") for op in
             [line.split()[0] if line.startswith(("ds_read", "global_load")) else
              "vm" if "s_waitcnt vmcnt(0)" in line else
              "lgkm" if line.startswith("s_waitcnt lgkmcnt(0)") else None] if op]
    text = " ".join(order)
    assert re.search(r"global_load_lds_dword ds_read_b32 (lgkm )?vm (lgkm )?ds_read_b32 lgkm "
                     r"global_load_lds_dword", text), text
    assert len(re.findall("ds_read", text)) == 2, text


def test_a_tile_waits_for_every_load_of_the_older_pair(asm):
    """The loop over the keys waits until the loads of one pair of tiles are left, as many as a
    pair has: the count of the instructions and the number in the wait agree."""
    for D, loads in ((64, 3), (128, 5)):
        for name in re.findall(r"^(_ZN3kda\S*attn4_kernelILi%dE\S*):" % D, asm, re.M):
            body = asm[asm.index(name + ":"):]
            body = body[:body.index(".Lfunc_end")]
            waits = {int(x) for x in re.findall(r"s_waitcnt vmcnt\((\d+)\)", body)}
            assert 2 * loads in waits, (name, waits)
            count = len(re.findall(r"global_load_lds_dword |buffer_load_dwordx4 .* lds", body))
            assert count % loads == 0 and count > 0, (name, count)
