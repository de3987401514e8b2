"""CPU guard on the attention kernels' loads from memory to LDS (inline assembly): what the
compiler knows of them, from the gfx950 assembly of small kernels around them.  Nothing runs."""
from __future__ import annotations

import re
import subprocess

import pytest

from gated_delta_rule_62_amd import _build

SOURCE = """
#include "attn_kernel.hip"
namespace kda {
__global__ void probe_m0(const u16* src, u16* out, int which) {
  __shared__ alignas(1024) u16 a[2][512];
  const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(src, 2048);
  auto to = (__attribute__((address_space(3))) void*)&a[which][0];
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, threadIdx.x * 4, 0, 0, 0);
  load_lds<ONCE>(rows_words(src, 512, 2, 128), &a[1 - which][0], threadIdx.x * 16);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, threadIdx.x * 4 + 256, 0, 0, 0);
  lds_barrier();
  out[threadIdx.x] = a[which][threadIdx.x];
}
__global__ void probe_waits(const u16* src, int* out) {
  __shared__ alignas(1024) int a[256];
  load_lds<ONCE>(rows_words(src, 512, 2, 128), (const u16*)a, threadIdx.x * 16);
  const int before = a[threadIdx.x];
  wait_loads();
  const int after = a[threadIdx.x];
  wait_lds();
  load_lds<ONCE>(rows_words(src, 512, 2, 128), (const u16*)a, threadIdx.x * 16);
  out[threadIdx.x] = before + 3 * after;
}
}
"""


@pytest.fixture(scope="module", params=["true", "false"])
def asm(request, tmp_path_factory):
    folder = tmp_path_factory.mktemp("lds")
    src, out = folder / "probe.hip", folder / "probe.s"
    src.write_text(SOURCE.replace("ONCE", request.param))
    subprocess.run([_build.hipcc()] + _build.HIP_FLAGS +
                   ["-I" + _build.CSRC, "--cuda-device-only", "-S", "-x", "hip", str(src), "-o",
                    str(out)], check=True, capture_output=True)
    return out.read_text()


def _kernel(asm, name):
    body = asm[re.search(r"^_ZN3kda\d+%s\w*:" % name, asm, re.M).end():]
    lines = [line.split(";")[0].strip() for line in body[:body.index("s_endpgm")].splitlines()]
    return [line for line in lines if line]


def test_the_address_register_is_known_to_change(asm):
    """A load to LDS by the compiler's own means, on both sides of one of ours to another place:
    the second has its address register written again."""
    loads, written = [], False
    for line in _kernel(asm, "probe_m0"):
        written |= line.startswith("s_mov_b32 m0")
        if line.startswith("buffer_load") and "lds" in line:
            loads.append(written)
            written = False
    assert loads == [True, True, True], loads


def test_no_access_moves_over_a_wait(asm):
    """LDS is read before and after the wait for the loads, and no load starts before the wait
    for the reads."""
    order = [op for line in _kernel(asm, "probe_waits") for op in
             [line.split()[0] if line.startswith(("ds_read", "buffer_load")) else
              "vm" if "s_waitcnt vmcnt(0)" in line else
              "lgkm" if line.startswith("s_waitcnt lgkmcnt(0)") else None] if op]
    text = " ".join(order)
    assert re.search(r"buffer_load_dwordx4 ds_read_b32 (lgkm )?vm (lgkm )?ds_read_b32 lgkm "
                     r"buffer_load_dwordx4", text), text
    assert len(re.findall("ds_read", text)) == 2, text
