"""Fills of LDS that go through M0, the register that says where they go: a
kernel that uses both kinds of them, compiled for gfx950 and read as assembly.
Each fill must find its own place there, whatever the other kind left."""
import importlib.util
import os
import re
import subprocess

import pytest

mod = pytest.importorskip("expert_grouping_dispatch_amd")
PKG = os.path.dirname(mod.LIB_PATH)
SOURCE = """
#include "lds_fill.h"
using namespace moe;
__global__ void both(const uint8_t* from, uint32_t* out) {
  __shared__ __align__(16) uint8_t a[2048], b[1024];
  const uint32_t off = threadIdx.x * 16;
  const __amdgpu_buffer_rsrc_t r = buffer_of(from, 4096);
  load_to_lds(r, off, 0, a);
  fill_lds(buffer_words(buffer_at(from, 4096)), off, 1024, lds_offset(b));
  load_to_lds(r, off, 2048, a);
  __builtin_amdgcn_s_waitcnt(kWaitLoads);
  __syncthreads();
  out[threadIdx.x] = a[threadIdx.x] + b[threadIdx.x];
}
"""


def test_each_fill_sets_its_own_place(tmp_path):
    spec = importlib.util.spec_from_file_location("build_lib_flags", os.path.join(PKG, "build_lib.py"))
    build_lib = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build_lib)
    source, asm = tmp_path / "both.hip", tmp_path / "both.s"
    source.write_text(SOURCE)
    r = subprocess.run([build_lib.hipcc(), *build_lib.HIPCC_FLAGS, "--offload-device-only", "-S", str(source), "-o", str(asm)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    places, m0 = [], None
    for line in asm.read_text().splitlines():
        if w := re.match(r"\s*s_\w+\s+m0,\s*(.*)", line):
            m0 = w.group(1).strip()
        elif re.match(r"\s*buffer_load_\S+ .*\blds\b", line):
            places.append(m0)
    assert len(places) == 3 and None not in places, places
    assert places[0] == places[2] != places[1], places
