"""The loads from memory to LDS that are written in assembly tell the compiler that
they write M0: a load of its own behind one sets M0 anew."""

import subprocess

from quantized_moe_expert_route_amd import build

SOURCE = """
#include "gemm_tile.h"
typedef const __attribute__((address_space(1))) int* from;
typedef __attribute__((address_space(3))) int* to;
__global__ void probe(const int* p, uint32_t lds) {
  __shared__ int l[4096];
  __builtin_amdgcn_global_load_lds((from)(p + threadIdx.x), (to)l, 4, 0, 0);
  qmoe::load_lds16(qmoe::buffer_at(p), threadIdx.x * 16, lds);
  __builtin_amdgcn_global_load_lds((from)(p + threadIdx.x + 256), (to)l, 4, 0, 0);
}
"""


def test_m0_is_set_anew(tmp_path):
    source, out = tmp_path / "probe.hip", tmp_path / "probe.s"
    source.write_text(SOURCE)
    r = subprocess.run([build._hipcc(), *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "--cuda-device-only", str(source),
                        "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    code = out.read_text()
    code = code[code.index("probe"):]
    own = code.index("buffer_load_dwordx4")
    second = code.index("global_load_lds_dword", own)
    assert "s_mov_b32 m0" in code[own:second]
    assert "inline asm clobber" not in r.stderr
