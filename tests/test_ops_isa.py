"""The delta rule's loads into LDS are written as assembly, which the compiler's own pass for wait
states does not look into.  gfx9 asks for 5 wait states between a vector instruction's write of a
scalar register and a memory instruction's read of it; these tests count them in the code that the
compiler makes of the sources.  No GPU needed."""
import os
import re
import subprocess

import pytest

from selective_state_space_msm_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")

# an extent that the lanes share, brought to a scalar register right before the load
PROBE = r"""
#include "ops_delta.hpp"
namespace msm {
__global__ void probe(const int* extent, const void* from, float* to) {
  __shared__ __attribute__((aligned(16))) float lds[256];
  const int n = uniform(extent[threadIdx.x]);
  load_lds(rsrc_words(from, (uint32_t)n), (MSM_LDS void*)lds, threadIdx.x * 16);
  sync_loads();
  to[threadIdx.x] = lds[threadIdx.x];
}
}
"""


def assembly(source, flags, tmp_path):
    out = str(tmp_path / "out.s")
    r = subprocess.run([build.HIPCC, *build.COMMON, *flags, "-S", "--cuda-device-only", source, "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0 and "warning:" not in r.stderr, r.stdout + r.stderr
    with open(out) as f:
        return f.read()


def scalars(token):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", token) or re.fullmatch(r"s((\d+))", token)
    return range(int(m[1]), int(m[2]) + 1) if m else ()


def short_waits(text):
    """(loads into LDS seen, memory instructions too close behind a vector write of their scalars)."""
    since, seen, short = {}, 0, []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if line.endswith(":"):
            if line.startswith("_Z"):
                since = {}
            continue
        if not line or line.startswith("."):
            continue
        op, _, rest = line.partition(" ")
        tokens = [x for t in re.split(r",\s*(?![^\[]*\])", rest.strip()) for x in t.split()]
        if op.startswith(("buffer_", "global_", "scratch_", "flat_")):
            seen += "lds" in tokens
            short += [(line, since[r]) for t in tokens for r in scalars(t) if since.get(r, 5) < 5]
        states = int(tokens[0]) + 1 if op == "s_nop" else 1
        since = {r: n + states for r, n in since.items() if n < 5}
        if op.startswith("v_") and tokens:
            since.update(dict.fromkeys(scalars(tokens[0]), 0))
    return seen, short


def test_counter_sees_a_short_wait():
    code = "_Zk:\n v_readfirstlane_b32 s6, v0\n s_mov_b32 m0, s9\n s_nop %d\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"
    assert short_waits(code % 2) == (1, [("buffer_load_dwordx4 v1, s[4:7], 0 offen lds", 4)])
    assert short_waits(code % 3) == (1, [])


def test_load_behind_a_vector_write(tmp_path):
    source = tmp_path / "probe.hip"
    source.write_text(PROBE)
    seen, short = short_waits(assembly(str(source), (), tmp_path))
    assert seen == 1 and not short, short


def test_walks(tmp_path):
    flags = build._DELTA[0]
    seen, short = short_waits(assembly(os.path.join(build.CSRC, "ops_delta.hip"), flags, tmp_path))
    assert seen > 10 and not short, short


def test_loads_alone_use_m0(tmp_path):
    """The loads change m0 behind the compiler's back, which is sound while nothing else has a use for it."""
    text = assembly(os.path.join(build.CSRC, "ops_delta.hip"), build._DELTA[4], tmp_path)
    seen, short = short_waits(text)
    uses = [line for line in text.splitlines() if re.search(r"\bm0\b", line.split(";")[0])]
    assert len(uses) == seen and all(re.match(r"\s*s_mov_b32 m0, ", u) for u in uses)
    assert not short, short
