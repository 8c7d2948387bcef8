"""Sizes and distances of these operators are 64-bit: nothing in their kernels narrows one by itself.  No GPU needed."""
import os
import re
import subprocess

import pytest

from selective_state_space_msm_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


def narrowed(source):
    r = subprocess.run([build.HIPCC, *build.COMMON, "-fsyntax-only", "--cuda-device-only", "-Wshorten-64-to-32", source],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return re.findall(r"^.*warning: implicit conversion loses integer precision.*$", r.stderr, re.M)


def test_a_narrowed_distance_is_seen(tmp_path):
    probe = tmp_path / "probe.hip"
    probe.write_text("#include \"ops_delta.hpp\"\n__device__ void at(uint16_t* p, int n);\n"
                     "__global__ void probe(uint16_t* p, int64_t plane) { at(p, plane); }\n")
    assert len(narrowed(str(probe))) == 1


@pytest.mark.parametrize("source", ["lm_xent.hip", "lm_embed.hip", "lm_block_norm.hip", "ops_norm.hip"])
def test_no_distance_is_narrowed(source):
    assert narrowed(os.path.join(build.CSRC, source)) == []
