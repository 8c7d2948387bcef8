"""The cross entropy's loads into LDS are written as assembly: their wait states, and m0, in the compiled code."""
import os
import re

import pytest

from selective_state_space_msm_amd import build
from test_ops_isa import assembly, short_waits

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


def test_loads_into_lds(tmp_path):
    text = assembly(os.path.join(build.CSRC, "lm_xent.hip"), (), tmp_path)
    seen, short = short_waits(text)
    assert seen > 100 and not short, short[:5]
    uses = [line for line in text.splitlines() if re.search(r"\bm0\b", line.split(";")[0])]
    assert len(uses) == seen and all(re.match(r"\s*s_mov_b32 m0, ", u) for u in uses)
