"""The sizes that the header names for the embedding, the block norm and the linear cross entropy are the ones that are
taken: the largest of each has a workspace, one more has none.  No GPU needed."""
import os
import re

import pytest

import selective_state_space_msm_amd as msm
from selective_state_space_msm_amd import build

EMBED = [((1 << 31) - 1, 1, 1), (1, (1 << 31) - 2, 1), (1, 1, 1 << 24), (1 << 24, 1, 1 << 24), (1, 1 << 24, 1 << 24)]
EMBED_PAST = [(1 << 31, 1, 1), (1, (1 << 31) - 1, 1), (1, 1, (1 << 24) + 1), ((1 << 24) + 1, 1, 1 << 24), (1, (1 << 24) + 1, 1 << 24)]
NORM = [((1 << 31) - 1, 1), (1, 1 << 30), (1 << 20, 1 << 30)]
NORM_PAST = [(1 << 31, 1), (1, (1 << 30) + 1), ((1 << 20) + 1, 1 << 30)]
XENT = [(1 << 22, 1, 1), (1, 1 << 22, 1), (1, 1, 1 << 16), (1 << 22, 1 << 15, 1), (1 << 15, 1 << 22, 1)]
XENT_PAST = [((1 << 22) + 1, 1, 1), (1, (1 << 22) + 1, 1), (1, 1, (1 << 16) + 1), (1 << 22, (1 << 15) + 1, 1)]


@pytest.mark.parametrize("io", [0, 1])
def test_largest_sizes(io):
    lib = msm.load_library()
    for size, past, query in ((EMBED, EMBED_PAST, lib.msm_embed_bwd_workspace_bytes),
                              (NORM, NORM_PAST, lambda *s: lib.msm_block_norm_bwd_workspace_bytes(*s, io)),
                              (XENT, XENT_PAST, lambda *s: lib.msm_linear_cross_entropy_fwd_workspace_bytes(*s, io)),
                              (XENT, XENT_PAST, lambda *s: lib.msm_linear_cross_entropy_bwd_workspace_bytes(*s, io))):
        for s in size:
            assert query(*s) > 0, s
        for s in past:
            assert query(*s) == 0, s


def test_header_names_them():
    with open(os.path.join(build.ROOT, "include", "msm.h")) as f:
        text = " ".join(re.sub(r"^ \* ?", "", line.rstrip()) for line in f.read().splitlines())
    for words in ("1 <= tokens < 2^31, 1 <= V < 2^31 - 1, 1 <= D <= 2^24, tokens D and V D <= 2^48",
                  "1 <= rows < 2^31, 1 <= D <= 2^30, rows D <= 2^50", "T and V <= 2^22, T V <= 2^37, D <= 2^16"):
        assert words in text, words
