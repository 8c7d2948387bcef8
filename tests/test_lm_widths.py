"""Widths at which the kernels of the embedding's gradient and of few rows' cross entropy take their other branches."""
import pytest
import torch

import lm_ref
from test_lm_xent import check as check_xent

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# a wavefront's share of k, in pieces of 32: held up to 8 for each of 16 wavefronts (D = 4096), which all share a tile
# from 65 pieces on (D = 2049)
@pytest.mark.parametrize("io,D", [("bf16", 2048), ("bf16", 2049), ("bf16", 4096), ("bf16", 4097), ("bf16", 6656), ("bf16", 9001),
                                  ("f32", 2048), ("f32", 2049), ("f32", 4099), ("f32", 8192)])
@pytest.mark.parametrize("T", [1, 16, 17, 32])
def test_few_rows_of_cross_entropy(io, D, T):
    check_xent(io, T, 500, D, weight_grad=False, on="cuda")


def gradient(io, table, T, V, D, ids=None):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T + V + D)
    if ids is None:
        ids = ((V + 1) ** torch.rand(T, generator=gen).double()).long() - 1  # frequent and rare ones
    ids = ids.clamp(0, V - 1)
    ids[torch.rand(T, generator=gen) < 0.1] = -1
    dy = torch.randn(T, D, generator=gen).to(DT[io])
    scale = 1.5
    d, size, n = lm_ref.embed_bwd(ids, dy.double(), V, scale)
    got = msm.msm_embed_bwd(ids.cuda(), dy.cuda(), V, scale, table_dtype=DT[table]).double().cpu()
    # sums of n terms in any order, the scaling, the rounding of the result
    tol = (n + 2) * 2.0 ** -24 * size
    tol = tol + (2.0 ** -8 if table == "bf16" else 2.0 ** -24) * (d.abs() + tol)
    assert bool(((got - d).abs() <= tol).all()), float(((got - d).abs() / (tol + 1e-300)).max())


# 256 threads take 16 bytes each: more columns than 2048 (bf16) or 1024 (fp32) are another workgroup's
@pytest.mark.parametrize("io,table,D", [("bf16", "bf16", 2048), ("bf16", "bf16", 2049), ("bf16", "f32", 2056), ("bf16", "bf16", 4096),
                                        ("bf16", "f32", 6151), ("f32", "f32", 1024), ("f32", "f32", 1025), ("f32", "bf16", 2049),
                                        ("f32", "f32", 4096)])
@pytest.mark.parametrize("T,V", [(1, 3), (40, 300), (700, 60), (700, 3000), (5000, 900), (9000, 9001)])
def test_embedding_gradient_of_wide_rows(io, table, D, T, V):
    gradient(io, table, T, V, D)


@pytest.mark.parametrize("io,D", [("bf16", 4099), ("f32", 2050)])
@pytest.mark.parametrize("T,V", [(3000, 50), (9000, 20000)])
def test_embedding_gradient_of_one_wide_word(io, D, T, V):
    gradient(io, io, T, V, D, ids=torch.full((T,), V - 1))
