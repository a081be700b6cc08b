"""The checks of the 4-bit calls' Python arguments (nothing is launched)."""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from routing_dispatch_expert_router_gb300.build import build

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def test_row_spacing_of_views():
    """Elements from row to row; a dimension of one has a stride that says nothing."""
    wide = torch.zeros(6, 4, 1024, dtype=BF)
    assert B._bf16_rows(wide, (6, 4, 1024), "x") == 1024
    assert B._bf16_rows(wide[:, :, 64:352], (6, 4, 288), "x") == 1024
    assert B._bf16_rows(wide[2:3, :, :288], (1, 4, 288), "x") == 1024
    assert B._bf16_rows(wide[2:3, 1:2, :288], (1, 1, 288), "x") == 288
    # groups of one row each: a row apart is a group apart
    rows = wide.view(24, 1024)
    for t in (rows[:, None, :288], rows[:, :288].unsqueeze(1), rows.view(24, 1, 1024)[:, :, :288]):
        assert B._bf16_rows(t, (24, 1, 288), "x") == 1024
    assert B._bf16_rows(wide[:, 1:2, :288], (6, 1, 288), "x") == 4096
    with pytest.raises(ValueError):
        B._bf16_rows(wide[:, :3, :288], (6, 3, 288), "x")  # groups four rows apart
    with pytest.raises(ValueError):
        B._bf16_rows(wide.transpose(0, 1)[:, :, :288], (4, 6, 288), "x")


def test_a_refused_quantisation_leaves_the_tensor_as_it_was():
    q = B.alloc_fp4(B.MOE_FP4_NV, 1, 4, 64, device="cpu", scale_log2=-3)
    for x, log2 in ((torch.zeros(1, 4, 32, dtype=BF), 5), (torch.zeros(1, 4, 64), 5),
                    (torch.zeros(1, 4, 64, dtype=BF), 65)):
        with pytest.raises((ValueError, B.MoEError)):
            B.moe_fp4_quantize(x, q, scale_log2=log2, stream=0)
        assert q.scale_log2 == -3
