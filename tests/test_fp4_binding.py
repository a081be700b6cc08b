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
