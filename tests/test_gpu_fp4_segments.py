"""Segments that the 4-bit FFN leaves out: reported, and no row of theirs written."""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from workloads import MoEShape

pytestmark = pytest.mark.gpu

T4 = pytest.importorskip("test_gpu_fp4")
DEV = "cuda"


@pytest.mark.parametrize("fmt", T4.FORMATS)
@pytest.mark.parametrize("T,counts,offsets", [
    (20, [5, 33], [0, 128]),            # more rows than the kernel of T <= 32 has room for
    (50, [5, 65], [0, 128]),            # than that of T <= 64
    (200, [5, 10 ** 6], [0, 128]), (200, [5, -1], [0, 128]), (200, [5, 5], [0, 130]),
    (200, [5, 5], [0, -128]), (2000, [5, 10 ** 6], [0, 128]), (2000, [5, 5], [0, 64])])
def test_ffn_reports_bad_segments(fmt, T, counts, offsets):
    rng = np.random.default_rng(3)
    H, F = 128, 128
    cfg = B.config(MoEShape("g", T=T, H=H, E=2, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    ex = T4.experts_of(fmt, rng, 2, H, F)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(R, H, device=DEV).bfloat16()
    y = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    ck = torch.full((R, 2 * F), 0x11, dtype=torch.uint8, device=DEV)
    cs = torch.full((R, 2 * F // 32), 0x11, dtype=torch.uint8, device=DEV)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).fwd_scratch_bytes)
    B.moe_fp4_ffn_fwd(cfg, ex[0], x, i32(counts), i32(offsets), ck, cs, y, sc)
    assert B.moe_last_device_status(sc) == 6               # MOE_ERR_DEVICE_CHECK
    assert (y[:5] != 7.0).any() and (y[5:] == 7.0).all()
    assert (ck[5:] == 0x11).all() and (cs[5:] == 0x11).all()
    good = y[:5].clone()
    B.moe_clear_device_status(sc)
    B.moe_fp4_ffn_fwd(cfg, ex[0], x, i32([5, 0]), i32([0, 128]), ck, cs, y, sc)
    assert B.moe_last_device_status(sc) == 0 and torch.equal(good, y[:5])
