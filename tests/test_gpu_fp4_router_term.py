"""The router's term of the 4-bit experts' backward: which rows and experts get it."""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O
from workloads import MoEShape

pytestmark = pytest.mark.gpu

H_ = pytest.importorskip("harness")
T4 = pytest.importorskip("test_gpu_fp4")
DEV = "cuda"
f64 = T4.f64


def test_padding_rows_are_zero_whatever_the_router_holds():
    """Rows that fill a segment's last 128-row block are zeros, an infinite or NaN router
    weight notwithstanding (their dlogits are none, not zero times that weight)."""
    rng = np.random.default_rng(5)
    H, F, counts = 128, 128, [5, 130]
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("p", T=len(rows), H=H, E=2, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    ex = T4.experts_of(B.MOE_FP4_NV, rng, 2, H, F)
    dO = torch.randn(R, H, device=DEV).bfloat16()
    ck = torch.full((R, 2 * F), 0x38, dtype=torch.uint8, device=DEV)
    cs = torch.full((R, 2 * F // 32), 120, dtype=torch.uint8, device=DEV)
    tok = np.full(R, -1, np.int32)
    tok[rows] = np.arange(len(rows))
    W_r = torch.randn(2, H, device=DEV)
    W_r[0, 3], W_r[1, 64], W_r[1, 65] = float("inf"), float("nan"), float("-inf")
    dl = torch.randn(len(rows), 2, device=DEV)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex[0], dO, ck, cs, cnt, offs, torch.from_numpy(tok).to(DEV), dl, W_r,
                      dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got = f64(dX)
    for g, c in enumerate(counts):
        pad = got[off[g] + c:off[g + 1]]
        assert len(pad) and (pad == 0).all()
        live = got[off[g]:off[g] + c]
        bad = ~np.isfinite(f64(W_r[g]))
        assert not np.isfinite(live[:, bad]).any() and np.isfinite(live[:, ~bad]).all()
