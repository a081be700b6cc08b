"""Which roundings the 4-bit experts' backward makes."""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O
from workloads import MoEShape

pytestmark = pytest.mark.gpu

T4 = pytest.importorskip("test_gpu_fp4")
DEV = "cuda"
f64 = T4.f64
# one rounding to bf16: errors even over a step of 2^-7 at values of 1 or more, so their norm is
# at most 2^-7 / sqrt(12) of the values'
ONE = 2.0 ** -7 / np.sqrt(12.0)


@pytest.mark.parametrize("fmt", T4.FORMATS)
@pytest.mark.parametrize("H,F,rows", [(256, 384, 600), (1024, 512, 130)])
def test_dgu_is_the_only_value_rounded_on_the_way(fmt, H, F, rows):
    """Against the formula with [dG|dU] rounded to bf16 (before alpha2) the gradient is off by its
    own rounding; against the formula without it by two."""
    rng = np.random.default_rng(H)
    cfg = B.config(MoEShape("r", T=rows, H=H, E=1, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    ex = T4.experts_of(fmt, rng, 1, H, F)
    a13, a2 = f64(ex[3])[0], f64(ex[4])[0]
    W13, W2 = ex[5][0] / a13, ex[6][0] / a2
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[:rows] = T4.rows_of(rng, rows, H, spread=False)
    codes = rng.integers(0, 120, (R, 2 * F), dtype=np.uint8)
    byte = np.full((R, 2 * F // 32), 119, np.uint8)
    dX = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).bwd_scratch_bytes)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)  # noqa: E731
    B.moe_fp4_ffn_bwd(cfg, ex[0], dO, torch.from_numpy(codes).to(DEV), torch.from_numpy(byte).to(DEV),
                      i32(rows), i32(0), None, None, None, dX, sc)
    assert B.moe_last_device_status(sc) == 0
    gu = O.checkpoint_values(codes[:rows], byte[:rows])
    _, dgu = O.ffn_bwd(f64(dO)[:rows], gu, W13, W2)
    got = f64(dX)[:rows]
    with_rounding = O.round_bf16(dgu) @ W13 * a13 * a2
    without = dgu @ W13 * a13 * a2
    rel = lambda ref: np.linalg.norm(got - ref) / np.linalg.norm(ref)  # noqa: E731
    print(f"with {rel(with_rounding):.5f}, without {rel(without):.5f}")
    assert rel(with_rounding) <= ONE
    assert rel(without) <= np.sqrt(2.0) * ONE
