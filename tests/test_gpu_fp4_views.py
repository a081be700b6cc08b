"""Views as arguments of the 4-bit quantiser and its inverse."""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O

pytestmark = pytest.mark.gpu

H_ = pytest.importorskip("harness")
T4 = pytest.importorskip("test_gpu_fp4")


@pytest.mark.parametrize("fmt", T4.FORMATS)
def test_groups_of_one_row_in_a_wider_tensor(fmt):
    wide = torch.randn(24, 1024, device="cuda").bfloat16()
    x = wide[:, None, 64:352]
    q = B.alloc_fp4(fmt, 24, 1, 288)
    B.moe_fp4_quantize(x, q)
    out = torch.full((24, 512), 7.0, device="cuda", dtype=torch.bfloat16)
    B.moe_fp4_dequantize(q, out[:, None, 64:352])
    H_.assert_equal("values", T4.f64(out[:, 64:352]), O.real(fmt, T4.f64(x[:, 0])))
    assert (out[:, :64] == 7.0).all() and (out[:, 352:] == 7.0).all()
