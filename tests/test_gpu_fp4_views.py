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


def test_the_tensor_scale_of_a_call_and_of_a_tensor():
    """A quantisation's scale stays with the tensor; an inverse's is the call's alone."""
    x = torch.randn(1, 40, 288, device="cuda").bfloat16()
    q = B.alloc_fp4(B.MOE_FP4_NV, 1, 40, 288, scale_log2=2)
    out = torch.empty_like(x)
    B.moe_fp4_quantize(x, q, scale_log2=-4)
    assert q.scale_log2 == -4
    B.moe_fp4_dequantize(q, out)
    H_.assert_equal("values", T4.f64(out), O.real(B.MOE_FP4_NV, T4.f64(x), -4))
    B.moe_fp4_dequantize(q, out, scale_log2=-3)
    assert q.scale_log2 == -4
    H_.assert_equal("twice the values", T4.f64(out), 2 * O.real(B.MOE_FP4_NV, T4.f64(x), -4))
