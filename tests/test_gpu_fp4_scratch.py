"""Scratch of the 4-bit calls that an earlier call left behind: results do not depend on it."""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B

pytestmark = pytest.mark.gpu

T4 = pytest.importorskip("test_gpu_fp4")
J = pytest.importorskip("test_gpu_fp4_joins")
FORMATS = T4.FORMATS
DEV = "cuda"
# arrival counters of cut tiles, behind the page of the status word
COUNTERS = slice(4096, 65536)


def leavings(sc):
    """What counters may hold after a call that gave up: some arrivals counted and others
    not; here any bits at all."""
    n = COUNTERS.stop - COUNTERS.start
    i32 = lambda v: torch.full((n // 4,), v, dtype=torch.int32, device=DEV).view(torch.uint8)  # noqa: E731
    g = torch.Generator(device=DEV).manual_seed(1)
    for what in (i32(1), i32(5), i32(-1), i32(0x01010101),
                 torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV, generator=g)):
        sc[COUNTERS] = what
        yield


@pytest.mark.parametrize("fmt", FORMATS)
def test_ffn_after_a_call_that_gave_up(fmt):
    """Both products' tiles are cut; the numbers are a fresh scratch's, on the next call and
    on the one after it."""
    counts, H, F = [1, 1], 4096, 4096
    assert J.cuts(counts, F // 128, H) and J.cuts(counts, H // 256, F)
    s = T4.run_ffn(fmt, counts, H, F)
    rows = s["rows"]
    y, ck, cs = s["y"][rows].clone(), s["ck"][rows].clone(), s["cs"][rows].clone()
    for _ in leavings(s["sc"]):
        for _ in range(2):
            s["y"].fill_(7.0)
            s["ck"].fill_(0x11)
            B.moe_fp4_ffn_fwd(s["cfg"], s["ex"][0], s["x"], s["cnt"], s["offs"], s["ck"], s["cs"],
                              s["y"], s["sc"])
            assert torch.equal(y, s["y"][rows])
            assert torch.equal(ck, s["ck"][rows]) and torch.equal(cs, s["cs"][rows])
    assert B.moe_last_device_status(s["sc"]) == 0


def test_product_after_a_call_that_gave_up():
    """The same for the product alone, and with a graph whose replays find the leavings."""
    counts, N, K = [7, 0, 3], 520, 7168
    assert J.cuts(counts, 3, K)
    off, rows, cnt, offs = T4.segments(counts)
    R = int(off[-1])
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(1, R, K, device=DEV, generator=g).bfloat16()
    w = torch.randn(3, N, K, device=DEV, generator=g).bfloat16()
    xq, wq = B.alloc_fp4(0, 1, R, K), B.alloc_fp4(0, 3, N, K)
    B.moe_fp4_quantize(x, xq)
    B.moe_fp4_quantize(w, wq)
    size = B.moe_fp4_query_sizes(None, 0).gemm_scratch_bytes
    first = torch.zeros(R, N, device=DEV, dtype=torch.bfloat16)
    B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, None, first, B.alloc_fp4_scratch(size))
    out, sc = torch.zeros_like(first), B.alloc_fp4_scratch(size)
    for _ in leavings(sc):
        out.zero_()
        B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, None, out, sc)
        assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, None, out, sc)
    for _ in leavings(sc):
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
    assert B.moe_last_device_status(sc) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_scratch_for_forward_product_and_backward(fmt):
    """Calls that follow each other may share scratch: what the backward keeps there lies
    behind the counters, and the forward's and the product's numbers are a fresh scratch's."""
    counts, H, F = [1, 1], 4096, 4096
    s = T4.run_ffn(fmt, counts, H, F)
    rows = s["rows"]
    y = s["y"][rows].clone()
    sz = B.moe_fp4_query_sizes(s["cfg"], fmt)
    sc = B.alloc_fp4_scratch(max(sz.gemm_scratch_bytes, sz.fwd_scratch_bytes, sz.bwd_scratch_bytes))
    dX = [torch.zeros_like(s["y"]) for _ in range(2)]
    for i in range(2):
        s["y"].fill_(7.0)
        B.moe_fp4_ffn_fwd(s["cfg"], s["ex"][0], s["x"], s["cnt"], s["offs"], s["ck"], s["cs"],
                          s["y"], sc)
        assert torch.equal(y, s["y"][rows])
        before = sc[COUNTERS].clone()
        # dO = the token rows: gradients of ordinary size
        B.moe_fp4_ffn_bwd(s["cfg"], s["ex"][0], s["x"], s["ck"], s["cs"], s["cnt"], s["offs"],
                          None, None, None, dX[i], sc)
        assert dX[i][rows].any()
        assert torch.equal(before, sc[COUNTERS])
    assert torch.equal(dX[0], dX[1])
    assert B.moe_last_device_status(sc) == 0
