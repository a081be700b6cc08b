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


class OnGpu(torch.Tensor):
    """A tensor that says it lies on the GPU: for checks that come before any launch."""
    is_cuda = property(lambda self: True)


def gpu(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def fp4(fmt, groups, rows, K):
    q = B.alloc_fp4(fmt, groups, rows, K, device="cpu")
    q.codes, q.scales = q.codes.as_subclass(OnGpu), q.scales.as_subclass(OnGpu)
    return q


I32, I64, F32 = torch.int32, torch.int64, torch.float32
T, H, E, K, F, S = 20, 128, 4, 2, 256, 1
G, R = E + S, T * K + E * 127 + 128


def layer_calls():
    cfg = B.MoEConfig(T=T, H=H, E=E, k=K, F=F, n_shared=S, n_groups=1, topk_groups=1,
                      route_scale=1.0, row_align=128)
    assert B.moe_query_sizes(cfg).rows_max == R
    W13, W2 = fp4(0, G, 2 * F, H), fp4(0, G, H, F)
    sz = B.moe_fp4_query_sizes(cfg, 0)
    both = dict(ckpt=gpu(R, 2 * F), ckpt_scale=gpu(R, 2 * F // 32), counts=gpu(G, dtype=I32),
                offsets=gpu(G + 1, dtype=I32))
    fwd = dict(both, x_perm=gpu(R, H, dtype=BF), y_perm=gpu(R, H, dtype=BF),
               scratch=gpu(sz.fwd_scratch_bytes))
    bwd = dict(both, dO_perm=gpu(R, H, dtype=BF), token_of=gpu(R, dtype=I32),
               dlogits=gpu(T, E, dtype=F32), W_r=gpu(E, H, dtype=F32),
               dX_perm=gpu(R, H, dtype=BF), scratch=gpu(sz.bwd_scratch_bytes))
    return cfg, W13, W2, fwd, bwd


def wrong(name, t):
    """Tensors that do not fit in t's place: other types, too few elements, gaps, the host."""
    yield t.to(I64 if t.dtype != I64 else I32)
    if t.dtype == BF:
        yield t.to(torch.float16)
    yield t[:-1]
    if t.dim() == 2 and name != "scratch":
        yield t[:, :-1]
        yield t.view(-1)
    yield torch.zeros(2 * t.shape[0], *t.shape[1:], dtype=t.dtype).as_subclass(OnGpu)[::2]
    yield torch.zeros(*t.shape, dtype=t.dtype)


def test_ffn_calls_refuse_tensors_that_do_not_fit():
    cfg, W13, W2, fwd, bwd = layer_calls()
    ex = B.fp4_experts(W13, W2)
    for call, args in ((B.moe_fp4_ffn_fwd, fwd), (B.moe_fp4_ffn_bwd, bwd)):
        for name, t in args.items():
            for bad in wrong(name, t):
                if name == "scratch" and bad.numel() * bad.element_size() >= t.numel() and \
                        bad.is_cuda and bad.is_contiguous():
                    continue                               # scratch has no type of its own
                if name == "offsets" and bad.dtype == I32 and bad.is_contiguous() and bad.is_cuda:
                    continue                               # its last element is not read
                with pytest.raises(ValueError, match=name):
                    call(cfg, ex, **{**args, name: bad}, stream=0)


def test_experts_refuse_scales_and_codes_that_do_not_fit():
    _, W13, W2, _, _ = layer_calls()
    one = gpu(G, dtype=F32)
    B.fp4_experts(W13, W2, one, one)
    for bad in (gpu(G, dtype=torch.float64), gpu(G - 1, dtype=F32), torch.ones(G),
                gpu(2 * G, dtype=F32)[::2]):
        with pytest.raises(ValueError, match="alpha13"):
            B.fp4_experts(W13, W2, bad, None)
        with pytest.raises(ValueError, match="alpha2"):
            B.fp4_experts(W13, W2, None, bad)
    q = B.Fp4Tensor(0, H, W13.codes.to(torch.int16), W13.scales)
    with pytest.raises(ValueError, match="uint8"):
        q.struct()
    with pytest.raises(ValueError, match="GPU"):
        B.fp4_experts(B.alloc_fp4(0, G, 2 * F, H, device="cpu"), W2)


def test_quantiser_and_product_refuse_tensors_that_do_not_fit():
    q, x = fp4(0, 1, 130, 256), gpu(1, 130, 256, dtype=BF)
    ok = gpu(2, dtype=I32)
    for bad in (gpu(2, dtype=I64), torch.zeros(2, dtype=I32), gpu(4, dtype=I32)[::2]):
        with pytest.raises(ValueError, match="counts"):
            B.moe_fp4_quantize(x, q, counts=bad, offsets=ok, stream=0)
        with pytest.raises(ValueError, match="offsets"):
            B.moe_fp4_quantize(x, q, counts=ok, offsets=bad, stream=0)
    with pytest.raises(ValueError, match="offsets"):
        B.moe_fp4_quantize(x, q, counts=ok, offsets=gpu(1, dtype=I32), stream=0)
    with pytest.raises(ValueError, match="scratch"):
        B.moe_fp4_quantize(x, q, scratch=gpu(3), stream=0)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_fp4_quantize(torch.zeros(1, 130, 256, dtype=BF), q, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_fp4_quantize(x, q, values=torch.zeros(1, 130, 256, dtype=BF), stream=0)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_fp4_dequantize(q, torch.zeros(1, 130, 256, dtype=BF), stream=0)
    with pytest.raises(ValueError, match="GPU"):
        B.moe_fp4_dequantize(B.alloc_fp4(0, 1, 130, 256, device="cpu"), x, stream=0)
    b, out = fp4(0, 2, 64, 256), gpu(130, 64, dtype=BF)
    sc = gpu(B.moe_fp4_query_sizes(None, 0).gemm_scratch_bytes)
    args = dict(counts=ok, offsets=gpu(3, dtype=I32), alpha=gpu(2, dtype=F32), out=out, scratch=sc)
    for name, bads in dict(counts=(gpu(2, dtype=I64), torch.zeros(2, dtype=I32)),
                           offsets=(gpu(3, dtype=I64), gpu(1, dtype=I32), gpu(6, dtype=I32)[::2]),
                           alpha=(gpu(2, dtype=torch.float64), gpu(1, dtype=F32), torch.ones(2)),
                           out=(torch.zeros(130, 64, dtype=BF), gpu(130, 64, dtype=torch.float16)),
                           scratch=(sc[:-1], torch.zeros(sc.shape, dtype=torch.uint8))).items():
        for bad in bads:
            with pytest.raises(ValueError, match=name):
                B.moe_fp4_grouped_gemm(q, b, **{**args, name: bad}, stream=0)


def test_experts_keep_their_tensors():
    """The structure holds addresses; tensors made for it alone live as long as it does."""
    import gc
    import weakref
    one = [gpu(G, dtype=F32), gpu(G, dtype=F32)]
    W = [fp4(0, G, 2 * F, H), fp4(0, G, H, F)]
    refs = [weakref.ref(t) for t in (W[0].codes, W[0].scales, W[1].codes, W[1].scales, *one)]
    ex = B.fp4_experts(*W, *one)
    one.clear(), W.clear()
    gc.collect()
    assert all(r() is not None for r in refs)
    del ex
    gc.collect()
    assert not any(r() is not None for r in refs)
