"""Refusals of the norm, the dispatch of 8-bit rows and the products of free form: what does not
fit is refused on the host (nothing is launched)."""
import ctypes

import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from routing_dispatch_expert_router_gb300.build import build

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


class OnGpu(torch.Tensor):
    """A tensor that says it lies on the GPU: for checks that come before any launch."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return torch.cuda.current_device() if torch.cuda.is_available() else 0


def gpu(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def wrong(t):
    """Tensors that do not fit in t's place: another type, too few elements, gaps, the host."""
    yield t.to(torch.float64)
    yield t[:-1]
    if t.dim() == 2:
        yield t[:, :-8]
    yield torch.zeros(*t.shape, dtype=t.dtype)


def refused(call, args, **bad):
    with pytest.raises((ValueError, B.MoEError)):
        call(**{**args, **bad}, stream=0)


T, H = 5, 256


def test_norm_refuses_tensors_that_do_not_fit():
    fwd = dict(x=gpu(T, H), gamma=gpu(H), out=gpu(T, H), residual=gpu(T, H), sum=gpu(T, H),
               rstd=gpu(T, dtype=F32), codes=gpu(T, H, dtype=U8), scales=gpu(T, H // 32, dtype=U8))
    for name in ("gamma", "out", "residual", "sum", "rstd", "codes", "scales"):
        for bad in wrong(fwd[name]):
            refused(B.moe_rmsnorm_fwd, fwd, **{name: bad})
    for name, bad in (("scales", None), ("codes", None), ("scales", gpu(T, H // 64, dtype=U8)),
                      ("residual", None), ("x", gpu(T, 2 * H)[:, ::2]), ("x", gpu(H, T).t()),
                      ("x", gpu(1, H).expand(T, H)), ("out", gpu(T, H, dtype=torch.float16)),
                      ("x", gpu(T, H + 4)[:, 4:])):
        refused(B.moe_rmsnorm_fwd, fwd, **{name: bad})
    refused(B.moe_rmsnorm_fwd, {**fwd, "codes": None, "scales": None}, out=None)
    for eps in (-1e-6, float("nan"), float("inf")):
        refused(B.moe_rmsnorm_fwd, fwd, eps=eps)
    bwd = dict(dy=gpu(T, H), h=gpu(T, H), rstd=gpu(T, dtype=F32), gamma=gpu(H), dx=gpu(T, H),
               dgamma=gpu(H, dtype=F32), dsum=gpu(T, H),
               scratch=gpu(B.rmsnorm_scratch_bytes(H), dtype=U8))
    for name in ("dy", "rstd", "gamma", "dx", "dgamma", "dsum"):
        for bad in wrong(bwd[name]):
            refused(B.moe_rmsnorm_bwd, bwd, **{name: bad})
    for bad in (None, gpu(B.rmsnorm_scratch_bytes(H) - 1, dtype=U8)):
        refused(B.moe_rmsnorm_bwd, bwd, scratch=bad)


def test_norm_entry_refuses_sizes_and_addresses():
    L, ok = B.lib(), 1024

    def fwd(T=4, H=256, x=ok, ldx=256, r=0, ldr=0, g=ok, kind=0, eps=0.0, s=0, lds=0, o=ok, ldo=256,
            c=0, sc=0, block=0, rstd=0):
        return L.moe_rmsnorm_fwd(T, H, x, ldx, r, ldr, g, kind, eps, s, lds, o, ldo, c, sc, block, rstd, 0)

    assert fwd(T=0) == 0
    for bad in (dict(T=-1), dict(H=0), dict(H=252), dict(x=0), dict(x=8), dict(ldx=248), dict(ldx=260),
                dict(r=8, ldr=256), dict(r=ok, ldr=8), dict(g=0), dict(g=4), dict(kind=2), dict(o=0),
                dict(s=ok, lds=256), dict(c=ok), dict(c=ok, sc=ok, block=64), dict(rstd=2),
                dict(H=264, ldx=264, ldo=264, c=ok, sc=ok, block=32)):
        assert fwd(**bad) == 1, bad
    assert fwd(H=32776, ldx=32776, ldo=32776) == 2
    n = ctypes.c_int64(0)
    assert L.moe_rmsnorm_scratch_bytes(4, ctypes.byref(n)) == 1
    assert L.moe_rmsnorm_scratch_bytes(32776, ctypes.byref(n)) == 2


def test_permute_fp8_refuses_what_does_not_fit():
    cfg = B.MoEConfig(T=20, H=256, E=4, k=2, F=256, n_groups=1, topk_groups=1, route_scale=1.0,
                      row_align=128, dtype=1)
    sz = B.moe_query_sizes(cfg)
    R = sz.rows_max
    args = dict(cfg=cfg, codes=gpu(20, 256, dtype=U8), scales=gpu(20, 2, dtype=U8), idx=gpu(20, 2, dtype=I32),
                counts=gpu(4, dtype=I32), offsets=gpu(5, dtype=I32), row_of=gpu(20, 2, dtype=I32),
                token_of=gpu(R, dtype=I32), sel_offsets=gpu(5, dtype=I32), sel_tokens=gpu(40, dtype=I32),
                scratch=gpu(sz.scratch_bytes, dtype=U8), codes_perm=gpu(R, 256, dtype=U8),
                scales_perm=gpu(-(-R // 128), 1, 512, dtype=U8))
    for name, t in args.items():
        if name in ("cfg", "scratch"):
            continue
        for bad in wrong(t):
            if bad.dim() == 3 and bad.is_cuda and bad.dtype == U8:
                bad = bad[:, :, :500]
            refused(B.moe_permute_fp8, args, **{name: bad})
    refused(B.moe_permute_fp8, args, scratch=gpu(4000, dtype=U8))
    refused(B.moe_permute_fp8, args, codes_perm=None)
    refused(B.moe_permute_fp8, {**args, "codes_perm": None, "scales_perm": None}, scratch=gpu(1 << 16, dtype=U8))
    bf = B.MoEConfig.from_buffer_copy(bytes(cfg))
    bf.dtype = 0
    refused(B.moe_permute_fp8, args, cfg=bf)
    bf.dtype, bf.stash_pool_pages = 1, 4
    refused(B.moe_permute_fp8, args, cfg=bf)


def int4(G, N, K, group, zeros=True):
    return B.Int4Tensor(gpu(G, N, K // 2, dtype=U8), gpu(G, K // group, N),
                        gpu(G, K // group, N, dtype=U8) if zeros else None)


def test_int4_tensor_refuses_what_does_not_fit():
    c, s, z = gpu(2, 32, 64, dtype=U8), gpu(2, 4, 32), gpu(2, 4, 32, dtype=U8)
    B.Int4Tensor(c, s, z)
    for bad in ((c.to(I32), s, z), (c[:, :, ::2], s, z), (c[0], s, z), (c, s.float(), z), (c, s[:1], z),
                (c, s[:, :, :16], z), (c, gpu(2, 3, 32), z), (c, s, z.to(I32)), (c, s, z[:1]),
                (torch.zeros(2, 32, 64, dtype=U8), s, z), (c, torch.zeros(2, 4, 32, dtype=BF), z)):
        with pytest.raises(ValueError):
            B.Int4Tensor(*bad)


def test_int4_calls_refuse_what_does_not_fit():
    args = dict(x=gpu(9, 128), w=int4(2, 32, 128, 32), counts=gpu(2, dtype=I32), offsets=gpu(2, dtype=I32),
                out=gpu(9, 32), scratch=gpu(B.product_scratch_bytes(), dtype=U8))
    for name in ("x", "counts", "offsets", "out", "scratch"):
        for bad in wrong(args[name]):
            if name == "scratch" and bad.element_size() == 8:
                continue                                   # (it has no type of its own)
            refused(B.moe_int4_grouped_gemm, args, **{name: bad})
    refused(B.moe_int4_grouped_gemm, args, counts=None)
    refused(B.moe_int4_grouped_gemm, args, counts=None, offsets=None)     # two groups
    refused(B.moe_int4_grouped_gemm, args, swiglu=True)                   # out is [9, 16] then
    refused(B.moe_int4_grouped_gemm, args, w=int4(2, 32, 128, 16))
    refused(B.moe_int4_grouped_gemm, {**args, "out": gpu(9, 40)}, w=int4(2, 40, 128, 32))
    refused(B.moe_int4_grouped_gemm, {**args, "out": gpu(9, 24)}, w=int4(2, 48, 128, 32), swiglu=True)
    refused(B.moe_int4_dequantize, dict(w=args["w"], out=gpu(2, 32, 120)))
    refused(B.moe_int4_dequantize, dict(w=args["w"], out=gpu(2, 32, 128, dtype=F32)))
    many = dict(args, w=int4(261, 32, 128, 32), counts=gpu(261, dtype=I32), offsets=gpu(261, dtype=I32))
    with pytest.raises(B.MoEError) as e:
        B.moe_int4_grouped_gemm(**many, stream=0)
    assert e.value.code == 2


def test_products_refuse_what_does_not_fit():
    seg = dict(counts=gpu(2, dtype=I32), offsets=gpu(2, dtype=I32), scratch=gpu(B.product_scratch_bytes(), dtype=U8))
    w = gpu(2, 32, 64)
    calls = ((B.moe_grouped_gemm, dict(seg, x=gpu(9, 64), w=w, out=gpu(9, 32), add=gpu(9, 32))),
             (B.moe_grouped_gemm_dgrad, dict(seg, dy=gpu(9, 32), w=w, dx=gpu(9, 64), add=gpu(9, 64))),
             (B.moe_grouped_gemm_wgrad, dict(seg, dy=gpu(9, 32), x=gpu(9, 64), dw=gpu(2, 32, 64))))
    for call, args in calls:
        for name, t in args.items():
            for bad in wrong(t):
                if name == "scratch" and bad.element_size() == 8:
                    continue                               # (it has no type of its own)
                refused(call, args, **{name: bad})
        refused(call, args, counts=None)
        refused(call, args, counts=None, offsets=None)     # two groups
        for name in ("w", "dw"):
            if name in args:
                refused(call, args, **{name: gpu(2, 64, 32).transpose(1, 2)})
                refused(call, args, **{name: gpu(32, 64)})
    refused(calls[0][0], calls[0][1], expected_rows=-1)
    odd = dict(calls[0][1], x=gpu(9, 68), w=gpu(2, 32, 68))
    refused(calls[0][0], odd)
    many = dict(calls[0][1], w=gpu(261, 32, 64), counts=gpu(261, dtype=I32), offsets=gpu(261, dtype=I32))
    with pytest.raises(B.MoEError) as e:
        B.moe_grouped_gemm(**many, stream=0)
    assert e.value.code == 2


def test_product_entries_refuse_sizes():
    L, ok = B.lib(), 1024

    def gemm(groups=1, rows=4, N=32, K=64, hint=0):
        return L.moe_grouped_gemm(groups, rows, N, K, ok, K, ok, ok, ok, 0, 0, ok, N, hint, ok, 0)

    assert gemm(rows=0) == 0
    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(groups=0), dict(N=0), dict(N=12), dict(K=4), dict(hint=-1)):
        assert gemm(**bad) == 1, bad
    for far in (dict(rows=2 ** 31 - 1), dict(rows=2 ** 31 - 1023), dict(groups=261)):
        assert gemm(**far) == 2, far
    assert gemm(rows=2 ** 31 - 1024, N=1 << 24, K=128) == 2            # more tiles than 32 bits hold
    w = B.MoEInt4Tensor(32, 261, 32, 64, ok, ok, ok)
    assert L.moe_int4_dequantize(w, ok, 0) == 2
    assert L.moe_int4_grouped_gemm(w, 4, ok, 64, ok, ok, 0, ok, 32, ok, 0) == 2
    w = B.MoEInt4Tensor(32, 1, 32, 64, ok, ok, ok)
    assert L.moe_int4_grouped_gemm(w, 2 ** 31 - 1, ok, 64, ok, ok, 0, ok, 32, ok, 0) == 2
