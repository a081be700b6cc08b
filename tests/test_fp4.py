"""The 4-bit experts on the CPU: the oracle against facts of the formats, the sizes
the library reports, and the refusals of its entry points (nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O
from routing_dispatch_expert_router_gb300.build import build
from workloads import MIXTRAL, TINY

VP = ctypes.c_void_p
I32, I64 = ctypes.c_int32, ctypes.c_int64
FORMATS = (O.NV, O.MX)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


# ------------------------------------------------------------------- the oracle
def test_grids_are_the_formats_values():
    assert len(O.E4M3) == 127 and O.E4M3[-1] == 448.0 and O.E4M3[8] == 2.0 ** -6
    byte = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(byte.view(torch.float8_e4m3fn).double().numpy(), O.E4M3)
    # ties go to the even code
    assert [int(i) for i in O.nearest([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], O.E2M1)] == \
        [0, 2, 2, 4, 4, 6, 6]


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantised_values_are_a_fixed_point(fmt):
    rng = np.random.default_rng(0)
    x = O.round_bf16(rng.standard_normal((5, 96)))
    v = O.real(fmt, x)
    if fmt == O.MX:
        assert np.array_equal(O.real(fmt, v), v)
    # no value is further from x than half the grid's widest step, in its block's scale
    c, b = O.quantise(fmt, x)
    unit = np.repeat(O.scale_values(fmt, b), O.BLOCK[fmt], 1)
    assert np.all(np.abs(v - x) <= unit * (1.0 if fmt == O.MX else 1.0 + 6.0 / 16))
    assert np.array_equal(O.unpack(O.pack(c)), c)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 32), (130, 288), (256, 512)])
def test_atoms_round_trip_and_sizes(fmt, rows, K):
    byte = np.random.default_rng(1).integers(1, 100, (2, rows, K // O.BLOCK[fmt]), dtype=np.uint8)
    a = O.to_atoms(fmt, byte, K)
    assert np.array_equal(O.from_atoms(fmt, a, rows, K), byte)
    assert a[0].size == B.fp4_scale_bytes(fmt, rows, K)
    assert a.sum() == byte.sum()                           # the rest is zero


def test_gradient_formula_against_differences():
    """ffn_bwd is the derivative of y = (silu(x Wg^T) x Wu^T) W2^T (no quantiser: they are
    passed straight through). Central differences with step 1e-5: the third derivative's
    share is below 1e-9 of unit-sized terms, rounding 1e-16 / 1e-5 = 1e-11."""
    rng = np.random.default_rng(2)
    H, F = 6, 5
    W13, W2 = rng.standard_normal((2 * F, H)) / 2, rng.standard_normal((H, F)) / 2
    x, dO = rng.standard_normal((3, H)), rng.standard_normal((3, H))

    def loss(x):
        gu = x @ W13.T
        return np.sum(dO * ((O.silu(gu[:, :F]) * gu[:, F:]) @ W2.T))

    dx, _ = O.ffn_bwd(dO, x @ W13.T, W13, W2)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        assert abs((loss(x + e) - loss(x - e)) / 2e-5 - dx[i]) < 1e-7


# ------------------------------------------------------------------ host checks
def tensor(fmt=0, log2=0, groups=1, rows=128, K=256, codes=4096, scales=4096):
    return B.MoEFp4Tensor(fmt, log2, groups, rows, K, codes, scales)


@pytest.mark.parametrize("bad", [
    dict(fmt=2), dict(fmt=-1), dict(log2=65), dict(fmt=1, log2=1), dict(K=48), dict(K=0),
    dict(rows=-1), dict(groups=-1), dict(codes=4104), dict(scales=4104), dict(codes=None),
    dict(scales=None), dict(groups=1 << 16, rows=1 << 16), dict(K=1 << 25),
])
def test_bad_tensors_are_refused(bad):
    q = tensor(**bad)
    ok = VP(4096)
    lib = B.lib()
    assert lib.moe_fp4_quantize(ctypes.byref(q), ok, I64(1 << 26), VP(None), VP(None), I32(0),
                                VP(None), VP(None), VP(None)) == 1
    assert lib.moe_fp4_dequantize(ctypes.byref(q), ok, I64(1 << 26), VP(None)) == 1
    good = tensor()
    for a, b in ((q, good), (good, q)):
        assert lib.moe_fp4_grouped_gemm(ctypes.byref(a), ctypes.byref(b), VP(None), VP(None),
                                        VP(None), ok, ok, VP(None)) == 1


def test_bad_quantise_arguments_are_refused():
    lib, q, ok = B.lib(), tensor(), VP(4096)

    def call(x=4096, ldx=256, counts=None, offsets=None, segments=0, values=None, scratch=None,
             q=q):
        return lib.moe_fp4_quantize(ctypes.byref(q), VP(x), I64(ldx), VP(counts), VP(offsets),
                                    I32(segments), VP(values), VP(scratch), VP(None))
    assert call(x=None) == 1 and call(x=4098) == 1
    assert call(ldx=248) == 1 and call(ldx=260) == 1
    assert call(counts=4096) == 1 and call(counts=4096, offsets=4096) == 1
    assert call(counts=4096, offsets=4096, segments=-1) == 1
    assert call(counts=4098, offsets=4096, segments=1) == 1
    assert call(counts=4096, offsets=4096, segments=2, q=tensor(groups=2)) == 1
    assert call(values=4100) == 1 and call(scratch=4098) == 1
    assert lib.moe_fp4_dequantize(ctypes.byref(q), VP(4104), I64(256), VP(None)) == 1
    assert lib.moe_fp4_dequantize(ctypes.byref(q), ok, I64(252), VP(None)) == 1
    # nothing to do: no launch
    assert call(x=None, q=tensor(rows=0, codes=None, scales=None)) == 0
    assert lib.moe_fp4_dequantize(ctypes.byref(tensor(groups=0, codes=None)), VP(None), I64(256),
                                  VP(None)) == 0


def test_bad_products_are_refused():
    lib = B.lib()

    def call(a=tensor(), b=tensor(), counts=None, offsets=None, alpha=None, out=4096,
             scratch=4096):
        return lib.moe_fp4_grouped_gemm(ctypes.byref(a), ctypes.byref(b), VP(counts), VP(offsets),
                                        VP(alpha), VP(out), VP(scratch), VP(None))
    assert call(a=tensor(fmt=1)) == 1                      # two formats
    assert call(a=tensor(K=512)) == 1                      # two reduction lengths
    assert call(a=tensor(groups=2)) == 1
    assert call(b=tensor(rows=100)) == 1                   # N a multiple of 8
    assert call(b=tensor(groups=2)) == 1                   # several groups without counts
    assert call(counts=4096) == 1 and call(offsets=4096) == 1
    assert call(alpha=4098) == 1 and call(out=4104) == 1 and call(out=None) == 1
    assert call(scratch=None) == 1 and call(scratch=4104) == 1
    assert call(b=tensor(groups=300), counts=4096, offsets=4096) == 2
    assert call(a=tensor(rows=0, codes=None, scales=None), out=None) == 0


def test_layer_calls_refuse_other_shapes_and_modes():
    lib = B.lib()
    cfg = B.config(TINY)                                   # E = 8, H = 128, F = 256

    def experts(**kw):
        e = dict(W13=tensor(groups=8, rows=512, K=128), W2=tensor(groups=8, rows=128, K=256),
                 alpha13=None, alpha2=None, x_scale_log2=0, h_scale_log2=0)
        return B.MoEFp4Experts(**{**e, **kw})

    def fwd(ex, cfg=cfg, x=4096, ckpt=4096, ckpt_scale=4096, y=4096, scratch=4096):
        return lib.moe_fp4_ffn_fwd(ctypes.byref(cfg), ctypes.byref(ex), VP(x), VP(4096), VP(4096),
                                   VP(ckpt), VP(ckpt_scale), VP(y), VP(scratch), VP(None))

    def bwd(ex, cfg=cfg, dO=4096, ckpt=4096, token_of=None, dlogits=None, W_r=None):
        return lib.moe_fp4_ffn_bwd(ctypes.byref(cfg), ctypes.byref(ex), VP(dO), VP(ckpt), VP(4096),
                                   VP(4096), VP(4096), VP(token_of), VP(dlogits), VP(W_r),
                                   VP(4096), VP(4096), VP(None))
    for bad in (dict(W13=tensor(groups=7, rows=512, K=128)), dict(W2=tensor(groups=8, rows=128, K=128)),
                dict(W13=tensor(groups=8, rows=256, K=128)),
                dict(W2=tensor(fmt=1, groups=8, rows=128, K=256)),
                dict(alpha13=4098), dict(x_scale_log2=100), dict(h_scale_log2=-65)):
        assert fwd(experts(**bad)) == 1, bad
        assert bwd(experts(**bad)) == 1, bad
    assert fwd(experts(), x=None) == 1 and fwd(experts(), y=4104) == 1
    assert fwd(experts(), scratch=None) == 1
    assert fwd(experts(), ckpt=None) == 1                  # one of the checkpoint's two
    assert bwd(experts(), dO=None) == 1 and bwd(experts(), ckpt=None) == 1
    assert bwd(experts(), dlogits=4096) == 1               # the router's term needs all three
    for mode in (dict(weights_in_expert=1), dict(stash_pool_pages=4), dict(dtype=1, H=256)):
        c = B.config(TINY.with_(**{k: v for k, v in mode.items() if k != "stash_pool_pages"}))
        c.stash_pool_pages = mode.get("stash_pool_pages", 0)
        assert fwd(experts(), cfg=c) == 2, mode
        assert bwd(experts(), cfg=c) == 2, mode
        with pytest.raises(B.MoEError) as e:
            B.moe_fp4_query_sizes(c, B.MOE_FP4_NV)
        assert e.value.code == 2


def test_scratch_sizes():
    with pytest.raises(B.MoEError):
        B.moe_fp4_query_sizes(None, 2)
    s = B.moe_fp4_query_sizes(None, B.MOE_FP4_NV)
    assert s.gemm_scratch_bytes >= 16 << 20 and s.fwd_scratch_bytes == 0
    for fmt in FORMATS:
        s = B.moe_fp4_query_sizes(MIXTRAL, fmt)
        R, H, F = 4096 * 2 + 8 * 127, 4096, 14336
        rows4 = R * (H + F) // 2 + B.fp4_scale_bytes(fmt, R, H) + B.fp4_scale_bytes(fmt, R, F)
        assert s.gemm_scratch_bytes + rows4 <= s.fwd_scratch_bytes <= \
            s.gemm_scratch_bytes + rows4 + 4096


def test_binding_checks_shapes():
    q = B.alloc_fp4(B.MOE_FP4_NV, 2, 130, 288, device="cpu")
    assert q.codes.shape == (2, 130, 144) and q.scales.shape == (2, 2, 8, 512)
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        B.moe_fp4_quantize(torch.zeros(2, 130, 256, dtype=bf), q, stream=0)
    with pytest.raises(ValueError):
        B.moe_fp4_quantize(torch.zeros(2, 130, 288), q, stream=0)
    with pytest.raises(ValueError):
        B.moe_fp4_quantize(torch.zeros(2, 140, 288, dtype=bf)[:, :130], q, stream=0)
    with pytest.raises(ValueError):
        B.moe_fp4_dequantize(q, torch.zeros(2, 288, 130, dtype=bf).transpose(1, 2), stream=0)
    with pytest.raises(ValueError):
        B.Fp4Tensor(B.MOE_FP4_NV, 256, q.codes, q.scales).struct()
    with pytest.raises(ValueError):
        B.Fp4Tensor(B.MOE_FP4_MX, 288, q.codes, q.scales).struct()
    with pytest.raises(ValueError):
        B.moe_fp4_grouped_gemm(B.alloc_fp4(0, 1, 4, 288, device="cpu"), q, None, None, None,
                               torch.zeros(4, 129, dtype=bf), None, stream=0)
