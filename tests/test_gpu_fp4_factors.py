"""Tensor scales over their whole accepted range, and experts' own scales (alpha) that bring
the results back into bf16's: against the fp64 oracle, with rows of zeros among the others."""
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


def quantised(rng, shape, log2, fmt=B.MOE_FP4_NV, zero_row=None, size=0.0):
    """bf16 numbers of about 2^(log2 + size) in 4 bits with that tensor scale, and their values."""
    x = rng.standard_normal(shape)
    if zero_row is not None:
        x[:, zero_row] = 0.0
    x = T4.bf(np.ldexp(x, int(log2 + size)))
    q = B.alloc_fp4(fmt, *shape, scale_log2=0 if fmt == B.MOE_FP4_MX else log2)
    B.moe_fp4_quantize(x, q)
    return q, x, O.real(fmt, f64(x), 0 if fmt == B.MOE_FP4_MX else log2)


# tensor scales of the two sides; alpha = m 2^e
FACTORS = [(64, 64, 1.5, -128), (64, 64, 1.25, -140), (64, 63, 1.75, -127), (-64, -64, 1.5, 127),
           (-64, -63, 1.25, 127), (-40, -40, 1.5, -20), (50, -50, 1.5, -130), (-64, 60, 1.5, 4),
           (60, 20, -1.5, 30)]


@pytest.mark.parametrize("rows,K", [(5, 288), (130, 288), (3, 8192), (900, 288)])
@pytest.mark.parametrize("xl,wl,m,e", FACTORS)
def test_product_over_the_range_of_scales(xl, wl, m, e, rows, K):
    """Whole tiles, cut ones (3 rows) and CTA pairs (900 rows)."""
    rng = np.random.default_rng(K + rows)
    xq, _, xv = quantised(rng, (1, rows, K), xl, zero_row=2)
    wq, _, wv = quantised(rng, (1, 136, K), wl)
    alpha = torch.tensor([np.ldexp(m, e)], dtype=torch.float32, device=DEV)
    assert float(alpha) == np.ldexp(m, e)
    out = torch.full((rows, 136), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, 0).gemm_scratch_bytes)
    cnt, offs = (torch.tensor([v], dtype=torch.int32, device=DEV) for v in (rows, 0))
    B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, alpha, out, sc)
    got, ref = f64(out), np.ldexp(m, e) * (xv[0] @ wv[0].T)
    mag = abs(np.ldexp(m, e)) * (np.abs(xv[0]) @ np.abs(wv[0]).T)
    assert (got[2] == 0).all()
    if e + xl + wl >= 100:                                 # past bf16: the infinity of its sign
        far = np.abs(ref) > 2.0 ** 128
        assert np.array_equal(got[far], np.copysign(np.inf, ref[far]))
        got, ref, mag = (np.where(far, 0.0, v) for v in (got, ref, mag))
    H_.assert_close("out", got, ref, atol=2.0 ** -134, rtol=1,
                    scale=2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag)


@pytest.mark.parametrize("xe,we,m,e", [(60, 60, 1.5, -130), (-60, -60, 1.5, 125), (0, 0, 1.25, -126)])
def test_mx_product_with_alphas_at_the_ends(xe, we, m, e):
    rng = np.random.default_rng(7)
    xq, _, xv = quantised(rng, (1, 5, 288), xe, B.MOE_FP4_MX, zero_row=2)
    wq, _, wv = quantised(rng, (1, 136, 288), we, B.MOE_FP4_MX)
    alpha = torch.tensor([np.ldexp(m, e)], dtype=torch.float32, device=DEV)
    out = torch.full((5, 136), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, 1).gemm_scratch_bytes)
    B.moe_fp4_grouped_gemm(xq, wq, None, None, alpha, out, sc)
    got, ref = f64(out), np.ldexp(m, e) * (xv[0] @ wv[0].T)
    assert (got[2] == 0).all()
    mag = np.ldexp(m, e) * (np.abs(xv[0]) @ np.abs(wv[0]).T)
    H_.assert_close("out", got, ref, atol=2.0 ** -134, rtol=1,
                    scale=2.0 ** -8 * np.abs(ref) + 288 * 2.0 ** -23 * mag)


# s: gate and up are of size 2^s, so h of 2^(2 s) (where gate is positive, for large s)
@pytest.mark.parametrize("x_log2,w13,s,h_log2,w2,e2", [
    (3, -3, 0, -5, -2, 0), (64, 64, 34, 64, 20, -80), (-64, -64, -31, -64, -64, 120),
    (-30, 30, 34, 64, 64, -128)])
@pytest.mark.parametrize("counts", [[1], [40, 0, 3], [1000, 900]])
def test_ffn_with_tensor_scales(counts, x_log2, w13, s, h_log2, w2, e2):
    """x and h quantised with tensor scales of their own, in every form of the products."""
    rng = np.random.default_rng(len(counts))
    H, F, G = 256, 256, len(counts)
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("s", T=sum(counts), H=H, E=G, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    x = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    x[rows] = T4.bf(np.ldexp(rng.standard_normal((len(rows), H)), x_log2 + 3))
    if len(rows) > 1:
        x[rows[-1]] = 0
    W13q, _, W13v = quantised(rng, (G, 2 * F, H), w13, size=3.0)
    W2q, _, W2v = quantised(rng, (G, H, F), w2, size=3.0)
    a13 = np.ldexp(1.0 + 0.5 * rng.random(G), s - (x_log2 + w13 + 10))
    a2 = np.ldexp(1.0 + 0.5 * rng.random(G), e2)
    dev = lambda a: torch.tensor(a, dtype=torch.float32, device=DEV)  # noqa: E731
    a13t, a2t = dev(a13), dev(a2)
    a13, a2 = f64(a13t), f64(a2t)
    ex = B.fp4_experts(W13q, W2q, a13t, a2t, x_scale_log2=x_log2, h_scale_log2=h_log2)
    y = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).fwd_scratch_bytes)
    B.moe_fp4_ffn_fwd(cfg, ex, x, cnt, offs, None, None, y, sc)
    assert B.moe_last_device_status(sc) == 0
    got, xv = f64(y), f64(x)
    assert len(rows) == 1 or not got[rows[-1]].any()
    for g, c in enumerate(counts):
        if c == 0:
            continue
        r = slice(off[g], off[g] + c)
        W13, W2 = W13v[g] * a13[g], W2v[g] * a2[g]
        gu, lo, hi, h4, slack = interval(xv[r], W13, x_log2, h_log2)
        ref, mag = h4 @ W2.T, np.abs(h4) @ np.abs(W2).T
        H_.assert_close(f"y of {g}", got[r], ref, atol=2.0 ** -134, rtol=1,
                        scale=2.0 ** -8 * np.abs(ref) + F * 2.0 ** -23 * mag + slack @ np.abs(W2).T)


def interval(x, W13, x_log2, h_log2):
    """h's 4-bit values as the oracle has them, and how far the bounds of G and U let the GPU's
    be from them (the tensor scales' form of test_gpu_fp4.h_interval)."""
    xv = O.real(B.MOE_FP4_NV, x, x_log2)
    gu = xv @ W13.T
    err = x.shape[1] * 2.0 ** -23 * (np.abs(xv) @ np.abs(W13).T)
    lo, hi = O.round_bf16(gu - err), O.round_bf16(gu + err)
    F = gu.shape[1] // 2
    c = np.stack([O.silu(g) * u for g in (lo[:, :F], hi[:, :F]) for u in (lo[:, F:], hi[:, F:])])
    h = O.round_bf16(O.silu(O.round_bf16(gu[:, :F])) * O.round_bf16(gu[:, F:]))
    hl = O.round_bf16(np.minimum(c.min(0) - 2.0 ** -20 * np.abs(c).max(0), h))
    hh = O.round_bf16(np.maximum(c.max(0) + 2.0 ** -20 * np.abs(c).max(0), h))
    h4, a, b = (O.real(B.MOE_FP4_NV, v, h_log2) for v in (h, hl, hh))
    amax = lambda v: np.abs(v).reshape(len(v), -1, 16).max(-1)  # noqa: E731
    same = np.where(np.sign(hl) == np.sign(hh), np.minimum(np.abs(hl), np.abs(hh)), 0.0)
    top = amax(np.maximum(np.abs(hl), np.abs(hh)))
    moved = np.repeat(amax(same) != top, 16, 1)
    # a scale that moved by a step (1/8, or 2^-9 of the tensor's unit below E4M3's normal
    # range) moves a value by at most one step of the grid (2 units of 6) more
    unit = np.repeat(np.maximum(top / 6.0 * 1.125, np.ldexp(1.0, h_log2 - 9)), 16, 1)
    slack = np.maximum(np.abs(a - h4), np.abs(b - h4)) + np.where(moved, 2.0 * unit, 0.0)
    return gu, lo, hi, h4, slack


@pytest.mark.parametrize("w13,w2,e13,e2", [(64, 64, -64, -64), (64, 64, -130, 2), (-64, -64, 64, 64),
                                           (-64, -64, 127, 1), (-3, 5, 0, 0), (0, 0, -70, -70)])
def test_backward_over_the_range_of_scales(w13, w2, e13, e2):
    """dX = alpha13 alpha2 2^(w13 + w2) times the codes' sums, whatever the factors' sizes."""
    rng = np.random.default_rng(31)
    H, F, counts = 256, 128, [40, 129]
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("b", T=len(rows), H=H, E=2, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    W13q, _, W13v = quantised(rng, (2, 2 * F, H), w13)
    W2q, _, W2v = quantised(rng, (2, H, F), w2)
    dev = lambda a: torch.tensor(a, dtype=torch.float32, device=DEV)  # noqa: E731
    a13t, a2t = dev(np.ldexp([1.0, 1.5], e13)), dev(np.ldexp([1.25, 1.0], e2))
    ex = B.fp4_experts(W13q, W2q, a13t, a2t)
    up = -(w13 + w2 + e13 + e2)                            # dO's size: dX of order one
    up = max(-60, min(60, up))
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[rows] = T4.bf(np.ldexp(rng.standard_normal((len(rows), H)), up))
    dO[rows[3]] = 0
    codes = rng.integers(0, 120, (R, 2 * F), dtype=np.uint8)
    byte = np.full((R, 2 * F // 32), 118, np.uint8)
    ck, cs = torch.from_numpy(codes).to(DEV), torch.from_numpy(byte).to(DEV)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex, dO, ck, cs, cnt, offs, None, None, None, dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got, dOv = f64(dX), f64(dO)
    assert not got[rows[3]].any()
    for g, c in enumerate(counts):
        r = slice(off[g], off[g] + c)
        W13, W2 = W13v[g] * float(a13t[g]), W2v[g] * float(a2t[g])
        gu = O.checkpoint_values(codes[r], byte[r])
        ref, dgu = O.ffn_bwd(dOv[r], gu, W13, W2)
        _, err = O.ffn_bwd(np.abs(dOv[r]), gu, np.abs(W13), np.abs(W2))
        d_err = 2.0 ** -8 * np.abs(dgu) + (H * 2.0 ** -23 + 2.0 ** -18) * np.abs(err)
        mag = np.abs(dgu) @ np.abs(W13)
        H_.assert_close(f"dX of {g}", got[r], ref, atol=2.0 ** -134, rtol=1,
                        scale=2.0 ** -8 * np.abs(ref) + d_err @ np.abs(W13) + 2 * F * 2.0 ** -23 * mag)
