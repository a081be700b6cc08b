"""The 4-bit experts on the GPU against the fp64 oracle.

Tolerances, derived from the formats and never from a run:
  quantiser, its inverse, the values            exact
  a bf16 result                                 half a step, 2^-8 of the value
  fp32 sums of K exact products                 K 2^-23 of the sum of magnitudes
  quantised h                                   the values that h's bounds allow: G, U within
                                                their sums' error, bf16's borders crossed or not
  [dG|dU] rounded to bf16 between the products  2^-8 of each term's magnitude
"""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O
from workloads import SIGMOID, TINY, MoEShape, make_inputs

pytestmark = pytest.mark.gpu

H_ = pytest.importorskip("harness")
FORMATS = (B.MOE_FP4_NV, B.MOE_FP4_MX)
DEV = "cuda"


def f64(t):
    return t.double().cpu().numpy()


def host(t):
    return t.cpu().numpy()


def bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(DEV).bfloat16()


def rows_of(rng, *shape, spread=True):
    """bf16 rows whose blocks differ in size, some zero."""
    x = rng.standard_normal(shape)
    if spread:
        x *= np.exp2(rng.integers(-6, 4, shape[:-1] + (1,)))
        x[..., ::7] *= 9.0
        x[..., : shape[-1] // 8] *= rng.random(shape[:-1] + (1,)) > 0.3
    return bf(x)


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("groups,rows,K,log2", [
    (1, 1, 32, 0), (1, 1, 7168, 0), (3, 130, 288, -3), (1, 127, 2080, 0), (2, 129, 512, 5),
    (1, 33, 544, -11), (5, 256, 64, 0)])
def test_quantise_equals_the_oracle(fmt, groups, rows, K, log2):
    rng = np.random.default_rng(rows + K)
    log2 = 0 if fmt == B.MOE_FP4_MX else log2
    x = rows_of(rng, groups, rows, K)
    q = B.alloc_fp4(fmt, groups, rows, K)
    q.scales.fill_(0xEE)
    values = torch.full_like(x, float("nan"))
    B.moe_fp4_quantize(x, q, scale_log2=log2, values=values)
    codes, byte = O.quantise(fmt, f64(x), log2)
    H_.assert_equal("scales", host(q.scales), O.to_atoms(fmt, byte, K))
    H_.assert_equal("codes", host(q.codes), O.pack(codes))
    ref = O.values(fmt, codes, byte, log2)
    H_.assert_equal("values", f64(values), ref)
    out = torch.full_like(x, float("nan"))
    B.moe_fp4_dequantize(q, out)
    H_.assert_equal("dequantised", f64(out), ref)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_at_the_borders_of_the_grid(fmt):
    """Every tie and its two neighbours in bf16, for every scale a block can get."""
    n = O.BLOCK[fmt]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    units = O.E4M3[1:] if fmt == B.MOE_FP4_NV else np.exp2(np.arange(-100, 100))
    rows = []
    for u in units:
        t = ties * u
        step = np.exp2(np.floor(np.log2(t)) - 7)           # bf16's step at t
        v = np.concatenate((t, t + step, t - step))
        for i in range(0, 21, n - 1):
            blk = np.zeros(n)
            part = v[i:i + n - 1]
            blk[:len(part)] = part * np.where(np.arange(len(part)) % 2, -1, 1)
            blk[-1] = 6.0 * u                              # amax: the block's scale is u
            rows.append(blk)
    a = np.concatenate(rows)
    K = -(-a.size // 32) * 32
    x = bf(np.pad(a, (0, K - a.size)))[None, None]
    q = B.alloc_fp4(fmt, 1, 1, K)
    B.moe_fp4_quantize(x, q)
    codes, byte = O.quantise(fmt, f64(x))
    H_.assert_equal("scales", host(q.scales), O.to_atoms(fmt, byte, K))
    H_.assert_equal("codes", host(q.codes), O.pack(codes))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_extremes(fmt):
    """bf16's largest and smallest values, infinities and NaN."""
    big, tiny = 3.3895313892515355e38, 2.0 ** -133
    x = torch.zeros(1, 8, 64)
    x[0, 0, :] = big
    x[0, 1, 3] = tiny
    x[0, 2, 5], x[0, 2, 40] = float("inf"), 1.0
    x[0, 3, 7], x[0, 3, 41] = float("nan"), -2.0
    x[0, 4, 8] = -float("inf")
    x[0, 5, :] = 2.0 ** -126
    x[0, 6, 1], x[0, 6, 2] = -0.0, 1.5
    x = x.to(DEV).bfloat16()
    q = B.alloc_fp4(fmt, 1, 8, 64)
    values = torch.empty_like(x)
    B.moe_fp4_quantize(x, q, values=values)
    codes, byte = O.quantise(fmt, f64(x))
    H_.assert_equal("scales", host(q.scales), O.to_atoms(fmt, byte, 64))
    H_.assert_equal("codes", host(q.codes), O.pack(codes))
    ref = O.values(fmt, codes, byte)
    ref[np.abs(ref) >= 2.0 ** 128] = np.inf                # past bf16's largest (4 x 2^126)
    got = f64(values)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    H_.assert_equal("values", np.nan_to_num(got), np.nan_to_num(ref))


def test_quantise_strided_rows_and_another_stream():
    wide = torch.randn(70, 1024, device=DEV).bfloat16()
    x = wide[:, 256:544][None]                             # rows 1024 apart
    q = B.alloc_fp4(B.MOE_FP4_NV, 1, 70, 288)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.moe_fp4_quantize(x, q, stream=s)
    out = torch.zeros(70, 512, device=DEV, dtype=torch.bfloat16)
    s.wait_stream(torch.cuda.current_stream())
    B.moe_fp4_dequantize(q, out[None, :, 64:352], stream=s)
    s.synchronize()
    H_.assert_equal("values", f64(out[:, 64:352]), O.real(B.MOE_FP4_NV, f64(x[0])))
    assert not out[:, :64].any() and not out[:, 352:].any()


def segments(counts):
    off = np.concatenate(([0], np.cumsum([-(-c // 128) * 128 for c in counts])))
    rows = np.concatenate([np.arange(o, o + c) for o, c in zip(off, counts)]).astype(np.int64)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    return off, rows, i32(counts), i32(off)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_segments_leaves_other_rows(fmt):
    counts = [0, 1, 130, 0, 128, 5, 0]
    off, rows, cnt, offs = segments(counts)
    R, K = int(off[-1]) + 77, 288
    x = rows_of(np.random.default_rng(3), 1, R, K)
    q = B.alloc_fp4(fmt, 1, R, K)
    q.codes.fill_(0x5A)
    sc = B.alloc_fp4_scratch(4096)
    B.moe_fp4_quantize(x, q, counts=cnt, offsets=offs, scratch=sc)
    codes, byte = O.quantise(fmt, f64(x)[0])
    got = host(q.codes)[0]
    H_.assert_equal("codes", got[rows], O.pack(codes)[rows])
    other = np.setdiff1d(np.arange(R), rows)
    assert (got[other] == 0x5A).all()
    H_.assert_equal("scales", O.from_atoms(fmt, host(q.scales), R, K)[0][rows], byte[rows])
    assert B.moe_last_device_status(sc) == 0
    for bad in ([0, 1, 130, 0, 128, R, 0], [0, -1, 130, 0, 128, 5, 0]):
        c = torch.tensor(bad, dtype=torch.int32, device=DEV)
        B.moe_clear_device_status(sc)
        B.moe_fp4_quantize(x, q, counts=c, offsets=offs, scratch=sc)
        assert B.moe_last_device_status(sc) == 6           # MOE_ERR_DEVICE_CHECK


# -------------------------------------------------------------------- product
def weights(fmt, rng, G, N, K, log2=0):
    """Weights in 4 bits, and the values they stand for."""
    w = rows_of(rng, G, N, K, spread=False)
    q = B.alloc_fp4(fmt, G, N, K)
    values = torch.empty_like(w)
    B.moe_fp4_quantize(w, q, scale_log2=log2, values=values)
    return q, f64(values)


PRODUCTS = [
    ([1], 8, 32), ([0], 64, 64), ([1, 0, 1, 3], 1000, 288), ([127, 128, 129, 0, 1], 264, 1504),
    # many rows an expert (CTA pairs): odd and even numbers of 128-row tiles, an empty one
    ([1700, 3, 0, 1900], 264, 800), ([812], 136, 96), ([1100, 900], 512, 2080),
    ([300, 2], 128, 4096), ([33], 512, 7168), ([600], 520, 544), ([31, 32, 64, 65, 96, 97], 256, 256),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,N,K", PRODUCTS)
def test_product_matches_oracle(fmt, counts, N, K):
    rng = np.random.default_rng(N + K)
    log2 = -2 if fmt == B.MOE_FP4_NV else 0
    off, rows, cnt, offs = segments(counts)
    R = max(int(off[-1]), 1) + 13
    x = rows_of(rng, 1, R, K)
    xq = B.alloc_fp4(fmt, 1, R, K)
    xq.scales.fill_(0xFF)                                  # rows without data: NaN scales
    xq.codes.fill_(0x77)
    B.moe_fp4_quantize(x, xq, counts=cnt, offsets=offs)
    wq, wv = weights(fmt, rng, len(counts), N, K, log2)
    alpha = torch.tensor(0.5 + rng.random(len(counts)), dtype=torch.float32, device=DEV)
    out = torch.full((R, N), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, fmt).gemm_scratch_bytes)
    B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, alpha, out, sc)
    assert B.moe_last_device_status(sc) == 0
    got, xv = f64(out), O.real(fmt, f64(x)[0])
    ref, mag = np.full((R, N), 7.0), np.zeros((R, N))
    for g, c in enumerate(counts):
        r = slice(off[g], off[g] + c)
        ref[r] = xv[r] @ wv[g].T * float(alpha[g])
        mag[r] = np.abs(xv[r]) @ np.abs(wv[g]).T * float(alpha[g])
    H_.assert_close("out", got, ref, atol=0, rtol=1, scale=2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag)
    again = torch.full_like(out, 7.0)
    B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, alpha, again, sc)
    assert torch.equal(out, again)                         # the counters were left at zero


@pytest.mark.parametrize("rows", [1, 20, 32, 50, 64, 200])
def test_product_dense_form_and_no_alpha(rows):
    rng = np.random.default_rng(5)
    x = rows_of(rng, 1, rows, 320)
    xq = B.alloc_fp4(B.MOE_FP4_NV, 1, rows, 320)
    B.moe_fp4_quantize(x, xq, scale_log2=1)
    wq, wv = weights(B.MOE_FP4_NV, rng, 1, 72, 320)
    out = torch.empty(rows, 72, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, 0).gemm_scratch_bytes)
    B.moe_fp4_grouped_gemm(xq, wq, None, None, None, out, sc)
    xv = O.real(B.MOE_FP4_NV, f64(x)[0], 1)
    ref, mag = xv @ wv[0].T, np.abs(xv) @ np.abs(wv[0]).T
    H_.assert_close("out", f64(out), ref, atol=0, rtol=1,
                    scale=2.0 ** -8 * np.abs(ref) + 320 * 2.0 ** -23 * mag)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_of_nonfinite_rows_stays_in_them(fmt):
    x = torch.randn(1, 40, 256, device=DEV).bfloat16()
    x[0, 3, 7], x[0, 20, 100] = float("nan"), float("inf")
    xq = B.alloc_fp4(fmt, 1, 40, 256)
    B.moe_fp4_quantize(x, xq)
    wq, wv = weights(fmt, np.random.default_rng(6), 1, 64, 256)
    out = torch.empty(40, 64, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, fmt).gemm_scratch_bytes)
    B.moe_fp4_grouped_gemm(xq, wq, None, None, None, out, sc)
    got = f64(out)
    bad = np.zeros(40, bool)
    bad[[3, 20]] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("counts,offsets", [
    ([5, 300], [0, 128]), ([5, -1], [0, 128]), ([5, 5], [0, 130]), ([5, 5], [0, -128])])
def test_product_reports_bad_segments(counts, offsets):
    """A segment outside the rows or off the 128-row grid is left out and reported."""
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(1, 256, 64, device=DEV).bfloat16()
    xq = B.alloc_fp4(0, 1, 256, 64)
    B.moe_fp4_quantize(x, xq)
    wq, wv = weights(0, np.random.default_rng(7), 2, 64, 64)
    out = torch.full((256, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, 0).gemm_scratch_bytes)
    B.moe_fp4_grouped_gemm(xq, wq, i32(counts), i32(offsets), None, out, sc)
    assert B.moe_last_device_status(sc) == 6
    got = f64(out)
    assert (got[5:] == 7.0).all() and (got[:5] != 7.0).any()


# ------------------------------------------------------------------------ FFN
def experts_of(fmt, rng, G, H, F):
    log2 = -3 if fmt == B.MOE_FP4_NV else 0
    W13q, W13 = weights(fmt, rng, G, 2 * F, H, log2)
    W2q, W2 = weights(fmt, rng, G, H, F, log2)
    a13 = torch.tensor((0.5 + rng.random(G)) / np.sqrt(H), dtype=torch.float32, device=DEV)
    a2 = torch.tensor((0.5 + rng.random(G)) / np.sqrt(F), dtype=torch.float32, device=DEV)
    ex = B.fp4_experts(W13q, W2q, a13, a2)
    return (ex, W13q, W2q, a13, a2, W13 * f64(a13)[:, None, None], W2 * f64(a2)[:, None, None])


def h_interval(fmt, x, W13):
    """h's 4-bit values as the oracle has them, and how far the bounds of G and U let the
    GPU's be from them; with G, U (bf16) and their bounds."""
    xv = O.real(fmt, x)
    K = x.shape[1]
    gu = xv @ W13.T
    err = K * 2.0 ** -23 * (np.abs(xv) @ np.abs(W13).T)
    lo, hi = O.round_bf16(gu - err), O.round_bf16(gu + err)
    F = gu.shape[1] // 2
    # silu on the special-function unit: a few fp32 ulp, taken as 2^-20
    c = np.stack([O.silu(g) * u for g in (lo[:, :F], hi[:, :F]) for u in (lo[:, F:], hi[:, F:])])
    h = O.round_bf16(O.silu(O.round_bf16(gu[:, :F])) * O.round_bf16(gu[:, F:]))
    hl = O.round_bf16(np.minimum(c.min(0) - 2.0 ** -20 * np.abs(c).max(0), h))
    hh = O.round_bf16(np.maximum(c.max(0) + 2.0 ** -20 * np.abs(c).max(0), h))
    h4 = O.real(fmt, h)
    # where some element of a block is uncertain, its scale may be too: the block's
    # elements may sit anywhere between the two quantisations
    a, b = O.real(fmt, hl), O.real(fmt, hh)
    n = O.BLOCK[fmt]
    amax = lambda v: np.abs(v).reshape(len(v), -1, n).max(-1)  # noqa: E731
    top_lo = amax(np.where(np.sign(hl) == np.sign(hh), np.minimum(np.abs(hl), np.abs(hh)), 0.0))
    top_hi = amax(np.maximum(np.abs(hl), np.abs(hh)))
    moved = np.repeat(top_lo != top_hi, n, 1)
    # a scale that moved by a step (1/8 for E4M3, 2 for a power of two) moves a value by at
    # most one step of the grid (6 - 4 = 2 units of 6) more
    unit = np.repeat(top_hi, n, 1) / 6.0 * (2.0 if fmt == B.MOE_FP4_MX else 1.125)
    slack = np.maximum(np.abs(a - h4), np.abs(b - h4)) + np.where(moved, 2.0 * unit, 0.0)
    return gu, lo, hi, h4, slack


FFNS = [([1], 128, 128), ([0, 3, 130, 0, 64], 128, 384), ([40, 129], 256, 640),
        # sums cut over the SMs: up to 64 rows, several parts of a tile
        ([1], 512, 2048), ([40, 0, 1, 64], 1024, 384), ([2, 33], 256, 4096),
        # CTA pairs
        ([1000, 612], 256, 384), ([2200, 0, 260], 384, 256)]


def run_ffn(fmt, counts, H, F, ckpt=True, seed=0, T=None):
    rng = np.random.default_rng(seed)
    off, rows, cnt, offs = segments(counts)
    G = len(counts)
    cfg = B.config(MoEShape("f", T=max(sum(counts), 1), H=H, E=G, k=1, F=F))
    R = B.moe_query_sizes(cfg).rows_max
    assert R >= off[-1]
    x = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    x[rows] = rows_of(rng, len(rows), H, spread=False)
    ex = experts_of(fmt, rng, G, H, F)
    y = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    ck = torch.full((R, 2 * F), 0x11, dtype=torch.uint8, device=DEV) if ckpt else None
    cs = torch.full((R, 2 * F // 32), 0x11, dtype=torch.uint8, device=DEV) if ckpt else None
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).fwd_scratch_bytes)
    B.moe_fp4_ffn_fwd(cfg, ex[0], x, cnt, offs, ck, cs, y, sc)
    assert B.moe_last_device_status(sc) == 0
    return dict(cfg=cfg, R=R, off=off, rows=rows, cnt=cnt, offs=offs, x=x, ex=ex, y=y, ck=ck,
                cs=cs, sc=sc)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,H,F", FFNS)
def test_ffn_forward_and_checkpoint_match_oracle(fmt, counts, H, F):
    s = run_ffn(fmt, counts, H, F)
    y, x = f64(s["y"]), f64(s["x"])
    W13, W2 = s["ex"][5], s["ex"][6]
    if len(s["rows"]):
        kept = O.checkpoint_values(host(s["ck"])[s["rows"]], host(s["cs"])[s["rows"]])
    at = 0
    for g, c in enumerate(counts):
        if c == 0:
            continue
        r = slice(s["off"][g], s["off"][g] + c)
        gu, lo, hi, h4, slack = h_interval(fmt, x[r], W13[g])
        ref, mag = h4 @ W2[g].T, np.abs(h4) @ np.abs(W2[g]).T
        H_.assert_close(f"y of {g}", y[r], ref, atol=0, rtol=1,
                        scale=2.0 ** -8 * np.abs(ref) + F * 2.0 ** -23 * mag + slack @ np.abs(W2[g]).T)
        # the checkpoint: half a step of E4M3 (2^-4 of the value, 2^-10 of the unit below its
        # normal range; the unit may be the next one where amax is uncertain)
        k = kept[at:at + c]
        at += c
        unit = 2.0 * np.repeat(O.checkpoint_unit(np.maximum(np.abs(lo), np.abs(hi))), 32, 1)
        bound = 2.0 ** -4 * np.maximum(np.abs(lo), np.abs(hi)) + 2.0 ** -10 * unit + (hi - lo)
        H_.assert_close(f"checkpoint of {g}", k, O.round_bf16(gu), atol=0, rtol=1, scale=bound)
    other = np.setdiff1d(np.arange(s["R"]), s["rows"])
    assert (y[other] == 7.0).all()
    assert (host(s["ck"])[other] == 0x11).all() and (host(s["cs"])[other] == 0x11).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_ffn_without_checkpoint_and_repeated(fmt):
    a = run_ffn(fmt, [3, 0, 200], 256, 384)
    b = run_ffn(fmt, [3, 0, 200], 256, 384, ckpt=False)
    assert torch.equal(a["y"], b["y"])
    B.moe_fp4_ffn_fwd(a["cfg"], a["ex"][0], a["x"], a["cnt"], a["offs"], a["ck"], a["cs"], b["y"], a["sc"])
    assert torch.equal(a["y"], b["y"])


def test_ffn_rows_do_not_depend_on_the_batch():
    """A token's row is the same alone (its sums cut over the SMs) as among others, up to the
    order of fp32 sums: y within two bf16 steps where no 4-bit rounding of h moved."""
    s = run_ffn(B.MOE_FP4_NV, [200], 512, 1024)
    cnt = torch.tensor([1], dtype=torch.int32, device=DEV)
    y = torch.zeros_like(s["y"])
    B.moe_fp4_ffn_fwd(s["cfg"], s["ex"][0], s["x"], cnt, s["offs"], None, None, y, s["sc"])
    gu, lo, hi, h4, slack = h_interval(B.MOE_FP4_NV, f64(s["x"])[:1], s["ex"][5][0])
    W2 = np.abs(s["ex"][6][0])
    bound = 2.0 ** -7 * np.abs(f64(s["y"])[:1]) + 2 * (slack + 1024 * 2.0 ** -23 * np.abs(h4)) @ W2.T
    H_.assert_close("row", f64(y)[:1], f64(s["y"])[:1], atol=0, rtol=1, scale=bound)


# ------------------------------------------------------------------- backward
def test_backward_reports_bad_segments():
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    rng = np.random.default_rng(12)
    cfg = B.config(MoEShape("b", T=200, H=128, E=2, k=1, F=128))
    R = B.moe_query_sizes(cfg).rows_max
    ex = experts_of(0, rng, 2, 128, 128)
    dO = torch.ones(R, 128, device=DEV, dtype=torch.bfloat16)
    ck = torch.full((R, 256), 0x38, dtype=torch.uint8, device=DEV)
    cs = torch.full((R, 8), 127, dtype=torch.uint8, device=DEV)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).bwd_scratch_bytes)
    for counts, offsets in (([5, R], [0, 128]), ([5, -2], [0, 128]), ([5, 5], [0, 64]),
                            ([5, 5], [0, -128])):
        B.moe_clear_device_status(sc)
        dX = torch.full((R, 128), 7.0, device=DEV, dtype=torch.bfloat16)
        B.moe_fp4_ffn_bwd(cfg, ex[0], dO, ck, cs, i32(counts), i32(offsets), None, None, None, dX, sc)
        assert B.moe_last_device_status(sc) == 6
        got = f64(dX)
        assert (got[:5] != 7.0).any() and (got[5:128] == 0).all() and (got[128:] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,H,F,router", [
    ([1], 128, 128, False), ([0, 3, 130, 0, 64], 128, 384, True), ([40, 129], 256, 640, False),
    ([700, 20], 256, 256, True), ([520, 600], 512, 256, False)])
def test_ffn_backward_matches_oracle(fmt, counts, H, F, router):
    rng = np.random.default_rng(11)
    off, rows, cnt, offs = segments(counts)
    G, n = len(counts), len(rows)
    cfg = B.config(MoEShape("b", T=max(n, 1), H=H, E=G, k=1, F=F))
    R = B.moe_query_sizes(cfg).rows_max
    ex = experts_of(fmt, rng, G, H, F)
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[rows] = rows_of(rng, n, H, spread=False)
    codes = rng.integers(0, 256, (R, 2 * F), dtype=np.uint8)
    codes = np.where(codes & 127 == 127, 0x38, codes).astype(np.uint8)     # no NaN code
    byte = rng.integers(117, 120, (R, 2 * F // 32), dtype=np.uint8)        # units 2^-10 .. 2^-8
    other = np.setdiff1d(np.arange(R), rows)
    codes[other], byte[other] = 0x7F, 0xFF                 # rows without data: NaN
    token_of = np.full(R, -1, np.int32)
    token_of[rows] = rng.permutation(n)
    dl = rng.standard_normal((max(n, 1), G)).astype(np.float32)
    Wr = rng.standard_normal((G, H)).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    ck, cs, tok, dlt, wrt = dev(codes), dev(byte), dev(token_of), dev(dl), dev(Wr)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).bwd_scratch_bytes)
    sc[4096:] = 0xFF                                       # NaN in whatever is not written first
    more = (tok, dlt, wrt) if router else (None, None, None)
    B.moe_fp4_ffn_bwd(cfg, ex[0], dO, ck, cs, cnt, offs, *more, dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got, dOv = f64(dX), f64(dO)
    W13, W2 = ex[5], ex[6]
    for g, c in enumerate(counts):
        if c == 0:
            continue
        r = slice(off[g], off[g] + c)
        gu = O.checkpoint_values(codes[r], byte[r])
        ref, dgu = O.ffn_bwd(dOv[r], gu, W13[g], W2[g])
        # dh's fp32 sum, the derivative's few fp32 roundings (2^-18), dGU's bf16 rounding
        _, dgu_err = O.ffn_bwd(np.abs(dOv[r]), gu, np.abs(W13[g]), np.abs(W2[g]))
        d_err = 2.0 ** -8 * np.abs(dgu) + (H * 2.0 ** -23 + 2.0 ** -18) * np.abs(dgu_err)
        if router:
            ref = ref + dl[token_of[r], g][:, None] * Wr[g]
        mag = np.abs(dgu) @ np.abs(W13[g])
        bound = 2.0 ** -8 * np.abs(ref) + d_err @ np.abs(W13[g]) + 2 * F * 2.0 ** -23 * mag
        H_.assert_close(f"dX of {g}", got[r], ref, atol=0, rtol=1, scale=bound)
        # the roundings are independent: their norm is that of one rounding of each kind,
        # 2^-8 / sqrt(3) of a value at most for dX and for dGU's terms
        rel = np.linalg.norm(got[r] - ref) / np.linalg.norm(ref)
        assert rel < 2.0 ** -8 * 1.2, rel
        pad = got[off[g] + c:off[g + 1]]
        assert (pad == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_repeated_passes_are_equal_bit_for_bit(fmt):
    """Thirty passes of every product over the same rows: whatever the order in which loads
    land and parts arrive, the results are the same numbers."""
    rng = np.random.default_rng(21)
    counts, H, F = [2520, 0, 600, 40], 512, 1024
    off, rows, cnt, offs = segments(counts)
    cfg = B.config(MoEShape("r", T=len(rows), H=H, E=4, k=1, F=F))
    R = B.moe_query_sizes(cfg).rows_max
    ex = experts_of(fmt, rng, 4, H, F)
    x = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    x[rows] = rows_of(rng, len(rows), H, spread=False)
    ck = torch.zeros(R, 2 * F, dtype=torch.uint8, device=DEV)
    cs = torch.zeros(R, 2 * F // 32, dtype=torch.uint8, device=DEV)
    sz = B.moe_fp4_query_sizes(cfg, fmt)
    sf, sb = B.alloc_fp4_scratch(sz.fwd_scratch_bytes), B.alloc_fp4_scratch(sz.bwd_scratch_bytes)
    few = torch.tensor([3, 0, 64, 1], dtype=torch.int32, device=DEV)      # sums cut over the SMs
    first = None
    for _ in range(30):
        y, z, dX = (torch.zeros(R, H, device=DEV, dtype=torch.bfloat16) for _ in range(3))
        B.moe_fp4_ffn_fwd(cfg, ex[0], x, few, offs, None, None, z, sf)
        B.moe_fp4_ffn_fwd(cfg, ex[0], x, cnt, offs, ck, cs, y, sf)
        B.moe_fp4_ffn_bwd(cfg, ex[0], y, ck, cs, cnt, offs, None, None, None, dX, sb)
        now = (y, z, dX, ck.clone(), cs.clone())
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    assert B.moe_last_device_status(sf) == 0 and B.moe_last_device_status(sb) == 0


# -------------------------------------------------------------- a layer, a graph
LAYER = MoEShape("fp4_layer", T=300, H=256, E=8, k=2, F=384, bias_kind="none")


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_with_4_bit_experts(fmt):
    """Route, dispatch, 4-bit experts with the checkpoint, combine, and the gradient at the
    layer's input: the framework's own stages around the new ones. Each is checked on its own
    elsewhere; here the whole against the oracle's experts on the GPU's own dispatched rows."""
    inp = {k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in make_inputs(LAYER, seed=0).items()}
    cfg = B.config(LAYER)
    bufs = B.alloc_buffers(cfg, DEV)
    f, b, sc = bufs.fwd, bufs.bwd, bufs.scratch
    B.moe_route(cfg, inp["x"], inp["W_r"], None, f["logits"], f["idx"], f["w"], sc)
    B.moe_permute(cfg, inp["x"], f["idx"], f["counts"], f["offsets"], f["row_of"], f["token_of"],
                  f["sel_offsets"], f["sel_tokens"], f["x_perm"], sc)
    G, H, F = LAYER.E, LAYER.H, LAYER.F
    log2 = -9 if fmt == B.MOE_FP4_NV else 0
    q13, q2 = B.alloc_fp4(fmt, G, 2 * F, H), B.alloc_fp4(fmt, G, H, F)
    v13, v2 = torch.empty_like(inp["W13"]), torch.empty_like(inp["W2"])
    B.moe_fp4_quantize(inp["W13"], q13, scale_log2=log2, values=v13)
    B.moe_fp4_quantize(inp["W2"], q2, scale_log2=log2, values=v2)
    ex = B.fp4_experts(q13, q2)
    sz = B.moe_fp4_query_sizes(cfg, fmt)
    sf, sb = B.alloc_fp4_scratch(sz.fwd_scratch_bytes), B.alloc_fp4_scratch(sz.bwd_scratch_bytes)
    R = bufs.sizes.rows_max
    ck = torch.empty(R, 2 * F, dtype=torch.uint8, device=DEV)
    cs = torch.empty(R, 2 * F // 32, dtype=torch.uint8, device=DEV)
    out, dx = torch.empty_like(inp["x"]), torch.empty_like(inp["x"])

    def step():
        B.moe_fp4_ffn_fwd(cfg, ex, f["x_perm"], f["counts"], f["offsets"], ck, cs, f["y_perm"], sf)
        B.moe_unpermute(cfg, f["y_perm"], f["row_of"], f["w"], f["offsets"], out)
        B.moe_unpermute_bwd(cfg, inp["dY"], f["y_perm"], f["row_of"], f["w"], f["counts"],
                            f["offsets"], b["dO_perm"], b["dw"], sc)
        B.moe_route_bwd(cfg, f["logits"], f["idx"], f["w"], b["dw"], b["dlogits"])
        B.moe_fp4_ffn_bwd(cfg, ex, b["dO_perm"], ck, cs, f["counts"], f["offsets"], f["token_of"],
                          b["dlogits"], inp["W_r"], b["dX_perm"], sb)
        B.moe_permute_bwd(cfg, b["dX_perm"], f["row_of"], f["offsets"], f["idx"], b["dlogits"],
                          inp["W_r"], dx)

    step()
    torch.cuda.synchronize()
    assert B.moe_last_device_status(sf) == 0 and B.moe_last_device_status(sb) == 0
    counts, off = host(f["counts"]), host(f["offsets"])
    x, y, dO, dX = (f64(t) for t in (f["x_perm"], f["y_perm"], b["dO_perm"], b["dX_perm"]))
    tok, dl, Wr = host(f["token_of"]), f64(b["dlogits"]), f64(inp["W_r"])
    for g in range(G):
        r = slice(off[g], off[g] + counts[g])
        W13, W2 = f64(v13[g]), f64(v2[g])
        _, _, _, ref = O.ffn_fwd(fmt, x[r], W13, W2)
        # one bf16 rounding of the result; a 4-bit rounding of h that fell the other way is rare
        assert np.linalg.norm(y[r] - ref) <= 2.0 ** -7 * np.linalg.norm(ref)
        gu = O.checkpoint_values(host(ck)[r], host(cs)[r])
        ref, _ = O.ffn_bwd(dO[r], gu, W13, W2)
        ref += dl[tok[r], g][:, None] * Wr[g]
        assert np.linalg.norm(dX[r] - ref) <= 2.0 ** -7 * np.linalg.norm(ref)
    # the same step captured in a graph, and replayed twice
    first = [t.clone() for t in (out, dx, ck, cs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for t in (out, dx):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    rows = np.concatenate([np.arange(o, o + c) for o, c in zip(off, counts)])
    assert torch.equal(out, first[0]) and torch.equal(dx, first[1])
    assert torch.equal(ck[rows], first[2][rows]) and torch.equal(cs[rows], first[3][rows])


def test_shared_experts_and_sigmoid_router_rows():
    """Groups past E are shared experts: one row per token, no router term."""
    shape = MoEShape("fp4_shared", T=70, H=128, E=4, k=2, F=128, n_shared=1, score_fn=SIGMOID)
    inp = {k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in make_inputs(shape, seed=0).items()}
    cfg = B.config(shape)
    bufs = B.alloc_buffers(cfg, DEV)
    f, sc = bufs.fwd, bufs.scratch
    B.moe_route(cfg, inp["x"], inp["W_r"], inp["bias"], f["logits"], f["idx"], f["w"], sc)
    B.moe_permute(cfg, inp["x"], f["idx"], f["counts"], f["offsets"], f["row_of"], f["token_of"],
                  f["sel_offsets"], f["sel_tokens"], f["x_perm"], sc)
    q13, q2 = B.alloc_fp4(0, 5, 256, 128), B.alloc_fp4(0, 5, 128, 128)
    v13, v2 = torch.empty_like(inp["W13"]), torch.empty_like(inp["W2"])
    B.moe_fp4_quantize(inp["W13"], q13, scale_log2=-9, values=v13)
    B.moe_fp4_quantize(inp["W2"], q2, scale_log2=-9, values=v2)
    sf = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).fwd_scratch_bytes)
    B.moe_fp4_ffn_fwd(cfg, B.fp4_experts(q13, q2), f["x_perm"], f["counts"], f["offsets"], None,
                      None, f["y_perm"], sf)
    assert B.moe_last_device_status(sf) == 0
    off = int(f["offsets"][4])
    assert int(f["counts"][4]) == 70
    x, y = f64(f["x_perm"])[off:off + 70], f64(f["y_perm"])[off:off + 70]
    _, _, _, ref = O.ffn_fwd(0, x, f64(v13[4]), f64(v2[4]))
    assert np.linalg.norm(y - ref) <= 2.0 ** -7 * np.linalg.norm(ref)


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_class_serves_and_trains(fmt):
    """The layer of the command: a serving step against the bf16 layer (4-bit weights and rows
    are about 0.1 away each; a wrong path would be 1 or more), and its gradients finite."""
    from routing_dispatch_expert_router_gb300 import fp4_layer as L
    shape = TINY.with_(T=70)
    inp = {k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in make_inputs(shape, seed=3).items()}
    layer = L.Fp4Layer(shape, inp, fmt, training=True)
    out = layer.forward(inp["x"])
    ref = L._bf16_output(shape, inp)
    dx, dW_r = layer.backward(inp["x"], inp["dY"])
    layer.check()
    a, b = f64(out), f64(ref)
    assert np.linalg.norm(a - b) < 0.4 * np.linalg.norm(b)
    assert np.isfinite(f64(dx)).all() and f64(dx).any() and np.isfinite(f64(dW_r)).all()
