"""Weights whose scales are at the ends of their formats, through the backward's own
conversion (codes times scale as bf16 values in shared memory)."""
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


def weights_of_bytes(fmt, rng, groups, rows, K, lo, hi):
    """Every code, with scale bytes of [lo, hi): the tensor and its values."""
    codes = rng.integers(0, 16, (groups, rows, K), dtype=np.uint8)
    byte = rng.integers(lo, hi, (groups, rows, K // O.BLOCK[fmt]), dtype=np.uint8)
    atoms = O.to_atoms(fmt, byte, K)
    q = B.Fp4Tensor(fmt, K, torch.from_numpy(O.pack(codes)).to(DEV), torch.from_numpy(atoms).to(DEV))
    return q, O.values(fmt, codes, byte)


# E4M3: subnormal scales (bytes 0..7, zero among them), all of them, the largest;
# powers of two: the smallest bf16 can multiply exactly, and a wide middle
BYTES = [(B.MOE_FP4_NV, 0, 8, 10), (B.MOE_FP4_NV, 0, 127, 0), (B.MOE_FP4_NV, 120, 127, -12),
         (B.MOE_FP4_MX, 64, 68, 62), (B.MOE_FP4_MX, 120, 135, 0)]


@pytest.mark.parametrize("fmt,lo,hi,up", BYTES)
def test_backward_at_the_ends_of_the_scales(fmt, lo, hi, up):
    """up: dO's size as a power of two, so that dX is of ordinary size."""
    rng = np.random.default_rng(lo + hi)
    H, F, counts = 256, 128, [70, 130]
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("w", T=len(rows), H=H, E=2, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    W13q, W13 = weights_of_bytes(fmt, rng, 2, 2 * F, H, lo, hi)
    W2q, W2 = weights_of_bytes(fmt, rng, 2, H, F, lo, hi)
    ex = B.fp4_experts(W13q, W2q)
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[rows] = T4.bf(np.ldexp(rng.standard_normal((len(rows), H)), up))
    codes = rng.integers(0, 120, (R, 2 * F), dtype=np.uint8)
    byte = np.full((R, 2 * F // 32), 118, np.uint8)
    ck, cs = torch.from_numpy(codes).to(DEV), torch.from_numpy(byte).to(DEV)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex, dO, ck, cs, cnt, offs, None, None, None, dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got, dOv = f64(dX), f64(dO)
    for g, c in enumerate(counts):
        r = slice(off[g], off[g] + c)
        gu = O.checkpoint_values(codes[r], byte[r])
        ref, dgu = O.ffn_bwd(dOv[r], gu, W13[g], W2[g])
        _, err = O.ffn_bwd(np.abs(dOv[r]), gu, np.abs(W13[g]), np.abs(W2[g]))
        d_err = 2.0 ** -8 * np.abs(dgu) + (H * 2.0 ** -23 + 2.0 ** -18) * np.abs(err)
        mag = np.abs(dgu) @ np.abs(W13[g])
        H_.assert_close(f"dX of {g}", got[r], ref, atol=0, rtol=1,
                        scale=2.0 ** -8 * np.abs(ref) + d_err @ np.abs(W13[g])
                        + 2 * F * 2.0 ** -23 * mag)


def test_each_weight_exact():
    """One-hot rows of dO through a W2 of the unit matrix, a gate of 128 (its sigmoid is 1 in
    fp32) and an up of 0 give dX = 128 times a row of W13: every code at every E4M3 scale,
    exact in bf16."""
    H, F = 128, 128
    # W13's up half: column h has code h % 16, row f the scale byte f (0 .. 126)
    codes13 = np.zeros((1, 2 * F, H), np.uint8)
    byte13 = np.zeros((1, 2 * F, H // 16), np.uint8)
    codes13[0, F:] = np.arange(H)[None] % 16
    byte13[0, F:] = np.arange(F)[:, None].clip(0, 126)
    W13 = O.values(O.NV, codes13, byte13)[0]
    codes2 = np.zeros((1, H, F), np.uint8)
    codes2[0] = np.eye(H, dtype=np.uint8) * 2              # 1.0 on the diagonal
    byte2 = np.full((1, H, F // 16), 0x38, np.uint8)       # scale 1
    q = lambda c, b, K: B.Fp4Tensor(O.NV, K, torch.from_numpy(O.pack(c)).to(DEV),  # noqa: E731
                                    torch.from_numpy(O.to_atoms(O.NV, b, K)).to(DEV))
    W13q, W2q = q(codes13, byte13, H), q(codes2, byte2, F)
    ex = B.fp4_experts(W13q, W2q)
    T = 128
    cfg = B.config(MoEShape("e", T=T, H=H, E=1, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[:T] = torch.eye(T, H, device=DEV)
    ck = torch.zeros(R, 2 * F, dtype=torch.uint8, device=DEV)
    ck[:, :F] = 0x70                                       # g = 128: s(g) is 1 in fp32; u = 0
    cs = torch.full((R, 2 * F // 32), 127, dtype=torch.uint8, device=DEV)
    dX = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)  # noqa: E731
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex, dO, ck, cs, i32(T), i32(0), None, None, None, dX, sc)
    # row f of dX: 128 times row f of W13's up half
    H_.assert_equal("dX", f64(dX)[:T], 128.0 * W13[F:])
