"""The router's term of the 4-bit experts' backward: which rows and experts get it."""
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


def test_padding_rows_are_zero_whatever_the_router_holds():
    """Rows that fill a segment's last 128-row block are zeros, an infinite or NaN router
    weight notwithstanding (their dlogits are none, not zero times that weight)."""
    rng = np.random.default_rng(5)
    H, F, counts = 128, 128, [5, 130]
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("p", T=len(rows), H=H, E=2, k=1, F=F))
    R = int(B.moe_query_sizes(cfg).rows_max)
    ex = T4.experts_of(B.MOE_FP4_NV, rng, 2, H, F)
    dO = torch.randn(R, H, device=DEV).bfloat16()
    ck = torch.full((R, 2 * F), 0x38, dtype=torch.uint8, device=DEV)
    cs = torch.full((R, 2 * F // 32), 120, dtype=torch.uint8, device=DEV)
    tok = np.full(R, -1, np.int32)
    tok[rows] = np.arange(len(rows))
    W_r = torch.randn(2, H, device=DEV)
    W_r[0, 3], W_r[1, 64], W_r[1, 65] = float("inf"), float("nan"), float("-inf")
    dl = torch.randn(len(rows), 2, device=DEV)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, 0).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex[0], dO, ck, cs, cnt, offs, torch.from_numpy(tok).to(DEV), dl, W_r,
                      dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got = f64(dX)
    for g, c in enumerate(counts):
        pad = got[off[g] + c:off[g + 1]]
        assert len(pad) and (pad == 0).all()
        live = got[off[g]:off[g] + c]
        bad = ~np.isfinite(f64(W_r[g]))
        assert not np.isfinite(live[:, bad]).any() and np.isfinite(live[:, ~bad]).all()


@pytest.mark.parametrize("fmt", T4.FORMATS)
@pytest.mark.parametrize("n_shared", [1, 2])
def test_backward_of_shared_experts_has_no_router_term(fmt, n_shared):
    """Groups past E: their dX is the FFN's alone, the routed groups' has dlogits W_r added.
    dlogits and W_r hold E experts and end where memory of other values begins."""
    rng = np.random.default_rng(17)
    E, H, F, T = 3, 256, 128, 150
    counts = [40, 0, 129] + [T] * n_shared
    G = E + n_shared
    off, rows, cnt, offs = T4.segments(counts)
    cfg = B.config(MoEShape("s", T=T, H=H, E=E, k=2, F=F, n_shared=n_shared))
    R = int(B.moe_query_sizes(cfg).rows_max)
    assert R >= off[-1]
    ex = T4.experts_of(fmt, rng, G, H, F)
    dO = torch.zeros(R, H, device=DEV, dtype=torch.bfloat16)
    dO[rows] = T4.rows_of(rng, len(rows), H, spread=False)
    codes = rng.integers(0, 120, (R, 2 * F), dtype=np.uint8) | \
        (rng.integers(0, 2, (R, 2 * F), dtype=np.uint8) << 7)
    byte = np.full((R, 2 * F // 32), 119, np.uint8)
    tok = np.full(R, -1, np.int32)
    for g, c in enumerate(counts):
        tok[off[g]:off[g] + c] = rng.permutation(T)[:c]
    # one buffer each; what follows dlogits and W_r is huge, so a term from there shows
    dl = np.full((T + 8, E), 1e30, np.float32)
    Wr = np.full((E + n_shared, H), 1e30, np.float32)
    dl[:T], Wr[:E] = rng.standard_normal((T, E)), rng.standard_normal((E, H))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    dlt, wrt = dev(dl), dev(Wr)
    dX = torch.full((R, H), 7.0, device=DEV, dtype=torch.bfloat16)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(cfg, fmt).bwd_scratch_bytes)
    B.moe_fp4_ffn_bwd(cfg, ex[0], dO, dev(codes), dev(byte), cnt, offs, dev(tok), dlt[:T], wrt[:E],
                      dX, sc)
    assert B.moe_last_device_status(sc) == 0
    got, dOv = f64(dX), f64(dO)
    for g, c in enumerate(counts):
        r = slice(off[g], off[g] + c)
        gu = O.checkpoint_values(codes[r], byte[r])
        W13, W2 = ex[5][g], ex[6][g]
        ref, dgu = O.ffn_bwd(dOv[r], gu, W13, W2)
        _, err = O.ffn_bwd(np.abs(dOv[r]), gu, np.abs(W13), np.abs(W2))
        d_err = 2.0 ** -8 * np.abs(dgu) + (H * 2.0 ** -23 + 2.0 ** -18) * np.abs(err)
        if g < E:
            ref = ref + dl[tok[r], g][:, None] * Wr[g]
        mag = np.abs(dgu) @ np.abs(W13)
        H_.assert_close(f"dX of {g}", got[r], ref, atol=0, rtol=1,
                        scale=2.0 ** -8 * np.abs(ref) + d_err @ np.abs(W13) + 2 * F * 2.0 ** -23 * mag)
