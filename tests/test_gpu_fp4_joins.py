"""Products of 4-bit experts whose k-blocks are shared over the SMs: tiles cut into parts
that are joined through scratch. Every case asserts that it is one (the kernel's rule,
restated here), so that a change of the rule cannot leave these paths without a test.
"""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from oracle import fp4_oracle as O

pytestmark = pytest.mark.gpu

H_ = pytest.importorskip("harness")
T4 = pytest.importorskip("test_gpu_fp4")
FORMATS = T4.FORMATS
DEV = "cuda"
f64, host = T4.f64, T4.host


def cuts(counts, n_tiles, K):
    """share_evenly of grouped_gemm_fp4.cu: whether tiles are cut (n_tiles: column tiles)."""
    grid = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum(-(-c // 128) for c in counts) * n_tiles
    nk, most = -(-K // 256), max(counts)
    slot_rows = min(128, -(-most // 32) * 32)
    if 2 * grid * slot_rows * 256 > (39 << 19) // 4 or tiles * 8 > 8192:
        return False
    m = tiles % grid
    whole = nk * (tiles // grid * 100 + (max(65, 100 * m // grid) if m else 0))
    return whole > tiles * nk * 100 // grid + 200 + most * 80


# counts, N, K: one row and several, odd numbers of them, empty groups, columns that end
# inside a tile, K that ends inside a k-block; up to 64 rows an expert (two 32-row boxes)
PRODUCTS = [([1], 256, 2048), ([7], 520, 7168), ([1, 0, 3, 2], 264, 4128), ([16, 9], 512, 14336),
            ([33, 1, 0, 20], 136, 14336), ([0, 40, 33], 256, 14368), ([1] * 9, 1000, 2080)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,N,K", PRODUCTS)
def test_cut_product_matches_oracle_again_and_again(fmt, counts, N, K):
    """The oracle's numbers, and the same bits on ten more passes over the same counters."""
    assert cuts(counts, -(-N // 256), K)
    rng = np.random.default_rng(N + K)
    off, rows, cnt, offs = T4.segments(counts)
    R = int(off[-1]) + 5
    x = T4.rows_of(rng, 1, R, K)
    xq = B.alloc_fp4(fmt, 1, R, K)
    xq.scales.fill_(0xFF)
    xq.codes.fill_(0x77)
    B.moe_fp4_quantize(x, xq, counts=cnt, offsets=offs)
    wq, wv = T4.weights(fmt, rng, len(counts), N, K)
    alpha = torch.tensor(0.5 + rng.random(len(counts)), dtype=torch.float32, device=DEV)
    sc = B.alloc_fp4_scratch(B.moe_fp4_query_sizes(None, fmt).gemm_scratch_bytes)
    out = torch.full((R, N), 7.0, device=DEV, dtype=torch.bfloat16)
    B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, alpha, out, sc)
    got, xv = f64(out), O.real(fmt, f64(x)[0])
    ref, mag = np.full((R, N), 7.0), np.zeros((R, N))
    for g, c in enumerate(counts):
        r = slice(off[g], off[g] + c)
        ref[r] = xv[r] @ wv[g].T * float(alpha[g])
        mag[r] = np.abs(xv[r]) @ np.abs(wv[g]).T * float(alpha[g])
    # half a step of bf16, and an fp32 sum of K exact products
    H_.assert_close("out", got, ref, atol=0, rtol=1,
                    scale=2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag)
    for _ in range(10):
        again = torch.full_like(out, 7.0)
        B.moe_fp4_grouped_gemm(xq, wq, cnt, offs, alpha, again, sc)
        assert torch.equal(out, again)
    assert B.moe_last_device_status(sc) == 0


# counts, H, F: the gate-up product is cut (h quantised and the checkpoint written row by
# row by the joining warp); the last one's rows an expert take the 128-row form
FFNS = [([1], 2048, 128), ([1, 0, 1], 4096, 384), ([9, 5], 8192, 256), ([33, 0, 2], 14336, 128),
        ([33, 32, 1], 14336, 128)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,H,F", FFNS)
def test_cut_ffn_and_checkpoint_match_oracle(fmt, counts, H, F):
    assert cuts(counts, F // 128, H)
    T4.test_ffn_forward_and_checkpoint_match_oracle(fmt, counts, H, F)


@pytest.mark.parametrize("fmt", FORMATS)
def test_both_products_cut_thirty_passes_equal(fmt):
    """Both products of an FFN cut, over and over on one scratch, with a whole-tile call of
    other sizes in between: the same bits, checkpoint included."""
    counts, H, F = [1, 1], 4096, 4096
    assert cuts(counts, F // 128, H) and cuts(counts, H // 256, F)
    s = T4.run_ffn(fmt, counts, H, F)
    rows = s["rows"]
    y, ck, cs = s["y"][rows].clone(), s["ck"][rows].clone(), s["cs"][rows].clone()
    for i in range(30):
        s["y"].fill_(7.0)
        s["ck"].fill_(0x11)
        s["cs"].fill_(0x11)
        B.moe_fp4_ffn_fwd(s["cfg"], s["ex"][0], s["x"], s["cnt"], s["offs"], s["ck"], s["cs"],
                          s["y"], s["sc"])
        assert torch.equal(y, s["y"][rows])
        assert torch.equal(ck, s["ck"][rows]) and torch.equal(cs, s["cs"][rows])
    assert B.moe_last_device_status(s["sc"]) == 0


def test_row_alone_and_among_others():
    """A token's row alone (both products cut) and among 200 (whole tiles): y within two bf16
    steps and the order of fp32 sums, where no 4-bit rounding of h moved."""
    H, F = 4096, 2048
    assert cuts([1], F // 128, H) and cuts([1], H // 256, F)
    assert not cuts([200], F // 128, H)
    s = T4.run_ffn(B.MOE_FP4_NV, [200], H, F)
    cnt = torch.tensor([1], dtype=torch.int32, device=DEV)
    y = torch.zeros_like(s["y"])
    B.moe_fp4_ffn_fwd(s["cfg"], s["ex"][0], s["x"], cnt, s["offs"], None, None, y, s["sc"])
    _, _, _, h4, slack = T4.h_interval(B.MOE_FP4_NV, f64(s["x"])[:1], s["ex"][5][0])
    W2 = np.abs(s["ex"][6][0])
    bound = 2.0 ** -7 * np.abs(f64(s["y"])[:1]) + 2 * (slack + F * 2.0 ** -23 * np.abs(h4)) @ W2.T
    H_.assert_close("row", f64(y)[:1], f64(s["y"])[:1], atol=0, rtol=1, scale=bound)
