"""Products with weights in 4-bit integers against the definition in 64 bits.

Tolerance of an element: its own rounding, 2^-8 |y|, and the fp32 sums'. The kernel sums (128 + q) x
and x of a group and subtracts (128 + z) times the latter; a group's sums are at most 24 additions
deep (a product of 16 terms, eight of those, two halves), each off by 2^-23 of its size at most (the
tensor cores cut instead of rounding), so a group is off by 48 2^-23 (128 + 127) s sum |x|, and the
groups' sum by one 2^-24 of their magnitudes each.
"""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def weights(G, N, K, group, zeros, seed=0, scale=0.01):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (G, N, K), generator=g, dtype=U8)
    codes = (q[:, :, 0::2] | (q[:, :, 1::2] << 4)).cuda()
    scales = (scale * (0.5 + torch.rand(G, K // group, N, generator=g))).to(BF).cuda()
    z = torch.randint(0, 16, scales.shape, generator=g, dtype=U8).cuda() if zeros else None
    return B.Int4Tensor(codes.contiguous(), scales, z), q.cuda()


def real(W, q, e):
    """Expert e's weights and their scales, both [N, K] in 64 bits."""
    group = q.shape[2] // W.scales.shape[1]
    s = W.scales[e].double().T.repeat_interleave(group, 1)
    z = W.zeros[e].double().T.repeat_interleave(group, 1) if W.zeros is not None else 8.0
    return (q[e].double() - z) * s, s


def place(counts, gap=0, order=None):
    """Offsets of segments one after the other (in `order`), with a gap between them."""
    off, at = [0] * len(counts), gap
    for e in order or range(len(counts)):
        off[e] = at
        at += counts[e] + gap
    return off, at


def dev(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def reference(W, q, x, e, swiglu):
    w, s = real(W, q, e)
    x = x.double()
    y = x @ w.T
    G = W.scales.shape[1]
    tol = 48 * 2.0 ** -23 * 255 * (x.abs() @ s.T) + G * 2.0 ** -24 * (x.abs() @ w.abs().T)
    if swiglu:
        a, b = y.chunk(2, 1)
        ta, tb = tol.chunk(2, 1)
        sa = a * torch.sigmoid(a)
        y = sa * b                                      # (|silu'| <= 1.1; its fp32 form a few ulp)
        tol = 1.1 * ta * b.abs() + (sa.abs() + 1.1 * ta) * tb + 2.0 ** -20 * y.abs()
    return y, tol + 2.0 ** -8 * y.abs()


def check(W, q, x, counts, off, out, swiglu=False, skip=()):
    err = norm = 0.0
    for e, n in enumerate(counts):
        if n == 0 or e in skip:
            continue
        y, tol = reference(W, q, x[off[e]:off[e] + n], e, swiglu)
        d = (out[off[e]:off[e] + n].double() - y).abs()
        assert bool((d <= tol).all()), (e, (d / tol).max().item())
        err, norm = err + d.square().sum().item(), norm + y.square().sum().item()
    # roundings of 2^-8 at most are 2^-8 of the norm at most; the sums' share is far below
    assert err <= 2.0 ** -16 * norm


CASES = [
    # counts, N, K, group, zeros, swiglu
    ([1], 16, 32, 32, False, False),
    ([2, 0, 1], 32, 64, 64, True, True),
    ([1, 8, 0, 9], 272, 288, 32, True, False),
    ([16, 17, 0, 33, 5], 1008, 1504, 32, True, False),
    ([3, 1], 480, 640, 128, False, True),
    ([0, 7, 0, 0, 2, 0], 1120, 1280, 64, False, True),
    ([1, 0, 1], 28672, 512, 128, False, True),
    ([5], 16, 14336, 128, True, False),                 # one unit, many CTAs
    ([70], 528, 4096, 128, True, False),                # five passes over the tokens
    ([0] * 200 + [3] + [0] * 58 + [1], 64, 128, 128, True, False),
]


@pytest.mark.parametrize("counts,N,K,group,zeros,swiglu", CASES)
def test_product(counts, N, K, group, zeros, swiglu):
    G = len(counts)
    W, q = weights(G, N, K, group, zeros)
    order = sorted(range(G), key=lambda e: (7 * e) % G)
    off, R = place(counts, gap=3, order=order)
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(R, K + 24, generator=g).to(BF).cuda()
    x = wide[:, 8:8 + K]
    cols = N // 2 if swiglu else N
    big = torch.full((R, cols + 16), 5.0, dtype=BF, device="cuda")
    out = big[:, 8:8 + cols]
    sc = B.alloc_product_scratch()
    B.moe_int4_grouped_gemm(x, W, dev(counts), dev(off), out, sc, swiglu=swiglu)
    check(W, q, x, counts, off, out, swiglu)
    mine = torch.zeros(R, dtype=torch.bool)
    for e, n in enumerate(counts):
        mine[off[e]:off[e] + n] = True
    assert bool((big[~mine] == 5).all()) and bool((big[:, :8] == 5).all()) and bool((big[:, 8 + cols:] == 5).all())
    # again on the same scratch: the same bits, and the counters left as they were
    first = out.clone()
    for _ in range(3):
        out.zero_()
        B.moe_int4_grouped_gemm(x, W, dev(counts), dev(off), out, sc, swiglu=swiglu)
        assert torch.equal(out[mine], first[mine])
    assert B.moe_last_device_status(sc) == 0 and bool((sc[:4096] == 0).all())


def test_one_group_of_all_rows_and_no_rows():
    W, q = weights(1, 96, 256, 64, True)
    x = torch.randn(11, 256, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    out, sc = torch.empty(11, 96, dtype=BF, device="cuda"), B.alloc_product_scratch()
    B.moe_int4_grouped_gemm(x, W, None, None, out, sc)
    check(W, q, x, [11], [0], out)
    B.moe_int4_grouped_gemm(x[:0], W, None, None, out[:0], sc)
    keep = out.clone()
    B.moe_int4_grouped_gemm(x, W, dev([0]), dev([4]), out, sc)
    assert torch.equal(out, keep)


def test_other_rows_values_stay_out():
    """NaN and infinities in rows between and beside the segments, and in a token of a segment."""
    counts, off, R, K = [3, 2], [2, 7], 12, 256
    W, q = weights(2, 64, K, 128, False)
    x = torch.randn(R, K, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    sc = B.alloc_product_scratch()
    clean = torch.zeros(R, 64, dtype=BF, device="cuda")
    B.moe_int4_grouped_gemm(x, W, dev(counts), dev(off), clean, sc)
    for r in (0, 1, 5, 6, 9, 10, 11):
        x[r] = float("nan") if r % 2 else float("inf")
    x[3, 7] = float("nan")
    out = torch.zeros_like(clean)
    B.moe_int4_grouped_gemm(x, W, dev(counts), dev(off), out, sc)
    assert bool(out[3].isnan().all())
    for r in (2, 4, 7, 8):
        assert torch.equal(out[r], clean[r])


def test_bad_segments_are_left_out():
    counts, off = [4, 3, 5, 2], [0, 30, -1, 6]
    W, q = weights(4, 64, 128, 32, False)
    x = torch.randn(32, 128, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    out, sc = torch.full((32, 64), 5.0, dtype=BF, device="cuda"), B.alloc_product_scratch()
    B.moe_int4_grouped_gemm(x, W, dev(counts), dev(off), out, sc)
    assert B.moe_last_device_status(sc) == 6
    check(W, q, x, counts, off, out, skip=(1, 2))
    assert bool((out[8:] == 5).all()) and bool((out[4:6] == 5).all())
    B.moe_clear_device_status(sc)
    B.moe_int4_grouped_gemm(x, W, dev([4, -2, 0, 2]), dev([0, 9, 40, 6]), out, sc)
    assert B.moe_last_device_status(sc) == 6


def test_rows_behind_2_to_the_31_elements():
    R, K, N = 600_000, 4096, 4096
    W, q = weights(2, N, K, 128, False)
    x = torch.zeros(R, K, dtype=BF, device="cuda")
    x[-9:] = torch.randn(9, K, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    out = torch.zeros(R, N, dtype=BF, device="cuda")
    B.moe_int4_grouped_gemm(x, W, dev([4, 5]), dev([R - 9, R - 5]), out, B.alloc_product_scratch())
    check(W, q, x, [4, 5], [R - 9, R - 5], out)
    assert bool((out[:-9] == 0).all())


@pytest.mark.parametrize("G,N,K,group,zeros", [(1, 16, 32, 32, True), (3, 80, 320, 64, False), (2, 1008, 1536, 128, True)])
def test_dequantised(G, N, K, group, zeros):
    W, q = weights(G, N, K, group, zeros)
    out = torch.empty(G, N, K, dtype=BF, device="cuda")
    B.moe_int4_dequantize(W, out)
    for e in range(G):
        assert torch.equal(out[e], real(W, q, e)[0].float().to(BF))


def test_zero_points_over_their_range():
    """0..127, and scales of both signs, huge and zero."""
    G, N, K = 1, 128, 64
    W, q = weights(G, N, K, 32, True)
    W.zeros.copy_(torch.arange(256, dtype=U8).view(1, 2, 128).cuda() & 127)
    W.scales[0, 0, :4] = torch.tensor([0.0, -1.0, 2.0 ** 60, -2.0 ** -60], dtype=BF)
    x = torch.randn(4, K, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    out = torch.empty(4, N, dtype=BF, device="cuda")
    B.moe_int4_grouped_gemm(x, W, None, None, out, B.alloc_product_scratch())
    w, s = real(W, q, 0)
    y, xa = x.double() @ w.T, x.double().abs()
    tol = 2.0 ** -8 * y.abs() + 48 * 2.0 ** -23 * 255 * (xa @ s.abs().T) + 2.0 ** -23 * (xa @ w.abs().T)
    assert bool(((out.double() - y).abs() <= tol).all())


def test_captured_and_replayed():
    """Gate-up and down products of a step, both on one scratch, on a side stream and replayed."""
    counts, off, R = [2, 0, 1, 3], [0, 4, 4, 9], 16
    W1, q1 = weights(4, 512, 384, 128, True, 1)
    W2, q2 = weights(4, 384, 256, 64, False, 2)
    x = torch.randn(R, 384, generator=torch.Generator().manual_seed(7)).to(BF).cuda()
    h, y = torch.zeros(R, 256, dtype=BF, device="cuda"), torch.zeros(R, 384, dtype=BF, device="cuda")
    sc, c, o = B.alloc_product_scratch(), dev(counts), dev(off)

    def step():
        B.moe_int4_grouped_gemm(x, W1, c, o, h, sc, swiglu=True)
        B.moe_int4_grouped_gemm(h, W2, c, o, y, sc)

    step()
    check(W1, q1, x, counts, off, h, True)
    check(W2, q2, h, counts, off, y)
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    y.zero_(), h.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # other counts on the device: the same graph
    c.copy_(dev([0, 3, 1, 0]))
    o.copy_(dev([0, 4, 8, 9]))
    graph.replay()
    torch.cuda.synchronize()
    check(W2, q2, h, [0, 3, 1, 0], [0, 4, 8, 9], y)
