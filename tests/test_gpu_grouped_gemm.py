"""Grouped products of ragged rows, forward, data gradient and weight gradient, against the
definition in 64 bits.

Tolerance of an element: its own rounding, 2^-8 of the value, and the fp32 sums': products of
bf16 numbers are exact, n of them are added in n / 16 steps of 16 on the tensor cores, each step
off by 2^-23 of what it holds at most (they cut instead of rounding): (n / 16 + 16) 2^-23 of the sum
of the magnitudes, the 16 for the sums inside a step and the parts' joining.
"""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def randn(*shape, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF).cuda()


def dev(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def place(counts, gap, order):
    off, at = [0] * len(counts), gap
    for e in order:
        off[e] = at
        at += counts[e] + gap
    return off, at


def within(got, ref, size, n, extra=None):
    """size: the sum of the magnitudes of the n terms."""
    tol = 2.0 ** -8 * ref.abs() + (n / 16 + 16) * 2.0 ** -23 * size
    d = (got.double() - ref).abs()
    assert bool((d <= tol).all()), (d / tol).max().item()
    assert d.square().sum() <= 2.0 ** -16 * ref.square().sum()


def check_rows(got, a, w, counts, off, add=None, dgrad=False):
    for e, n in enumerate(counts):
        if not n:
            continue
        r = slice(off[e], off[e] + n)
        m = w[e].double() if dgrad else w[e].double().T
        ref, size = a[r].double() @ m, a[r].double().abs() @ m.abs()
        if add is not None:
            ref, size = ref + add[r].double(), size + add[r].double().abs()
        within(got[r], ref, size, m.shape[0])


def check_wgrad(dw, dy, x, counts, off):
    for e, n in enumerate(counts):
        r = slice(off[e], off[e] + n)
        a, b = dy[r].double(), x[r].double()
        if n == 0:
            assert bool((dw[e] == 0).all())
        else:
            within(dw[e], a.T @ b, a.abs().T @ b.abs(), n)


CASES = [
    # counts, N, K
    ([1], 8, 8),
    ([3, 0, 1, 2], 24, 40),
    ([1, 128, 0, 129, 63, 64, 65], 136, 72),
    ([300, 5, 0, 517], 520, 16),
    ([40, 41], 16, 1032),
    ([1000, 0, 24], 264, 2040),
    ([2500], 1000, 328),
    ([700, 650, 130, 20], 4096, 264),
    ([0, 0], 64, 64),
    ([0] * 250 + [70, 1] + [0] * 7 + [30], 72, 128),
    # short reductions
    ([700, 0, 33, 5, 128], 1000, 48),
    ([50, 2000, 1], 56, 328),
    ([129, 16, 15], 64, 64),
    ([0, 1], 24, 30000),
    # few outputs of many rows, forward and data gradient
    ([3000, 0, 3, 1160], 8, 4104),
    ([17, 2257, 256, 1, 2900], 4104, 8),
    ([14600], 1032, 16),
    ([0, 9000, 90, 6000], 16, 1096),
    # few tiles, a long reduction: several pairs share a tile
    ([17, 0, 30], 200, 4104),
    ([420], 4104, 120),
    ([3363], 456, 184),
    ([2, 4000, 0, 640], 264, 40),
]


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("add", [False, True])
def test_products(counts, N, K, add):
    G = len(counts)
    order = sorted(range(G), key=lambda e: (5 * e + 3) % G)
    off, R = place(counts, 1, order)
    w = randn(G, N, K, seed=1, scale=0.1)
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    mine = torch.zeros(R, dtype=torch.bool)
    for e, n in enumerate(counts):
        mine[off[e]:off[e] + n] = True
    for dgrad in (False, True):
        ka, kc = (N, K) if dgrad else (K, N)
        a = randn(R, ka + 16, seed=2)[:, 8:8 + ka]
        more = randn(R, kc, seed=3) if add else None
        wide = torch.full((R, kc + 16), 5.0, dtype=BF, device="cuda")
        out = wide[:, 8:8 + kc]

        def call(**kw):
            if dgrad:
                B.moe_grouped_gemm_dgrad(a, w, c, o, out, sc, add=more, **kw)
            else:
                B.moe_grouped_gemm(a, w, c, o, out, sc, add=more, **kw)

        call()
        check_rows(out, a, w, counts, off, more, dgrad)
        assert bool((wide[~mine] == 5).all())
        assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + kc:] == 5).all())
        first = out.clone()
        call()
        assert torch.equal(out, first)
        if not dgrad:                                      # the kernel for few rows
            call(expected_rows=1)
            check_rows(out, a, w, counts, off, more)
            assert bool((wide[~mine] == 5).all()) and bool((wide[:, 8 + kc:] == 5).all())
        if add:                                            # in place of what is added
            out.copy_(more)
            more = out
            call()
            assert torch.equal(out[mine], first[mine])
    assert B.moe_last_device_status(sc) == 0 and bool((sc[:8192] == 0).all())


@pytest.mark.parametrize("counts,N,K", CASES)
def test_weight_gradient(counts, N, K):
    G = len(counts)
    off, R = place(counts, 0, range(G))
    R += 3
    dy, x = randn(R, N + 8, seed=4)[:, :N], randn(R, K + 8, seed=5)[:, 8:]
    sc = B.alloc_product_scratch()
    out = torch.full((G * N * K + 64,), 5.0, dtype=BF, device="cuda")
    dw = out[:G * N * K].view(G, N, K)
    B.moe_grouped_gemm_wgrad(dy, x, dev(counts), dev(off), dw, sc)
    check_wgrad(dw, dy, x, counts, off)
    assert bool((out[G * N * K:] == 5).all()) and bool((sc[:8192] == 0).all())
    first = dw.clone()
    B.moe_grouped_gemm_wgrad(dy, x, dev(counts), dev(off), dw, sc)
    assert torch.equal(dw, first)


def test_gradients_against_differences():
    """sum(dy * f(x, w)) moved along one direction at a time, in 64 bits."""
    counts, off, R, N, K = [3, 2], [0, 3], 5, 16, 24
    x, w, dy = randn(R, K, seed=6), randn(2, N, K, seed=7), randn(R, N, seed=8)
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    B.moe_grouped_gemm_dgrad(dy, w, c, o, dx, sc)
    B.moe_grouped_gemm_wgrad(dy, x, c, o, dw, sc)

    def f(xx, ww):
        return sum((dy[off[e]:off[e] + n].double() * (xx[off[e]:off[e] + n] @ ww[e].T)).sum()
                   for e, n in enumerate(counts))

    base, d = f(x.double(), w.double()), 1e-3
    for got, t, both in ((dx, x, False), (dw, w, True)):
        flat = got.double().reshape(-1)
        for i in range(0, flat.numel(), 7):
            moved = t.double().clone()
            moved.view(-1)[i] += d
            slope = (f(x.double(), moved) if both else f(moved, w.double())) - base
            assert abs(flat[i].item() - slope.item() / d) <= 2.0 ** -8 * abs(slope.item() / d) + 1e-6


@pytest.mark.parametrize("N,K", [(136, 200), (1024, 512)])
def test_other_rows_values_stay_out(N, K):
    """NaN and infinities in the rows of other groups and of none."""
    counts, off, R = [70, 130, 65], [1, 71, 202], 270
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    x, dy, w = randn(R, K, seed=9), randn(R, N, seed=10), randn(3, N, K, seed=11)
    want = [torch.zeros(R, N, dtype=BF, device="cuda"), torch.zeros(R, K, dtype=BF, device="cuda"),
            torch.empty_like(w)]
    got = [t.clone() for t in want]

    def run(out):
        B.moe_grouped_gemm(x, w, c, o, out[0], sc)
        B.moe_grouped_gemm_dgrad(dy, w, c, o, out[1], sc)
        B.moe_grouped_gemm_wgrad(dy, x, c, o, out[2], sc)

    run(want)
    for t in (x, dy):
        t[0], t[201], t[267:] = float("nan"), float("inf"), float("nan")
        t[71:201] = float("nan")                           # the whole second group
    w[1] = float("inf")
    run(got)
    for e in (0, 2):
        r = slice(off[e], off[e] + counts[e])
        assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][r], want[1][r])
        assert torch.equal(got[2][e], want[2][e])
    assert bool(got[2][1].isnan().all())
    few = torch.zeros_like(want[0])
    B.moe_grouped_gemm(x, w, c, o, few, sc, expected_rows=1)
    check_rows(few, x, w, [70, 0, 65], off)


@pytest.mark.parametrize("N,K,times", [(1000, 24, 1), (40, 1000, 1), (16, 4104, 17), (4104, 8, 17)])
def test_other_values_stay_out_of_short_and_narrow_products(N, K, times):
    """The same where the reduction is short or the outputs few, and NaN behind every row's end."""
    counts = [70 * times, 130 * times, 65 * times]
    off, R = [1, 1 + counts[0], 2 + counts[0] + counts[1]], 5 + sum(counts)
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    w = randn(3, N, K, seed=11)
    for dgrad in (False, True):
        ka, kc = (N, K) if dgrad else (K, N)
        wide, more = randn(R, ka + 8, seed=9), randn(R, kc, seed=12)
        want, got = torch.zeros(R, kc, dtype=BF, device="cuda"), torch.zeros(R, kc, dtype=BF, device="cuda")
        call = B.moe_grouped_gemm_dgrad if dgrad else B.moe_grouped_gemm
        call(wide[:, :ka], w, c, o, want, sc, add=more)
        check_rows(want, wide[:, :ka], w, counts, off, more, dgrad)
        wide[:, ka:] = float("nan")
        wide[0], wide[off[2] - 1], wide[-3:] = float("nan"), float("inf"), float("nan")
        wide[off[1]:off[2]] = float("nan")
        bad = w.clone()
        bad[1] = float("nan")
        call(wide[:, :ka], bad, c, o, got, sc, add=more)
        for e in (0, 2):
            r = slice(off[e], off[e] + counts[e])
            assert torch.equal(got[r], want[r])
        assert bool((got[0] == 0).all()) and bool((got[-3:] == 0).all())


def test_one_group_of_all_rows_and_no_rows():
    x, w, dy = randn(130, 64, seed=12), randn(1, 72, 64, seed=13), randn(130, 72, seed=14)
    sc = B.alloc_product_scratch()
    y, dx, dw = (torch.empty(130, 72, dtype=BF, device="cuda"), torch.empty_like(x), torch.empty_like(w))
    B.moe_grouped_gemm(x, w, None, None, y, sc)
    B.moe_grouped_gemm_dgrad(dy, w, None, None, dx, sc)
    B.moe_grouped_gemm_wgrad(dy, x, None, None, dw, sc)
    check_rows(y, x, w, [130], [0])
    check_rows(dx, dy, w, [130], [0], dgrad=True)
    check_wgrad(dw, dy, x, [130], [0])
    B.moe_grouped_gemm(x[:0], w, None, None, y[:0], sc)
    B.moe_grouped_gemm_dgrad(dy[:0], w, None, None, dx[:0], sc)
    B.moe_grouped_gemm_wgrad(dy[:0], x[:0], None, None, dw, sc)
    assert bool((dw == 0).all())
    dw.fill_(1)
    B.moe_grouped_gemm_wgrad(dy[:0], x[:0], dev([0]), dev([0]), dw, sc)
    assert bool((dw == 0).all()) and B.moe_last_device_status(sc) == 0


def test_bad_segments_are_left_out():
    counts, off = [40, 30, 5, 20], [0, 80, -1, 45]
    x, w, dy = randn(100, 64, seed=15), randn(4, 72, 64, seed=16), randn(100, 72, seed=17)
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    good = [40, 0, 0, 20]
    for few in (0, 1):
        y = torch.full((100, 72), 5.0, dtype=BF, device="cuda")
        B.moe_grouped_gemm(x, w, c, o, y, sc, expected_rows=few)
        assert B.moe_last_device_status(sc) == 6
        B.moe_clear_device_status(sc)
        check_rows(y, x, w, good, off)
        assert bool((y[65:] == 5).all())
    dx, dw = torch.full((100, 64), 5.0, dtype=BF, device="cuda"), torch.empty_like(w)
    B.moe_grouped_gemm_dgrad(dy, w, c, o, dx, sc)
    assert B.moe_last_device_status(sc) == 6 and bool((dx[65:] == 5).all())
    check_rows(dx, dy, w, good, off, dgrad=True)
    B.moe_clear_device_status(sc)
    B.moe_grouped_gemm_wgrad(dy, x, c, o, dw, sc)
    assert B.moe_last_device_status(sc) == 6
    check_wgrad(dw, dy, x, good, off)


def test_rows_behind_2_to_the_31_elements():
    R, K, N = 600_000, 4096, 4096
    x = torch.zeros(R, K, dtype=BF, device="cuda")
    x[-140:] = randn(140, K, seed=18)
    w, out = randn(2, N, K, seed=19, scale=0.02), torch.zeros(R, N, dtype=BF, device="cuda")
    counts, off = [135, 5], [R - 140, R - 5]
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    for few in (0, 8):
        out.zero_()
        B.moe_grouped_gemm(x, w, c, o, out, sc, expected_rows=few)
        check_rows(out, x, w, counts, off)
        assert bool((out[:-140] == 0).all())
    dw = torch.empty_like(w)
    B.moe_grouped_gemm_wgrad(out, x, c, o, dw, sc)
    check_wgrad(dw, out, x, counts, off)


@pytest.mark.parametrize("R,N,K", [(600_000, 16, 4096), (600_000, 4096, 16), (140_000_000, 24, 16)])
def test_narrow_products_of_rows_behind_2_to_the_31_elements(R, N, K):
    w, counts, off = randn(2, N, K, seed=19, scale=0.1), [135, 5], [R - 140, R - 5]
    c, o, sc = dev(counts), dev(off), B.alloc_product_scratch()
    for dgrad in (False, True):
        ka, kc = (N, K) if dgrad else (K, N)
        a = torch.zeros(R, ka, dtype=BF, device="cuda")
        a[-140:] = randn(140, ka, seed=18)
        out = torch.zeros(R, kc, dtype=BF, device="cuda")
        if dgrad:
            B.moe_grouped_gemm_dgrad(a, w, c, o, out, sc, add=out)
        else:
            B.moe_grouped_gemm(a, w, c, o, out, sc, add=out)
        check_rows(out, a, w, counts, off, dgrad=dgrad)
        assert bool((out[:-140] == 0).all()) and B.moe_last_device_status(sc) == 0
        del a, out


def test_captured_and_replayed_with_other_counts():
    R, N, K = 400, 256, 320
    x, w, dy = randn(R, K, seed=20), randn(3, N, K, seed=21), randn(R, N, seed=22)
    c, o, sc = dev([100, 200, 50]), dev([0, 100, 300]), B.alloc_product_scratch()
    y, dx, dw = torch.zeros(R, N, dtype=BF, device="cuda"), torch.zeros_like(x), torch.empty_like(w)

    def step():
        B.moe_grouped_gemm(x, w, c, o, y, sc)
        B.moe_grouped_gemm_dgrad(dy, w, c, o, dx, sc, add=x)
        B.moe_grouped_gemm_wgrad(dy, x, c, o, dw, sc)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for counts, off in (([100, 200, 50], [0, 100, 300]), ([0, 1, 390], [0, 399, 0])):
        c.copy_(dev(counts))
        o.copy_(dev(off))
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_rows(y, x, w, counts, off)
        check_rows(dx, dy, w, counts, off, add=x, dgrad=True)
        check_wgrad(dw, dy, x, counts, off)
