"""Products with 4-bit integer weights whose tokens have a few channels far above the others, as
the channels in front of experts do: a code that is its zero point takes such a channel out of the
result whatever its size.

Tolerance of an element: its own rounding, 2^-8 |y|, and the fp32 sums' of what the weights leave. A
group's sum of (code - zero) x is at most 24 additions deep (a product of 16 terms, eight of those),
each off by 2^-23 of the magnitudes' sum at most (the tensor cores cut instead of rounding); scaling
and adding the groups' sums is off by 2^-24 of them each.
"""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8


def weights(N, K, group, zeros, channels, above, seed):
    """Codes whose value at `channels` is the zero point plus `above`; w in 64 bits beside them."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randint(3, 12, (1, K // group, N), generator=g, dtype=U8)
    if not zeros:
        z.fill_(8)
    q = torch.randint(0, 16, (1, N, K), generator=g, dtype=U8)
    zk = z[0].T.repeat_interleave(group, 1)                          # [N, K]
    q[0][:, channels] = zk[:, channels] + above
    s = (0.01 * (0.5 + torch.rand(1, K // group, N, generator=g))).to(BF)
    w = (q[0].double() - zk.double()) * s[0].double().T.repeat_interleave(group, 1)
    codes = (q[:, :, 0::2] | (q[:, :, 1::2] << 4)).contiguous().cuda()
    return B.Int4Tensor(codes, s.cuda(), z.cuda() if zeros else None), w.cuda()


def product(W, x, cols, swiglu=False):
    out = torch.empty(x.shape[0], cols, dtype=BF, device="cuda")
    B.moe_int4_grouped_gemm(x, W, None, None, out, B.alloc_product_scratch(), swiglu=swiglu)
    return out.double()


def sums(x, w, groups):
    x = x.double()
    return x @ w.T, (24 * 2.0 ** -23 + (groups + 1) * 2.0 ** -24) * (x.abs() @ w.abs().T)


@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("group,zeros", [(32, True), (32, False), (64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 14, 2.0 ** 40])
def test_a_channel_far_above_the_others(rows, group, zeros, size):
    N, K = 272, 640                                     # (a short last slab, a short last step)
    W, w = weights(N, K, group, zeros, [5, 200, 511], 0, seed=group)
    x = torch.randn(rows, K, generator=torch.Generator().manual_seed(1)).to(BF)
    x[:, [5, 200, 511]] = torch.tensor([size, -1.5 * size, 0.75 * size]).to(BF)
    x = x.cuda()
    y, tol = sums(x, w, K // group)
    d = (product(W, x, N) - y).abs()
    assert bool((d <= tol + 2.0 ** -8 * y.abs()).all()), (d / (tol + 2.0 ** -8 * y.abs())).max().item()


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_a_channel_far_above_the_others_behind_swiglu(group, zeros):
    N, K = 320, 512
    W, w = weights(N, K, group, zeros, [7, 300], 0, seed=3)
    x = torch.randn(3, K, generator=torch.Generator().manual_seed(2)).to(BF)
    x[:, [7, 300]] = torch.tensor([2.0 ** 14, -(2.0 ** 13)]).to(BF)
    x = x.cuda()
    y, tol = sums(x, w, K // group)
    (a, b), (ta, tb) = y.chunk(2, 1), tol.chunk(2, 1)
    sa = a * torch.sigmoid(a)
    y = sa * b                                          # (|silu'| <= 1.1; its fp32 form a few ulp)
    tol = 1.1 * ta * b.abs() + (sa.abs() + 1.1 * ta) * tb + (2.0 ** -20 + 2.0 ** -8) * y.abs()
    assert bool(((product(W, x, N // 2, swiglu=True) - y).abs() <= tol).all())


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_values_near_the_end_of_fp32(group, zeros):
    """2^124 times one: a group's sum of (code - zero) x is finite, and so is the result."""
    N, K = 64, 256
    W, w = weights(N, K, group, zeros, [40], 1, seed=4)
    x = torch.randn(2, K, generator=torch.Generator().manual_seed(3)).to(BF)
    x[:, 40] = 2.0 ** 124
    x = x.cuda()
    y, tol = sums(x, w, K // group)
    got = product(W, x, N)
    assert bool(got.isfinite().all())
    assert bool(((got - y).abs() <= tol + 2.0 ** -8 * y.abs()).all())


def test_codes_at_their_zero_points_give_zero():
    W, _ = weights(96, 384, 128, True, list(range(384)), 0, seed=5)
    x = (100 * torch.randn(5, 384, generator=torch.Generator().manual_seed(4))).to(BF).cuda()
    assert bool((product(W, x, 96) == 0).all())
