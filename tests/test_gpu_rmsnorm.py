"""RMS norm with the residual's addition, its 8-bit output and its backward, against the formulas
in 64 bits.

Tolerances. A rounding to bf16 is off by 2^-8 of the value at most. fp32 sums of n terms in any
order are off by n 2^-24 of the sum of their magnitudes; a thread adds 32 squares at most and
two trees of five levels join them, so the sum of squares is off by 42 2^-24 of itself, and its
inverse root by half of that and the roundings of quotient, sum and root: 24 2^-24.
"""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B

pytestmark = pytest.mark.gpu
BF, U = torch.bfloat16, 2.0 ** -24
EPS = 1e-5


def rows(T, H, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * torch.exp(0.5 * torch.randn(H, generator=g)) * scale
    return x.to(BF).cuda()


def gamma_of(H, f32, seed=5):
    g = 1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(seed))
    return (g if f32 else g.to(BF)).cuda()


def near(got, ref, tol):
    d = (got.double() - ref).abs()
    assert bool((d <= tol).all()), (d - tol).max().item()


def check_fwd(x, res, gamma, y, s, rstd):
    h = x.double()
    if res is not None:
        h = h + res.double()
        near(s, h, (2.0 ** -8 + U) * h.abs())
        h = s.double()
    r = (h.square().mean(1) + EPS).rsqrt()
    near(rstd, r, 24 * U * r)
    ref = h * r[:, None] * gamma.double()
    near(y, ref, (2.0 ** -8 + 32 * U) * ref.abs())


def codes_of(y, block):
    """E4M3 codes and scale bytes of bf16 rows, from the definition."""
    b = y.double().unflatten(-1, (-1, block))
    amax = b.abs().amax(-1)
    # ceil(log2 q), q = m 2^e with 1/2 <= m < 1 (a logarithm need not be whole at powers of two)
    m, e = torch.frexp(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448)
    e = (e - (m == 0.5).int()).clamp(min=-127)
    v = (b * torch.exp2(-e).unsqueeze(-1)).float().to(torch.float8_e4m3fn)
    return v.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (9, 520), (700, 1024), (5, 1032), (1, 4096),
                                 (333, 4096), (130, 7168), (2, 8200), (3, 16384), (2, 16392),
                                 (2, 32768)])
@pytest.mark.parametrize("residual,f32", [(True, False), (False, True)])
def test_forward(T, H, residual, f32):
    x, gamma = rows(T, H, 1), gamma_of(H, f32)
    res = rows(T, H, 2, 3.0) if residual else None
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    s = torch.empty_like(x) if residual else None
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, sum=s, rstd=rstd, eps=EPS)
    check_fwd(x, res, gamma, y, s, rstd)
    # without the sum and the root, the same bits
    y2 = torch.empty_like(x)
    B.moe_rmsnorm_fwd(x, gamma, y2, residual=res, eps=EPS)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T,H,block", [(1, 32, 32), (7, 128, 128), (33, 1024, 32), (5, 1056, 32),
                                       (4, 4096, 128), (3, 7168, 32), (2, 16512, 128)])
def test_forward_in_8_bits(T, H, block):
    x, res, gamma = rows(T, H, 3), rows(T, H, 4), gamma_of(H, False)
    x[0], res[0] = 0, 0                                    # a row of empty blocks
    if H > 32:
        x[-1, :32], res[-1, :32] = 0, 0                    # an empty block beside others
    y = torch.empty_like(x)
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // block, dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, codes=codes, scales=scales, eps=EPS)
    c, e = codes_of(y, block)
    assert torch.equal(scales, e)
    assert torch.equal(codes & 127, c & 127) and torch.equal(codes[c & 127 > 0], c[c & 127 > 0])
    only = torch.empty_like(codes), torch.empty_like(scales)
    B.moe_rmsnorm_fwd(x, gamma, None, residual=res, codes=only[0], scales=only[1], eps=EPS)
    assert torch.equal(only[0], codes) and torch.equal(only[1], scales)


def test_in_place_strided_and_what_lies_beside():
    T, H, wide = 37, 2056, 2176
    x, res, gamma = rows(T, H, 6), rows(T, H, 7), gamma_of(H, False)
    y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, sum=s, rstd=rstd, eps=EPS)
    # rows of wider tensors; the sum over the residual, the output over x
    bx = torch.full((T + 2, wide), 7.0, dtype=BF, device="cuda")
    br = bx.clone()
    bx[1:-1, 64:64 + H], br[1:-1, 8:8 + H] = x, res
    vx, vr = bx[1:-1, 64:64 + H], br[1:-1, 8:8 + H]
    B.moe_rmsnorm_fwd(vx, gamma, vx, residual=vr, sum=vr, eps=EPS)
    assert torch.equal(vx, y) and torch.equal(vr, s)
    vx.fill_(7.0), vr.fill_(7.0)
    assert bool((bx == 7).all()) and bool((br == 7).all())
    # the backward over dy and over dsum
    dy, ds = rows(T, H, 8), rows(T, H, 9)
    dx, dg = torch.empty_like(x), torch.empty(H, device="cuda")
    sc = torch.empty(B.rmsnorm_scratch_bytes(H), dtype=torch.uint8, device="cuda").fill_(255)
    B.moe_rmsnorm_bwd(dy, s, rstd, gamma, dx, dg, dsum=ds, scratch=sc)
    for name in ("dy", "dsum"):
        t = dict(dy=dy.clone(), dsum=ds.clone())
        B.moe_rmsnorm_bwd(t["dy"], s, rstd, gamma, t[name], dsum=t["dsum"])
        assert torch.equal(t[name], dx)


def test_special_values_stay_in_their_rows():
    T, H = 6, 4096
    x, gamma = rows(T, H, 10), gamma_of(H, False)
    clean, y = torch.empty_like(x), torch.empty_like(x)
    B.moe_rmsnorm_fwd(x, gamma, clean, eps=EPS)
    x[1, 5], x[3, 9], x[4] = float("nan"), float("inf"), 0
    rstd = torch.empty(T, device="cuda")
    B.moe_rmsnorm_fwd(x, gamma, y, rstd=rstd, eps=EPS)
    assert bool(y[1].isnan().all()) and bool(y[3, 9].isnan()) and bool((y[3, :9] == 0).all())
    assert bool((y[4] == 0).all()) and abs(rstd[4].item() - EPS ** -0.5) < 1e-3
    for t in (0, 2, 5):
        assert torch.equal(y[t], clean[t])


@pytest.mark.parametrize("T,H", [(1, 8), (9, 64), (100, 512), (70, 1024), (3, 1032), (700, 2048),
                                 (1, 4096), (333, 4096), (60, 8192), (7, 8200), (5, 16384), (3, 32768)])
@pytest.mark.parametrize("residual,f32", [(True, True), (False, False)])
def test_backward(T, H, residual, f32):
    h, dy, gamma = rows(T, H, 11), rows(T, H, 12), gamma_of(H, f32)
    ds = rows(T, H, 13) if residual else None
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dg = torch.empty_like(h), torch.empty(H, device="cuda")
    sc = torch.empty(B.rmsnorm_scratch_bytes(H), dtype=torch.uint8, device="cuda").fill_(255)
    B.moe_rmsnorm_bwd(dy, h, rstd, gamma, dx, dg, dsum=ds, scratch=sc)
    r = rstd.double()[:, None]
    n, t = h.double() * r, dy.double() * gamma.double()
    ref = r * (t - n * (t * n).mean(1, keepdim=True))
    big = r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
    if residual:
        ref, big = ref + ds.double(), big + ds.double().abs()
    # the mean of t n: 42 additions deep and four roundings; the rest a few
    near(dx, ref, 2.0 ** -8 * ref.abs() + 64 * U * big)
    near(dg, (dy.double() * n).sum(0), (T + 4) * U * (dy.double() * n).abs().sum(0))
    dx2, dg2 = torch.empty_like(h), torch.empty(H, device="cuda")
    B.moe_rmsnorm_bwd(dy, h, rstd, gamma, dx2, dg2, dsum=ds, scratch=sc.fill_(1))
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_backward_against_differences():
    """The formula itself: (f(h + d) - f(h - d)) / 2 in 64 bits."""
    T, H = 3, 16
    h, dy, gamma = rows(T, H, 14), rows(T, H, 15), gamma_of(H, True)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dg = torch.empty_like(h), torch.empty(H, device="cuda")
    sc = torch.empty(B.rmsnorm_scratch_bytes(H), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_bwd(dy, h, rstd, gamma, dx, dg, scratch=sc)

    def f(hh, gg):
        return (dy.double() * hh * (hh.square().mean(1, keepdim=True) + EPS).rsqrt() * gg).sum()

    d = 1e-5
    for i in range(H):
        e = torch.zeros(H, dtype=torch.float64, device="cuda")
        e[i] = d
        slope = (f(h.double(), gamma.double() + e) - f(h.double(), gamma.double() - e)) / (2 * d)
        assert abs(dg[i].item() - slope.item()) <= 1e-5 * (1 + abs(slope.item()))
        for t in range(T):
            step = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            step[t, i] = d
            slope = ((f(h.double() + step, gamma.double()) - f(h.double() - step, gamma.double()))
                     / (2 * d)).item()
            assert abs(dx[t, i].item() - slope) <= 2.0 ** -8 * abs(slope) + 1e-5


def test_no_rows_and_a_held_gamma():
    H = 256
    e = torch.empty(0, H, dtype=BF, device="cuda")
    gamma, dg = gamma_of(H, False), torch.ones(H, device="cuda")
    none = torch.empty(0, device="cuda")
    sc = torch.empty(B.rmsnorm_scratch_bytes(H), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_fwd(e, gamma, e, rstd=none)
    B.moe_rmsnorm_bwd(e, e, none, gamma, e, dg, scratch=sc)
    assert bool((dg == 0).all())


def test_captured_and_on_another_stream():
    T, H = 65, 4096
    x, res, gamma, dy = rows(T, H, 16), rows(T, H, 17), gamma_of(H, False), rows(T, H, 18)
    out = [torch.empty_like(x) for _ in range(3)]
    rstd, dg = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    sc = torch.empty(B.rmsnorm_scratch_bytes(H), dtype=torch.uint8, device="cuda")

    def step():
        B.moe_rmsnorm_fwd(x, gamma, out[0], residual=res, sum=out[1], rstd=rstd)
        B.moe_rmsnorm_bwd(dy, out[1], rstd, gamma, out[2], dg, dsum=out[0], scratch=sc)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, rstd, dg)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
    for t in (*out, rstd, dg):
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (*out, rstd, dg)))
