"""The norm's kernels of many rows. Those that keep rows in flight have more rows to every CTA than its
ring has slots, so that each slot is filled and read again: every width that has a form of its own,
the 8-bit output, in place, strided, and beside rows of NaN. Against the formulas in 64 bits, with the tolerances of the
short cases (their sums are no deeper here; dgamma's grow with the rows).
"""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from test_gpu_rmsnorm import BF, EPS, U, check_fwd, codes_of, gamma_of, near, rows

pytestmark = pytest.mark.gpu

# rows, columns: eight rows a CTA or more where CTAs are persistent (three an SM at 4096 columns, two at
# 7168 and 8200, one above; on 152 SMs), and no whole number of rounds
WIDTHS = [(8301, 2056), (4201, 4096), (2501, 7168), (2501, 8200), (1301, 16384)]


@pytest.mark.parametrize("T,H", [(15001, 1032), *WIDTHS])
@pytest.mark.parametrize("residual,f32", [(True, False), (False, True)])
def test_forward(T, H, residual, f32):
    x, gamma = rows(T, H, 21), gamma_of(H, f32)
    res = rows(T, H, 22, 3.0) if residual else None
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    s = torch.empty_like(x) if residual else None
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, sum=s, rstd=rstd, eps=EPS)
    check_fwd(x, res, gamma, y, s, rstd)
    for _ in range(3):
        y2 = torch.empty_like(x)
        B.moe_rmsnorm_fwd(x, gamma, y2, residual=res, eps=EPS)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("T,H,block", [(8301, 2080, 32), (4201, 4096, 128), (2501, 7168, 32), (2501, 8320, 128),
                                       (1301, 16384, 32)])
def test_forward_in_8_bits(T, H, block):
    x, res, gamma = rows(T, H, 23), rows(T, H, 24), gamma_of(H, False)
    x[T // 2], res[T // 2] = 0, 0                          # a row of empty blocks
    y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // block, dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, sum=s, rstd=rstd, codes=codes, scales=scales, eps=EPS)
    check_fwd(x, res, gamma, y, s, rstd)
    c, e = codes_of(y, block)
    assert torch.equal(scales, e)
    assert torch.equal(codes & 127, c & 127) and torch.equal(codes[c & 127 > 0], c[c & 127 > 0])
    only = torch.empty_like(codes), torch.empty_like(scales)
    B.moe_rmsnorm_fwd(x, gamma, None, residual=res, codes=only[0], scales=only[1], eps=EPS)
    assert torch.equal(only[0], codes) and torch.equal(only[1], scales)


@pytest.mark.parametrize("T,H", [(8301, 2056), (2501, 8200)])
def test_in_place_and_strided(T, H):
    x, res, gamma = rows(T, H, 25), rows(T, H, 26), gamma_of(H, False)
    y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    B.moe_rmsnorm_fwd(x, gamma, y, residual=res, sum=s, rstd=rstd, eps=EPS)
    check_fwd(x, res, gamma, y, s, rstd)
    bx = torch.full((T + 2, H + 120), 7.0, dtype=BF, device="cuda")
    br = bx.clone()
    vx, vr = bx[1:-1, 64:64 + H], br[1:-1, 8:8 + H]
    vx.copy_(x), vr.copy_(res)
    B.moe_rmsnorm_fwd(vx, gamma, vx, residual=vr, sum=vr, eps=EPS)     # the sum over the residual, the output over x
    assert torch.equal(vx, y) and torch.equal(vr, s)
    vx.copy_(x), vr.copy_(res)
    y2 = torch.empty_like(x)
    B.moe_rmsnorm_fwd(vx, gamma, y2, residual=vr, sum=vx, eps=EPS)     # the sum over x
    assert torch.equal(y2, y) and torch.equal(vx, s) and torch.equal(vr, res)
    vx.fill_(7.0), vr.fill_(7.0)
    assert bool((bx == 7).all()) and bool((br == 7).all())


@pytest.mark.parametrize("T,H", [(4201, 4096), (1301, 16384)])
def test_special_values_stay_in_their_rows(T, H):
    x, gamma = rows(T, H, 27), gamma_of(H, False)
    clean, y = torch.empty_like(x), torch.empty_like(x)
    B.moe_rmsnorm_fwd(x, gamma, clean, eps=EPS)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[3::7] = True
    x[bad] = float("nan")
    B.moe_rmsnorm_fwd(x, gamma, y, eps=EPS)
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("T,H", [(17301, 512), (17301, 40), (6101, 1024), (4201, 2056), (4201, 4096), (2501, 8192),
                                 (1301, 8200), (1301, 16384), (701, 32768)])
@pytest.mark.parametrize("residual,f32", [(True, True), (False, False)])
def test_backward(T, H, residual, f32):
    h, dy, gamma = rows(T, H, 31), rows(T, H, 32), gamma_of(H, f32)
    ds = rows(T, H, 33) if residual else None
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
    near(dx, ref, 2.0 ** -8 * ref.abs() + 64 * U * big)
    # a CTA's rows, its eight warps, 32 shares a thread and 16 of those, one addition each, on
    # terms of four roundings
    terms = dy.double() * n
    near(dg, terms.sum(0), (T // 152 + 64) * U * terms.abs().sum(0))
    for name in ("dy", "dsum") if residual else ("dy",):
        d = dict(dy=dy.clone(), dsum=None if ds is None else ds.clone())
        dg2 = torch.empty_like(dg)
        B.moe_rmsnorm_bwd(d["dy"], h, rstd, gamma, d[name], dg2, dsum=d["dsum"], scratch=sc.fill_(1))
        assert torch.equal(d[name], dx) and torch.equal(dg2, dg)
