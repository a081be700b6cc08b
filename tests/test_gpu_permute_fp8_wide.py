"""The dispatch of tokens in 8 bits at the widths of real layers: rows of several pieces of 2 KB, the
scale words dealt among them, and more pieces than the grid has warps."""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from test_gpu_permute_fp8 import BF, I32, U8, maps, normed, scale_bytes, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("T,E,k,H,cf", [(61, 128, 8, 7168, 0.0), (300, 11, 3, 2304, 0.0), (300, 11, 3, 2048, 0.0),
                                        (520, 4, 2, 4096, 0.6), (33, 8, 2, 16384, 0.0), (8192, 64, 4, 4096, 0.0),
                                        (4099, 32, 8, 7168, 1.25)])
def test_rows_and_maps(T, E, k, H, cf, dtype):
    cfg = B.config(shape_of(T, E, k, dtype, cf, H))
    g = torch.Generator().manual_seed(T + H)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(I32).contiguous().cuda()
    y, codes, scales = normed(cfg, 3)
    sz = B.moe_query_sizes(cfg)
    R, n = int(sz.rows_max), scales.shape[1]
    want, sc = maps(cfg), torch.zeros(int(sz.scratch_bytes), dtype=U8, device="cuda")
    x_perm = torch.empty(R, H, dtype=BF, device="cuda")
    B.moe_permute(cfg, y, idx, *want.values(), x_perm, sc)
    del x_perm
    got = maps(cfg)
    xq = torch.full((R, H), 9, dtype=U8, device="cuda")
    xs = torch.full((-(-R // 128), -(-n // 4), 512), 9, dtype=U8, device="cuda")
    B.moe_permute_fp8(cfg, codes, scales, idx, *got.values(), sc, codes_perm=xq, scales_perm=xs)
    for name in want:
        assert torch.equal(want[name], got[name]), name
    if cf:
        assert T != 520 or int((got["row_of"] < 0).sum()) > 0
    last, token = int(got["offsets"][E]), got["token_of"][:R]
    live = (token[:last] >= 0).nonzero()[:, 0]
    source = token[live].long()
    # every kept assignment has its row
    assert live.numel() == int((got["row_of"] >= 0).sum())
    assert torch.equal(xq[live], codes[source])
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[live] = False
    assert bool((xq[rest] == 9).all())
    bytes_ = scale_bytes(xs, n)
    assert torch.equal(bytes_[live], scales[source])
    assert bool((bytes_[:R][rest] == 9).all())
    assert B.moe_last_device_status(sc) == 0
