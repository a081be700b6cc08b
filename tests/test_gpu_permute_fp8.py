"""The dispatch of tokens in 8 bits: the same maps, codes and scales as the dispatch that
quantises bf16 tokens, and an FP8 layer served from the norm's codes."""
import pytest
import torch

import routing_dispatch_expert_router_gb300.binding as B
from workloads import MoEShape, make_inputs

pytestmark = pytest.mark.gpu
U8, I32, BF = torch.uint8, torch.int32, torch.bfloat16


def shape_of(T, E, k, dtype, cf=0.0, H=512):
    return MoEShape("s", T=T, H=H, E=E, k=k, F=256, dtype=dtype, capacity_factor=cf)


def maps(cfg):
    sz = B.moe_query_sizes(cfg)
    T, E, k, R = cfg.T, cfg.E, cfg.k, int(sz.rows_max)
    n = dict(counts=E, offsets=E + 1, row_of=T * k, token_of=R, sel_offsets=E + 1, sel_tokens=T * k)
    return {a: torch.full((max(b, 1),), -7, dtype=I32, device="cuda") for a, b in n.items()}


def normed(cfg, seed):
    """A norm's output in bf16 and in 8 bits."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(cfg.T, cfg.H, generator=g).to(BF).cuda()
    block = 32 if cfg.dtype == 2 else 128
    y, codes = torch.empty_like(x), torch.empty(cfg.T, cfg.H, dtype=U8, device="cuda")
    scales = torch.empty(cfg.T, cfg.H // block, dtype=U8, device="cuda")
    B.moe_rmsnorm_fwd(x, torch.ones(cfg.H, device="cuda"), y, codes=codes, scales=scales)
    return y, codes, scales


def scale_bytes(atoms, n):
    """[rows, n] scale bytes out of their atoms [row blocks, atoms, 512]."""
    a = atoms.view(atoms.shape[0], -1, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return a.reshape(atoms.shape[0] * 128, -1)[:, :n]


@pytest.mark.parametrize("dtype", [1, 2])
@pytest.mark.parametrize("T,E,k,cf", [(0, 8, 2, 0.0), (1, 8, 2, 0.0), (61, 128, 8, 0.0), (300, 11, 3, 0.0),
                                      (520, 4, 2, 0.6), (1, 1, 1, 0.0)])
def test_rows_and_maps(T, E, k, cf, dtype):
    H = 512 if T != 300 else 768                       # (768: the last atom holds two blocks)
    shape = shape_of(T, E, k, dtype, cf, H)
    cfg = B.config(shape)
    g = torch.Generator().manual_seed(T + E)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(I32).contiguous().cuda()
    y, codes, scales = normed(cfg, 3)
    R, n = int(B.moe_query_sizes(cfg).rows_max), scales.shape[1]
    want, sc = maps(cfg), torch.zeros(int(B.moe_query_sizes(cfg).scratch_bytes), dtype=U8, device="cuda")
    x_perm = torch.empty(R, H, dtype=BF, device="cuda")
    B.moe_permute(cfg, y, idx, *want.values(), x_perm, sc)
    got = maps(cfg)
    xq = torch.full((R, H), 9, dtype=U8, device="cuda")
    xs = torch.full((-(-R // 128), -(-n // 4), 512), 9, dtype=U8, device="cuda")
    small = torch.zeros(4352 + 4 * E * (-(-T // 256)), dtype=U8, device="cuda")
    B.moe_permute_fp8(cfg, codes, scales, idx, *got.values(), small, codes_perm=xq, scales_perm=xs)
    for name in want:
        assert torch.equal(want[name], got[name]), name
    token = got["token_of"][:R]
    if cf:
        assert int((got["row_of"] < 0).sum()) > 0      # some were dropped
    # (past the last segment token_of is not written)
    last = int(got["offsets"][E])
    live = (token[:last] >= 0).nonzero()[:, 0]
    assert torch.equal(xq[live], codes[token[live].long()])
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[live] = False
    assert bool((xq[rest] == 9).all())
    bytes_ = scale_bytes(xs, n)
    assert torch.equal(bytes_[live], scales[token[live].long()])
    assert bool((bytes_[:R][rest] == 9).all())
    assert B.moe_last_device_status(small) == 0


def layer(shape, x_bf16, codes, scales, W, capture=False):
    """Route (on the bf16 rows), dispatch (bf16 rows, or their codes), experts, combine."""
    cfg = B.config(shape)
    bufs = B.alloc_buffers(cfg, "cuda", backward=False)
    for t in bufs.fwd.values():
        t.zero_()
    f, sc = bufs.fwd, bufs.scratch
    out = torch.empty_like(x_bf16)
    B.moe_quantize_weights(cfg, W["W13"], W["W2"], sc)

    def step():
        B.moe_route(cfg, x_bf16, W["W_r"], W["bias"], f["logits"], f["idx"], f["w"], sc)
        m = [f[n] for n in ("counts", "offsets", "row_of", "token_of", "sel_offsets", "sel_tokens")]
        if codes is None:
            B.moe_permute(cfg, x_bf16, f["idx"], *m, f["x_perm"], sc)
        else:
            B.moe_permute_fp8(cfg, codes, scales, f["idx"], *m, sc)
        B.moe_grouped_ffn_fwd(cfg, f["x_perm"] if codes is None else None, f["counts"], f["offsets"],
                              W["W13"], W["W2"], f["GU"], f["h"], f["y_perm"], sc)
        B.moe_unpermute(cfg, f["y_perm"], f["row_of"], f["w"], f["offsets"], out)

    step()
    if capture:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        out.zero_()
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert B.moe_last_device_status(sc) == 0
    return out


@pytest.mark.parametrize("dtype", [1, 2])
def test_an_fp8_layer_served_from_the_norms_codes(dtype):
    """Bit for bit the layer that quantises the norm's bf16 output in its dispatch."""
    shape = shape_of(200, 8, 2, dtype)
    W = make_inputs(shape, seed=1, device="cuda")
    y, codes, scales = normed(B.config(shape), 5)
    want = layer(shape, y, None, None, W)
    assert torch.equal(layer(shape, y, codes, scales, W), want)
    assert torch.equal(layer(shape, y, codes, scales, W, capture=True), want)


def test_a_bad_expert_is_left_out():
    shape = shape_of(5, 4, 2, 1)
    cfg = B.config(shape)
    idx = torch.tensor([[0, 1], [2, 9], [3, 3], [-1, 0], [1, 2]], dtype=I32, device="cuda")
    _, codes, scales = normed(cfg, 6)
    m, sc = maps(cfg), torch.zeros(int(B.moe_query_sizes(cfg).scratch_bytes), dtype=U8, device="cuda")
    B.moe_permute_fp8(cfg, codes, scales, idx, *m.values(), sc)
    assert B.moe_last_device_status(sc) == 6
    assert m["counts"].tolist() == [2, 2, 2, 1]
    assert (m["row_of"] < 0).tolist() == [False, False, False, True, False, True, True, False, False, False]
