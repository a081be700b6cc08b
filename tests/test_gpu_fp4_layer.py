"""The layer of the fp4_layer command, served and trained, against the fp64 oracle: its output,
the gradient of the tokens and the router's.

Each result is compared with the formula on the layer's own routing, dispatched outputs and
checkpoint, so that only the roundings behind those are left: bf16 results half a step (2^-8),
[dG|dU], dO and dX_perm rounded to bf16 in between, fp32 sums."""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as O4
from oracle import moe_oracle as O
from routing_dispatch_expert_router_gb300 import fp4_layer as L
from workloads import SIGMOID, TINY, MoEShape, make_inputs

pytestmark = pytest.mark.gpu

H_ = pytest.importorskip("harness")
T4 = pytest.importorskip("test_gpu_fp4")
DEV = "cuda"
f64, host = T4.f64, T4.host
SHAPES = [TINY.with_(T=70),
          MoEShape("fp4_sig", T=150, H=256, E=8, k=2, F=384, n_shared=1, score_fn=SIGMOID,
                   n_groups=4, topk_groups=2, bias_kind="normal"),
          MoEShape("fp4_one", T=1, H=2048, E=8, k=2, F=512, bias_kind="none")]


def weight_values(q, rows):
    g = q.codes.shape[0]
    byte = O4.from_atoms(q.format, host(q.scales).reshape(g, -(-rows // 128), -1, 512), rows, q.K)
    return O4.values(q.format, O4.unpack(host(q.codes)), byte, q.scale_log2)


@pytest.mark.parametrize("fmt", T4.FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.name)
def test_layer_serves_and_trains_as_the_oracle(fmt, shape):
    inp = {k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in make_inputs(shape, seed=4).items()}
    layer = L.Fp4Layer(shape, inp, fmt, training=True)
    out = layer.forward(inp["x"])
    dx, dW_r = layer.backward(inp["x"], inp["dY"])
    layer.check()
    T, H, E, k, F, S = shape.T, shape.H, shape.E, shape.k, shape.F, shape.n_shared
    x, dY, Wr = f64(inp["x"]), f64(inp["dY"]), f64(inp["W_r"])
    idx, logits = H_.i64(layer.idx), f64(layer.logits)
    idx_ref, w = O.route(logits, shape, None if inp["bias"] is None else f64(inp["bias"]))
    H_.assert_equal("idx", idx, idx_ref)
    m = O.permutation_maps(idx, shape)
    off, cnt, row = m["offsets"], m["counts"], m["row_of"]
    W13, W2 = weight_values(layer.W13, 2 * F), weight_values(layer.W2, H)
    y, ck, cs = f64(layer.y_perm), host(layer.ckpt), host(layer.ckpt_scale)
    x_rows = O.permute(x, m)
    dX = np.zeros((m["R"], H))
    dO = np.zeros((m["R"], H))
    for j in range(k):
        dO[row[:, j]] = w[:, j:j + 1] * dY
    for s in range(S):
        dO[off[E + s]:off[E + s] + T] = dY
    for g in range(E + S):
        r = slice(off[g], off[g] + cnt[g])
        if cnt[g] == 0:
            continue
        gu, _, _, ref = O4.ffn_fwd(fmt, x_rows[r], W13[g], W2[g])
        # one rounding of y; a gate, up or h that fell the other way moves few terms
        assert np.linalg.norm(y[r] - ref) <= 2.0 ** -7 * np.linalg.norm(ref), g
        kept = O4.checkpoint_values(ck[r], cs[r])
        # half a step of E4M3's three bits, on values whose own rounding may differ by one of bf16
        assert np.linalg.norm(kept - gu) <= 2.0 ** -4 * np.linalg.norm(gu), g
        dX[r], _ = O4.ffn_bwd(dO[r], kept, W13[g], W2[g])
    # combine: fp32 sum of k + S bf16 rows, rounded once
    acc = sum(w[:, j:j + 1] * y[row[:, j]] for j in range(k))
    mag = sum(w[:, j:j + 1] * np.abs(y[row[:, j]]) for j in range(k))
    for s in range(S):
        acc = acc + y[off[E + s]:off[E + s] + T]
        mag = mag + np.abs(y[off[E + s]:off[E + s] + T])
    # weights of the router's own precision (1e-5 relative, as its stage is held to)
    H_.assert_close("out", f64(out), acc, atol=0, rtol=1, scale=2.0 ** -8 * np.abs(acc) + 2e-5 * mag)
    # router: dw = <dY, y> in fp32, its way through the scores, dW_r summed over the tokens
    dw = np.stack([(dY * y[row[:, j]]).sum(1) for j in range(k)], 1)
    dw_mag = np.stack([(np.abs(dY) * np.abs(y[row[:, j]])).sum(1) for j in range(k)], 1)
    dl = O.router_dlogits(shape, logits, idx, w, dw)
    # a dw off by 1e-5 of its magnitudes moves a dlogit by at most twice that (the scores'
    # derivatives are weights of at most route_scale)
    dl_err = 1e-5 * np.abs(dl) + 2e-5 * shape.route_scale * dw_mag.max(1, keepdims=True)
    dl_err = np.where(dl != 0, dl_err, 0.0)
    ref = dl.T @ x
    H_.assert_close("dW_r", f64(dW_r), ref, atol=0, rtol=1,
                    scale=1e-5 * np.abs(dl).T @ np.abs(x) + dl_err.T @ np.abs(x))
    # tokens: the rows of their experts and the router's term
    ref = sum(dX[row[:, j]] for j in range(k)) + dl @ Wr
    for s in range(S):
        ref = ref + dX[off[E + s]:off[E + s] + T]
    rows_norm = np.sqrt(sum(np.linalg.norm(dX[row[:, j]]) ** 2 for j in range(k))
                        + sum(np.linalg.norm(dX[off[E + s]:off[E + s] + T]) ** 2 for s in range(S))
                        + np.linalg.norm(dl @ Wr) ** 2)
    # dO, [dG|dU], dX_perm and dx: four bf16 roundings of independent signs, each at most
    # 2^-9 / sqrt(3) x 2 of its operand's norm on average
    assert np.linalg.norm(f64(dx) - ref) <= 4 * 2.0 ** -9 * max(rows_norm, np.linalg.norm(ref))
    far = np.abs(f64(dx) - ref).max()
    assert far <= 2.0 ** -5 * np.abs(ref).max(), far
