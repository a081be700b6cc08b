"""The layer of the int4_layer command, served and trained, against the formulas in 64 bits.

Each result is compared with the formula on the layer's own routing, dispatched rows and
intermediates, so that only the roundings behind those are left: bf16 results half a step (2^-8 of
the value), fp32 sums of at most 2^-14 of their terms' magnitudes. Experts that became bf16 have one
rounding more of every weight."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from routing_dispatch_expert_router_gb300 import int4_layer as L
from workloads import SIGMOID, MoEShape, make_inputs

pytestmark = pytest.mark.gpu
H_ = pytest.importorskip("harness")
f64 = H_.f64
STEP, SUM = 2.0 ** -8, 2.0 ** -14
# tokens that stream the codes and tokens for which the experts become bf16
SHAPES = [MoEShape("int4_few", T=37, H=256, E=8, k=2, F=384, bias_kind="none"),
          MoEShape("int4_one", T=1, H=512, E=4, k=2, F=128, bias_kind="none"),
          MoEShape("int4_sig", T=150, H=256, E=8, k=2, F=384, n_shared=1, score_fn=SIGMOID,
                   n_groups=4, topk_groups=2, bias_kind="normal"),
          MoEShape("int4_many", T=420, H=384, E=4, k=2, F=256, bias_kind="none")]


def values(W):
    """The weights that an Int4Tensor's codes stand for."""
    q = W.codes.cpu().numpy()
    code = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], q.shape[1], -1).astype(np.float64)
    group = code.shape[2] // W.scales.shape[1]
    wide = lambda t: np.repeat(f64(t).transpose(0, 2, 1), group, axis=2)
    return wide(W.scales) * (code - (8 if W.zeros is None else wide(W.zeros)))


def close(name, got, ref, tol):
    H_.assert_close(name, got, ref, atol=1e-30, rtol=1, scale=tol)


def prepared(shape, training, rank=24, group=64):
    inp = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in make_inputs(shape, seed=4).items()}
    layer = L.Int4Layer(shape, inp, group=group, rank=rank, training=training)
    g = torch.Generator().manual_seed(9)
    layer.B.copy_(torch.randn(layer.B.shape, generator=g) * 0.05)
    layer.gamma.copy_(torch.rand(shape.H, generator=g) + 0.5)
    more = torch.randn(shape.T, shape.H, generator=g).to(torch.bfloat16).cuda()
    return layer, inp, more


def segments(layer, shape):
    m = O.permutation_maps(H_.i64(layer.idx), shape)
    return m, [slice(o, o + c) for o, c in zip(m["offsets"], m["counts"])]


def check_forward(layer, shape, x, residual):
    T, E, k, F, S = shape.T, shape.E, shape.k, shape.F, shape.n_shared
    s = f64(x)
    if residual is not None:
        s = s + f64(residual)
        close("sum", f64(layer.sum), s, STEP * np.abs(s))
        s = f64(layer.sum)
    rstd = (np.mean(s * s, 1) + 1e-6) ** -0.5
    close("rstd", f64(layer.rstd), rstd, 1e-5 * rstd)
    n = s * rstd[:, None] * f64(layer.gamma)
    close("normed", f64(layer.normed), n, (STEP + 1e-5) * np.abs(n))
    n = f64(layer.normed)
    idx_ref, w = O.route(f64(layer.logits), shape, None if layer.bias is None else f64(layer.bias))
    H_.assert_equal("idx", H_.i64(layer.idx), idx_ref)
    m, seg = segments(layer, shape)
    X = O.permute(n, m)
    W13, W2, A, Bm = values(layer.W13), values(layer.W2), f64(layer.A), f64(layer.B)
    h, a, y = f64(layer.h), f64(layer.a), f64(layer.y_perm)
    # roundings of h's and y's operands and of themselves, of independent signs: in norm
    n_h, n_y = (2, 3) if layer.streams else (6, 4)
    for e, r in enumerate(seg):
        if r.start == r.stop:
            continue
        H_.assert_equal("x_perm", f64(layer.x_perm[r]), X[r])
        gu = X[r] @ W13[e].T
        ref = O.silu(gu[:, :F]) * gu[:, F:]
        assert np.linalg.norm(h[r] - ref) <= n_h * STEP * np.linalg.norm(ref), e
        ref, mag = X[r] @ A[e].T, np.abs(X[r]) @ np.abs(A[e]).T
        close("a", a[r], ref, STEP * np.abs(ref) + SUM * mag)
        base, low = h[r] @ W2[e].T, a[r] @ Bm[e].T
        assert np.linalg.norm(y[r] - base - low) <= n_y * STEP * np.linalg.norm(np.abs(base) + np.abs(base + low)), e
    row, off = m["row_of"], m["offsets"]
    parts = [w[:, j:j + 1] * y[row[:, j]] for j in range(k)]
    parts += [y[off[E + i]:off[E + i] + T] for i in range(S)]
    ref = sum(parts)
    # weights of the router's own precision (1e-5 relative, as its stage is held to)
    close("out", f64(layer.out), ref, STEP * np.abs(ref) + 2e-5 * sum(np.abs(p) for p in parts))
    return m, seg, X, w


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.name)
def test_served(shape, with_residual):
    layer, inp, more = prepared(shape, training=False)
    assert layer.streams == (shape.name in ("int4_few", "int4_one"))
    residual = more if with_residual else None
    out = layer.forward(inp["x"], residual)
    layer.check()
    check_forward(layer, shape, inp["x"], residual)
    # a captured step, replayed on other tokens and back
    first = out.clone()
    x = inp["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, residual)
    x.copy_(more)
    g.replay()
    check_forward(layer, shape, more, residual)
    x.copy_(inp["x"])
    g.replay()
    assert torch.equal(layer.out, first)
    layer.check()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.name)
def test_trained(shape):
    layer, inp, more = prepared(shape, training=True)
    T, E, k, F, S = shape.T, shape.E, shape.k, shape.F, shape.n_shared
    x, dY = inp["x"], inp["dY"]
    past = torch.randn(T, shape.H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    layer.forward(x, more)
    dx = layer.backward(x, dY, dsum=past, residual=more)
    layer.check()
    m, seg, X, w = check_forward(layer, shape, x, more)
    row, off = m["row_of"], m["offsets"]
    W13, W2, A, Bm = values(layer.W13), values(layer.W2), f64(layer.A), f64(layer.B)
    GU, a, y, dYd = f64(layer.GU), f64(layer.a), f64(layer.y_perm), f64(dY)
    dO = np.zeros((m["R"], shape.H))
    dX = np.zeros_like(dO)
    for j in range(k):
        dO[row[:, j]] = w[:, j:j + 1] * dYd
    for i in range(S):
        dO[off[E + i]:off[E + i] + T] = dYd
    got_A, got_B = f64(layer.dA), f64(layer.dB)
    for e, r in enumerate(seg):
        if r.start == r.stop:
            assert (got_A[e] == 0).all() and (got_B[e] == 0).all()
            continue
        # dO is rounded (and its weight off by 1e-5), so is da, and each result
        ref, mag = dO[r].T @ a[r], np.abs(dO[r]).T @ np.abs(a[r])
        close("dB", got_B[e], ref, (2 * STEP + SUM) * mag)
        da, damag = dO[r] @ Bm[e], np.abs(dO[r]) @ np.abs(Bm[e])
        ref, mag = da.T @ X[r], damag.T @ np.abs(X[r])
        close("dA", got_A[e], ref, (3.1 * STEP + SUM) * mag)
        dX[r] = O.expert_fc1_dgrad(O.expert_fc2_dgrad_swiglu(dO[r], W2[e], GU[r], False), W13[e], False)
        dX[r] += da @ A[e]
    dw = np.stack([(dYd * y[row[:, j]]).sum(1) for j in range(k)], 1)
    dl = O.router_dlogits(shape, f64(layer.logits), H_.i64(layer.idx), w, dw)
    terms = [dX[row[:, j]] for j in range(k)] + [dX[off[E + i]:off[E + i] + T] for i in range(S)]
    terms.append(dl @ f64(layer.W_r))
    dn = sum(terms)
    # dO, [dG|dU], both weights, dX_perm twice and dn: seven roundings of independent signs, in norm
    tol = 8 * STEP * np.sqrt(sum(np.linalg.norm(t) ** 2 for t in terms))
    assert np.linalg.norm(f64(layer.dn) - dn) <= tol
    # the norm's backward on the layer's own dn
    dn, s, rstd, gamma = f64(layer.dn), f64(layer.sum), f64(layer.rstd), f64(layer.gamma)
    xhat = s * rstd[:, None]
    gdy = dn * gamma
    mean = np.mean(gdy * xhat, 1, keepdims=True)
    ref = rstd[:, None] * (gdy - xhat * mean) + f64(past)
    mag = rstd[:, None] * (np.abs(gdy) + np.abs(xhat) * np.mean(np.abs(gdy * xhat), 1, keepdims=True))
    close("dx", f64(dx), ref, STEP * np.abs(ref) + 1e-5 * (mag + np.abs(f64(past))))
    ref, mag = (dn * xhat).sum(0), np.abs(dn * xhat).sum(0)
    close("dgamma", f64(layer.dgamma), ref, SUM * mag)
    # captured, with an eager step between
    want = [t.clone() for t in (dx, layer.dA, layer.dB, layer.dgamma, layer.dW_r)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, more)
        layer.backward(x, dY, dsum=past, residual=more)
    layer.forward(more)
    layer.backward(more, past)
    g.replay()
    for t, v in zip((dx, layer.dA, layer.dB, layer.dgamma, layer.dW_r), want):
        assert torch.equal(t, v)
    layer.check()


def test_quantised_weights():
    """Every weight within half a step of its group's scale (and the scale's own rounding)."""
    W = torch.randn(2, 48, 256, generator=torch.Generator().manual_seed(3)).cuda()
    W[0, 0] = 0
    W[1, 5] = W[1, 5].abs()
    for group in (32, 64, 128):
        for zeros in (True, False):
            q = L.quantize_int4(W, group, zeros)
            step = np.repeat(f64(q.scales).transpose(0, 2, 1), group, axis=2)
            # a scale off by 2^-8 of itself moves the outermost of 15 codes (8 of them from zero)
            # by that much more, and the zero point by half a step of the lower end
            assert (np.abs(values(q) - f64(W)) <= step * (0.5 + 15 * 2.0 ** -8 + (0.5 if zeros else 0)) + 1e-6).all()


def test_two_layers_at_once():
    """A serving and a training layer on streams of their own, with buffers of their own, give the bits
    that they give alone."""
    serve, inp, more = prepared(SHAPES[0], training=False)
    train, inp2, more2 = prepared(SHAPES[3], training=True)

    def step():
        train.forward(inp2["x"], more2)
        return train.backward(inp2["x"], inp2["dY"], residual=more2)

    out = serve.forward(inp["x"], more).clone()
    kept = [t.clone() for t in (step(), train.out, train.dA, train.dB, train.dgamma, train.dW_r)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for t in (serve.out, train.out, train.dA, train.dB, train.dgamma, train.dx):
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            with torch.cuda.stream(a):
                serve.forward(inp["x"], more)
            with torch.cuda.stream(b):
                step()
        torch.cuda.synchronize()
        assert torch.equal(serve.out, out)
        for t, v in zip((train.dx, train.out, train.dA, train.dB, train.dgamma, train.dW_r), kept):
            assert torch.equal(t, v)
    serve.check()
    train.check()
