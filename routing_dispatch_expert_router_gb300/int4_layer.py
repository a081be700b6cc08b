"""One MoE layer behind its norm, the experts held in 4-bit integers, an adapter beside each:
serving steps and a training step of the adapters.

    python -m routing_dispatch_expert_router_gb300.int4_layer [workload] [--group 32|64|128]
        [--rank R] [--tokens 1,16,..] [--steps N]

    s = x + residual,  n = RMS norm of s,  out = combine over the router's choice of
    expert(n) + B (A n),  A [R, H] and B [H, R] of every expert

The experts (workloads.make_inputs) are quantised once, with a zero point and a scale for every
group along the input. For every token count of --tokens (default 1,16,256,4096) a serving step is
captured in a CUDA graph and timed; the last count also runs a training step, whose backward gives
the gradients of the tokens, the adapters, the norm and the router. One JSON line each: microseconds
a step, the bytes of 4-bit weights against bf16's, and how far the layer's output is from that of
the bf16 experts (relative 2-norm).
"""
from __future__ import annotations

import json
import sys

import torch

from . import binding as B
from .fp4_layer import ROOT, _time_graph

# Rows an expert expects up to which the products read the codes once for every 16 rows. Beyond it
# the experts become bf16 first, which costs 4.5 bytes of traffic a weight, eight readings of codes.
# (A step of eight experts 28672 x 4096, 2 of them a token, us, streamed and not: 128 tokens 464 and
# 1099, 256: 808 and 1103, 384: 1132 and 1103, 512: 1443 and 1193.)
STREAM_ROWS = 96


def quantize_int4(W: torch.Tensor, group: int = 128, zeros: bool = True) -> B.Int4Tensor:
    """[groups, N, K] in 4 bits, group after group of K from the smallest to the largest value;
    without zero points: from -8 to 7 times the scale."""
    G, N, K = W.shape
    codes = torch.empty(G, N, K // 2, dtype=torch.uint8, device=W.device)
    scales = torch.empty(G, K // group, N, dtype=torch.bfloat16, device=W.device)
    zero = torch.empty(G, K // group, N, dtype=torch.uint8, device=W.device) if zeros else None
    for g in range(G):
        w = W[g].float().view(N, -1, group)
        if zeros:
            lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            s = ((hi - lo) / 15).to(torch.bfloat16)
        else:
            s = (w.abs().amax(2) / 7).to(torch.bfloat16)
        s = torch.where(s > 0, s, torch.ones_like(s))
        z = (-lo / s.float()).round().clamp(0, 15) if zeros else torch.full_like(s, 8, dtype=torch.float32)
        q = ((w / s.float().unsqueeze(2)).round() + z.unsqueeze(2)).clamp(0, 15).to(torch.uint8)
        q = q.view(N, K)
        codes[g] = q[:, ::2] | q[:, 1::2] << 4
        scales[g] = s.T
        if zeros:
            zero[g] = z.T.to(torch.uint8)
    return B.Int4Tensor(codes, scales, zero)


class Int4Layer:
    """A layer's norm and router, its experts in 4 bits, an adapter for each of them and the buffers
    of up to `shape.T` tokens (bf16)."""

    def __init__(self, shape, inputs: dict, group: int = 128, rank: int = 16, training: bool = False):
        self.cfg = cfg = B.config(shape)
        self.training = training
        self.W_r, self.bias = inputs["W_r"], inputs["bias"]
        G, H, F = cfg.E + cfg.n_shared, cfg.H, cfg.F
        self.W13 = quantize_int4(inputs["W13"], group)
        self.W2 = quantize_int4(inputs["W2"], group)
        R, T, E, k = int(B.moe_query_sizes(cfg).rows_max), cfg.T, cfg.E, cfg.k

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.gamma = torch.ones(H, dtype=f32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(17)
        self.A = (torch.randn(G, rank, H, device="cuda", generator=g) * H ** -0.5).to(torch.bfloat16)
        self.B = torch.zeros(G, H, rank, dtype=torch.bfloat16, device="cuda")
        self.sum, self.normed, self.rstd = empty(T, H), empty(T, H), empty(T, dtype=f32)
        self.logits, self.idx, self.w = empty(T, E, dtype=f32), empty(T, k, dtype=i32), empty(T, k, dtype=f32)
        self.counts, self.offsets = empty(G, dtype=i32), empty(G + 1, dtype=i32)
        self.row_of, self.token_of = empty(T, k, dtype=i32), empty(R, dtype=i32)
        self.sel_offsets, self.sel_tokens = empty(E + 1, dtype=i32), empty(T * k, dtype=i32)
        self.x_perm, self.h, self.y_perm = empty(R, H), empty(R, F), empty(R, H)
        self.a, self.out = empty(R, rank), empty(T, H)
        self.scratch = torch.zeros(int(B.moe_query_sizes(cfg).scratch_bytes), dtype=u8, device="cuda")
        self.product_scratch = B.alloc_product_scratch()
        self.streams = not training and max(T if cfg.n_shared else 0, T * k / E) <= STREAM_ROWS
        if not self.streams:                       # (a model's layers share the two)
            self.W13_bf16, self.W2_bf16, self.GU = empty(G, 2 * F, H), empty(G, H, F), empty(R, 2 * F)
        if training:
            self.dO_perm, self.dX_perm, self.dGU = empty(R, H), empty(R, H), empty(R, 2 * F)
            self.dw, self.dlogits = empty(T, k, dtype=f32), empty(T, E, dtype=f32)
            self.da, self.dn, self.dx = empty(R, rank), empty(T, H), empty(T, H)
            self.dA, self.dB = torch.empty_like(self.A), torch.empty_like(self.B)
            self.dgamma, self.dW_r = empty(H, dtype=f32), empty(E, H, dtype=f32)
            self.norm_scratch = empty(B.rmsnorm_scratch_bytes(H), dtype=u8)

    def _segments(self):
        return self.counts, self.offsets[:-1]

    def _bf16_experts(self):
        B.moe_int4_dequantize(self.W13, self.W13_bf16)
        B.moe_int4_dequantize(self.W2, self.W2_bf16)

    def forward(self, x, residual=None):
        """The layer's output for its input x (+ residual): what the next norm takes as x, with
        `sum` (or x, without a residual) as its residual."""
        c, s = self.cfg, self.product_scratch
        B.moe_rmsnorm_fwd(x, self.gamma, self.normed, residual=residual,
                          sum=None if residual is None else self.sum, rstd=self.rstd)
        B.moe_route(c, self.normed, self.W_r, self.bias, self.logits, self.idx, self.w, self.scratch)
        B.moe_permute(c, self.normed, self.idx, self.counts, self.offsets, self.row_of, self.token_of,
                      self.sel_offsets, self.sel_tokens, self.x_perm, self.scratch)
        if self.streams:
            B.moe_int4_grouped_gemm(self.x_perm, self.W13, *self._segments(), self.h, s, swiglu=True)
            B.moe_int4_grouped_gemm(self.h, self.W2, *self._segments(), self.y_perm, s)
        else:
            self._bf16_experts()
            B.moe_grouped_ffn_fwd(c, self.x_perm, self.counts, self.offsets, self.W13_bf16,
                                  self.W2_bf16, self.GU, self.h, self.y_perm, self.scratch)
        B.moe_grouped_gemm(self.x_perm, self.A, *self._segments(), self.a, s, expected_rows=c.T)
        B.moe_grouped_gemm(self.a, self.B, *self._segments(), self.y_perm, s, add=self.y_perm,
                           expected_rows=c.T)
        B.moe_unpermute(c, self.y_perm, self.row_of, self.w, self.offsets, self.out)
        return self.out

    def backward(self, x, dY, dsum=None, residual=None):
        """The gradient of x (and of the residual); dA, dB, dgamma and dW_r beside it. dsum: the
        gradient that reaches `sum` past the layer."""
        c, s = self.cfg, self.product_scratch
        B.moe_unpermute_bwd(c, dY, self.y_perm, self.row_of, self.w, self.counts, self.offsets,
                            self.dO_perm, self.dw, self.scratch)
        B.moe_route_bwd(c, self.logits, self.idx, self.w, self.dw, self.dlogits)
        B.moe_grouped_gemm_dgrad(self.dO_perm, self.B, *self._segments(), self.da, s)
        B.moe_grouped_gemm_wgrad(self.dO_perm, self.a, *self._segments(), self.dB, s)
        B.moe_grouped_gemm_wgrad(self.da, self.x_perm, *self._segments(), self.dA, s)
        self._bf16_experts()
        B.moe_grouped_ffn_dgrad(c, self.dO_perm, self.GU, None, self.counts, self.offsets,
                                self.token_of, self.dlogits, self.W_r, self.W13_bf16, self.W2_bf16,
                                self.dGU, self.dX_perm, self.scratch)
        B.moe_grouped_gemm_dgrad(self.da, self.A, *self._segments(), self.dX_perm, s,
                                 add=self.dX_perm)
        B.moe_permute_bwd(c, self.dX_perm, self.row_of, self.offsets, self.idx, self.dlogits,
                          self.W_r, self.dn)
        B.moe_router_wgrad(c, self.normed, self.sel_offsets, self.sel_tokens, self.dlogits, self.dW_r,
                           self.scratch)
        B.moe_rmsnorm_bwd(self.dn, x if residual is None else self.sum, self.rstd, self.gamma, self.dx,
                          dgamma=self.dgamma, dsum=dsum, scratch=self.norm_scratch)
        return self.dx

    def check(self):
        """Raises if a kernel recorded a problem (synchronises)."""
        for s in (self.scratch, self.product_scratch):
            code = B.moe_last_device_status(s)
            if code:
                raise B.MoEError("device status", code)


def _bf16_output(shape, inp, x):
    cfg = B.config(shape)
    bufs = B.alloc_buffers(cfg, "cuda", backward=False)
    out = torch.empty_like(x)
    B.moe_layer_fwd(cfg, B.params(inp["W_r"], inp["bias"], inp["W13"], inp["W2"]), x, out,
                    bufs.fwd_struct, bufs.scratch)
    return out


def main(argv=None) -> None:
    sys.path.insert(0, ROOT)
    import workloads as W
    argv = list(sys.argv[1:] if argv is None else argv)

    def option(name, default):
        if name not in argv:
            return default
        i = argv.index(name)
        value = argv[i + 1]
        del argv[i:i + 2]
        return value

    group, rank = int(option("--group", "128")), int(option("--rank", "16"))
    tokens = [int(t) for t in option("--tokens", "1,16,256,4096").split(",")]
    steps = int(option("--steps", "20"))
    shapes = {n: s for n, s in W.SHAPES.items() if s.dtype == W.DT_BF16}
    name = argv[0] if argv else "mixtral"
    if name not in shapes:
        raise SystemExit(f"workload: one of {', '.join(shapes)}")
    for T in tokens:
        shape = shapes[name].with_(T=T)
        inp = W.make_inputs(shape, seed=0, device="cuda")
        layer = Int4Layer(shape, inp, group, rank)
        us = _time_graph(lambda: layer.forward(inp["x"]), steps)
        layer.check()
        ref = _bf16_output(shape, inp, layer.normed).float()
        far = ((layer.out.float() - ref).norm() / ref.norm()).item()
        size = sum(t.numel() * t.element_size() for w in (layer.W13, layer.W2)
                   for t in (w.codes, w.scales, w.zeros))
        print(json.dumps(dict(
            layer=name, group=group, rank=rank, tokens=T, step="serve", us=round(us, 1),
            streamed=layer.streams, weight_bytes=size,
            bf16_weight_bytes=2 * (inp["W13"].numel() + inp["W2"].numel()),
            rel_to_bf16=round(far, 4))), flush=True)
        del layer
        if T == tokens[-1]:
            layer = Int4Layer(shape, inp, group, rank, training=True)

            def train():
                layer.forward(inp["x"])
                layer.backward(inp["x"], inp["dY"])

            us = _time_graph(train, steps)
            layer.check()
            print(json.dumps(dict(layer=name, group=group, rank=rank, tokens=T, step="train",
                                  us=round(us, 1))), flush=True)
            del layer
        del inp
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
