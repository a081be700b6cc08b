"""One MoE layer with its experts in 4 bits: serving steps and a training step around them.

    python -m routing_dispatch_expert_router_gb300.fp4_layer [workload] [--format nv|mx]
        [--tokens 1,16,..] [--steps N]

The layer's weights (workloads.make_inputs) are quantised once with moe_fp4_quantize.
For every token count of --tokens (default 1,16,256,4096) a serving step -- route, dispatch,
the experts' FFN in 4 bits, combine -- is captured in a CUDA graph and timed; the last
count also runs a training step around the frozen experts, whose forward keeps the 8-bit
checkpoint and whose backward gives the gradients of the tokens and of the router. One
JSON line each: microseconds a step, the bytes of 4-bit weights against bf16's, and how far
the layer's output is from the bf16 layer's (relative 2-norm).
"""
from __future__ import annotations

import json
import os
import sys

import torch

from . import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# weights of standard deviation 0.02: block maxima over 6 2^-9 lie well inside E4M3's range
NV_SCALE_LOG2 = -9


class Fp4Layer:
    """A layer's router, its experts in 4 bits and the buffers of up to `shape.T` tokens."""

    def __init__(self, shape, inputs: dict, fmt: int, training: bool = False):
        self.cfg = cfg = B.config(shape)
        self.W_r, self.bias = inputs["W_r"], inputs["bias"]
        G, H, F = cfg.E + cfg.n_shared, cfg.H, cfg.F
        log2 = NV_SCALE_LOG2 if fmt == B.MOE_FP4_NV else 0
        self.W13 = B.alloc_fp4(fmt, G, 2 * F, H, scale_log2=log2)
        self.W2 = B.alloc_fp4(fmt, G, H, F, scale_log2=log2)
        B.moe_fp4_quantize(inputs["W13"], self.W13)
        B.moe_fp4_quantize(inputs["W2"], self.W2)
        self.experts = B.fp4_experts(self.W13, self.W2)
        sz, s4 = B.moe_query_sizes(cfg), B.moe_fp4_query_sizes(cfg, fmt)
        R, T, E, k = int(sz.rows_max), cfg.T, cfg.E, cfg.k

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.logits, self.idx, self.w = empty(T, E, dtype=f32), empty(T, k, dtype=i32), empty(T, k, dtype=f32)
        self.counts, self.offsets = empty(G, dtype=i32), empty(G + 1, dtype=i32)
        self.row_of, self.token_of = empty(T, k, dtype=i32), empty(R, dtype=i32)
        self.sel_offsets, self.sel_tokens = empty(E + 1, dtype=i32), empty(T * k, dtype=i32)
        self.x_perm, self.y_perm, self.out = empty(R, H), empty(R, H), empty(T, H)
        self.scratch = torch.zeros(int(sz.scratch_bytes), dtype=u8, device="cuda")
        self.fwd_scratch = B.alloc_fp4_scratch(s4.fwd_scratch_bytes)
        self.ckpt = self.ckpt_scale = None
        if training:
            self.ckpt, self.ckpt_scale = empty(R, 2 * F, dtype=u8), empty(R, 2 * F // 32, dtype=u8)
            self.bwd_scratch = B.alloc_fp4_scratch(s4.bwd_scratch_bytes)
            self.dO_perm, self.dX_perm, self.dx = empty(R, H), empty(R, H), empty(T, H)
            self.dw, self.dlogits = empty(T, k, dtype=f32), empty(T, E, dtype=f32)
            self.dW_r = empty(E, H, dtype=f32)

    def forward(self, x):
        B.moe_route(self.cfg, x, self.W_r, self.bias, self.logits, self.idx, self.w, self.scratch)
        B.moe_permute(self.cfg, x, self.idx, self.counts, self.offsets, self.row_of, self.token_of,
                      self.sel_offsets, self.sel_tokens, self.x_perm, self.scratch)
        B.moe_fp4_ffn_fwd(self.cfg, self.experts, self.x_perm, self.counts, self.offsets, self.ckpt,
                          self.ckpt_scale, self.y_perm, self.fwd_scratch)
        B.moe_unpermute(self.cfg, self.y_perm, self.row_of, self.w, self.offsets, self.out)
        return self.out

    def backward(self, x, dY):
        """Gradients of the tokens (dx) and of the router's weight (dW_r); the experts are held."""
        c = self.cfg
        B.moe_unpermute_bwd(c, dY, self.y_perm, self.row_of, self.w, self.counts, self.offsets,
                            self.dO_perm, self.dw, self.scratch)
        B.moe_route_bwd(c, self.logits, self.idx, self.w, self.dw, self.dlogits)
        B.moe_fp4_ffn_bwd(c, self.experts, self.dO_perm, self.ckpt, self.ckpt_scale, self.counts,
                          self.offsets, self.token_of, self.dlogits, self.W_r, self.dX_perm,
                          self.bwd_scratch)
        B.moe_permute_bwd(c, self.dX_perm, self.row_of, self.offsets, self.idx, self.dlogits,
                          self.W_r, self.dx)
        B.moe_router_wgrad(c, x, self.sel_offsets, self.sel_tokens, self.dlogits, self.dW_r,
                           self.scratch)
        return self.dx, self.dW_r

    def check(self):
        """Raises if a kernel recorded a problem (synchronises)."""
        words = [self.scratch, self.fwd_scratch] + ([self.bwd_scratch] if self.ckpt is not None else [])
        for s in words:
            code = B.moe_last_device_status(s)
            if code:
                raise B.MoEError("device status", code)


def _time_graph(step, steps: int) -> float:
    """Microseconds a step of a captured step, L2 flushed before each."""
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    times = []
    for i in range(3 + steps):
        flush.fill_(i & 1)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        if i >= 3:
            times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[len(times) // 2]


def _bf16_output(shape, inp):
    cfg = B.config(shape)
    bufs = B.alloc_buffers(cfg, "cuda", backward=False)
    out = torch.empty_like(inp["x"])
    B.moe_layer_fwd(cfg, B.params(inp["W_r"], inp["bias"], inp["W13"], inp["W2"]), inp["x"], out,
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

    fmt = {"nv": B.MOE_FP4_NV, "mx": B.MOE_FP4_MX}[option("--format", "nv")]
    tokens = [int(t) for t in option("--tokens", "1,16,256,4096").split(",")]
    steps = int(option("--steps", "20"))
    shapes = {n: s for n, s in W.SHAPES.items() if s.dtype == W.DT_BF16}
    name = argv[0] if argv else "mixtral"
    if name not in shapes:
        raise SystemExit(f"workload: one of {', '.join(shapes)}")
    for T in tokens:
        shape = shapes[name].with_(T=T)
        inp = W.make_inputs(shape, seed=0, device="cuda")
        last = T == tokens[-1]
        layer = Fp4Layer(shape, inp, fmt)
        us = _time_graph(lambda: layer.forward(inp["x"]), steps)
        layer.check()
        ref = _bf16_output(shape, inp).float()
        far = ((layer.out.float() - ref).norm() / ref.norm()).item()
        size = sum(t.numel() for t in (layer.W13.codes, layer.W13.scales, layer.W2.codes,
                                       layer.W2.scales))
        print(json.dumps(dict(
            layer=name, format=("nv", "mx")[fmt], tokens=T, step="serve", us=round(us, 1),
            weight_bytes=size, bf16_weight_bytes=2 * (inp["W13"].numel() + inp["W2"].numel()),
            rel_to_bf16=round(far, 4))), flush=True)
        if last:
            del layer
            layer = Fp4Layer(shape, inp, fmt, training=True)

            def train():
                layer.forward(inp["x"])
                layer.backward(inp["x"], inp["dY"])

            us = _time_graph(train, steps)
            layer.check()
            rows = layer.ckpt.shape[0]
            print(json.dumps(dict(
                layer=name, format=("nv", "mx")[fmt], tokens=T, step="train", us=round(us, 1),
                checkpoint_bytes=layer.ckpt.numel() + layer.ckpt_scale.numel(),
                bf16_gate_up_and_h_bytes=rows * 3 * shape.F * 2)), flush=True)
        del layer, inp
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
