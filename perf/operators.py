"""The 4-bit expert operators, as cases that can be timed and checked.

The operators are those of a Mixture-of-Experts layer whose experts are kept in
microscaled 4-bit floating point:

  quantize    rows of bf16 -> E2M1 codes with a scale per block (and, where the
              caller asks for them, the bf16 values that the codes stand for);
  dequantize  the bf16 values of such codes;
  product     y[r] = alpha[g] * x4[r] W4[g]^T for the rows r of every expert g,
              the bf16 rows quantised in the call;
  ffn         the experts' SwiGLU FFN in 4 bits, with the 8-bit checkpoint of its
              gate and up values where a backward will follow;
  ffn_bwd     the gradient at the FFN's input, through the 4-bit weights, from
              the 8-bit checkpoint.

Two formats: "nv" (blocks of 16 along K, one E4M3 scale each) and "mx" (blocks
of 32, one power-of-two scale each). Codes are packed two to a byte, the even
element in the low four bits. Scale bytes lie in atoms of 512 bytes, one per 128
rows and four consecutive blocks: byte (r % 32) * 16 + (r % 128) // 32 * 4 + j
holds the scale of row r's j-th block; each 128-row slab has whole 256-element
steps of K, the atoms past K's end being zero.

`run` computes a case in elementary torch operations where `own` is false and
through the framework's entry points where it is true; `prepare` does not depend
on it.
"""
import math

import torch

own = False

NV, MX = "nv", "mx"
BLOCK = {NV: 16, MX: 32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # the magnitudes of E2M1


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token's hidden row, the smallest call: latency
        dict(name="quantize_one_token", op="quantize", fmt=NV, groups=1, rows=1, K=7168, log2=0),
        # a ragged batch of activations of an odd width, straight-through training
        dict(name="quantize_odd_mx", op="quantize", fmt=MX, groups=1, rows=4091, K=2080, log2=0),
        # a layer's gate and up weights, quantised when a checkpoint is loaded or trained on
        dict(name="quantize_weights", op="quantize", fmt=NV, groups=8, rows=14336, K=4096, log2=-11),
        # a layer's weights as bf16 again, for a path that multiplies in bf16
        dict(name="dequantize_weights", op="dequantize", fmt=NV, groups=8, rows=4096, K=14336, log2=-11),
        # a small slab of odd height
        dict(name="dequantize_odd_mx", op="dequantize", fmt=MX, groups=5, rows=331, K=1504, log2=0),
        # a projection of odd sizes over few tokens, some experts without any
        dict(name="product_odd_mx", op="product", fmt=MX, T=300, E=11, k=2, N=1000, K=1504),
        # the second projection of a layer with eight large experts, a long prompt
        dict(name="product_prompt", op="product", fmt=NV, T=4096, E=8, k=2, N=4096, K=14336),
        # one token through a layer of eight large experts: every byte read is a weight
        dict(name="ffn_one_token", op="ffn", fmt=NV, T=1, E=8, k=2, H=4096, F=14336, ckpt=False),
        # a decoding batch over many small experts: nearly all of the weights, few rows each
        dict(name="ffn_decode_batch", op="ffn", fmt=NV, T=64, E=64, k=8, H=4096, F=2048, ckpt=False),
        # a training batch: the same layer, keeping the checkpoint
        dict(name="ffn_train", op="ffn", fmt=NV, T=4096, E=64, k=8, H=4096, F=2048, ckpt=True),
        # its backward
        dict(name="ffn_bwd_train", op="ffn_bwd", fmt=NV, T=4096, E=64, k=8, H=4096, F=2048),
        # a small step, odd batch: launches and tile edges count
        dict(name="ffn_bwd_small_mx", op="ffn_bwd", fmt=MX, T=333, E=8, k=2, H=512, F=896),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _drawn(rng)
        if 3072 not in case.values():                    # a size of no layer here
            return case


def _drawn(rng):
    op = rng.choice(["quantize", "dequantize", "product", "ffn", "ffn_bwd"])
    fmt = rng.choice([NV, MX])
    if op in ("quantize", "dequantize"):
        while True:
            K = 32 * _between(rng, 2, 448)
            groups, rows = rng.choice([1, 1, 3, 8]), _between(rng, 1, 14336)
            if groups * rows * K <= 8 * 14336 * 4096:
                return dict(op=op, fmt=fmt, groups=groups, rows=rows, K=K,
                            log2=rng.choice([-11, -3, 0]) if fmt == NV else 0)
    while True:
        E = rng.choice([1, 4, 8, 11, 32, 64])
        k = rng.choice([x for x in (1, 2, 4, 8) if x <= E])
        T = _between(rng, 1, 4096)
        if op == "product":
            N, K = 8 * _between(rng, 8, 512), 32 * _between(rng, 4, 448)
            if E * N * K <= 8 * 4096 * 14336 and T * k * N * K <= 4096 * 2 * 4096 * 14336:
                return dict(op=op, fmt=fmt, T=T, E=E, k=k, N=N, K=K)
            continue
        H, F = 128 * _between(rng, 1, 32), 128 * _between(rng, 1, 112)
        if E * H * F <= 64 * 4096 * 2048 and T * k * H * F <= 4096 * 8 * 4096 * 2048:
            case = dict(op=op, fmt=fmt, T=T, E=E, k=k, H=H, F=F)
            if op == "ffn":
                case["ckpt"] = rng.random() < 0.5
            return case


# ----------------------------------------------------------- sizes and layouts
def _up(a, b):
    return -(-a // b) * b


def _atoms(fmt, K):
    """Atoms of a 128-row slab: whole 256-element steps of K."""
    return _up(K, 256) // (4 * BLOCK[fmt])


def _to_atoms(fmt, s, K):
    """Scale bytes [groups, rows, K / block] in their atoms [groups, slabs, atoms, 512]."""
    g, rows, nb = s.shape
    ka, slabs = _atoms(fmt, K), _up(rows, 128) // 128
    full = s.new_zeros(g, slabs * 128, ka * 4)
    full[:, :rows, :nb] = s
    return full.view(g, slabs, 4, 32, ka, 4).permute(0, 1, 4, 3, 2, 5).reshape(g, slabs, ka, 512)


def _from_atoms(fmt, a, rows, K):
    """The inverse of _to_atoms."""
    g, slabs, ka, _ = a.shape
    full = a.view(g, slabs, ka, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(g, slabs * 128, ka * 4)
    return full[:, :rows, :K // BLOCK[fmt]]


# -------------------------------------------------------- elementary operations
def _scale_value(fmt, byte):
    """What a scale byte stands for, in 32 bits."""
    if fmt == NV:
        return byte.view(torch.float8_e4m3fn).float()
    v = torch.exp2(byte.float() - 127.0)
    return torch.where(byte == 255, torch.full_like(v, math.nan), v)


def _quantise(fmt, x, log2):
    """bf16 [..., K] -> signed E2M1 values and scale bytes [..., K / block].

    nv: scale = E4M3(amax / (6 * 2^log2)), to nearest, at most 448;
    mx: scale = 2^ceil(log2(amax / 6)), 1 for an empty block.
    Values: x / (scale * 2^log2) to the nearest of the grid, ties to the even
    code, at most 6; zero where the scale is zero. A block that holds an infinity
    or a NaN gets the scale NaN.
    """
    b = x.float().unflatten(-1, (-1, BLOCK[fmt]))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    amax = amax.masked_fill(bad, 0.0)
    if fmt == NV:
        # (a tensor for 6: torch takes a number's reciprocal, which moves ties)
        byte = (amax * 2.0 ** -log2 / amax.new_tensor(6.0)).clamp(max=448.0)
        byte = byte.to(torch.float8_e4m3fn).view(torch.uint8)
        byte = byte.masked_fill(bad, 127)
        step = byte.masked_fill(bad, 0).view(torch.float8_e4m3fn).float() * 2.0 ** log2
    else:
        m, e = torch.frexp(amax)                        # amax = m 2^e, 1/2 <= m < 1
        code = (e - 3 + (m > 0.75).int() + 127).clamp(min=0)
        code = torch.where(amax > 0, code, torch.full_like(code, 127))
        byte = code.masked_fill(bad, 255).to(torch.uint8)
        step = torch.exp2((code - 127).float())
    step = step.unsqueeze(-1)
    # the quotient of few-bit numbers: 32 bits keep it clear of the grid's borders
    a = torch.where(step > 0, b.abs() / step, torch.zeros_like(b))
    a = torch.where(bad.unsqueeze(-1), torch.zeros_like(a), a)
    q = (0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
         + (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float())
    return torch.copysign(q, b).flatten(-2), byte


def _values(fmt, q, byte, log2):
    """What quantised values stand for, in 32 bits."""
    s = _scale_value(fmt, byte) * 2.0 ** log2
    return (q.unflatten(-1, (-1, BLOCK[fmt])) * s.unsqueeze(-1)).flatten(-2)


def _pack(q):
    """Signed E2M1 values -> codes, two to a byte."""
    a = q.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for m in GRID[1:]:
        code += (a >= m).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(codes):
    """Packed codes -> signed E2M1 values, in 32 bits."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return grid[both.int()]


def _weights(fmt, w, rows, K):
    """Packed weights with their atoms -> values in 32 bits."""
    return _values(fmt, _unpack(w["codes"]), _from_atoms(fmt, w["scales"], rows, K), 0)


# -------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1 + seed)


def _activations(rows, K, g):
    """Rows whose sizes spread as a norm's outputs do, a few channels being large."""
    x = torch.randn(rows, K, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(K, device="cuda", generator=g))
    x *= torch.exp(0.3 * torch.randn(rows, 1, device="cuda", generator=g))
    return x.bfloat16()


def _fp4_weights(fmt, groups, rows, K, g):
    """A layer's weights as they are kept: N(0, 0.02^2), quantised expert by expert
    (nv: in units of 2^-11, which the product's alpha holds)."""
    codes = torch.empty(groups, rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(groups, _up(rows, 128) // 128, _atoms(fmt, K), 512, dtype=torch.uint8,
                         device="cuda")
    for e in range(groups):
        w = (torch.randn(rows, K, device="cuda", generator=g)
             * (0.02 * 2.0 ** 11 if fmt == NV else 0.02)).bfloat16()
        q, byte = _quantise(fmt, w, 0)
        codes[e] = _pack(q)
        scales[e] = _to_atoms(fmt, byte[None], K)[0]
    return {"codes": codes, "scales": scales}


def _alpha(fmt, E, g):
    """The experts' own scales: a tensor scale each (nv), or 1."""
    one = torch.ones(E, device="cuda")
    if fmt == MX:
        return one
    return one * 2.0 ** -11 * (0.75 + 0.5 * torch.rand(E, device="cuda", generator=g))


def _routing(T, E, k, g):
    """Rows of every expert: a router's choice, uneven; segments start at multiples of 128."""
    bias = 0.5 * torch.randn(E, device="cuda", generator=g)
    score = torch.randn(T, E, device="cuda", generator=g) + bias
    idx = score.argsort(dim=1, descending=True)[:, :k]
    counts = (idx.reshape(-1, 1) == torch.arange(E, device="cuda")).sum(0)
    n = counts.tolist()
    off = [0]
    for c in n:
        off.append(off[-1] + _up(c, 128))
    R = T * k + E * 127                                  # the layer's worst case
    rows = torch.cat([torch.arange(o, o + c) for o, c in zip(off, n)]).cuda()
    return dict(R=R, n=n, off=off, rows=rows, counts=counts.int(),
                offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))


def _rows_in(R, rows, x):
    """The dispatched rows in their segments, the padding zero."""
    out = torch.zeros(R, x.shape[1], dtype=x.dtype, device="cuda")
    out[rows] = x
    return out


def prepare(case, seed):
    g = _gen(seed)
    c, fmt = case, case["fmt"]
    s = {"case": c}
    if c["op"] == "quantize":
        n = c["groups"] * c["rows"]
        x = torch.randn(n, c["K"], device="cuda", generator=g) * 0.02 if c["log2"] <= -11 \
            else _activations(n, c["K"], g)
        s["x"] = x.bfloat16().view(c["groups"], c["rows"], c["K"])
        s["q"] = _empty_fp4(fmt, c["groups"], c["rows"], c["K"])
        s["values"] = torch.empty_like(s["x"])
    elif c["op"] == "dequantize":
        s["q"] = _fp4_weights(fmt, c["groups"], c["rows"], c["K"], g)
        s["values"] = torch.empty(c["groups"], c["rows"], c["K"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "product":
        s["map"] = m = _routing(c["T"], c["E"], c["k"], g)
        x = _activations(c["T"], c["K"], g)
        s["x"] = _rows_in(m["R"], m["rows"], x[torch.randint(c["T"], (len(m["rows"]),), device="cuda", generator=g)])
        s["W"] = _fp4_weights(fmt, c["E"], c["N"], c["K"], g)
        s["alpha"] = _alpha(fmt, c["E"], g)
        s["xq"] = _empty_fp4(fmt, 1, m["R"], c["K"])
        s["y"] = torch.zeros(m["R"], c["N"], dtype=torch.bfloat16, device="cuda")
    else:
        H, F = c["H"], c["F"]
        s["map"] = m = _routing(c["T"], c["E"], c["k"], g)
        s["W13"] = _fp4_weights(fmt, c["E"], 2 * F, H, g)
        s["W2"] = _fp4_weights(fmt, c["E"], H, F, g)
        s["alpha13"], s["alpha2"] = _alpha(fmt, c["E"], g), _alpha(fmt, c["E"], g)
        x = _activations(c["T"], H, g)
        x = x[torch.randint(c["T"], (len(m["rows"]),), device="cuda", generator=g)]
        s["x"] = _rows_in(m["R"], m["rows"], x)          # dO's rows, in the backward
        s["y"] = torch.zeros(m["R"], H, dtype=torch.bfloat16, device="cuda")
        if c["op"] == "ffn_bwd":
            gu = (1.5 * torch.randn(len(m["rows"]), 2 * F, device="cuda", generator=g)).bfloat16()
            code, byte = _checkpoint(gu)
            s["ckpt"] = _rows_in(m["R"], m["rows"], code.view(torch.uint8))
            s["ckpt_scale"] = _rows_in(m["R"], m["rows"], byte)
        elif c["ckpt"]:
            s["ckpt"] = torch.zeros(m["R"], 2 * F, dtype=torch.uint8, device="cuda")
            s["ckpt_scale"] = torch.zeros(m["R"], 2 * F // 32, dtype=torch.uint8, device="cuda")
    if "map" in s:
        s["scratch"] = torch.zeros(_scratch_bytes(c, s["map"]["R"]), dtype=torch.uint8, device="cuda")
    return s


def _empty_fp4(fmt, groups, rows, K):
    return {"codes": torch.zeros(groups, rows, K // 2, dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros(groups, _up(rows, 128) // 128, _atoms(fmt, K), 512,
                                  dtype=torch.uint8, device="cuda")}


def _scratch_bytes(c, R):
    """What a caller sets aside for a call, generously: room for sums in parts, and for an
    FFN the rows in 4 bits or (backward) the weights and two row tensors in bf16."""
    n = 20 << 20
    if c["op"] not in ("ffn", "ffn_bwd"):
        return n
    H, F, E = c["H"], c["F"], c["E"]
    n += _up(R, 128) * (_up(H, 256) + _up(F, 256))
    if c["op"] == "ffn_bwd":
        n += 6 * E * H * F + 8 * R * F + (1 << 16)
    return n


# ------------------------------------------------------------------ the plain form
def _checkpoint(gu):
    """bf16 [rows, 2F] -> E4M3 codes and a power-of-two scale byte per 32 values."""
    b = gu.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                            # amax / 448 = m / 0.875 2^(e - 9)
    code = (e - 9 + (m > 0.875).int() + 127).clamp(min=0)
    code = torch.where(amax > 0, code, torch.full_like(code, 127))
    v = b * torch.exp2(127.0 - code.float()).unsqueeze(-1)
    return v.to(torch.float8_e4m3fn).flatten(-2), code.to(torch.uint8)


def _of_checkpoint(codes, byte):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (v * torch.exp2(byte.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _padded(m):
    """The experts that have rows, and where their rows lie in a [experts, most rows] array."""
    live = [e for e, c in enumerate(m["n"]) if c]
    e = torch.tensor(live, device="cuda")
    most = max(m["n"])
    c = torch.tensor([m["n"][i] for i in live], device="cuda")
    start = torch.tensor([m["off"][i] for i in live], device="cuda")
    at = torch.arange(most, device="cuda")
    return e, (start[:, None] + at).clamp(max=m["R"] - 1), at < c[:, None]


def _pick(w, e):
    return {"codes": w["codes"][e], "scales": w["scales"][e]}


def _plain_product(x, w, alpha):
    """[experts, rows, K] by [experts, N, K], each expert's product by its alpha."""
    return torch.bmm(x, w.transpose(1, 2)) * alpha[:, None, None]


def _plain_ffn(s, c, fmt):
    m, H, F = s["map"], c["H"], c["F"]
    e, at, ok = _padded(m)
    x = _values(fmt, *_quantise(fmt, s["x"][at], 0), 0)
    gu = _plain_product(x, _weights(fmt, _pick(s["W13"], e), 2 * F, H), s["alpha13"][e]).bfloat16()
    g, u = gu.float().split(F, -1)
    h = (g / (1.0 + torch.exp(-g)) * u).bfloat16()
    y = _plain_product(_values(fmt, *_quantise(fmt, h, 0), 0),
                       _weights(fmt, _pick(s["W2"], e), H, F), s["alpha2"][e]).bfloat16()
    out = {"y": torch.zeros_like(s["y"])}
    out["y"][at[ok]] = y[ok]
    if c["ckpt"]:
        code, byte = _checkpoint(gu[ok])
        out["ckpt"], out["ckpt_scale"] = torch.zeros_like(s["ckpt"]), torch.zeros_like(s["ckpt_scale"])
        out["ckpt"][at[ok]], out["ckpt_scale"][at[ok]] = code.view(torch.uint8), byte
        out["ckpt"] = out["ckpt"].view(torch.float8_e4m3fn)
        out["ckpt_scale"] = out["ckpt_scale"].view(torch.float8_e8m0fnu)
    return out


def _plain_ffn_bwd(s, c, fmt):
    m, H, F = s["map"], c["H"], c["F"]
    e, at, ok = _padded(m)
    dO = s["x"][at].float()
    dh = torch.bmm(dO, _weights(fmt, _pick(s["W2"], e), H, F)) * s["alpha2"][e, None, None]
    g, u = _of_checkpoint(s["ckpt"][at], s["ckpt_scale"][at]).split(F, -1)
    sg = 1.0 / (1.0 + torch.exp(-g))
    dgu = torch.cat((dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg), -1)
    dx = torch.bmm(dgu, _weights(fmt, _pick(s["W13"], e), 2 * F, H)) * s["alpha13"][e, None, None]
    out = torch.zeros_like(s["y"])
    out[at[ok]] = dx[ok].bfloat16()
    return out


def _run_plain(s):
    c, fmt = s["case"], s["case"]["fmt"]
    if c["op"] == "quantize":
        return _values(fmt, *_quantise(fmt, s["x"], c["log2"]), c["log2"]).bfloat16()
    if c["op"] == "dequantize":
        q = s["q"]
        return _values(fmt, _unpack(q["codes"]), _from_atoms(fmt, q["scales"], c["rows"], c["K"]),
                       c["log2"]).bfloat16()
    if c["op"] == "product":
        e, at, ok = _padded(s["map"])
        x = _values(fmt, *_quantise(fmt, s["x"][at], 0), 0)
        y = _plain_product(x, _weights(fmt, _pick(s["W"], e), c["N"], c["K"]), s["alpha"][e])
        out = torch.zeros_like(s["y"])
        out[at[ok]] = y[ok].bfloat16()
        return out
    return _plain_ffn(s, c, fmt) if c["op"] == "ffn" else _plain_ffn_bwd(s, c, fmt)


# ----------------------------------------------------------- the framework's calls
def _run_own(s):
    import routing_dispatch_expert_router_gb300.binding as B
    c = s["case"]
    fmt = B.MOE_FP4_NV if c["fmt"] == NV else B.MOE_FP4_MX

    def fp4(t, K):
        return B.Fp4Tensor(fmt, K, t["codes"], t["scales"])

    if c["op"] == "quantize":
        B.moe_fp4_quantize(s["x"], fp4(s["q"], c["K"]), scale_log2=c["log2"], values=s["values"])
        return s["values"]
    if c["op"] == "dequantize":
        B.moe_fp4_dequantize(fp4(s["q"], c["K"]), s["values"], scale_log2=c["log2"])
        return s["values"]
    m = s["map"]
    if c["op"] == "product":
        xq = fp4(s["xq"], c["K"])
        B.moe_fp4_quantize(s["x"][None], xq, counts=m["counts"], offsets=m["offsets"],
                           scratch=s["scratch"])
        B.moe_fp4_grouped_gemm(xq, fp4(s["W"], c["K"]), m["counts"], m["offsets"], s["alpha"],
                               s["y"], s["scratch"])
        return s["y"]
    cfg = B.MoEConfig(T=c["T"], H=c["H"], E=c["E"], k=c["k"], F=c["F"], n_groups=1, topk_groups=1,
                      route_scale=1.0, row_align=128)
    ex = B.fp4_experts(fp4(s["W13"], c["H"]), fp4(s["W2"], c["F"]), s["alpha13"], s["alpha2"])
    if c["op"] == "ffn":
        B.moe_fp4_ffn_fwd(cfg, ex, s["x"], m["counts"], m["offsets"], s.get("ckpt"),
                          s.get("ckpt_scale"), s["y"], s["scratch"])
        out = {"y": s["y"]}
        if c["ckpt"]:
            out["ckpt"] = s["ckpt"].view(torch.float8_e4m3fn)
            out["ckpt_scale"] = s["ckpt_scale"].view(torch.float8_e8m0fnu)
        return out
    B.moe_fp4_ffn_bwd(cfg, ex, s["x"], s["ckpt"], s["ckpt_scale"], m["counts"], m["offsets"],
                      None, None, None, s["y"], s["scratch"])
    return s["y"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------- what a pass cannot do without
def _live(T, E, k):
    """Experts with a row, expected for an even router: a count that needs no data."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    c = case
    bits = 0.5 + 1.0 / BLOCK[c["fmt"]]                   # bytes of an element in 4 bits
    if c["op"] in ("quantize", "dequantize"):
        n = c["groups"] * c["rows"] * c["K"]
        # codes and scales one way, bf16 in and (quantize) the bf16 values out
        return {"bytes": n * (bits + (4 if c["op"] == "quantize" else 2)), "flops": 0}
    rows, live = c["T"] * c["k"], _live(c["T"], c["E"], c["k"])
    if c["op"] == "product":
        return {"bytes": live * c["N"] * c["K"] * bits + rows * 2 * (c["K"] + c["N"]),
                "flops": 2.0 * rows * c["N"] * c["K"]}
    HF = c["H"] * c["F"]
    kept = 2 * c["F"] * (1 + 1 / 32) if c["op"] == "ffn_bwd" or c["ckpt"] else 0
    return {"bytes": live * 3 * HF * bits + rows * (4 * c["H"] + kept), "flops": 6.0 * rows * HF}


# ------------------------------------------------------------ the definition, in 64 bits
def _nearest64(v, grid):
    """The element of an ascending grid nearest to v >= 0, the even index on a tie."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = (grid[hi] - v).abs(), (v - grid[lo]).abs()
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, grid[hi], grid[lo])


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                                                for m in range(8) if e < 15 or m < 7]


def _real64(fmt, x, log2=0):
    """The values that quantised rows stand for."""
    n = BLOCK[fmt]
    b = x.double().reshape(-1, n)
    top = b.abs().max(dim=1, keepdim=True).values
    top = top / torch.full_like(top, 6.0)
    if fmt == NV:
        unit = _nearest64((top / 2.0 ** log2).clamp(max=448), _e4m3_grid()) * 2.0 ** log2
    else:
        up = torch.frexp(top).exponent.double()          # 2^(up - 1) <= top < 2^up
        unit = torch.where(top == torch.exp2(up - 1), torch.exp2(up - 1), torch.exp2(up))
        unit = torch.where(top > 0, unit, torch.ones_like(top)).clamp(min=2.0 ** -127)
    safe = torch.where(unit > 0, unit, torch.ones_like(unit))
    v = _nearest64((b.abs() / safe).clamp(max=6.0), GRID) * unit
    return (torch.sign(b) * v).reshape(x.shape)


def _kept64(fmt, codes, atoms, K):
    """One expert's weights: every code's value times its block's scale, by index."""
    rows = codes.shape[0]
    n = BLOCK[fmt]
    k = torch.arange(K, device="cuda")
    nib = (codes[:, k // 2].int() >> (4 * (k % 2))) & 15
    mag = torch.tensor(GRID, dtype=torch.float64, device="cuda")[nib & 7] * (1 - 2 * (nib >> 3))
    r, b = torch.arange(rows, device="cuda")[:, None], (k // n)[None, ::n]
    byte = atoms[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].long()
    if fmt == NV:
        table = torch.tensor(_e4m3_grid() + [math.nan], dtype=torch.float64, device="cuda")
    else:
        table = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan],
                             dtype=torch.float64, device="cuda")
    return mag * table[byte].repeat_interleave(n, dim=1)


def exact(case, seed):
    c, fmt = case, case["fmt"]
    w = work(c)
    if w["flops"] > 4e12 or (w["flops"] == 0 and w["bytes"] > 3e9):
        return None
    s = prepare(case, seed)
    if c["op"] == "quantize":
        return _real64(fmt, s["x"], c["log2"])
    if c["op"] == "dequantize":
        q = s["q"]
        return torch.stack([_kept64(fmt, q["codes"][e], q["scales"][e], c["K"]) * 2.0 ** c["log2"]
                            for e in range(c["groups"])])
    m = s["map"]
    out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for e, n in enumerate(m["n"]):
        if n == 0:
            continue
        r = slice(m["off"][e], m["off"][e] + n)
        if c["op"] == "product":
            W = _kept64(fmt, s["W"]["codes"][e], s["W"]["scales"][e], c["K"])
            out[r] = _real64(fmt, s["x"][r]) @ W.T * s["alpha"][e].double()
            continue
        H, F = c["H"], c["F"]
        W13 = _kept64(fmt, s["W13"]["codes"][e], s["W13"]["scales"][e], H) * s["alpha13"][e].double()
        W2 = _kept64(fmt, s["W2"]["codes"][e], s["W2"]["scales"][e], F) * s["alpha2"][e].double()
        if c["op"] == "ffn":
            # the gate and up values and h are defined as bf16 numbers
            gu = (_real64(fmt, s["x"][r]) @ W13.T).bfloat16().double()
            h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            out[r] = _real64(fmt, h.bfloat16()) @ W2.T
        else:
            sc = torch.exp2(s["ckpt_scale"][r].double() - 127).repeat_interleave(32, dim=1)
            gu = s["ckpt"][r].view(torch.float8_e4m3fn).double() * sc
            g, u = gu[:, :F], gu[:, F:]
            dh = s["x"][r].double() @ W2
            sig = torch.sigmoid(g)
            d = torch.cat((dh * u * (sig + g * sig * (1 - sig)), dh * g * sig), dim=1)
            out[r] = d @ W13
    if c["op"] == "ffn":
        # the checkpoint's codes have no value between two of theirs
        return {"y": out, "ckpt": None, "ckpt_scale": None} if c["ckpt"] else {"y": out}
    return out
