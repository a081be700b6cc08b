"""The operators around and inside experts of free form, as cases that can be timed and checked.

  norm_fwd    h = bf16(x + residual), y = bf16(h * rstd * gamma), and where the
              caller asks for it y in E4M3 with a power-of-two scale per block;
  norm_bwd    the gradients at x (and at the residual, the same) and at gamma;
  dispatch    rows in E4M3, with their scales, copied into the experts' segments
              with the maps of the dispatch;
  gemm        y[r] = x[r] w[g]^T (+ what is there to add) for the rows r of every
              group g, rows of one group following the other's without padding;
  gemm_dgrad  dx[r] = dy[r] w[g] (+ ...);
  gemm_wgrad  dw[g] = sum over the group's rows of dy[r]^T x[r];
  int4        y[r] = x[r] w4[g]^T with the experts' weights in 4-bit integers,
              w = scale * (code - zero) with a scale (and a zero point) for
              `group` consecutive elements along K; or h = silu(gate) * up of
              such a product, whose first half of columns is the gate.

`run` computes a case in elementary torch operations where `own` is false and
through the framework's entry points where it is true; `prepare` does not depend
on it.
"""
import math

import torch

own = False

EPS = 1e-6
SCRATCH = 32 << 20                           # what a caller sets aside for a product


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token between two layers, the smallest call: latency
        dict(name="norm_one_token", op="norm_fwd", T=1, H=4096, residual=True, gamma="bf16", block=0),
        # a long prompt in front of a layer with MXFP8 experts: bf16 for the router, 8 bits for them
        dict(name="norm_prompt_mx", op="norm_fwd", T=8192, H=7168, residual=True, gamma="bf16", block=32),
        # a training batch's backward, the residual's gradient coming in beside the norm's
        dict(name="norm_bwd_train", op="norm_bwd", T=8191, H=4096, residual=True, gamma="f32"),
        # a decoding batch into MXFP8 experts, nothing dropped, many experts without a row
        dict(name="dispatch_decode", op="dispatch", T=61, H=4096, E=128, k=8, block=32, cf=0.0),
        # a long prompt into FP8 experts with a capacity limit
        dict(name="dispatch_prompt", op="dispatch", T=8192, H=7168, E=256, k=8, block=128, cf=1.25),
        # the second half of low-rank adapters, added to what the experts gave
        dict(name="gemm_adapter", op="gemm", T=4096, E=8, k=2, N=4096, K=16, add=True),
        # a few decoded tokens through bf16 experts: every byte read is a weight
        dict(name="gemm_few_rows", op="gemm", T=4, E=8, k=2, N=4096, K=14336, add=False),
        # a training batch through many experts of odd width: data gradient
        dict(name="gemm_dgrad_train", op="gemm_dgrad", T=4096, E=64, k=8, N=4096, K=2040, add=False),
        # and weight gradient
        dict(name="gemm_wgrad_train", op="gemm_wgrad", T=4096, E=64, k=8, N=4096, K=2040),
        # one token through the gate and up weights of eight large experts
        dict(name="int4_one_token", op="int4", T=1, E=8, k=2, N=28672, K=4096, group=128, zeros=False, swiglu=True),
        # a decoding batch over many small experts: nearly all of the weights, few rows each
        dict(name="int4_decode_batch", op="int4", T=64, E=64, k=8, N=4096, K=2048, group=128, zeros=True, swiglu=False),
        # odd sizes, small groups, some experts without a row
        dict(name="int4_odd", op="int4", T=19, E=11, k=2, N=1008, K=1504, group=32, zeros=True, swiglu=False),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _experts(rng, most):
    E = rng.choice([e for e in (1, 4, 8, 11, 32, 64, 128, 256) if e <= most])
    return E, rng.choice([x for x in (1, 2, 4, 8) if x <= E])


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "dispatch", "gemm", "gemm_dgrad", "gemm_wgrad", "int4"])
    while True:
        if op in ("norm_fwd", "norm_bwd"):
            block = rng.choice([0, 32, 128]) if op == "norm_fwd" else 0
            unit = max(block, 8)
            T, H = _between(rng, 1, 8192), unit * _between(rng, max(1, 64 // unit), 16384 // unit)
            if T * H <= 8192 * 7168:
                case = dict(op=op, T=T, H=H, residual=rng.random() < 0.7, gamma=rng.choice(["bf16", "f32"]))
                return {**case, "block": block} if op == "norm_fwd" else case
        elif op == "dispatch":
            E, k = _experts(rng, 256)
            T, H = _between(rng, 1, 8192), 256 * _between(rng, 1, 28)
            if T * k * H <= 8192 * 8 * 7168:
                return dict(op=op, T=T, H=H, E=E, k=k, block=rng.choice([32, 128]),
                            cf=rng.choice([0.0, 1.25]))
        elif op == "int4":
            E, k = _experts(rng, 64)
            T, group = _between(rng, 1, 64), rng.choice([32, 64, 128])
            N, K = 16 * _between(rng, 4, 1792), group * _between(rng, 1, 14336 // group)
            if E * N * K <= 8 * 28672 * 4096:
                return dict(op=op, T=T, E=E, k=k, N=N, K=K, group=group, zeros=rng.random() < 0.5,
                            swiglu=N % 32 == 0 and rng.random() < 0.5)
        else:
            E, k = _experts(rng, 64)
            T = _between(rng, 1, 4096)
            N, K = 8 * _between(rng, 2, 1792), 8 * _between(rng, 2, 1792)
            if E * N * K <= 64 * 4096 * 2040 and T * k * N * K <= 4096 * 8 * 4096 * 2040:
                case = dict(op=op, T=T, E=E, k=k, N=N, K=K)
                return case if op == "gemm_wgrad" else {**case, "add": rng.random() < 0.3}


# -------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1 + seed)


def _randn(*shape, g):
    return torch.randn(*shape, device="cuda", generator=g)


def _activations(rows, K, g):
    """Rows whose sizes spread as a layer's do, a few channels being large."""
    x = _randn(rows, K, g=g)
    x *= torch.exp(0.5 * _randn(K, g=g))
    x *= torch.exp(0.3 * _randn(rows, 1, g=g))
    return x.bfloat16()


def _up(a, b):
    return -(-a // b) * b


def _choice(T, E, k, g):
    """A router's choice, uneven: every token's k experts, best first."""
    bias = 0.5 * _randn(E, g=g)
    return (_randn(T, E, g=g) + bias).argsort(dim=1, descending=True)[:, :k]


def _segments(c, g, align):
    """Rows of every expert; segments begin at multiples of `align` and some rows behind the
    last belong to none."""
    idx = _choice(c["T"], c["E"], c["k"], g)
    n = (idx.reshape(-1, 1) == torch.arange(c["E"], device="cuda")).sum(0).tolist()
    off = [0]
    for rows in n:
        off.append(off[-1] + _up(rows, align))
    R = c["T"] * c["k"] + c["E"] * (align - 1) + 5
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(R=R, n=n, off=off, counts=torch.tensor(n, **i32), offsets=torch.tensor(off, **i32))


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = {"case": c}
    bf = dict(dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    if op in ("norm_fwd", "norm_bwd"):
        T, H = c["T"], c["H"]
        gamma = 1.0 + 0.2 * _randn(H, g=g)
        s["gamma"] = gamma.bfloat16() if c["gamma"] == "bf16" else gamma
        if op == "norm_fwd":
            s["x"] = _activations(T, H, g)
            s["y"], s["rstd"] = torch.empty(T, H, **bf), torch.empty(T, **f32)
            if c["residual"]:
                s["residual"], s["sum"] = (3.0 * _randn(T, H, g=g)).bfloat16(), torch.empty(T, H, **bf)
            if c["block"]:
                s["codes"] = torch.empty(T, H, **u8)
                s["scales"] = torch.empty(T, H // c["block"], **u8)
        else:
            s["dy"], s["h"] = _randn(T, H, g=g).bfloat16(), _activations(T, H, g)
            s["rstd"] = 1.0 / torch.sqrt(s["h"].float().square().mean(1) + EPS)
            if c["residual"]:
                s["dsum"] = _randn(T, H, g=g).bfloat16()
            s["dx"], s["dgamma"] = torch.empty(T, H, **bf), torch.empty(H, **f32)
            s["scratch"] = torch.zeros(4096 + 512 * H * 4, **u8)
    elif op == "dispatch":
        T, H, E, k, n = c["T"], c["H"], c["E"], c["k"], c["block"]
        x = _activations(T, H, g).float().unflatten(-1, (-1, n))
        byte = _scale_byte(x.abs().amax(-1))
        s["codes"] = _codes(x, byte)
        s["scales"] = byte
        s["idx"] = _choice(T, E, k, g).int().contiguous()
        R = _rows(c)
        atoms = H // 128 if n == 32 else -(-H // 512)
        for name, size in (("counts", E), ("offsets", E + 1), ("row_of", T * k), ("token_of", R),
                           ("sel_offsets", E + 1), ("sel_tokens", T * k)):
            s[name] = torch.empty(size, **i32)
        s["token_of"].fill_(-1)
        s["xq"], s["xsf"] = torch.zeros(R, H, **u8), torch.zeros(_up(R, 128) // 128, atoms, 512, **u8)
        s["scratch"] = torch.zeros(1 << 20, **u8)
    elif op == "int4":
        E, N, K, n = c["E"], c["N"], c["K"], c["group"]
        s["map"] = m = _segments(c, g, 128)
        s["x"] = _activations(m["R"], K, g)
        s["codes"] = torch.empty(E, N, K // 2, **u8)
        for e in range(E):
            q = (8 + 2.5 * _randn(N, K, g=g)).round().clamp(0, 15).to(torch.uint8)
            s["codes"][e] = q[:, 0::2] | (q[:, 1::2] << 4)
        s["scales"] = (0.008 * (0.5 + torch.rand(E, K // n, N, device="cuda", generator=g))).bfloat16()
        s["zeros"] = torch.randint(6, 11, (E, K // n, N), generator=g, **u8) if c["zeros"] else None
        s["y"] = torch.zeros(m["R"], N // 2 if c["swiglu"] else N, **bf)
        s["scratch"] = torch.zeros(SCRATCH, **u8)
    else:
        E, N, K = c["E"], c["N"], c["K"]
        s["map"] = m = _segments(c, g, 1)
        if op != "gemm_dgrad":
            s["x"] = _activations(m["R"], K, g)
        if op != "gemm":
            s["dy"] = _randn(m["R"], N, g=g).bfloat16()
        if op == "gemm_wgrad":
            s["out"] = torch.empty(E, N, K, **bf)
        else:
            s["w"] = torch.empty(E, N, K, **bf)
            for e in range(E):
                s["w"][e] = _randn(N, K, g=g) * 0.02
            cols = N if op == "gemm" else K
            s["add"] = _randn(m["R"], cols, g=g).bfloat16() if c["add"] else None
            s["out"] = torch.zeros(m["R"], cols, **bf)
        s["scratch"] = torch.zeros(SCRATCH, **u8)
    return s


# ------------------------------------------------------------------ the plain form
def _scale_byte(amax):
    """The byte of 2^ceil(log2(amax / 448)), a bias of 127; 1 for an empty block."""
    m, e = torch.frexp(amax)                            # amax / 448 = m / 0.875 2^(e - 9)
    code = (e - 9 + (m > 0.875).int() + 127).clamp(min=0)
    return torch.where(amax > 0, code, torch.full_like(code, 127)).to(torch.uint8)


def _codes(blocks, byte):
    """E4M3 codes of blocks [.., block] over their scales."""
    v = blocks * torch.exp2(127.0 - byte.float()).unsqueeze(-1)
    return v.to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)


def _values8(out):
    """Codes and scale bytes as the numbers that they stand for."""
    return {**out, "codes": out["codes"].view(torch.float8_e4m3fn),
            "scales": out["scales"].view(torch.float8_e8m0fnu)}


def _plain_norm_fwd(s, c):
    h = s["x"]
    out = {}
    if c["residual"]:
        h = out["sum"] = (h.float() + s["residual"].float()).bfloat16()
    f = h.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + EPS)
    out["y"] = y = (f * rstd[:, None] * s["gamma"].float()).bfloat16()
    out["rstd"] = rstd
    if c["block"]:
        b = y.float().unflatten(-1, (-1, c["block"]))
        out["scales"] = _scale_byte(b.abs().amax(-1))
        out["codes"] = _codes(b, out["scales"])
        return _values8(out)
    return out


def _plain_norm_bwd(s, c):
    h, r = s["h"].float(), s["rstd"][:, None]
    dy = s["dy"].float()
    n = h * r
    t = dy * s["gamma"].float()
    dx = (t - n * (t * n).mean(1, keepdim=True)) * r
    if c["residual"]:
        dx = dx + s["dsum"].float()
    return {"dx": dx.bfloat16(), "dgamma": (dy * n).sum(0)}


def _capacity(c):
    """Rows that an expert keeps; 0 without a limit."""
    return _up(math.ceil(c["cf"] * c["T"] * c["k"] / c["E"]), 128) if c["cf"] else 0


def _rows(c):
    return c["E"] * _capacity(c) if c["cf"] else c["T"] * c["k"] + c["E"] * 127


def _plain_dispatch(s, c):
    T, H, E, k, C, R = c["T"], c["H"], c["E"], c["k"], _capacity(c), _rows(c)
    e = s["idx"].reshape(-1).long()
    order = torch.argsort(e, stable=True)               # by expert, then by token
    total = (e[None] == torch.arange(E, device="cuda")[:, None]).sum(1)
    first = total.cumsum(0) - total
    rank = torch.empty_like(e)
    rank[order] = torch.arange(T * k, device="cuda") - first[e[order]]
    kept = total.clamp(max=C) if C else total
    size = torch.full_like(total, C) if C else (total + 127) // 128 * 128
    start = size.cumsum(0) - size
    row = start[e] + rank
    if C:
        row = torch.where(rank < C, row, torch.full_like(row, -1))
    live = (row >= 0).nonzero()[:, 0]
    token_of = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    token_of[row[live]] = (live // k).int()
    xq, xsf = torch.zeros_like(s["xq"]), torch.zeros_like(s["xsf"])
    xq[row[live]] = s["codes"][live // k]
    # scales: atoms of 128 rows (rows without a token are left as they were)
    n = H // c["block"]
    byte = torch.zeros(_up(R, 128), n, dtype=torch.uint8, device="cuda")
    byte[row[live]] = s["scales"][live // k]
    full = byte.new_zeros(byte.shape[0], xsf.shape[1] * 4)
    full[:, :n] = byte
    xsf = full.view(-1, 4, 32, xsf.shape[1], 4).permute(0, 3, 2, 1, 4).reshape(xsf.shape)
    out = {"codes": xq, "scales": xsf, "counts": kept.int(), "row_of": row.int(),
           "offsets": torch.cat((start, start[-1:] + size[-1:])).int(), "token_of": token_of}
    return _values8(out)


def _padded(m):
    """The groups that have rows, and where their rows lie in a [groups, most rows] array."""
    live = [e for e, n in enumerate(m["n"]) if n]
    e = torch.tensor(live, device="cuda")
    n = torch.tensor([m["n"][i] for i in live], device="cuda")
    start = torch.tensor([m["off"][i] for i in live], device="cuda")
    at = torch.arange(max(m["n"]), device="cuda")
    return e, (start[:, None] + at).clamp(max=m["R"] - 1), at < n[:, None]


def _int4_weights(s, e):
    """The weights of the experts e, [experts, N, K] in 32 bits."""
    q = s["codes"][e]
    q = torch.stack((q & 15, q >> 4), -1).flatten(-2).float()
    n = q.shape[2] // s["scales"].shape[1]
    z = s["zeros"][e].transpose(1, 2).float() if s["zeros"] is not None else torch.full((1, 1, 1), 8.0, device="cuda")
    q = q.unflatten(-1, (-1, n)) - z.unsqueeze(-1)
    return (q * s["scales"][e].transpose(1, 2).float().unsqueeze(-1)).flatten(-2)


def _plain_gemm(s, c):
    op, m = c["op"], s["map"]
    e, at, ok = _padded(m)
    if op == "gemm_wgrad":
        dy = s["dy"][at].float() * ok[..., None]
        out = torch.zeros_like(s["out"])
        out[e] = torch.bmm(dy.transpose(1, 2), s["x"][at].float()).bfloat16()
        return out
    a, w = (s["x"], s["w"][e].float().transpose(1, 2)) if op == "gemm" else (s["dy"], s["w"][e].float())
    y = torch.bmm(a[at].float(), w)
    if c["add"]:
        y += s["add"][at].float()
    out = torch.zeros_like(s["out"])
    out[at[ok]] = y[ok].bfloat16()
    return out


def _plain_int4(s, c):
    e, at, ok = _padded(s["map"])
    y = torch.bmm(s["x"][at].float(), _int4_weights(s, e).transpose(1, 2))
    if c["swiglu"]:
        gate, up = y.split(c["N"] // 2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    out = torch.zeros_like(s["y"])
    out[at[ok]] = y[ok].bfloat16()
    return out


def _run_plain(s):
    c = s["case"]
    plain = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "dispatch": _plain_dispatch,
             "int4": _plain_int4}
    return plain.get(c["op"], _plain_gemm)(s, c)


# ----------------------------------------------------------- the framework's calls
def _run_own(s):
    import routing_dispatch_expert_router_gb300.binding as B
    c = s["case"]
    op, m = c["op"], s.get("map")
    if op == "norm_fwd":
        B.moe_rmsnorm_fwd(s["x"], s["gamma"], s["y"], residual=s.get("residual"), sum=s.get("sum"),
                          rstd=s["rstd"], codes=s.get("codes"), scales=s.get("scales"), eps=EPS)
        out = {"y": s["y"], "rstd": s["rstd"]}
        if c["residual"]:
            out["sum"] = s["sum"]
        return _values8({**out, "codes": s["codes"], "scales": s["scales"]}) if c["block"] else out
    if op == "norm_bwd":
        B.moe_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["gamma"], s["dx"], s["dgamma"],
                          dsum=s.get("dsum"), scratch=s["scratch"])
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if op == "dispatch":
        cfg = B.MoEConfig(T=c["T"], H=c["H"], E=c["E"], k=c["k"], F=256, n_groups=1, topk_groups=1,
                          route_scale=1.0, capacity_factor=c["cf"], row_align=128,
                          dtype=2 if c["block"] == 32 else 1)
        B.moe_permute_fp8(cfg, s["codes"], s["scales"], s["idx"], s["counts"], s["offsets"],
                          s["row_of"], s["token_of"], s["sel_offsets"], s["sel_tokens"], s["scratch"],
                          codes_perm=s["xq"], scales_perm=s["xsf"])
        return _values8({"codes": s["xq"], "scales": s["xsf"], "counts": s["counts"],
                         "row_of": s["row_of"], "offsets": s["offsets"], "token_of": s["token_of"]})
    if op == "int4":
        W = B.Int4Tensor(s["codes"], s["scales"], s["zeros"])
        B.moe_int4_grouped_gemm(s["x"], W, m["counts"], m["offsets"], s["y"], s["scratch"],
                                swiglu=c["swiglu"])
        return s["y"]
    if op == "gemm":
        B.moe_grouped_gemm(s["x"], s["w"], m["counts"], m["offsets"], s["out"], s["scratch"],
                           add=s["add"], expected_rows=c["T"])
    elif op == "gemm_dgrad":
        B.moe_grouped_gemm_dgrad(s["dy"], s["w"], m["counts"], m["offsets"], s["out"], s["scratch"],
                                 add=s["add"])
    else:
        B.moe_grouped_gemm_wgrad(s["dy"], s["x"], m["counts"], m["offsets"], s["out"], s["scratch"])
    return s["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------- what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "norm_fwd":
        n = c["T"] * c["H"]
        return {"bytes": n * ((8 if c["residual"] else 4) + (1 + 1 / c["block"] if c["block"] else 0)),
                "flops": 4 * n}
    if op == "norm_bwd":
        n = c["T"] * c["H"]
        return {"bytes": n * (8 if c["residual"] else 6), "flops": 8 * n}
    if op == "dispatch":
        rows = c["T"] * c["k"]
        if c["cf"]:
            rows = min(rows, _rows(c))
        return {"bytes": (c["T"] + rows) * c["H"] * (1 + 1 / c["block"]) + 12 * c["T"] * c["k"], "flops": 0}
    rows, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
    live = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])      # groups with a row, for an even router
    flops = 2.0 * rows * N * K
    if op == "int4":
        weights = live * N * K * (0.5 + (3 if c["zeros"] else 2) / c["group"])
        return {"bytes": weights + 2 * rows * (K + (N // 2 if c["swiglu"] else N)), "flops": flops}
    if op == "gemm_wgrad":
        return {"bytes": 2 * (E * N * K + rows * (N + K)), "flops": flops}
    add = (N if op == "gemm" else K) if c["add"] else 0
    return {"bytes": 2 * (live * N * K + rows * (N + K + add)), "flops": flops}


# ------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    c, op = case, case["op"]
    if op == "dispatch" or (op != "norm_fwd" and work(c)["flops"] > 4e12):
        return None                                      # (a dispatch moves codes)
    s = prepare(case, seed)
    if op == "norm_fwd":
        h = s["x"].double()
        out = {}
        if c["residual"]:
            out["sum"] = h + s["residual"].double()
            h = out["sum"].bfloat16().double()           # the stream is held in bf16, and normed so
        out["rstd"] = (h.pow(2).sum(1) / c["H"] + EPS).pow(-0.5)
        out["y"] = h * s["gamma"].double() * out["rstd"].unsqueeze(1)
        if c["block"]:
            out["codes"] = out["scales"] = None          # no value between two of theirs
        return out
    if op == "norm_bwd":
        h, dy, ga, r = s["h"].double(), s["dy"].double(), s["gamma"].double(), s["rstd"].double()
        r = r.unsqueeze(1)
        dot = (dy * ga * h).sum(1, keepdim=True)
        dx = r * dy * ga - r.pow(3) * h * dot / c["H"]
        if c["residual"]:
            dx = s["dsum"].double() + dx
        return {"dx": dx, "dgamma": torch.einsum("th,th->h", dy, h * r)}
    m = s["map"]
    out = torch.zeros((s["y"] if op == "int4" else s["out"]).shape, dtype=torch.float64, device="cuda")
    for e, n in enumerate(m["n"]):
        if n == 0:
            continue
        r = slice(m["off"][e], m["off"][e] + n)
        if op == "gemm_wgrad":
            out[e] = s["dy"][r].double().T @ s["x"][r].double()
            continue
        if op == "gemm":
            out[r] = s["x"][r].double() @ s["w"][e].double().T
        elif op == "gemm_dgrad":
            out[r] = s["dy"][r].double() @ s["w"][e].double()
        else:
            k = torch.arange(c["K"], device="cuda")
            code = (s["codes"][e][:, k // 2].int() >> (4 * (k % 2))) & 15
            zero = s["zeros"][e][k // c["group"]].T.int() if c["zeros"] else 8
            w = (code - zero).double() * s["scales"][e][k // c["group"]].T.double()
            y = s["x"][r].double() @ w.T
            if c["swiglu"]:
                half = c["N"] // 2
                y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
            out[r] = y
        if op != "int4" and c["add"]:
            out[r] += s["add"][r].double()
    return out
