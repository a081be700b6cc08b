"""Thin ctypes binding of libmoe_gb300.so: argument marshalling only.

Every function here has the name of the C entry point it calls and takes
torch tensors (device memory) where the C call takes device pointers. There is
no compute in Python and no fallback: if the library is missing, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from .build import LIB_PATH

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
                6: "MOE_ERR_DEVICE_CHECK", 7: "MOE_ERR_STASH_FULL"}

# every exported entry point of include/moe_abi.h
ENTRY_POINTS = (
    "moe_query_sizes", "moe_route", "moe_route_replay", "moe_route_aux", "moe_route_aux_bwd",
    "moe_permute", "moe_permute_noalloc", "moe_permute_noalloc_status",
    "moe_quantize_weights", "moe_load_fp8_weights", "moe_grouped_ffn_fwd", "moe_unpermute",
    "moe_unpermute_bwd", "moe_grouped_ffn_dgrad", "moe_grouped_ffn_wgrad", "moe_grouped_ffn_bwd",
    "moe_grouped_ffn_fwd_reordered", "moe_unpermute_bwd_reordered",
    "moe_grouped_ffn_dgrad_reordered", "moe_route_bwd", "moe_permute_bwd",
    "moe_router_wgrad", "moe_layer_fwd", "moe_layer_bwd", "moe_stash_release",
    "moe_fp4_query_sizes", "moe_fp4_scale_bytes", "moe_fp4_quantize", "moe_fp4_dequantize",
    "moe_fp4_grouped_gemm", "moe_fp4_ffn_fwd", "moe_fp4_ffn_bwd",
    "moe_last_device_status",
    "moe_clear_device_status", "moe_check_bounded_wait", "moe_status_string",
)


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} returned {STATUS_NAMES.get(code, code)}: {status_string(code)}")


class MoEConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("F", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("score_fn", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("row_align", ctypes.c_int32),
                ("weights_in_expert", ctypes.c_int32), ("recompute_h", ctypes.c_int32),
                ("stash_pool_pages", ctypes.c_int32)]


class MoESizes(ctypes.Structure):
    _fields_ = [("rows_max", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("capacity", ctypes.c_int64), ("scratch_bytes", ctypes.c_int64),
                ("stash_table_len", ctypes.c_int64)]


_P = ctypes.c_void_p


class MoEParams(ctypes.Structure):
    _fields_ = [("W_r", _P), ("bias", _P), ("W13", _P), ("W2", _P)]


FWD_FIELDS = ("logits", "idx", "w", "counts", "offsets", "row_of", "token_of", "sel_offsets",
              "sel_tokens", "x_perm", "GU", "h", "y_perm")
BWD_FIELDS = ("dO_perm", "dw", "dlogits", "dGU", "dX_perm")


# the paged stash's per-layer page table and the pool's page counter
STASH_FIELDS = ("stash_table", "stash_top")


class MoEFwdState(ctypes.Structure):
    _fields_ = [(n, _P) for n in FWD_FIELDS + STASH_FIELDS]


class MoEBwdState(ctypes.Structure):
    _fields_ = [(n, _P) for n in BWD_FIELDS]


_lib = None


def lib():
    """Loads the library once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m routing_dispatch_expert_router_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name in ENTRY_POINTS:
            f = getattr(L, name)
            f.restype = ctypes.c_int
        for name, args in _FP4_ARGS.items():
            getattr(L, name).argtypes = args
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def _check(name: str, code: int):
    if code != MOE_OK:
        raise MoEError(name, code)


def config(shape) -> MoEConfig:
    """moe_config from any object with the layer's fields (e.g. workloads.MoEShape)."""
    return MoEConfig(T=shape.T, H=shape.H, E=shape.E, k=shape.k, F=shape.F,
                     n_shared=getattr(shape, "n_shared", 0),
                     score_fn=getattr(shape, "score_fn", 0),
                     n_groups=getattr(shape, "n_groups", 1),
                     topk_groups=getattr(shape, "topk_groups", 1),
                     group_score=getattr(shape, "group_score", 0),
                     route_scale=getattr(shape, "route_scale", 1.0),
                     dtype=getattr(shape, "dtype", 0),
                     capacity_factor=getattr(shape, "capacity_factor", 0.0),
                     row_align=getattr(shape, "row_align", 128),
                     weights_in_expert=getattr(shape, "weights_in_expert", 0),
                     recompute_h=getattr(shape, "recompute_h", 0),
                     stash_pool_pages=getattr(shape, "stash_pool_pages", 0))


def _cfg(c) -> MoEConfig:
    return c if isinstance(c, MoEConfig) else config(c)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # (the handle alone: a Stream object takes a microsecond, some calls eight)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, *args):
    f = getattr(lib(), name)
    conv = []
    for a in args:
        if isinstance(a, ctypes.Structure):
            conv.append(ctypes.byref(a))
        elif isinstance(a, float):
            conv.append(ctypes.c_float(a))
        elif a is None or isinstance(a, int):
            conv.append(ctypes.c_void_p(a))
        else:
            conv.append(ctypes.c_void_p(_ptr(a)))
    _check(name, f(*conv))


# ------------------------------------------------------------------ entry points
def moe_query_sizes(cfg) -> MoESizes:
    out = MoESizes()
    _check("moe_query_sizes", lib().moe_query_sizes(ctypes.byref(_cfg(cfg)), ctypes.byref(out)))
    return out


def moe_route(cfg, x, W_r, bias, logits, idx, w, scratch, stream=None):
    _call("moe_route", _cfg(cfg), x, W_r, bias, logits, idx, w, scratch, _stream(stream))


def moe_route_replay(cfg, x, W_r, bias, idx, logits, w, scratch, stream=None):
    """Router Replay: the given experts idx [T,k] (input) instead of the top-k."""
    _call("moe_route_replay", _cfg(cfg), x, W_r, bias, idx, logits, w, scratch, _stream(stream))


def moe_route_aux(cfg, logits, bias, idx, coeff, bias_rate, sel_counts, p_mean, loss, bias_out,
                  scratch, stream=None):
    """Load-balancing loss statistics, loss and (bias_out not None) the bias update."""
    _call("moe_route_aux", _cfg(cfg), logits, bias, idx, float(coeff), float(bias_rate),
          sel_counts, p_mean, loss, bias_out, scratch, _stream(stream))


def moe_route_aux_bwd(cfg, x, logits, bias, W_r, sel_counts, coeff, dloss, dlogits_aux, dx,
                      dW_r, scratch, stream=None):
    """The loss's gradient: writes dlogits_aux, adds into dx and dW_r."""
    _call("moe_route_aux_bwd", _cfg(cfg), x, logits, bias, W_r, sel_counts, float(coeff),
          float(dloss), dlogits_aux, dx, dW_r, scratch, _stream(stream))


def moe_permute(cfg, x, idx, counts, offsets, row_of, token_of, sel_offsets, sel_tokens, x_perm,
                scratch, stream=None):
    _call("moe_permute", _cfg(cfg), x, idx, counts, offsets, row_of, token_of, sel_offsets,
          sel_tokens, x_perm, scratch, _stream(stream))


def moe_permute_noalloc(cfg, x, idx, counts, offsets, row_of, token_of, sel_offsets, sel_tokens,
                        x_perm, stream=None):
    """moe_permute with the library's own fixed scratch array (allocates nothing)."""
    _call("moe_permute_noalloc", _cfg(cfg), x, idx, counts, offsets, row_of, token_of,
          sel_offsets, sel_tokens, x_perm, _stream(stream))


def moe_quantize_weights(cfg, W13, W2, scratch, stream=None):
    """FP8 mode: the E4M3 weights (and scales) in scratch; no-op in bf16 mode."""
    _call("moe_quantize_weights", _cfg(cfg), W13, W2, scratch, _stream(stream))


def moe_load_fp8_weights(cfg, W13_e4m3, W13_scale, W2_e4m3, W2_scale, scratch, stream=None):
    _call("moe_load_fp8_weights", _cfg(cfg), W13_e4m3, W13_scale, W2_e4m3, W2_scale, scratch,
          _stream(stream))


def moe_permute_noalloc_status(stream=None) -> int:
    """The status word the last moe_permute_noalloc call left (synchronises)."""
    code = ctypes.c_int32(0)
    _check("moe_permute_noalloc_status",
           lib().moe_permute_noalloc_status(ctypes.byref(code), ctypes.c_void_p(_stream(stream))))
    return code.value


def moe_grouped_ffn_fwd(cfg, x_perm, counts, offsets, W13, W2, GU, h, y_perm, scratch,
                        stream=None):
    _call("moe_grouped_ffn_fwd", _cfg(cfg), x_perm, counts, offsets, W13, W2, GU, h, y_perm,
          scratch, _stream(stream))


def moe_unpermute(cfg, y_perm, row_of, w, offsets, out, stream=None):
    _call("moe_unpermute", _cfg(cfg), y_perm, row_of, w, offsets, out, _stream(stream))


def moe_unpermute_bwd(cfg, dY, y_perm, row_of, w, counts, offsets, dO_perm, dw, scratch,
                      stream=None):
    _call("moe_unpermute_bwd", _cfg(cfg), dY, y_perm, row_of, w, counts, offsets, dO_perm, dw,
          scratch, _stream(stream))


def moe_grouped_ffn_bwd(cfg, dO_perm, x_perm, GU, h, counts, offsets, token_of, dlogits, W_r,
                        W13, W2, dGU, dX_perm, dW13, dW2, scratch, stream=None):
    _call("moe_grouped_ffn_bwd", _cfg(cfg), dO_perm, x_perm, GU, h, counts, offsets, token_of,
          dlogits, W_r, W13, W2, dGU, dX_perm, dW13, dW2, scratch, _stream(stream))


def moe_grouped_ffn_dgrad(cfg, dO_perm, GU, h, counts, offsets, token_of, dlogits, W_r, W13, W2,
                          dGU, dX_perm, scratch, stream=None):
    """h: None, or the buffer to rewrite h into from GU (fine-grained recompute)."""
    _call("moe_grouped_ffn_dgrad", _cfg(cfg), dO_perm, GU, h, counts, offsets, token_of, dlogits,
          W_r, W13, W2, dGU, dX_perm, scratch, _stream(stream))


def moe_grouped_ffn_wgrad(cfg, dO_perm, x_perm, h, dGU, counts, offsets, dW13, dW2, scratch,
                          stream=None):
    _call("moe_grouped_ffn_wgrad", _cfg(cfg), dO_perm, x_perm, h, dGU, counts, offsets, dW13,
          dW2, scratch, _stream(stream))


def moe_grouped_ffn_fwd_reordered(cfg, x_perm, counts, offsets, token_of, row_of, w, W13, W2,
                                  GU, h, y_perm, scratch, stream=None):
    """Forward GEMMs with the routing weight inside the expert (h = w silu(G) U)."""
    _call("moe_grouped_ffn_fwd_reordered", _cfg(cfg), x_perm, counts, offsets, token_of, row_of,
          w, W13, W2, GU, h, y_perm, scratch, _stream(stream))


def moe_unpermute_bwd_reordered(cfg, dY, row_of, counts, offsets, dO_perm, stream=None):
    _call("moe_unpermute_bwd_reordered", _cfg(cfg), dY, row_of, counts, offsets, dO_perm,
          _stream(stream))


def moe_grouped_ffn_dgrad_reordered(cfg, dO_perm, GU, h, counts, offsets, token_of, row_of,
                                    logits, idx, w, W_r, W13, W2, dGU, dX_perm, dw, dlogits,
                                    scratch, stream=None):
    _call("moe_grouped_ffn_dgrad_reordered", _cfg(cfg), dO_perm, GU, h, counts, offsets,
          token_of, row_of, logits, idx, w, W_r, W13, W2, dGU, dX_perm, dw, dlogits, scratch,
          _stream(stream))


def moe_route_bwd(cfg, logits, idx, w, dw, dlogits, stream=None):
    _call("moe_route_bwd", _cfg(cfg), logits, idx, w, dw, dlogits, _stream(stream))


def moe_permute_bwd(cfg, dX_perm, row_of, offsets, idx, dlogits, W_r, dx, stream=None):
    _call("moe_permute_bwd", _cfg(cfg), dX_perm, row_of, offsets, idx, dlogits, W_r, dx,
          _stream(stream))


def moe_router_wgrad(cfg, x, sel_offsets, sel_tokens, dlogits, dW_r, scratch, stream=None):
    _call("moe_router_wgrad", _cfg(cfg), x, sel_offsets, sel_tokens, dlogits, dW_r, scratch,
          _stream(stream))


def moe_layer_fwd(cfg, params: MoEParams, x, out, fwd: MoEFwdState, scratch, stream=None):
    _call("moe_layer_fwd", _cfg(cfg), params, x, out, fwd, scratch, _stream(stream))


def moe_layer_bwd(cfg, params: MoEParams, x, dY, fwd: MoEFwdState, bwd: MoEBwdState, dx, dW_r,
                  dW13, dW2, scratch, stream=None):
    _call("moe_layer_bwd", _cfg(cfg), params, x, dY, fwd, bwd, dx, dW_r, dW13, dW2, scratch,
          _stream(stream))


def moe_stash_release(cfg, fwd: MoEFwdState, stream=None):
    _call("moe_stash_release", _cfg(cfg), fwd, _stream(stream))


# ------------------------------------------------------------------ 4-bit experts
MOE_FP4_NV, MOE_FP4_MX = 0, 1
_FP4_BLOCK = (16, 32)


class MoEFp4Tensor(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("scale_log2", ctypes.c_int32),
                ("groups", ctypes.c_int64), ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("codes", _P), ("scales", _P)]


class MoEFp4Experts(ctypes.Structure):
    _fields_ = [("W13", MoEFp4Tensor), ("W2", MoEFp4Tensor), ("alpha13", _P), ("alpha2", _P),
                ("x_scale_log2", ctypes.c_int32), ("h_scale_log2", ctypes.c_int32)]


class MoEFp4Sizes(ctypes.Structure):
    _fields_ = [("gemm_scratch_bytes", ctypes.c_int64), ("fwd_scratch_bytes", ctypes.c_int64),
                ("bwd_scratch_bytes", ctypes.c_int64)]


# with the argument types declared, a call converts its integers (addresses, sizes)
# without wrapping each: these calls can be shorter than that
_T = ctypes.POINTER(MoEFp4Tensor)
_I32, _I64 = ctypes.c_int32, ctypes.c_int64
_FP4_ARGS = {
    "moe_fp4_quantize": [_T, _P, _I64, _P, _P, _I32, _P, _P, _P],
    "moe_fp4_dequantize": [_T, _P, _I64, _P],
    "moe_fp4_grouped_gemm": [_T, _T, _P, _P, _P, _P, _P, _P],
    "moe_fp4_ffn_fwd": [ctypes.POINTER(MoEConfig), ctypes.POINTER(MoEFp4Experts)] + [_P] * 8,
    "moe_fp4_ffn_bwd": [ctypes.POINTER(MoEConfig), ctypes.POINTER(MoEFp4Experts)] + [_P] * 11,
}


class Fp4Tensor:
    """A tensor [groups, rows, K] in 4 bits: packed codes [groups, rows, K / 2] and
    scale atoms [groups, slabs, atoms, 512] (include/moe_abi.h has the layout)."""
    __slots__ = ("format", "K", "codes", "scales", "scale_log2")

    def __init__(self, format: int, K: int, codes: torch.Tensor, scales: torch.Tensor,
                 scale_log2: int = 0):
        self.format, self.K, self.codes, self.scales = format, K, codes, scales
        self.scale_log2 = scale_log2

    def struct(self) -> MoEFp4Tensor:
        codes, scales, u8 = self.codes, self.scales, torch.uint8
        g, rows, kb = codes.shape
        if kb * 2 != self.K:
            raise ValueError(f"codes hold {2 * kb} elements a row, K is {self.K}")
        # ceil(K / 256) steps of 4 (NV) or 2 (MX) atoms per 128 rows
        if self.format not in (0, 1) or scales.numel() != \
                g * -(-rows // 128) * -(-self.K // 256) * (2048 >> self.format):
            raise ValueError("scales do not have the atoms of the codes' shape")
        if codes.dtype is not u8 or scales.dtype is not u8 or \
                not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales are contiguous uint8")
        if not (codes.is_cuda and scales.is_cuda):
            raise ValueError("codes and scales are on the GPU")
        return MoEFp4Tensor(self.format, self.scale_log2, g, rows, self.K, codes.data_ptr(),
                            scales.data_ptr())


def fp4_scale_bytes(fmt: int, rows: int, K: int) -> int:
    """moe_fp4_scale_bytes: bytes of the scale atoms of one group of rows x K."""
    n = ctypes.c_int64(0)
    _check("moe_fp4_scale_bytes",
           lib().moe_fp4_scale_bytes(ctypes.c_int32(fmt), ctypes.c_int64(rows),
                                     ctypes.c_int64(K), ctypes.byref(n)))
    return n.value


def alloc_fp4(fmt: int, groups: int, rows: int, K: int, device="cuda",
              scale_log2: int = 0) -> Fp4Tensor:
    """Uninitialised room for [groups, rows, K] in 4 bits."""
    atoms = fp4_scale_bytes(fmt, rows, K) // 512
    slabs = -(-rows // 128)
    u8 = torch.uint8
    return Fp4Tensor(fmt, K, torch.empty(groups, rows, K // 2, dtype=u8, device=device),
                     torch.empty(groups, slabs, atoms // max(slabs, 1), 512, dtype=u8,
                                 device=device), scale_log2)


def fp4_experts(W13: Fp4Tensor, W2: Fp4Tensor, alpha13=None, alpha2=None, x_scale_log2: int = 0,
                h_scale_log2: int = 0) -> MoEFp4Experts:
    """The experts' 4-bit weights for the FFN calls; alpha13, alpha2: None, or their own scales
    (fp32, one per expert). The result keeps the tensors alive."""
    a, b = W13.struct(), W2.struct()
    ex = MoEFp4Experts(a, b, _vector(alpha13, a.groups, torch.float32, "alpha13"),
                       _vector(alpha2, b.groups, torch.float32, "alpha2"), x_scale_log2,
                       h_scale_log2)
    ex.tensors = (W13.codes, W13.scales, W2.codes, W2.scales, alpha13, alpha2)
    return ex


def moe_fp4_query_sizes(cfg, fmt: int) -> MoEFp4Sizes:
    out = MoEFp4Sizes()
    c = None if cfg is None else ctypes.byref(_cfg(cfg))
    _check("moe_fp4_query_sizes",
           lib().moe_fp4_query_sizes(c, ctypes.c_int32(fmt), ctypes.byref(out)))
    return out


def alloc_fp4_scratch(nbytes: int, device="cuda") -> torch.Tensor:
    """Scratch of the 4-bit calls: zero-filled once (status word, arrival counters)."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device)


def _bf16_rows(t, shape, what: str) -> int:
    """Elements from row to row of a bf16 tensor of this shape whose rows are evenly spaced."""
    if t.shape != shape or t.dtype != torch.bfloat16:
        raise ValueError(f"{what} is bf16 {tuple(shape)}")
    if t.is_contiguous():
        return shape[2]
    sg, ld, one = t.stride()
    if shape[1] == 1:
        ld = sg                                            # the stride of a single row says nothing
    if one != 1 or (shape[0] > 1 and sg != ld * shape[1]):
        raise ValueError(f"{what} has contiguous rows, its groups following each other row by row")
    return ld if shape[0] > 1 or shape[1] > 1 else shape[2]


# Addresses of the calls' tensors. A kernel can see neither a tensor's type nor its size: what
# does not fit is refused here. None passes, to be refused (or taken) by the C entry.
def _vector(t, n: int, dtype, what: str):
    """At least n elements in a row."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what} is contiguous {dtype} of {n} elements, on the GPU")
    return t.data_ptr()


def _rows(t, rows: int, cols: int, dtype, what: str):
    """[at least rows, cols]; dtype None: any of one byte."""
    if t is None:
        return None
    if t.dim() != 2 or t.shape[1] != cols or t.shape[0] < rows or not t.is_contiguous() or \
            not t.is_cuda or (t.dtype is not dtype if dtype else t.element_size() != 1):
        raise ValueError(f"{what} is contiguous {dtype or 'bytes'} [{rows}, {cols}], on the GPU")
    return t.data_ptr()


def _scratch(t, nbytes: int):
    if t is None:
        return None
    if t.numel() * t.element_size() < nbytes or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"scratch has {nbytes} bytes on the GPU")
    return t.data_ptr()


_gemm_scratch_bytes = 0


def _gemm_scratch(t):
    global _gemm_scratch_bytes
    if not _gemm_scratch_bytes:                            # of any shape and format
        _gemm_scratch_bytes = moe_fp4_query_sizes(None, MOE_FP4_NV).gemm_scratch_bytes
    return _scratch(t, _gemm_scratch_bytes)


def moe_fp4_quantize(x, q: Fp4Tensor, scale_log2: int | None = None, counts=None, offsets=None,
                     values=None, scratch=None, stream=None):
    """x [groups, rows, K] bf16 into q; with counts and offsets only those rows of
    x [1, rows, K]. values: the bf16 values that the codes stand for. scale_log2: the tensor
    scale to quantise with; it is part of what the codes mean, so q keeps it (a call that is
    refused leaves q as it was). None: q's own."""
    s = q.struct()
    if scale_log2 is not None:
        s.scale_log2 = scale_log2
    ldx = _bf16_rows(x, (s.groups, s.rows, s.K), "x")
    if values is not None and not (values.is_contiguous() and values.shape == x.shape
                                   and values.dtype == torch.bfloat16):
        raise ValueError("values is contiguous bf16 of x's shape")
    n = 0 if counts is None else counts.numel()
    if not x.is_cuda or (values is not None and not values.is_cuda):
        raise ValueError("x and values are on the GPU")
    rc = lib().moe_fp4_quantize(s, x.data_ptr(), ldx,
                                _vector(counts, n, torch.int32, "counts"),
                                _vector(offsets, n, torch.int32, "offsets"), n,
                                None if values is None else values.data_ptr(),
                                _scratch(scratch, 4), _stream(stream))
    _check("moe_fp4_quantize", rc)
    q.scale_log2 = s.scale_log2


def moe_fp4_dequantize(q: Fp4Tensor, out, scale_log2: int | None = None, stream=None):
    """out [groups, rows, K] bf16 = the values that q's codes stand for, with q's tensor scale
    or, in this call alone, with scale_log2."""
    s = q.struct()
    if scale_log2 is not None:
        s.scale_log2 = scale_log2
    ldo = _bf16_rows(out, (s.groups, s.rows, s.K), "out")
    if not out.is_cuda:
        raise ValueError("out is on the GPU")
    _check("moe_fp4_dequantize",
           lib().moe_fp4_dequantize(s, out.data_ptr(), ldo, _stream(stream)))


def moe_fp4_grouped_gemm(a: Fp4Tensor, b: Fp4Tensor, counts, offsets, alpha, out, scratch,
                         stream=None):
    """out [rows, N] bf16: every group's rows of a [1, rows, K] by b [G, N, K]."""
    sa, sb = a.struct(), b.struct()
    if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.shape != (sa.rows, sb.rows) \
            or not out.is_cuda:
        raise ValueError("out is contiguous bf16 [rows of a, rows of b], on the GPU")
    if counts is not None and counts.numel() != sb.groups:
        raise ValueError("one count per group of b")
    _check("moe_fp4_grouped_gemm",
           lib().moe_fp4_grouped_gemm(sa, sb,
                                      _vector(counts, sb.groups, torch.int32, "counts"),
                                      _vector(offsets, sb.groups, torch.int32, "offsets"),
                                      _vector(alpha, sb.groups, torch.float32, "alpha"),
                                      out.data_ptr(), _gemm_scratch(scratch), _stream(stream)))


@functools.lru_cache(maxsize=64)
def _layer_sizes(config: bytes, fmt: int):
    """Rows of a layer's buffers and the scratch of its 4-bit calls: rows, forward, backward.
    By the configuration's bytes: asking the library takes as long as checking every tensor."""
    c = MoEConfig.from_buffer_copy(config)
    s = moe_fp4_query_sizes(c, fmt)
    return moe_query_sizes(c).rows_max, s.fwd_scratch_bytes, s.bwd_scratch_bytes


def moe_fp4_ffn_fwd(cfg, experts: MoEFp4Experts, x_perm, counts, offsets, ckpt, ckpt_scale,
                    y_perm, scratch, stream=None):
    """The experts' FFN in 4 bits on x_perm's rows [R, H] (bf16, R = rows_max at least) into
    y_perm's; counts, offsets: int32, one per group at least. ckpt [R, 2F], ckpt_scale
    [R, 2F / 32]: None, or the 8-bit checkpoint."""
    c = _cfg(cfg)
    R, need, _ = _layer_sizes(bytes(c), experts.W13.format)
    G, H, F2, bf16 = c.E + c.n_shared, c.H, 2 * c.F, torch.bfloat16
    _check("moe_fp4_ffn_fwd",
           lib().moe_fp4_ffn_fwd(c, experts, _rows(x_perm, R, H, bf16, "x_perm"),
                                 _vector(counts, G, torch.int32, "counts"),
                                 _vector(offsets, G, torch.int32, "offsets"),
                                 _rows(ckpt, R, F2, None, "ckpt"),
                                 _rows(ckpt_scale, R, F2 // 32, None, "ckpt_scale"),
                                 _rows(y_perm, R, H, bf16, "y_perm"),
                                 _scratch(scratch, need), _stream(stream)))


def moe_fp4_ffn_bwd(cfg, experts: MoEFp4Experts, dO_perm, ckpt, ckpt_scale, counts, offsets,
                    token_of, dlogits, W_r, dX_perm, scratch, stream=None):
    """The gradient at the FFN's input, the tensors as moe_fp4_ffn_fwd's; token_of (int32, R),
    dlogits [T, E], W_r [E, H] (fp32): None, or the router's term."""
    c = _cfg(cfg)
    R, _, need = _layer_sizes(bytes(c), experts.W13.format)
    G, H, F2, bf16, f32 = c.E + c.n_shared, c.H, 2 * c.F, torch.bfloat16, torch.float32
    _check("moe_fp4_ffn_bwd",
           lib().moe_fp4_ffn_bwd(c, experts, _rows(dO_perm, R, H, bf16, "dO_perm"),
                                 _rows(ckpt, R, F2, None, "ckpt"),
                                 _rows(ckpt_scale, R, F2 // 32, None, "ckpt_scale"),
                                 _vector(counts, G, torch.int32, "counts"),
                                 _vector(offsets, G, torch.int32, "offsets"),
                                 _vector(token_of, R, torch.int32, "token_of"),
                                 _rows(dlogits, c.T, c.E, f32, "dlogits"),
                                 _rows(W_r, c.E, H, f32, "W_r"),
                                 _rows(dX_perm, R, H, bf16, "dX_perm"),
                                 _scratch(scratch, need), _stream(stream)))


def moe_last_device_status(scratch, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check("moe_last_device_status",
           lib().moe_last_device_status(ctypes.c_void_p(_ptr(scratch)), ctypes.byref(code),
                                        ctypes.c_void_p(_stream(stream))))
    return code.value


def moe_check_bounded_wait(scratch, budget_cycles: int, stream=None):
    f = lib().moe_check_bounded_wait
    _check("moe_check_bounded_wait",
           f(ctypes.c_void_p(_ptr(scratch)), ctypes.c_int64(int(budget_cycles)),
             ctypes.c_void_p(_stream(stream))))


def moe_clear_device_status(scratch, stream=None):
    _call("moe_clear_device_status", scratch, _stream(stream))


# ------------------------------------------------------------------ buffers
@dataclass
class LayerBuffers:
    """Caller-owned device buffers of one layer, sized by moe_query_sizes."""
    sizes: MoESizes
    fwd: dict
    bwd: dict
    scratch: torch.Tensor
    fwd_struct: MoEFwdState
    bwd_struct: MoEBwdState


@dataclass
class StashPool:
    """The rows layers keep for their backward, in pages of 128 rows shared by
    the layers of a step: x_perm, GU, h, y_perm with (pages + 1) * 128 rows
    (the last page is the spill page) and the device page counter."""
    pages: int
    tensors: dict
    top: torch.Tensor


def alloc_stash_pool(cfg, pages: int, device="cuda") -> StashPool:
    c = _cfg(cfg)
    if int(pages) < 1:
        raise ValueError("a stash pool has at least one page (stash_pool_pages = 0 means no pool)")
    rows = (int(pages) + 1) * 128
    bf = torch.bfloat16
    e = lambda *s: torch.empty(*s, dtype=bf, device=device)  # noqa: E731
    t = dict(x_perm=e(rows, c.H), GU=e(rows, 2 * c.F), h=e(rows, c.F), y_perm=e(rows, c.H))
    return StashPool(int(pages), t, torch.zeros(1, dtype=torch.int32, device=device))


def alloc_buffers(cfg, device="cuda", backward: bool = True,
                  pool: StashPool | None = None) -> LayerBuffers:
    """Allocates (torch.empty / zeros) every buffer the layer calls need; with
    a stash pool (cfg.stash_pool_pages == pool.pages) the four stashed row
    tensors are the pool's and the layer gets its own page table."""
    c = _cfg(cfg)
    sz = moe_query_sizes(c)
    R, G = int(sz.rows_max), int(sz.groups)
    T, H, E, k, F = c.T, c.H, c.E, c.k, c.F
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    e = lambda *s, dt: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
    fwd = dict(logits=e(T, E, dt=f32), idx=e(T, k, dt=i32), w=e(T, k, dt=f32),
               counts=e(G, dt=i32), offsets=e(G + 1, dt=i32), row_of=e(T, k, dt=i32),
               token_of=e(R, dt=i32), sel_offsets=e(E + 1, dt=i32),
               sel_tokens=e(max(T * k, 1), dt=i32))
    if pool is None:
        fwd.update(x_perm=e(R, H, dt=bf), GU=e(R, 2 * F, dt=bf), h=e(R, F, dt=bf),
                   y_perm=e(R, H, dt=bf))
    else:
        if c.stash_pool_pages < 1 or c.stash_pool_pages != pool.pages:
            raise ValueError("cfg.stash_pool_pages must equal the pool's pages (at least 1)")
        fwd.update(pool.tensors)
        fwd.update(stash_table=e(int(sz.stash_table_len), dt=i32), stash_top=pool.top)
    bwd = {}
    if backward:
        bwd = dict(dO_perm=e(R, H, dt=bf), dw=e(T, k, dt=f32), dlogits=e(T, E, dt=f32),
                   dGU=e(R, 2 * F, dt=bf), dX_perm=e(R, H, dt=bf))
    scratch = torch.zeros(int(sz.scratch_bytes), dtype=torch.uint8, device=device)
    fs = MoEFwdState(**{n: (fwd[n].data_ptr() if n in fwd else 0)
                        for n in FWD_FIELDS + STASH_FIELDS})
    bs = MoEBwdState(**{n: (bwd[n].data_ptr() if bwd else 0) for n in BWD_FIELDS})
    return LayerBuffers(sz, fwd, bwd, scratch, fs, bs)


def params(W_r, bias, W13, W2) -> MoEParams:
    return MoEParams(W_r=_ptr(W_r), bias=_ptr(bias), W13=_ptr(W13), W2=_ptr(W2))
