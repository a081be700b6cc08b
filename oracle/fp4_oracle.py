"""Plain fp64 oracle of the 4-bit experts -- test infrastructure only.

It shares no code with the CUDA path. Formats (include/moe_abi.h): E2M1 codes with
a scale per block along K, "nv" (blocks of 16, E4M3 scales) and "mx" (blocks of
32, power-of-two scales); the scale bytes in 512-byte atoms. Rounding is to the
nearest, ties to the even code, by search in the list of a format's values.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import round_bf16

NV, MX = 0, 1
BLOCK = {NV: 16, MX: 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# E4M3's non-negative finite values, by code 0 .. 126 (127 is NaN)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])


def nearest(v, grid):
    """Index of the grid's value nearest to v >= 0 (ties to the even index)."""
    v = np.asarray(v, np.float64)
    hi = np.clip(np.searchsorted(grid, v), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(grid[hi] - v), np.abs(v - grid[lo])
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(fmt, x, scale_log2=0):
    """x [.., K] -> codes [.., K] (0..15) and scale bytes [.., K / block]."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, BLOCK[fmt])
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    amax = np.where(bad, 0.0, amax)
    if fmt == NV:
        byte = nearest(np.minimum(amax / 6.0 / 2.0 ** scale_log2, 448.0), E4M3)
        unit = E4M3[byte] * 2.0 ** scale_log2
        byte = np.where(bad, 127, byte)
    else:
        m, e = np.frexp(amax / 6.0)                     # amax / 6 = m 2^e, 1/2 <= m < 1
        code = np.where(m == 0.5, e - 1, e) + 127
        code = np.where(amax > 0, np.maximum(code, 0), 127)
        unit = np.exp2(code - 127.0)
        byte = np.where(bad, 255, code)
    ok = (unit > 0) & ~bad
    with np.errstate(invalid="ignore"):
        q = np.where(ok[..., None], np.abs(b) / np.where(ok, unit, 1.0)[..., None], 0.0)
    codes = nearest(np.minimum(np.nan_to_num(q), 6.0), E2M1)
    codes = codes + 8 * (np.signbit(b) & ok[..., None])
    return codes.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def scale_values(fmt, byte):
    table = np.append(E4M3, np.nan) if fmt == NV else \
        np.append(np.exp2(np.arange(255) - 127.0), np.nan)
    return table[byte]


def values(fmt, codes, byte, scale_log2=0):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = scale_values(fmt, byte) * 2.0 ** scale_log2
    return (v.reshape(*byte.shape, BLOCK[fmt]) * s[..., None]).reshape(codes.shape)


def real(fmt, x, scale_log2=0):
    """The values that x's 4-bit form stands for."""
    return values(fmt, *quantise(fmt, x, scale_log2), scale_log2)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def atoms_k(fmt, K):
    return -(-K // 256) * 256 // (4 * BLOCK[fmt])


def to_atoms(fmt, byte, K):
    """Scale bytes [groups, rows, K / block] -> [groups, slabs, atoms, 512], element by element."""
    g, rows, nb = byte.shape
    out = np.zeros((g, -(-rows // 128), atoms_k(fmt, K), 512), np.uint8)
    r, b = np.arange(rows)[:, None], np.arange(nb)[None]
    out[:, r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte
    return out


def from_atoms(fmt, atoms, rows, K):
    r, b = np.arange(rows)[:, None], np.arange(K // BLOCK[fmt])[None]
    return atoms[:, r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def silu(g):
    return g / (1.0 + np.exp(-g))


def checkpoint_values(codes, byte):
    """E4M3 codes (with sign) [.., n] and UE8M0 bytes [.., n / 32] -> what they stand for."""
    mag = np.append(E4M3, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return (mag.reshape(*byte.shape, 32) * scale_values(MX, byte)[..., None]).reshape(codes.shape)


def checkpoint_unit(gu):
    """The power-of-two unit of every 32 values: 2^ceil(log2(amax / 448)), 1 for zeros."""
    amax = np.abs(gu.reshape(*gu.shape[:-1], -1, 32)).max(-1)
    m, e = np.frexp(amax / 448.0)
    return np.where(amax > 0, np.exp2(np.maximum(np.where(m == 0.5, e - 1, e), -127)), 1.0)


def ffn_fwd(fmt, x, W13, W2, x_log2=0, h_log2=0):
    """One expert's rows: W13 [2F, H], W2 [H, F] the values of its 4-bit weights (alpha
    included). Returns GU (bf16 numbers), h (bf16 numbers), h4 and y (not rounded)."""
    F = W2.shape[1]
    gu = round_bf16(real(fmt, x, x_log2) @ W13.T)
    h = round_bf16(silu(gu[:, :F]) * gu[:, F:])
    h4 = real(fmt, h, h_log2)
    return gu, h, h4, h4 @ W2.T


def ffn_bwd(dO, gu, W13, W2):
    """dX (not rounded) and [dG | dU] of one expert's rows from its gate and up values."""
    F = W2.shape[1]
    g, u = gu[:, :F], gu[:, F:]
    s = 1.0 / (1.0 + np.exp(-g))
    dh = dO @ W2
    dgu = np.concatenate((dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s), 1)
    return dgu @ W13, dgu
