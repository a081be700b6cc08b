// Storage of 4-bit operands: E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) packed two to a byte along K, the even element in the low four
// bits, and one scale byte per block of consecutive K elements:
//   MOE_FP4_NV  blocks of 16, E4M3 scales (the sign bit never set);
//   MOE_FP4_MX  blocks of 32, UE8M0 scales (byte e means 2^(e - 127)).
// Scale bytes lie the way the block-scaled tensor-core MMA reads them, in the
// 512-byte atoms of fp8_layout.cuh: one atom per 128 rows and 4 consecutive
// blocks (64 elements of K for NV, 128 for MX), the scale of row r's j-th block
// at byte (r % 32) * 16 + (r % 128) / 32 * 4 + j. An atom's 32 lines of 16 bytes
// go into four tensor-memory columns of each lane quarter, where the MMA of a
// 64-wide K slice reads all four bytes of a row (scale_vec::4X, NV) or the two
// that its scale-factor id names (scale_vec::2X, MX). A 128-row slab's atoms follow each
// other along K and fill whole 256-element steps (one GEMM k-block = 128 bytes
// of codes); bytes of blocks past K are zero.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace moe {
namespace f4 {

constexpr int kStep = 256;                       // elements of a GEMM k-block
constexpr int kAtomBytes = 512;

__host__ __device__ constexpr int block_of(int fmt) { return fmt == MOE_FP4_NV ? 16 : 32; }
__host__ __device__ constexpr int step_atoms(int fmt) { return kStep / (4 * block_of(fmt)); }
// atoms of a 128-row slab of a K-long operand
__host__ __device__ constexpr int64_t atoms_k(int fmt, int64_t K) {
  return (K + kStep - 1) / kStep * step_atoms(fmt);
}
__host__ __device__ constexpr int64_t slabs(int64_t rows) { return (rows + 127) / 128; }
__host__ __device__ constexpr int64_t sf_bytes(int fmt, int64_t rows, int64_t K) {
  return slabs(rows) * atoms_k(fmt, K) * kAtomBytes;
}
// byte of (row r of the slab, block b) counted from the slab's first atom
__host__ __device__ constexpr int64_t sf_byte(int r, int64_t b) {
  return (b >> 2) * kAtomBytes + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

}  // namespace f4

// ------------------------------------------------------- the factor of a product
// What a fp32 sum is multiplied with, x y 2^log2 (the experts' own scales and the tensors'
// powers of two): `by`, and then, as a bf16 pair for the rounded values, `rest`: a power of
// two that is 1 unless the product lies outside fp32's normal numbers. It may without the
// result doing so: two tensor scales of 2^64 and an alpha of 2^-128, sums that are zero, an
// alpha below 2^-126. (Taking account of these costs a single token's FFN 0.3 of 50.0 us and
// a training forward 2.7 of 560.)
struct Fp4Factor {
  float by;
  uint32_t rest;
};
constexpr uint32_t kFp4One = 0x3F803F80u;          // a `rest` of 1

__device__ __forceinline__ bool fp4_normal(float v) {
  return ((__float_as_uint(v) >> 23 & 255u) - 1u) < 254u;
}

// The mantissas times as much of the power as stays far inside the range, and the rest: both
// go the same way, so that an infinity or a zero after the first is the result's too. (Not
// inlined: hardly any call reaches it.)
static __device__ __noinline__ Fp4Factor fp4_factor_far(float x, float y, int log2) {
  if (!(fabsf(x) > 0.f && fabsf(y) > 0.f && isfinite(x) && isfinite(y)))
    return Fp4Factor{x * y, kFp4One};
  int ex, ey;
  const float m = frexpf(x, &ex) * frexpf(y, &ey);
  const int e = ex + ey + log2, near = min(max(e, -100), 100);
  const uint32_t rest = (uint32_t)(min(max(e - near, -126), 127) + 127) << 7;
  return Fp4Factor{ldexpf(m, near), rest | rest << 16};
}

// unit = 2^log2, which may be past fp32's range.
__device__ __forceinline__ Fp4Factor fp4_factor(float x, float y, float unit, int log2) {
  const float xy = x * y, by = xy * unit;
  if (fp4_normal(xy) && fp4_normal(unit) && fp4_normal(by)) return Fp4Factor{by, kFp4One};
  return fp4_factor_far(x, y, log2);
}

// Eight rounded values times `rest`.
__device__ __forceinline__ void fp4_times(uint4& v, uint32_t rest) {
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v.x) : "r"(rest));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v.y) : "r"(rest));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v.z) : "r"(rest));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v.w) : "r"(rest));
}

// ------------------------------------------------------ producing the 4-bit form
// A block's scale byte and the factor that its elements are multiplied with
// before they are rounded to E2M1.
struct Fp4Scale {
  uint32_t byte;
  float inv;
};

// To 12 significant bits, to nearest.
__device__ __forceinline__ float fp4_snap(float q) {
  return __uint_as_float((__float_as_uint(q) + 0x800u) & 0xFFFFF000u);
}

// amax: the block's largest magnitude, a bf16 number; finite: whether every
// element of the block is. down = 2^-scale_log2 (NV).
// NV: the scale is amax / (6 2^scale_log2) rounded to E4M3 (to nearest, at most
// 448). MX: 2^ceil(log2(amax / 6)); amax = 2^E M gives E - 2 for M <= 1.5, else
// E - 1; amax = 0 gives 1, and scales below 2^-127 are raised to it.
// A block with an infinity or a NaN gets the scale NaN, so that whatever is
// computed from it is NaN too and not silently finite.
template <int FMT>
__device__ __forceinline__ Fp4Scale fp4_scale(float amax, bool finite, float down) {
  Fp4Scale s;
  if (FMT == MOE_FP4_NV) {
    // a sixth as a product: amax has 8 significant bits and a border between two
    // scales 5, so a quotient that is not on one is 2^-10 away; rounding the product
    // (within 2^-23) to 12 bits puts those that are exactly there (a tie)
    const float a = fp4_snap(amax * down * (1.f / 6.f));
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(a));
    uint32_t half2;                              // the scale's value, as an fp16 pair
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(h));
    float v;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}"
        : "=f"(v) : "r"(half2));
    s.byte = finite ? (h & 0xffu) : 0x7Fu;
    s.inv = (finite && v > 0.f) ? down * ptx::rcp_approx(v) : 0.f;
  } else {
    const uint32_t b = __float_as_uint(amax);
    int code = (int)(b >> 23) - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    if (b < 0x00800000u) code = b ? 0 : 127;     // subnormal amax: the smallest scale
    code = code < 0 ? 0 : code;
    s.byte = finite ? (uint32_t)code : 0xFFu;
    s.inv = finite ? __uint_as_float((254u - (uint32_t)code) << 23) : 0.f;
  }
  return s;
}

// x times the scale's reciprocal, so near to the real quotient that rounding it
// to the E2M1 grid rounds the quotient itself. MX: the product is exact. NV: x
// has 8 significant bits, the scale 4 and a border of the grid 3, so a quotient
// that is not on a border is at least 2^-9 (relative) away from it; the product
// is within 2^-22, and rounding it to 12 significant bits puts the quotients
// that are on a border exactly there (the E2M1 conversion then sees a tie).
template <int FMT>
__device__ __forceinline__ float fp4_quotient(float x, float inv) {
  const float q = x * inv;
  if (FMT == MOE_FP4_MX) return q;
  return fp4_snap(q);
}

// E2M1 codes of eight quotients (to nearest, ties to even, at most 6): 4 bytes
// in element order.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r) : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]),
        "f"(f[7]));
  return r;
}

// Eight codes -> eight fp16 values (four packed pairs).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
}

// What a scale byte stands for.
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
  if (FMT == MOE_FP4_NV) {
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"((uint16_t)byte));
    float v;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}"
        : "=f"(v) : "r"(half2));
    return v;
  }
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Largest magnitude of eight bf16 values, as its bits (magnitudes order as integers; NaN
// counts as more than infinite).
__device__ __forceinline__ uint32_t amax_bits8(const uint4& v) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag));
  return max(m & 0xFFFFu, m >> 16);
}

}  // namespace moe
