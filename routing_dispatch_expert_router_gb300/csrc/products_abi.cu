// C entry points of the norm before a layer, the dispatch of rows in 8 bits and the products
// of free form: argument checks and launches.
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "fp8_layout.cuh"
#include "internal.h"

using namespace moe;

namespace {

#define OP_TRY(expr)                   \
  do {                                 \
    const moe_status _s = (expr);      \
    if (_s != MOE_OK) return _s;       \
  } while (0)

#define OP_CUDA(expr)                                                         \
  do {                                                                        \
    const cudaError_t _e = (expr);                                            \
    if (_e != cudaSuccess)                                                    \
      return _e == cudaErrorInvalidValue ? MOE_ERR_INVALID_ARG : MOE_ERR_CUDA; \
  } while (0)

#define OP_REQUIRE(cond)                       \
  do {                                         \
    if (!(cond)) return MOE_ERR_INVALID_ARG;   \
  } while (0)

bool al16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
bool al16_or_null(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
bool al4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Rows of `cols` bf16 elements, ld apart, where the 16-byte accesses want them.
bool rows_ok(const void* p, int64_t ld, int64_t cols) {
  return al16(p) && ld >= cols && ld % 8 == 0 && ld <= INT_MAX;
}
bool rows_or_null(const void* p, int64_t ld, int64_t cols) { return !p || rows_ok(p, ld, cols); }

moe_status check_norm(int64_t T, int64_t H, const void* gamma, int32_t gamma_dtype) {
  OP_REQUIRE(T >= 0 && T <= INT_MAX && H >= 8 && H % 8 == 0);
  if (H > 32768) return MOE_ERR_UNSUPPORTED;
  OP_REQUIRE(gamma_dtype == MOE_GAMMA_BF16 || gamma_dtype == MOE_GAMMA_F32);
  OP_REQUIRE(al16(gamma));
  return MOE_OK;
}

// Scratch of a product: the status word, the parts' counters (of each kernel its own), the parts.
constexpr int64_t kArrivedOffset = 1024;
constexpr int64_t kRaggedArrivedOffset = kArrivedOffset + kFewCtas * 4;
constexpr int64_t kPartsOffset = 8192;
constexpr int64_t kFewBytes = 2LL * kFewCtas * kFewPart * 4, kRaggedBytes = kRaggedPairs * (256LL << 10);
constexpr int64_t kProductScratch = kPartsOffset + (kFewBytes > kRaggedBytes ? kFewBytes : kRaggedBytes);
static_assert(kRaggedArrivedOffset + kRaggedPairs / 2 * 16 * 4 <= kPartsOffset, "counters before the parts");

// (a tile past the last row is counted in 32 bits)
constexpr int64_t kMaxRows = INT_MAX - 1023;

moe_status check_segments(int64_t groups, int64_t rows, const int32_t* counts,
                          const int32_t* offsets) {
  OP_REQUIRE(groups >= 1 && rows >= 0 && rows <= INT_MAX);
  if (groups > kMaxGroups || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (counts || offsets) OP_REQUIRE(al4(counts) && al4(offsets));
  else OP_REQUIRE(groups == 1);
  return MOE_OK;
}

// Sizes that the maps' and kernels' 32-bit numbers hold.
bool matrix_ok(int64_t N, int64_t K, int unit) {
  return N >= unit && K >= unit && N % unit == 0 && K % unit == 0 && N <= (1 << 24) &&
         K <= (1 << 24);
}

moe_status check_int4(const moe_int4_tensor* w) {
  OP_REQUIRE(w && (w->group == 32 || w->group == 64 || w->group == 128));
  OP_REQUIRE(w->groups >= 1 && w->groups <= INT_MAX);
  OP_REQUIRE(matrix_ok(w->N, w->K, 16) && w->K % w->group == 0);
  OP_REQUIRE(al16(w->codes) && al16(w->scales) && al16_or_null(w->zeros));
  return MOE_OK;
}

FewProduct few_product(int64_t groups, int64_t rows, int64_t N, int64_t K, const int32_t* counts,
                       const int32_t* offsets, void* out, int64_t ldo, void* scratch) {
  uint8_t* sc = static_cast<uint8_t*>(scratch);
  FewProduct p{};
  p.G = (int)groups;
  p.rows = rows;
  p.N = (int)N;
  p.K = (int)K;
  p.counts = counts;
  p.offsets = offsets;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.parts = reinterpret_cast<float*>(sc + kPartsOffset);
  p.arrived = reinterpret_cast<uint32_t*>(sc + kArrivedOffset);
  p.status = reinterpret_cast<int32_t*>(sc);
  return p;
}

moe_status check_product(int64_t groups, int64_t rows, int64_t N, int64_t K, const void* w,
                         const int32_t* counts, const int32_t* offsets, const void* scratch) {
  OP_TRY(check_segments(groups, rows, counts, offsets));
  OP_REQUIRE(matrix_ok(N, K, 8) && al16(w) && al16(scratch));
  return MOE_OK;
}

RaggedProduct ragged_product(int64_t groups, int64_t rows, const int32_t* counts,
                             const int32_t* offsets, const void* add, int64_t ldadd, void* out,
                             int64_t ldo, void* scratch) {
  uint8_t* sc = static_cast<uint8_t*>(scratch);
  RaggedProduct p{};
  p.G = (int)groups;
  p.rows = rows;
  p.counts = counts;
  p.offsets = offsets;
  p.add = static_cast<const __nv_bfloat16*>(add);
  p.ldadd = ldadd;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.parts = reinterpret_cast<float*>(sc + kPartsOffset);
  p.arrived = reinterpret_cast<uint32_t*>(sc + kRaggedArrivedOffset);
  p.status = static_cast<int32_t*>(scratch);
  return p;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(void* p) { return static_cast<__nv_bfloat16*>(p); }

}  // namespace

extern "C" {

moe_status moe_rmsnorm_fwd(int64_t T, int64_t H, const void* x, int64_t ldx, const void* residual,
                           int64_t ldr, const void* gamma, int32_t gamma_dtype, float eps,
                           void* sum, int64_t lds, void* out, int64_t ldo, void* codes,
                           void* scales, int32_t block, float* rstd, void* stream) {
  OP_TRY(check_norm(T, H, gamma, gamma_dtype));
  OP_REQUIRE(isfinite(eps) && eps >= 0.f && !codes == !scales && (out || codes || T == 0));
  if (codes) {
    OP_REQUIRE((block == 32 || block == 128) && H % block == 0);
    OP_REQUIRE(al16(codes));
  }
  if (T == 0) return MOE_OK;
  OP_REQUIRE(rows_ok(x, ldx, H) && rows_or_null(residual, ldr, H) && rows_or_null(sum, lds, H));
  OP_REQUIRE(rows_or_null(out, ldo, H) && al4_or_null(rstd) && (residual || !sum));
  const RmsNormFwd p{T, (int)H, bf(x), ldx, bf(residual), ldr, gamma,
                     gamma_dtype == MOE_GAMMA_F32, eps, bf(sum), lds, bf(out), ldo,
                     static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                     codes ? block : 32, rstd};
  OP_CUDA(launch_rmsnorm_fwd(p, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_rmsnorm_scratch_bytes(int64_t H, int64_t* bytes) {
  OP_REQUIRE(bytes && H >= 8 && H % 8 == 0);
  if (H > 32768) return MOE_ERR_UNSUPPORTED;
  *bytes = (int64_t)kRmsNormParts * H * 4;
  return MOE_OK;
}

moe_status moe_rmsnorm_bwd(int64_t T, int64_t H, const void* dy, int64_t lddy, const void* h,
                           int64_t ldh, const float* rstd, const void* gamma, int32_t gamma_dtype,
                           const void* dsum, int64_t ldds, void* dx, int64_t lddx, float* dgamma,
                           void* scratch, void* stream) {
  OP_TRY(check_norm(T, H, gamma, gamma_dtype));
  OP_REQUIRE(!dgamma || (al4(dgamma) && al16(scratch)));
  if (T > 0) {
    OP_REQUIRE(rows_ok(dy, lddy, H) && rows_ok(h, ldh, H) && al4(rstd) && rows_ok(dx, lddx, H));
    OP_REQUIRE(rows_or_null(dsum, ldds, H));
  }
  const RmsNormBwd p{T, (int)H, bf(dy), lddy, bf(h), ldh, rstd, gamma,
                     gamma_dtype == MOE_GAMMA_F32, bf(dsum), ldds, bf(dx), lddx,
                     dgamma ? static_cast<float*>(scratch) : nullptr};
  OP_CUDA(launch_rmsnorm_bwd(p, dgamma, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_permute_fp8(const moe_config* cfg, const void* codes, const void* scales,
                           const int32_t* idx, int32_t* counts, int32_t* offsets, int32_t* row_of,
                           int32_t* token_of, int32_t* sel_offsets, int32_t* sel_tokens,
                           void* codes_perm, void* scales_perm, void* scratch, void* stream) {
  OP_TRY(check_config(cfg));
  OP_REQUIRE(cfg->dtype == MOE_DTYPE_FP8_E4M3_BLOCK || cfg->dtype == MOE_DTYPE_MXFP8);
  if (cfg->stash_pool_pages) return MOE_ERR_UNSUPPORTED;
  OP_REQUIRE(al4(counts) && al4(offsets) && al4(token_of) && al4(sel_offsets) && al16(scratch));
  OP_REQUIRE(!codes_perm == !scales_perm && al16_or_null(codes_perm) && al16_or_null(scales_perm));
  if (cfg->T > 0)
    OP_REQUIRE(al16(codes) && scales && al4(idx) && al4(row_of) && al4(sel_tokens));
  if (!codes_perm) {
    const Fp8Scratch f = fp8_scratch(*cfg, scratch);
    codes_perm = f.xq;
    scales_perm = f.xsf;
  }
  OP_CUDA(launch_permute_fp8(*cfg, static_cast<const uint8_t*>(codes),
                             static_cast<const uint8_t*>(scales), idx, counts, offsets, row_of,
                             token_of, sel_offsets, sel_tokens, static_cast<uint8_t*>(codes_perm),
                             static_cast<uint8_t*>(scales_perm), static_cast<uint8_t*>(scratch),
                             (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_product_scratch_bytes(int64_t* bytes) {
  OP_REQUIRE(bytes);
  *bytes = kProductScratch;
  return MOE_OK;
}

moe_status moe_int4_grouped_gemm(const moe_int4_tensor* w, int64_t rows, const void* x, int64_t ldx,
                                 const int32_t* counts, const int32_t* offsets, int32_t swiglu,
                                 void* out, int64_t ldo, void* scratch, void* stream) {
  OP_TRY(check_int4(w));
  OP_TRY(check_segments(w->groups, rows, counts, offsets));
  OP_REQUIRE(swiglu == 0 || (swiglu == 1 && w->N % 32 == 0));
  OP_REQUIRE(al16(scratch));
  if (!few_fits(rows, (int)w->groups, w->N, w->K)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  OP_REQUIRE(rows_ok(x, ldx, w->K) && rows_ok(out, ldo, swiglu ? w->N / 2 : w->N));
  FewProduct p = few_product(w->groups, rows, w->N, w->K, counts, offsets, out, ldo, scratch);
  p.group = w->group;
  OP_CUDA(launch_product_few(p, x, ldx, w->codes, w->scales, w->zeros, swiglu != 0,
                             (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_int4_dequantize(const moe_int4_tensor* w, void* out, void* stream) {
  OP_TRY(check_int4(w));
  if (w->groups > kMaxGroups) return MOE_ERR_UNSUPPORTED;
  OP_REQUIRE(al16(out));
  OP_CUDA(launch_int4_dequantize(w->codes, w->scales, w->zeros, (int)w->groups, (int)w->N,
                                 (int)w->K, w->group, out, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_grouped_gemm(int64_t groups, int64_t rows, int64_t N, int64_t K, const void* x,
                            int64_t ldx, const void* w, const int32_t* counts,
                            const int32_t* offsets, const void* add, int64_t ldadd, void* out,
                            int64_t ldo, int64_t expected_rows, void* scratch, void* stream) {
  OP_TRY(check_product(groups, rows, N, K, w, counts, offsets, scratch));
  OP_REQUIRE(expected_rows >= 0);
  if (rows == 0) return MOE_OK;
  OP_REQUIRE(rows_ok(x, ldx, K) && rows_ok(out, ldo, N) && rows_or_null(add, ldadd, N));
  const int64_t most = expected_rows > 0 && expected_rows < rows ? expected_rows : rows;
  const RaggedProduct rp = ragged_product(groups, rows, counts, offsets, add, ldadd, out, ldo, scratch);
  if (short_fits(rows, (int)groups, N, K, add != nullptr)) {
    OP_CUDA(launch_product_short(rp, 0, x, ldx, w, (int)N, (int)K, (cudaStream_t)stream));
    return MOE_OK;
  }
  FewProduct p = few_product(groups, rows, N, K, counts, offsets, out, ldo, scratch);
  p.add = bf(add);
  p.ldadd = ldadd;
  if (few_rows(most) && few_fits(rows, (int)groups, N, K)) {
    OP_CUDA(launch_product_few(p, x, ldx, w, nullptr, nullptr, false, (cudaStream_t)stream));
    return MOE_OK;
  }
  if (narrow_fits(rows, (int)groups, N, K)) {
    OP_CUDA(launch_product_narrow(p, 0, x, ldx, w, (int)N, (int)K, (cudaStream_t)stream));
    return MOE_OK;
  }
  if (!ragged_fits(rows, (int)groups, N, 0)) return MOE_ERR_UNSUPPORTED;
  OP_CUDA(launch_ragged_gemm(rp, 0, x, ldx, w, (int)N, (int)K, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_grouped_gemm_dgrad(int64_t groups, int64_t rows, int64_t N, int64_t K,
                                  const void* dy, int64_t lddy, const void* w,
                                  const int32_t* counts, const int32_t* offsets, const void* add,
                                  int64_t ldadd, void* dx, int64_t lddx, void* scratch,
                                  void* stream) {
  OP_TRY(check_product(groups, rows, N, K, w, counts, offsets, scratch));
  if (rows == 0) return MOE_OK;
  OP_REQUIRE(rows_ok(dy, lddy, N) && rows_ok(dx, lddx, K) && rows_or_null(add, ldadd, K));
  const RaggedProduct rp =
      ragged_product(groups, rows, counts, offsets, add, ldadd, dx, lddx, scratch);
  if (short_fits(rows, (int)groups, K, N, add != nullptr)) {
    OP_CUDA(launch_product_short(rp, 1, dy, lddy, w, (int)N, (int)K, (cudaStream_t)stream));
    return MOE_OK;
  }
  if (narrow_fits(rows, (int)groups, K, N)) {
    FewProduct p = few_product(groups, rows, N, K, counts, offsets, dx, lddx, scratch);
    p.add = bf(add);
    p.ldadd = ldadd;
    OP_CUDA(launch_product_narrow(p, 1, dy, lddy, w, (int)N, (int)K, (cudaStream_t)stream));
    return MOE_OK;
  }
  if (!ragged_fits(rows, (int)groups, K, 0)) return MOE_ERR_UNSUPPORTED;
  OP_CUDA(launch_ragged_gemm(rp, 1, dy, lddy, w, (int)N, (int)K, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_grouped_gemm_wgrad(int64_t groups, int64_t rows, int64_t N, int64_t K,
                                  const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                  const int32_t* counts, const int32_t* offsets, void* dw,
                                  void* scratch, void* stream) {
  OP_TRY(check_product(groups, rows, N, K, dw, counts, offsets, scratch));
  if (rows > 0) OP_REQUIRE(rows_ok(dy, lddy, N) && rows_ok(x, ldx, K));
  if (!ragged_fits(rows, (int)groups, N, K)) return MOE_ERR_UNSUPPORTED;
  OP_CUDA(launch_ragged_wgrad(
      ragged_product(groups, rows, counts, offsets, nullptr, 0, dw, K, scratch), dy, lddy, x, ldx,
      (int)N, (int)K, (cudaStream_t)stream));
  return MOE_OK;
}

}  // extern "C"
