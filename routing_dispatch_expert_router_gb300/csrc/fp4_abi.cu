// C entry points of the 4-bit experts: argument checks and launches.
#include <limits.h>

#include "fp4_layout.cuh"
#include "internal.h"

using namespace moe;

namespace {

// Scratch of a product: the status word, each CTA's count of its launches, the arrival
// counters of the parts of cut tiles (8 epilogue warps each), then the fp32 parts.
constexpr int64_t kLaunchesOffset = 1024;
constexpr int64_t kArrivedOffset = 4096;
constexpr int kArrived = 8192;
constexpr int64_t kPartOffset = 65536;
constexpr int64_t kPartBytes = 39LL << 19;       // 64 rows in two parts per SM
constexpr int64_t kGemmScratch = kPartOffset + kPartBytes;
static_assert(kLaunchesOffset + kFp4SplitCtas * 4 <= kArrivedOffset, "launches before the counters");
static_assert(kArrivedOffset + kArrived * 4 <= kPartOffset, "counters before the parts");

#define FP4_TRY(expr)                  \
  do {                                 \
    const moe_status _s = (expr);      \
    if (_s != MOE_OK) return _s;       \
  } while (0)

#define FP4_CUDA(expr)                                                        \
  do {                                                                        \
    const cudaError_t _e = (expr);                                            \
    if (_e != cudaSuccess)                                                    \
      return _e == cudaErrorInvalidValue ? MOE_ERR_INVALID_ARG : MOE_ERR_CUDA; \
  } while (0)

#define FP4_REQUIRE(cond)                      \
  do {                                         \
    if (!(cond)) return MOE_ERR_INVALID_ARG;   \
  } while (0)

bool al16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
bool al16_or_null(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
bool al4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

bool format_ok(int f) { return f == MOE_FP4_NV || f == MOE_FP4_MX; }
bool scale_ok(int f, int log2) { return f == MOE_FP4_NV ? log2 >= -64 && log2 <= 64 : log2 == 0; }

int32_t* status_of(void* scratch) { return static_cast<int32_t*>(scratch); }

// Sizes that the kernels' 32-bit coordinates and grids hold.
moe_status check_tensor(const moe_fp4_tensor* q) {
  FP4_REQUIRE(q && format_ok(q->format) && scale_ok(q->format, q->scale_log2));
  FP4_REQUIRE(q->groups >= 0 && q->rows >= 0 && q->K >= 32 && q->K % 32 == 0);
  FP4_REQUIRE(q->K <= (1 << 24) && q->groups <= INT_MAX && q->rows <= INT_MAX);
  FP4_REQUIRE(q->groups == 0 || q->rows <= (INT_MAX - 1024) / q->groups - 128);
  if (q->groups == 0 || q->rows == 0) return MOE_OK;
  FP4_REQUIRE(al16(q->codes) && al16(q->scales));
  return MOE_OK;
}

Fp4Split split_of(void* scratch) {
  uint8_t* p = static_cast<uint8_t*>(scratch);
  return Fp4Split{reinterpret_cast<float*>(p + kPartOffset), kPartBytes / 4,
                  reinterpret_cast<uint32_t*>(p + kArrivedOffset), kArrived,
                  reinterpret_cast<uint32_t*>(p + kLaunchesOffset)};
}

// What an FFN call keeps behind a product's scratch.
struct FwdScratch {
  uint8_t *xq, *xsf, *hq, *hsf;
};
int64_t fwd_region(const moe_config& c, int fmt, void* scratch, FwdScratch* f) {
  const int64_t R = rows_max(c);
  const int64_t sizes[4] = {R * c.H / 2, f4::sf_bytes(fmt, R, c.H), R * c.F / 2,
                            f4::sf_bytes(fmt, R, c.F)};
  int64_t off = kGemmScratch;
  uint8_t* ptr[4];
  for (int i = 0; i < 4; ++i) {
    ptr[i] = scratch ? static_cast<uint8_t*>(scratch) + off : nullptr;
    off += up256(sizes[i]);
  }
  if (f) *f = FwdScratch{ptr[0], ptr[1], ptr[2], ptr[3]};
  return off;
}

// The backward's: [dG | dU] between the products, without the weights' scales; behind the
// counters of a forward that the caller runs on the same scratch.
constexpr int64_t kDguOffset = kPartOffset;
int64_t bwd_region(const moe_config& c) {
  return kDguOffset + up256(rows_max(c) * 2 * c.F * 2);
}

moe_status check_layer(const moe_config* cfg, const moe_fp4_experts* ex) {
  FP4_TRY(check_config(cfg));
  if (cfg->dtype != MOE_DTYPE_BF16 || cfg->weights_in_expert || cfg->stash_pool_pages)
    return MOE_ERR_UNSUPPORTED;
  FP4_REQUIRE(ex && ex->W13.format == ex->W2.format);
  FP4_TRY(check_tensor(&ex->W13));
  FP4_TRY(check_tensor(&ex->W2));
  const int64_t G = cfg->E + cfg->n_shared;
  FP4_REQUIRE(ex->W13.groups == G && ex->W13.rows == 2LL * cfg->F && ex->W13.K == cfg->H);
  FP4_REQUIRE(ex->W2.groups == G && ex->W2.rows == cfg->H && ex->W2.K == cfg->F);
  FP4_REQUIRE(al4_or_null(ex->alpha13) && al4_or_null(ex->alpha2));
  FP4_REQUIRE(scale_ok(ex->W13.format, ex->x_scale_log2) &&
              scale_ok(ex->W13.format, ex->h_scale_log2));
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_fp4_query_sizes(const moe_config* cfg, int32_t format, moe_fp4_sizes* out) {
  FP4_REQUIRE(out && format_ok(format));
  *out = moe_fp4_sizes{kGemmScratch, 0, 0};
  if (!cfg) return MOE_OK;
  FP4_TRY(check_config(cfg));
  if (cfg->dtype != MOE_DTYPE_BF16 || cfg->weights_in_expert || cfg->stash_pool_pages)
    return MOE_ERR_UNSUPPORTED;
  out->fwd_scratch_bytes = fwd_region(*cfg, format, nullptr, nullptr);
  out->bwd_scratch_bytes = bwd_region(*cfg);
  return MOE_OK;
}

moe_status moe_fp4_scale_bytes(int32_t format, int64_t rows, int64_t K, int64_t* bytes) {
  FP4_REQUIRE(bytes && format_ok(format) && rows >= 0 && K >= 32 && K % 32 == 0);
  FP4_REQUIRE(rows <= INT_MAX && K <= (1 << 24));
  *bytes = f4::sf_bytes(format, rows, K);
  return MOE_OK;
}

moe_status moe_fp4_quantize(const moe_fp4_tensor* q, const void* x, int64_t ldx,
                            const int32_t* counts, const int32_t* offsets, int32_t segments,
                            void* values, void* scratch, void* stream) {
  FP4_TRY(check_tensor(q));
  FP4_REQUIRE(ldx >= q->K && ldx % 8 == 0 && al4_or_null(scratch));
  if (counts || offsets || segments) {
    FP4_REQUIRE(al4(counts) && al4(offsets) && segments > 0 && q->groups <= 1);
  }
  if (q->groups == 0 || q->rows == 0) return MOE_OK;
  FP4_REQUIRE(al16(x) && al16_or_null(values));
  FP4_CUDA(launch_fp4_quantize(q->format, x, ldx, q->groups, q->rows, q->K, q->scale_log2, counts,
                               offsets, segments, static_cast<uint8_t*>(q->codes),
                               static_cast<uint8_t*>(q->scales), values, status_of(scratch),
                               (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_fp4_dequantize(const moe_fp4_tensor* q, void* out, int64_t ldo, void* stream) {
  FP4_TRY(check_tensor(q));
  FP4_REQUIRE(ldo >= q->K && ldo % 8 == 0);
  if (q->groups == 0 || q->rows == 0) return MOE_OK;
  FP4_REQUIRE(al16(out));
  FP4_CUDA(launch_fp4_dequantize(q->format, static_cast<const uint8_t*>(q->codes),
                                 static_cast<const uint8_t*>(q->scales), q->groups, q->rows, q->K,
                                 q->scale_log2, out, ldo, (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_fp4_grouped_gemm(const moe_fp4_tensor* a, const moe_fp4_tensor* b,
                                const int32_t* counts, const int32_t* offsets, const float* alpha,
                                void* out, void* scratch, void* stream) {
  FP4_TRY(check_tensor(a));
  FP4_TRY(check_tensor(b));
  FP4_REQUIRE(a->format == b->format && a->K == b->K && a->groups == 1 && b->groups >= 1);
  FP4_REQUIRE(b->rows % 8 == 0 && al4_or_null(alpha) && al16(scratch));
  if (b->groups > kMaxGroups) return MOE_ERR_UNSUPPORTED;
  if (counts || offsets) FP4_REQUIRE(al4(counts) && al4(offsets));
  else FP4_REQUIRE(b->groups == 1);
  if (a->rows == 0 || b->rows == 0) return MOE_OK;
  FP4_REQUIRE(al16(out));
  const Fp4Problem p{a->format, (int)b->groups, a->rows, b->rows, a->K,
                     static_cast<const uint8_t*>(a->codes), static_cast<const uint8_t*>(a->scales),
                     static_cast<const uint8_t*>(b->codes), static_cast<const uint8_t*>(b->scales),
                     counts, offsets, alpha, a->scale_log2 + b->scale_log2, false,
                     a->rows, a->rows / b->groups};
  FP4_CUDA(launch_fp4_gemm(p, out, split_of(scratch), status_of(scratch), (cudaStream_t)stream));
  return MOE_OK;
}

moe_status moe_fp4_ffn_fwd(const moe_config* cfg, const moe_fp4_experts* ex, const void* x_perm,
                           const int32_t* counts, const int32_t* offsets, void* ckpt,
                           void* ckpt_scale, void* y_perm, void* scratch, void* stream) {
  FP4_TRY(check_layer(cfg, ex));
  FP4_REQUIRE(al16(x_perm) && al4(counts) && al4(offsets) && al16(y_perm) && al16(scratch));
  FP4_REQUIRE(!ckpt == !ckpt_scale && al16_or_null(ckpt) && al16_or_null(ckpt_scale));
  cudaStream_t s = (cudaStream_t)stream;
  const int fmt = ex->W13.format, G = cfg->E + cfg->n_shared;
  const int64_t per_expert = (int64_t)cfg->T * cfg->k / cfg->E;
  const int64_t R = rows_max(*cfg), H = cfg->H, F = cfg->F;
  FwdScratch w;
  fwd_region(*cfg, fmt, scratch, &w);
  const Fp4Split sp = split_of(scratch);
  int32_t* st = status_of(scratch);
  FP4_CUDA(launch_fp4_quantize(fmt, x_perm, H, 1, R, H, ex->x_scale_log2, counts, offsets, G, w.xq,
                               w.xsf, nullptr, st, s));
  const Fp4Problem up{fmt, G, R, 2 * F, H, w.xq, w.xsf,
                      static_cast<const uint8_t*>(ex->W13.codes),
                      static_cast<const uint8_t*>(ex->W13.scales), counts, offsets, ex->alpha13,
                      ex->x_scale_log2 + ex->W13.scale_log2, true, cfg->T, per_expert};
  FP4_CUDA(launch_fp4_swiglu(up, w.hq, w.hsf, ex->h_scale_log2, static_cast<uint8_t*>(ckpt),
                             static_cast<uint8_t*>(ckpt_scale), sp, st, s));
  const Fp4Problem down{fmt, G, R, H, F, w.hq, w.hsf, static_cast<const uint8_t*>(ex->W2.codes),
                        static_cast<const uint8_t*>(ex->W2.scales), counts, offsets, ex->alpha2,
                        ex->h_scale_log2 + ex->W2.scale_log2, true, cfg->T, per_expert};
  FP4_CUDA(launch_fp4_gemm(down, y_perm, sp, st, s));
  return MOE_OK;
}

moe_status moe_fp4_ffn_bwd(const moe_config* cfg, const moe_fp4_experts* ex, const void* dO_perm,
                           const void* ckpt, const void* ckpt_scale, const int32_t* counts,
                           const int32_t* offsets, const int32_t* token_of, const float* dlogits,
                           const float* W_r, void* dX_perm, void* scratch, void* stream) {
  FP4_TRY(check_layer(cfg, ex));
  FP4_REQUIRE(al16(dO_perm) && al16(ckpt) && al16(ckpt_scale) && al4(counts) && al4(offsets));
  FP4_REQUIRE(al16(dX_perm) && al16(scratch));
  if (dlogits) FP4_REQUIRE(al4(dlogits) && al4(token_of) && al16(W_r));
  cudaStream_t s = (cudaStream_t)stream;
  const int fmt = ex->W13.format, G = cfg->E + cfg->n_shared;
  const int64_t per_expert = (int64_t)cfg->T * cfg->k / cfg->E;
  const int64_t R = rows_max(*cfg), H = cfg->H, F = cfg->F;
  uint8_t* dGU = static_cast<uint8_t*>(scratch) + kDguOffset;
  int32_t* st = status_of(scratch);
  const Fp4Problem down{fmt, G, R, F, H, static_cast<const uint8_t*>(dO_perm), nullptr,
                        static_cast<const uint8_t*>(ex->W2.codes),
                        static_cast<const uint8_t*>(ex->W2.scales), counts, offsets, nullptr, 0,
                        false, cfg->T, per_expert};
  FP4_CUDA(launch_fp4_dgrad_swiglu(down, static_cast<const uint8_t*>(ckpt),
                                   static_cast<const uint8_t*>(ckpt_scale), dGU, st, s));
  const Fp4Problem up{fmt, G, R, H, 2 * F, dGU, nullptr,
                      static_cast<const uint8_t*>(ex->W13.codes),
                      static_cast<const uint8_t*>(ex->W13.scales), counts, offsets, ex->alpha13,
                      ex->W13.scale_log2 + ex->W2.scale_log2, true, cfg->T, per_expert};
  FP4_CUDA(launch_fp4_dgrad_out(up, ex->alpha2, dX_perm, token_of, dlogits, W_r, cfg->E, cfg->T,
                                st, s));
  return MOE_OK;
}

}  // extern "C"
