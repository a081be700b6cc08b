// Host-side launchers shared between the translation units of the library.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_abi.h"
#include "per_device.h"

namespace moe {

moe_status check_config(const moe_config* c);
int64_t scratch_bytes(const moe_config& c);
int64_t capacity_rows(const moe_config& c);
int64_t rows_max(const moe_config& c);
int n_chunks(const moe_config& c);
int num_sms();
// The calling thread's device, -1 without one.
inline int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}
// A kernel's dynamic shared memory, set at its first launch on each device.
template <class Kernel>
cudaError_t set_smem_once(PerDevice& set, Kernel kern, int bytes) {
  int done = 0;
  return set.get(current_device(), &done, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}
// A launch that may be made ready while the kernel before it on the stream still runs (programmatic
// dependent launch). Every thread of such a kernel waits for that one's end (ptx::grid_dependency_wait)
// before its first access to memory: results are as in a plain launch, without its latency.
template <class... Params, class... Args>
cudaError_t launch_early(void (*kern)(Params...), unsigned grid, dim3 block, int smem, cudaStream_t s,
                         Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, static_cast<Params>(args)...);
}
// set_smem_once for a kernel of CTA pairs, and as many CTAs as can be resident at once (its tile
// loop strides over the pairs, so every launched pair must run).
template <class Kernel>
cudaError_t pair_grid_once(PerDevice& set, Kernel kern, int threads, int smem, int* grid) {
  return set.get(current_device(), grid, [&](int* v) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    lc.blockDim = dim3(threads, 1, 1);
    lc.dynamicSmemBytes = smem;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &lc);
    if (e != cudaSuccess || clusters <= 0) {
      (void)cudaGetLastError();
      clusters = num_sms() / 2;
    }
    *v = 2 * clusters;
    return cudaSuccess;
  });
}

cudaError_t launch_route(const moe_config& c, const void* x, const float* W_r, const float* bias,
                         float* logits, int32_t* idx, float* w, uint8_t* scratch, cudaStream_t s);
cudaError_t launch_route_replay(const moe_config& c, const void* x, const float* W_r,
                                const float* bias, const int32_t* idx, float* logits, float* w,
                                uint8_t* scratch, cudaStream_t s);

// Where a layer keeps the rows its backward reads (x_perm, GU, h, y_perm):
// row r is row pages[r / 128] * 128 + r % 128 of pool tensors of `rows` rows
// (paged stash), or row r of the layer's own rows_max-row buffers
// (pages == nullptr, rows == 0).
struct StashMap {
  const int32_t* pages = nullptr;
  int64_t rows = 0;
};
int64_t stash_rows(const moe_config& c, const StashMap& sm);
// The paged stash's allocation, done by the dispatch once the segment
// offsets are known: the layer's page table and the pool's page counter.
struct StashAlloc {
  int32_t* table;
  int32_t* top;
  int pool_pages;
};
// Gives the layer's pages back: *top = table[rows_max / 128 + 1].
cudaError_t launch_stash_release(const moe_config& c, const int32_t* table, int32_t* top,
                                 cudaStream_t s);

struct Fp8Scratch;
// fp8 (FP8 configuration, optional): also write x_perm's 1-byte form there.
// alloc (optional): take the layer's stash pages and write x_perm into them.
cudaError_t launch_permute(const moe_config& c, const void* x, const int32_t* idx,
                           int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* token_of,
                           int32_t* sel_offsets, int32_t* sel_tokens, void* x_perm,
                           uint8_t* scratch, cudaStream_t s, const Fp8Scratch* fp8 = nullptr,
                           const StashAlloc* alloc = nullptr);

// The dispatch of rows in 8 bits: the maps, and the rows and scale atoms alone (no bf16 rows).
cudaError_t launch_permute_fp8(const moe_config& c, const uint8_t* codes, const uint8_t* scales,
                               const int32_t* idx, int32_t* counts, int32_t* offsets,
                               int32_t* row_of, int32_t* token_of, int32_t* sel_offsets,
                               int32_t* sel_tokens, uint8_t* xq, uint8_t* xsf, uint8_t* scratch,
                               cudaStream_t s);

// pages (optional): y_perm is paged (StashMap).
cudaError_t launch_unpermute(const moe_config& c, const void* y_perm, const int32_t* row_of,
                             const float* w, const int32_t* offsets, void* out, cudaStream_t s,
                             const int32_t* pages = nullptr);

// dOq, dOsf (FP8 configuration, optional): also write dO_perm's 1-byte form.
// pages (optional): y_perm is paged; dO_perm is not.
cudaError_t launch_unpermute_bwd(const moe_config& c, const void* dY, const void* y_perm,
                                 const int32_t* row_of, const float* w, const int32_t* counts,
                                 const int32_t* offsets, void* dO_perm, float* dw, cudaStream_t s,
                                 uint8_t* dOq = nullptr, uint8_t* dOsf = nullptr,
                                 const int32_t* pages = nullptr);

// The layer with the routing weight inside the expert: the unweighted copy of
// dY into the expert rows (dO_perm), the routing weight of every permuted row,
// and dw from the FC2 data gradient's per-tile partial dot products.
cudaError_t launch_unpermute_bwd_copy(const moe_config& c, const void* dY, const int32_t* row_of,
                                      const int32_t* counts, const int32_t* offsets,
                                      void* dO_perm, cudaStream_t s);
cudaError_t launch_row_weights(const moe_config& c, const int32_t* token_of,
                               const int32_t* row_of, const float* w, const int32_t* offsets,
                               float* row_w, cudaStream_t s);
cudaError_t launch_dw_reduce(const moe_config& c, const float* dw_part, const int32_t* row_of,
                             float* dw, cudaStream_t s);
// Where the layer with the weight inside the expert keeps its per-row weights
// ([rows_max] fp32) and the partial dot products ([rows_max][dw_tiles] fp32).
struct ReorderScratch {
  float* row_w;
  float* dw_part;
};
ReorderScratch reorder_scratch(const moe_config& c, void* scratch);

cudaError_t launch_route_bwd(const moe_config& c, const float* logits, const int32_t* idx,
                             const float* w, const float* dw, float* dlogits, cudaStream_t s);

cudaError_t launch_permute_bwd(const moe_config& c, const void* dX_perm, const int32_t* row_of,
                               const int32_t* offsets, const int32_t* idx, const float* dlogits,
                               const float* W_r, void* dx, cudaStream_t s);

// dW_r (= or, with accumulate, +=) sum over tokens of dlogits[t,e] x[t,:]; with
// sel_offsets == sel_tokens == NULL every token counts for every expert
// (dense dlogits), else only the tokens that selected e.
cudaError_t launch_router_wgrad(const moe_config& c, const void* x, const int32_t* sel_offsets,
                                const int32_t* sel_tokens, const float* dlogits, float* dW_r,
                                uint8_t* scratch, cudaStream_t s, bool accumulate = false);

// Load-balancing loss: statistics, loss and bias update in one launch; its
// gradient into dlogits_aux, dx and dW_r.
cudaError_t launch_route_aux(const moe_config& c, const float* logits, const float* bias,
                             const int32_t* idx, float coeff, float rate, int32_t* counts,
                             float* p_mean, float* loss, float* bias_out, uint8_t* scratch,
                             cudaStream_t s);
cudaError_t launch_route_aux_bwd(const moe_config& c, const void* x, const float* logits,
                                 const float* bias, const float* W_r, const int32_t* counts,
                                 float coeff, float dloss, float* dl, void* dx, float* dW_r,
                                 uint8_t* scratch, cudaStream_t s);
int64_t aux_partial_bytes(const moe_config& c);    // the aux-loss region of scratch
int64_t aux_partial_offset(const moe_config& c);   // its byte offset in scratch

// FP8 block quantisation (E4M3 values with power-of-two block scales):
// 1-byte codes with UE8M0 scale atoms (fp8_layout.cuh) for the FP8 GEMMs --
// weights in 128x128 tiles (atoms for both orientations of the weight),
// activations in 1x128 slices along their rows -- and, for the bf16-path
// weight gradients, the dequantised values of 128x1 slices along the tokens.
cudaError_t launch_quant_tiles8(const void* W, uint8_t* Wq, uint8_t* sf_f, uint8_t* sf_d, int G,
                                int rows, int cols, cudaStream_t s);
// mx: 32-element blocks and the MX atom layout (MXFP8), else 128.
// pages (optional): X is a paged stash tensor (StashMap); the outputs are not.
cudaError_t launch_quant_cols8(const void* X, uint8_t* Xq, uint8_t* sf, const int32_t* offsets,
                               const int32_t* counts, int G, int64_t rows_max, int cols,
                               cudaStream_t s, bool mx = false, const int32_t* pages = nullptr);
// Both forms of one tensor from a single read: 1xBLK rows (Xr, sfr) and
// BLKx1 columns (Xc, sfc).
cudaError_t launch_quant_rows_cols8(const void* X, uint8_t* Xr, uint8_t* sfr, uint8_t* Xc,
                                    uint8_t* sfc, const int32_t* offsets, const int32_t* counts,
                                    int G, int64_t rows_max, int cols, cudaStream_t s,
                                    bool mx = false);
// The atoms of caller-quantised E4M3 weights from one UE8M0 code per 128x128 tile.
cudaError_t launch_load_fp8_scales(const uint8_t* scale, uint8_t* sf_f, uint8_t* sf_d, int G,
                                   int rows, int cols, cudaStream_t s);
// MXFP8 weights: forward (1x32 along cols) and data-gradient (32x1 along rows) forms.
cudaError_t launch_quant_wmx(const void* W, uint8_t* Wf, uint8_t* Wd, uint8_t* sf_f, uint8_t* sf_d,
                             int G, int rows, int cols, cudaStream_t s);

// Where the FP8 mode keeps its quantised tensors inside `scratch`.
struct Fp8Scratch {
  bool mx;          // MXFP8: 32-element blocks, MX atom layout, two weight forms
  uint8_t* W13q;    // [G,2F,H] E4M3 (forward form)
  uint8_t* W13qd;   // data-gradient form (MX), else W13q
  uint8_t* W13sf;   // atoms, N = W13 rows, K = H (forward)
  uint8_t* W13sft;  // atoms, N = H, K = W13 rows (FC1 data gradient)
  uint8_t* W2q;     // [G,H,F] E4M3 (forward form)
  uint8_t* W2qd;    // data-gradient form (MX), else W2q
  uint8_t* W2sf;    // atoms, N = H, K = F (forward)
  uint8_t* W2sft;   // atoms, N = F, K = H (FC2 data gradient)
  uint8_t* xq;      // [R,H] x_perm, 1x128 slices
  uint8_t* xsf;
  uint8_t* hq;      // [R,F] h
  uint8_t* hsf;
  uint8_t* dOq;     // [R,H] dO
  uint8_t* dOsf;
  uint8_t* dGq;     // [R,2F] dGU
  uint8_t* dGsf;
  // 128x1 slices along the tokens (weight gradients): E4M3 codes, then atoms
  // [columns / 128][row blocks / 4]
  uint8_t* cHq;     // [R,H]  dO
  uint8_t* cHsf;
  uint8_t* bFq;     // [R,F]  h
  uint8_t* bFsf;
  uint8_t* d2Fq;    // [R,2F] dGU
  uint8_t* d2Fsf;
  uint8_t* aHq;     // [R,H]  x_perm
  uint8_t* aHsf;
};
Fp8Scratch fp8_scratch(const moe_config& c, void* scratch);

// The 4-bit experts (fp4_layout.cuh, grouped_gemm_fp4.cu).
// bf16 rows to codes and scale atoms: groups x rows dense, or (counts != null,
// groups = 1) the rows [offsets[i], offsets[i] + counts[i]) of `segments`
// segments that start at multiples of 128. values (optional): what they stand for.
cudaError_t launch_fp4_quantize(int fmt, const void* x, int64_t ldx, int64_t groups, int64_t rows,
                                int64_t K, int scale_log2, const int32_t* counts,
                                const int32_t* offsets, int segments, uint8_t* codes,
                                uint8_t* scales, void* values, int32_t* status, cudaStream_t s);
cudaError_t launch_fp4_dequantize(int fmt, const uint8_t* codes, const uint8_t* scales,
                                  int64_t groups, int64_t rows, int64_t K, int scale_log2,
                                  void* out, int64_t ldo, cudaStream_t s);
// One grouped product: A [rows, K] by B [G, N, K], codes and scale atoms.
struct Fp4Problem {
  int fmt;
  int G;
  int64_t rows, N, K;
  const uint8_t* a;
  const uint8_t* sfa;
  const uint8_t* b;
  const uint8_t* sfb;
  const int32_t* counts;      // null: one group of all rows
  const int32_t* offsets;
  const float* alpha;         // [G] or null
  int unit_log2;              // the operands' tensor scales, as a power of two
  // The kernel before this one on the stream is one of this library's that
  // writes only A, and counts, offsets and alpha were complete before that one
  // began: this one may start while it runs (programmatic dependent launch).
  bool early;
  int64_t most_rows;          // no group has more rows than this
  int64_t mean_rows;          // about how many a group has
};
// Scratch of the products that cut K: fp32 parts, their arrival counters, and how often
// each CTA's index has run on this scratch (zero at first; the same number for every CTA
// of a launch).
struct Fp4Split {
  float* part;
  int64_t part_floats;
  uint32_t* arrived;
  int arrived_n;
  uint32_t* launches;
};
// The most CTAs that may share tiles: a counter has eight bits for a tile's parts.
constexpr int kFp4SplitCtas = 255;
cudaError_t launch_fp4_gemm(const Fp4Problem& q, void* out, const Fp4Split& sp, int32_t* status,
                            cudaStream_t s);
// The gate-up product with SwiGLU: h in 4 bits (hq, hsf), and the checkpoint of
// gate and up (E4M3 codes and UE8M0 bytes) where ckpt is given.
cudaError_t launch_fp4_swiglu(const Fp4Problem& q, uint8_t* hq, uint8_t* hsf, int h_scale_log2,
                              uint8_t* ckpt, uint8_t* ckpt_sf, const Fp4Split& sp, int32_t* status,
                              cudaStream_t s);

// Their data gradients: A bf16 [rows, K] by the 4-bit weights [G, K, N] (q.a is A;
// q.sfa is not used). FC2's, times SwiGLU's derivative from the 8-bit
// checkpoint -> dGU [rows, 2N] bf16, without the weights' scales; FC1's, with both
// products' scales (q.alpha, alpha_b, q.unit_log2) and the router's term where
// dlogits is given -> dX [rows, N] bf16.
cudaError_t launch_fp4_dgrad_swiglu(const Fp4Problem& q, const uint8_t* ckpt,
                                    const uint8_t* ckpt_sf, void* dGU, int32_t* status,
                                    cudaStream_t s);
cudaError_t launch_fp4_dgrad_out(const Fp4Problem& q, const float* alpha_b, void* dX,
                                 const int32_t* token_of, const float* dlogits, const float* W_r,
                                 int router_E, int router_T, int32_t* status, cudaStream_t s);

// RMS norm with the residual's addition (norm.cu): bf16 rows [T, H], ld* elements from row to
// row. residual, sum, out, rstd: or null; codes, scales: the output in E4M3 with a UE8M0 byte
// per `block` (32 or 128) values, contiguous, or null.
struct RmsNormFwd {
  int64_t T;
  int H;
  const __nv_bfloat16* x;
  int64_t ldx;
  const __nv_bfloat16* residual;
  int64_t ldr;
  const void* gamma;
  bool gamma_f32;
  float eps;
  __nv_bfloat16* sum;
  int64_t lds;
  __nv_bfloat16* out;
  int64_t ldo;
  uint8_t* codes;
  uint8_t* scales;
  int block;
  float* rstd;
};
cudaError_t launch_rmsnorm_fwd(const RmsNormFwd& p, cudaStream_t s);
// Its backward; dsum: or null. parts: [kRmsNormParts, H] fp32, null with dgamma.
struct RmsNormBwd {
  int64_t T;
  int H;
  const __nv_bfloat16* dy;
  int64_t lddy;
  const __nv_bfloat16* h;
  int64_t ldh;
  const float* rstd;
  const void* gamma;
  bool gamma_f32;
  const __nv_bfloat16* dsum;
  int64_t ldds;
  __nv_bfloat16* dx;
  int64_t lddx;
  float* parts;
};
constexpr int kRmsNormParts = 512;
cudaError_t launch_rmsnorm_bwd(const RmsNormBwd& p, float* dgamma, cudaStream_t s);

// Grouped products of few rows (product_few.cu): out[r] = x[r] W[g]^T (+ add) for the rows of
// every group g (counts, offsets; null: one group of all rows). W [G, N, K] in bf16 (scales null),
// or codes with scales [G, K / group, N] bf16 and zero points (null: 8) u8; swiglu (4-bit):
// out [rows, N / 2] = silu(first half) second half.
struct FewProduct {
  int G;
  int64_t rows;
  int N, K;
  const int32_t* counts;
  const int32_t* offsets;
  int group;                  // elements of K that share a scale (4-bit)
  const __nv_bfloat16* add;
  int64_t ldadd;
  __nv_bfloat16* out;
  int64_t ldo;
  float* parts;               // [2 kFewCtas][kFewPart] fp32
  uint32_t* arrived;          // [kFewCtas], zero before and after every launch
  int32_t* status;
  // set by the launcher
  int F, slabs, steps, groups_per_step;
  bool has_zeros, x_whole;
};
constexpr int kFewCtas = 256;
constexpr int kFewPart = 256 * 16;
// steps of K a CTA takes at least (they must weigh more than one; us, with two and with four: 4 rows
// of six experts through 4-bit 1008 x 1504 9.2 and 11.1, a row through 1024 x 1024 7.7 and 8.6; with bf16
// weights the same within 2 %)
constexpr int kFewLeast = 2;
// steps that joining a unit's parts takes the time of (us, with none, two and six: 128 rows of 64
// experts, bf16 512 x 512, 10.5, 7.9 and 7.8; the 4-bit cases above 9.2, 9.2, 11.6 and 7.8, 7.7, 8.5)
constexpr int kFewJoin = 2;
bool few_fits(int64_t rows, int G, int64_t N, int64_t K);
// Whether bf16 weights are streamed, groups having about `most` rows at most.
bool few_rows(int64_t most);
cudaError_t launch_product_few(FewProduct p, const void* x, int64_t ldx, const void* w,
                               const void* scales, const void* zeros, bool swiglu, cudaStream_t s);

// The same kernel for few outputs: the rows stream, the weights are what few there is of.
bool narrow_fits(int64_t rows, int G, int64_t outputs, int64_t reduction);
cudaError_t launch_product_narrow(FewProduct p, int dgrad, const void* x, int64_t ldx, const void* w,
                                  int N, int K, cudaStream_t s);

// The bf16 weights that 4-bit codes stand for: out [G, N, K].
cudaError_t launch_int4_dequantize(const void* codes, const void* scales, const void* zeros, int G,
                                   int N, int K, int group, void* out, cudaStream_t s);

// Grouped products of ragged rows (grouped_gemm_ragged.cu): W [G, N, K] bf16; forward
// [rows, K] -> [rows, N], data gradient [rows, N] -> [rows, K] (both + add, or null), weight
// gradient -> [G, N, K] (zeros for an empty group).
struct RaggedProduct {
  int G;
  int64_t rows;
  const int32_t* counts;      // null: one group of all rows
  const int32_t* offsets;
  const __nv_bfloat16* add;
  int64_t ldadd;
  __nv_bfloat16* out;
  int64_t ldo;
  float* parts;               // [kRaggedPairs][256 x 256] fp32
  uint32_t* arrived;          // [kRaggedPairs / 2][16], zero before and after every launch
  int32_t* status;
  // set by the launchers: features (the output's columns; the weight gradient's rows), the length
  // reduced over (not the weight gradient's), the weight gradient's columns, columns of a tile
  int feat, red, cols, tile;
};
constexpr int kRaggedPairs = 80;   // pairs of SMs, at most, that share reductions
// cols: of a weight gradient, else 0.
bool ragged_fits(int64_t rows, int G, int64_t feat, int64_t cols);
cudaError_t launch_ragged_gemm(RaggedProduct p, int dgrad, const void* x, int64_t ldx,
                               const void* w, int N, int K, cudaStream_t s);
// The two of a reduction of 64 at most (product_short.cu).
bool short_fits(int64_t rows, int G, int64_t feat, int64_t red, bool add);
cudaError_t launch_product_short(RaggedProduct p, int dgrad, const void* x, int64_t ldx,
                                 const void* w, int N, int K, cudaStream_t s);
cudaError_t launch_ragged_wgrad(RaggedProduct p, const void* dy, int64_t lddy, const void* x,
                                int64_t ldx, int N, int K, cudaStream_t s);

// Router logits for E % 128 == 0 on the tensor cores (W3 = W_r split in three bf16 parts).
cudaError_t launch_router_logits_tc(const moe_config& c, const void* x, const void* W3,
                                    float* logits, int32_t* status, cudaStream_t s);
cudaError_t launch_router_wgrad_tc(const moe_config& c, const void* x, const void* D3,
                                   long long Tp, float* P, int chunk, int32_t* status,
                                   cudaStream_t s);
// dx [T,H] bf16 += A3 [T,K3] . B3 [H,K3]^T (bf16 operands, K-major), on the tensor cores.
cudaError_t launch_router_dx_tc(const moe_config& c, const void* A3, const void* B3, int K3,
                                void* dx, int32_t* status, cudaStream_t s);
bool router_on_tensor_cores(const moe_config& c);
// tensor-core router weight gradient: tokens per chunk (<= 271 chunks), and
// the byte offset of the chunk partial sums after the split dlogits in the
// router region of scratch
int router_wgrad_chunk(const moe_config& c);
int64_t router_wgrad_split_bytes(const moe_config& c);
int64_t router_split_bytes(const moe_config& c);   // the router region of scratch
int64_t aux_dx_split_bytes(const moe_config& c);   // the loss's split dx operands in it
int64_t router_split_offset(const moe_config& c);   // byte offset of the split in scratch
int64_t permute_scratch_bytes(const moe_config& c); // scratch the dispatch needs

// Grouped GEMMs (tcgen05). Return cudaErrorInvalidValue when a tensor map
// cannot be encoded for the given pointers. sm: where x_perm, GU, h and y_perm
// live (the other row tensors are the layer's own, at their rows).
// row_w (the routing weight inside the expert, optional): h = w_row silu(G) U.
cudaError_t launch_ffn_fc1(const moe_config& c, const void* x_perm, const int32_t* counts,
                           const int32_t* offsets, const void* W13, void* GU, void* h,
                           int32_t* status, cudaStream_t s, const float* row_w = nullptr,
                           const StashMap& sm = StashMap());
cudaError_t launch_ffn_fc2(const moe_config& c, const void* h, const int32_t* counts,
                           const int32_t* offsets, const void* W2, void* y_perm,
                           int32_t* status, cudaStream_t s, const StashMap& sm = StashMap());
// row_w, dw_part (optional): the weight inside the expert -- dh = w_row dh_s,
// and dw_part[r * dw_tiles(c) + n-tile] = the row's <dh_s, h> over that tile.
// h_out (optional): h [rows, F] rewritten from GU (fine-grained recompute).
cudaError_t launch_ffn_fc2_dgrad(const moe_config& c, const void* dO_perm, const int32_t* counts,
                                 const int32_t* offsets, const void* W2, const void* GU,
                                 void* dGU, int32_t* status, cudaStream_t s,
                                 const float* row_w = nullptr, float* dw_part = nullptr,
                                 void* h_out = nullptr, const StashMap& sm = StashMap());
int dw_tiles(const moe_config& c);
cudaError_t launch_ffn_fc1_dgrad(const moe_config& c, const void* dGU, const int32_t* counts,
                                 const int32_t* offsets, const void* W13, const int32_t* token_of,
                                 const float* dlogits, const float* W_r, void* dX_perm,
                                 int32_t* status, cudaStream_t s);
cudaError_t launch_ffn_wgrad_fc2(const moe_config& c, const void* dO_perm, const void* h,
                                 const int32_t* counts, const int32_t* offsets, void* dW2,
                                 int32_t* status, cudaStream_t s, const StashMap& sm = StashMap());
cudaError_t launch_ffn_wgrad_fc1(const moe_config& c, const void* dGU, const void* x_perm,
                                 const int32_t* counts, const int32_t* offsets, void* dW13,
                                 int32_t* status, cudaStream_t s, const StashMap& sm = StashMap());

// The FP8 configuration's forward and data-gradient GEMMs on the block-scaled
// FP8 tensor cores (tcgen05 kind::mxf8f6f4): E4M3 operands with UE8M0 scale
// atoms; the same epilogues and outputs as the bf16 launches above.
cudaError_t launch_ffn_fc1_fp8(const moe_config& c, const uint8_t* xq, const uint8_t* xsf,
                               const int32_t* counts, const int32_t* offsets, const uint8_t* W13q,
                               const uint8_t* W13sf, void* GU, void* h, uint8_t* hq, uint8_t* hsf,
                               int32_t* status, cudaStream_t s, const StashMap& sm = StashMap());
cudaError_t launch_ffn_fc2_fp8(const moe_config& c, const uint8_t* hq, const uint8_t* hsf,
                               const int32_t* counts, const int32_t* offsets, const uint8_t* W2q,
                               const uint8_t* W2sf, void* y_perm, int32_t* status,
                               cudaStream_t s, const StashMap& sm = StashMap());
cudaError_t launch_ffn_fc2_dgrad_fp8(const moe_config& c, const uint8_t* dOq, const uint8_t* dOsf,
                                     const int32_t* counts, const int32_t* offsets,
                                     const uint8_t* W2q, const uint8_t* W2sf_t, const void* GU,
                                     void* dGU, int32_t* status, cudaStream_t s,
                                     void* h_out = nullptr, const StashMap& sm = StashMap());
cudaError_t launch_ffn_fc1_dgrad_fp8(const moe_config& c, const uint8_t* dGq, const uint8_t* dGsf,
                                     const int32_t* counts, const int32_t* offsets,
                                     const uint8_t* W13q, const uint8_t* W13sf_t,
                                     const int32_t* token_of, const float* dlogits,
                                     const float* W_r, void* dX_perm, int32_t* status,
                                     cudaStream_t s);
// Weight gradients over the 128x1-slice operands (K = each group's rows):
// dW2[g] = dO^T h, dW13[g] = dGU^T x_perm (bf16; zero for empty groups).
cudaError_t launch_ffn_wgrad_fc2_fp8(const moe_config& c, const uint8_t* dOq, const uint8_t* dOsf,
                                     const uint8_t* hq, const uint8_t* hsf, const int32_t* counts,
                                     const int32_t* offsets, void* dW2, int32_t* status,
                                     cudaStream_t s);
cudaError_t launch_ffn_wgrad_fc1_fp8(const moe_config& c, const uint8_t* dGq, const uint8_t* dGsf,
                                     const uint8_t* xq, const uint8_t* xsf, const int32_t* counts,
                                     const int32_t* offsets, void* dW13, int32_t* status,
                                     cudaStream_t s);

}  // namespace moe
