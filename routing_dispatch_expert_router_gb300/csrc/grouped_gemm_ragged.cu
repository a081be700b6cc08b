// Grouped products of ragged rows on the fifth-generation tensor cores: for the rows r of every
// group g, which follow each other without padding at any offset,
//   forward          y[r] = x[r] W[g]^T         (A x, B W, both K-major)
//   data gradient    dx[r] = dy[r] W[g]         (B MN-major: W read as it lies)
//   weight gradient  dW[g] = sum of dy[r]^T x[r] (both MN-major, the rows reduced over)
// in one kernel, a persistent CTA per SM: TMA producer, MMA issuer, four epilogue warps, two
// accumulators in tensor memory, as in the experts' FFN. What the raggedness adds:
//   - the weights' maps have the expert as a dimension of their own, so that a box that passes
//     an expert's last row or column reads zeros and not the next expert's;
//   - a tile's rows past its group's end are the next group's (each row of A makes its own row
//     of the product alone); the epilogue leaves them out: 32 rows that are all the group's go
//     by TMA, the last few lane by lane;
//   - the weight gradient's last block of rows holds the next group's rows in both operands:
//     the issuing warp zeroes them in shared memory (both: zero times a NaN is one).
#include "gemm_common.cuh"

namespace moe {
namespace {

using gg::BK;
using gg::BM;
using gg::kThreads;
using gg::kWaitBudget;

enum Mode : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kCtrl = 5120;
constexpr int kOutBox = 32 * 128;               // 32 rows x 64 bf16

template <int BN>
struct Cfg {
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int STAGE = A_BYTES + BN * BK * 2;
  static constexpr int SMEM = STAGES * STAGE + kCtrl + 4 * kOutBox + 1024;
};
static_assert(Cfg<256>::SMEM <= 232448 && Cfg<128>::SMEM <= 232448 && Cfg<64>::SMEM <= 232448,
              "shared memory");

// 64 columns of 32 rows, one row a lane, from tensor memory to the output.
template <int MODE>
__device__ __forceinline__ void store64(const RaggedProduct& p, const CUtensorMap* tmC,
                                        uint32_t taddr, bool zero, int g, int64_t row, int rows_left,
                                        int out_row, int col, int lane, uint8_t* stage,
                                        uint32_t stage_u32) {
  uint32_t r0[32], r1[32];
  if (zero) {
#pragma unroll
    for (int i = 0; i < 32; ++i) r0[i] = r1[i] = 0u;
  } else {
    ptx::tmem_ld32(taddr, r0);
    ptx::tmem_ld32(taddr + 32, r1);
    ptx::tmem_ld_wait();
  }
  if (MODE != kWgrad && p.add && lane < rows_left) {
    const __nv_bfloat16* src = p.add + (row + lane) * p.ldadd + col;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      if (col + 8 * v >= p.cols) break;
      float f[8];
      unpack8(*reinterpret_cast<const uint4*>(src + 8 * v), f);
      uint32_t* r = v < 4 ? r0 + 8 * v : r1 + 8 * (v - 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + f[i]);
    }
  }
  uint4 o[8];
  {
    uint4 a[4], b[4];
    gg::pack_slice(r0, a);
    gg::pack_slice(r1, b);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      o[v] = a[v];
      o[4 + v] = b[v];
    }
  }
  if (MODE != kWgrad && rows_left < 32) {
    if (lane < rows_left) {
      __nv_bfloat16* dst = p.out + (row + lane) * p.ldo + col;
#pragma unroll
      for (int v = 0; v < 8; ++v)
        if (col + 8 * v < p.cols) stg_v4(dst + 8 * v, o[v]);
    }
    return;
  }
  // the staging box is free once TMA has read the previous one
  if (lane == 0) ptx::tma_store_wait_read();
  __syncwarp();
  uint8_t* rowp = stage + lane * 128;             // chunk j of row r at j ^ (r & 7)
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(rowp + ((j ^ (lane & 7)) << 4)) = o[j];
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (MODE == kWgrad) ptx::tma_store_3d(tmC, stage_u32, col, out_row, g);
    else ptx::tma_store_2d(tmC, stage_u32, col, (int)row);
    ptx::tma_store_commit();
  }
}

template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1)
ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmC, const RaggedProduct p) {
  using C = Cfg<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* out_stage = smem_raw + (base - raw) + STAGES * C::STAGE;
  const uint32_t out_stage_u32 = base + STAGES * C::STAGE;
  uint8_t* ctrl = out_stage + 4 * kOutBox;
  const uint32_t ctrl_u = out_stage_u32 + 4 * kOutBox;
  const uint32_t bar_full = ctrl_u, bar_empty = ctrl_u + 64;       // [STAGES] each
  const uint32_t bar_tfull = ctrl_u + 128, bar_tempty = ctrl_u + 144, bar_drain = ctrl_u + 160;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 196);
  int* prefix = reinterpret_cast<int*>(ctrl + 256);       // [kMaxGroups + 1] tiles
  int* s_off = reinterpret_cast<int*>(ctrl + 1536);       // [kMaxGroups]
  int* s_cnt = reinterpret_cast<int*>(ctrl + 2688);       // [kMaxGroups]
  int* tmp = reinterpret_cast<int*>(ctrl + 3840);         // [33]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NT = (p.cols + BN - 1) / BN;
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(bar_tfull + 8 * a, 1);
      ptx::mbar_init(bar_tempty + 8 * a, 128);
    }
    ptx::mbar_init(bar_drain, 1);
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
    ptx::tma_prefetch_desc(&tmC);
  }
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  for (int g = tid; g < p.G; g += kThreads) {
    int c = (int)p.rows, o = 0;
    if (p.counts) {
      c = p.counts[g];
      o = p.offsets[g];
      if (c < 0 || o < 0 || (int64_t)o + c > p.rows) {
        if (blockIdx.x == 0) record_status(p.status, MOE_ERR_DEVICE_CHECK);
        c = 0;
      }
    }
    s_cnt[g] = c;
    s_off[g] = o;
    prefix[g] = ((MODE == kWgrad ? p.out_rows : c) + BM - 1) / BM * NT;
  }
  __syncthreads();
  const int total = block_exclusive_scan(prefix, p.G, tmp);
  if (tid == 0) prefix[p.G] = total;
  __syncthreads();
  if ((int)blockIdx.x >= total) return;

  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 2 * BN);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  struct Tile {
    int g, mt, nt, nk;
  };
  auto tile_at = [&](int tile) {
    Tile t;
    t.g = gg::find_group(prefix, p.G, tile);
    const int local = tile - prefix[t.g];
    if (MODE == kWgrad) {
      // n fastest: tiles that run together share A's columns
      t.nt = local % NT;
      t.mt = local / NT;
      t.nk = (s_cnt[t.g] + BK - 1) / BK;
    } else {
      // m fastest: they share the expert's weights
      const int mt = (s_cnt[t.g] + BM - 1) / BM;
      t.mt = local % mt;
      t.nt = local / mt;
      t.nk = (p.red + BK - 1) / BK;
    }
    return t;
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = tile_at(tile);
        for (int kb = 0; kb < t.nk; ++kb) {
          if (!ptx::mbar_wait(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * stage;
          ptx::mbar_arrive_expect_tx(fb, C::STAGE);
          const uint32_t sA = base + stage * C::STAGE, sB = sA + C::A_BYTES;
          const int k0 = kb * BK;
          if (MODE == kWgrad) {
            const int r = s_off[t.g] + k0;
#pragma unroll
            for (int j = 0; j < BM / 64; ++j)
              ptx::tma_load_2d(sA + j * 8192, &tmA, fb, t.mt * BM + 64 * j, r);
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              ptx::tma_load_2d(sB + j * 8192, &tmB, fb, t.nt * BN + 64 * j, r);
          } else {
            ptx::tma_load_2d(sA, &tmA, fb, k0, s_off[t.g] + t.mt * BM);
            if (MODE == kFwd) {
              ptx::tma_load_3d(sB, &tmB, fb, k0, t.nt * BN, t.g);
            } else {
#pragma unroll
              for (int j = 0; j < BN / 64; ++j)
                ptx::tma_load_3d(sB + j * 8192, &tmB, fb, t.nt * BN + 64 * j, k0, t.g);
            }
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every load issued must land before the CTA may exit
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s))
          ptx::mbar_wait(bar_full + 8 * s, (issued_phase >> s) & 1u, kWaitBudget, nullptr);
    }
  } else if (warp == 1) {
    // the whole warp walks the blocks (a weight gradient's last one is zeroed by all lanes),
    // one lane issues
    constexpr int A_MN = MODE == kWgrad, B_MN = MODE != kFwd;
    constexpr uint32_t IDESC = ptx::idesc_bf16(BM, BN, A_MN, B_MN);
    uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
    bool ok = true, issued = false;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_tempty + 8 * acc, acc_phase ^ 1u, kWaitBudget,
                                                  abort_flag));
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem_base + acc * BN;
      for (int kb = 0; kb < t.nk; ++kb) {
        ok = __all_sync(0xffffffffu,
                        ptx::mbar_wait(bar_full + 8 * stage, phase, kWaitBudget, abort_flag));
        if (!ok) break;
        const uint32_t sA = base + stage * C::STAGE, sB = sA + C::A_BYTES;
        if (MODE == kWgrad) {
          const int valid = s_cnt[t.g] - kb * BK;
          if (valid < BK) {
            // rows valid .. 63 of every 64-column chunk of A and B (128 bytes a row)
            for (int j = 0; j < (BM + BN) / 64; ++j)
              for (int b = valid * 128 + lane * 16; b < 8192; b += 512)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};"
                             :: "r"(sA + j * 8192 + b), "r"(0u) : "memory");
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
        }
        ptx::tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = A_MN ? ptx::smem_desc_sw128(sA + kk * 2048, 8192, 1024)
                                     : ptx::smem_desc_sw128(sA + kk * 32, 16, 1024);
            const uint64_t bd = B_MN ? ptx::smem_desc_sw128(sB + kk * 2048, 8192, 1024)
                                     : ptx::smem_desc_sw128(sB + kk * 32, 16, 1024);
            ptx::mma_bf16(d, ad, bd, IDESC, (kb | kk) ? 1u : 0u);
          }
          ptx::mma_commit(bar_empty + 8 * stage);
        }
        __syncwarp();
        issued = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) {
        if (t.nk > 0) ptx::mma_commit(bar_tfull + 8 * acc);
        else ptx::mbar_arrive(bar_tfull + 8 * acc);     // an empty group: nothing to wait for
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // every MMA issued by this thread is waited for before tensor memory is freed
    if (issued && lane == 0) {
      ptx::mma_commit(bar_drain);
      ptx::mbar_wait(bar_drain, 0, kWaitBudget, nullptr);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;                              // tensor-memory lane quarter
    uint8_t* stage = out_stage + (warp - 2) * kOutBox;
    const uint32_t stage_u32 = out_stage_u32 + (warp - 2) * kOutBox;
    uint32_t acc = 0, acc_phase = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      bool ok = ptx::mbar_wait(bar_tfull + 8 * acc, acc_phase, kWaitBudget, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      ptx::tc_fence_after();
      const int m0 = t.mt * BM + q * 32;
      const int rows_left = (MODE == kWgrad ? p.out_rows : s_cnt[t.g]) - m0;
      const int64_t row = (int64_t)s_off[t.g] + m0;
      const uint32_t tbase = tmem_base + acc * BN + ((uint32_t)(q * 32) << 16);
      if (rows_left > 0) {
#pragma unroll 1
        for (int c = 0; c < BN; c += 64) {
          const int col = t.nt * BN + c;
          if (col >= p.cols) break;
          store64<MODE>(p, &tmC, tbase + c, t.nk == 0, t.g, row, rows_left, m0, col, lane, stage,
                        stage_u32);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar_tempty + 8 * acc);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) ptx::tma_store_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 2 * BN);
  }
}

// bf16 rows [rows, cols], ld elements apart; a matrix per group behind each other.
bool map2(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t b0,
          uint32_t b1) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = gg::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {b0, b1};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map3(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t groups,
          uint32_t b0, uint32_t b1) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = gg::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, groups};
  cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  cuuint32_t box[3] = {b0, b1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int BN>
cudaError_t run_ragged(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                       const RaggedProduct& p, cudaStream_t s) {
  auto kern = ragged_gemm_kernel<MODE, BN>;
  static PerDevice set;
  const cudaError_t e = set_smem_once(set, kern, Cfg<BN>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)num_sms(), dim3(kThreads, 1, 1), Cfg<BN>::SMEM, s, a, b, c, p);
}

// Columns of a tile: as wide as fills the SMs (a wider tile reads A less often, but few tiles
// leave SMs without one, and a narrow output multiplies nothing by padding).
int tile_columns(int cols, int64_t row_tiles) {
  const int sms = num_sms();
  for (int bn = 256; bn > 64; bn /= 2)
    if (cols > bn / 2 && row_tiles * ((cols + bn - 1) / bn) >= sms) return bn;
  return 64;
}

}  // namespace

// Tiles of 128 rows and 64 columns at least, in 32 bits.
bool ragged_fits(int64_t rows, int G, int64_t cols, int64_t out_rows) {
  const int64_t m = out_rows ? (out_rows + 127) / 128 * G : rows / 128 + G;
  return m * ((cols + 63) / 64) < (1LL << 31);
}

cudaError_t launch_ragged_gemm(RaggedProduct p, int dgrad, const void* x, int64_t ldx,
                               const void* w, int N, int K, cudaStream_t s) {
  p.cols = dgrad ? K : N;
  p.red = dgrad ? N : K;
  p.out_rows = 0;
  const int64_t tiles = p.rows / BM + (p.rows < p.G ? p.rows : p.G);
  const int bn = tile_columns(p.cols, tiles);
  CUtensorMap a, b, c;
  if (!map2(&a, x, p.red, p.rows, ldx, 64, BM) || !map2(&c, p.out, p.cols, p.rows, p.ldo, 64, 32) ||
      !map3(&b, w, K, N, p.G, 64, dgrad ? 64 : bn))
    return cudaErrorInvalidValue;
  if (dgrad)
    return bn == 256   ? run_ragged<kDgrad, 256>(a, b, c, p, s)
           : bn == 128 ? run_ragged<kDgrad, 128>(a, b, c, p, s)
                       : run_ragged<kDgrad, 64>(a, b, c, p, s);
  return bn == 256   ? run_ragged<kFwd, 256>(a, b, c, p, s)
         : bn == 128 ? run_ragged<kFwd, 128>(a, b, c, p, s)
                     : run_ragged<kFwd, 64>(a, b, c, p, s);
}

cudaError_t launch_ragged_wgrad(RaggedProduct p, const void* dy, int64_t lddy, const void* x,
                                int64_t ldx, int N, int K, cudaStream_t s) {
  p.cols = K;
  p.out_rows = N;
  p.red = 0;
  p.add = nullptr;
  const int bn = tile_columns(K, (int64_t)p.G * ((N + BM - 1) / BM));
  CUtensorMap a, b, c;
  // (without rows nothing is loaded: the maps are then of any valid extent)
  const int64_t rows = p.rows > 0 ? p.rows : 1;
  if (!map2(&a, p.rows > 0 ? dy : p.out, N, rows, p.rows > 0 ? lddy : (N + 7) / 8 * 8, 64, 64) ||
      !map2(&b, p.rows > 0 ? x : p.out, K, rows, p.rows > 0 ? ldx : (K + 7) / 8 * 8, 64, 64) ||
      !map3(&c, p.out, K, N, p.G, 64, 32))
    return cudaErrorInvalidValue;
  return bn == 256   ? run_ragged<kWgrad, 256>(a, b, c, p, s)
         : bn == 128 ? run_ragged<kWgrad, 128>(a, b, c, p, s)
                     : run_ragged<kWgrad, 64>(a, b, c, p, s);
}

}  // namespace moe
