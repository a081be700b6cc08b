// Quantisation of bf16 rows to 4 bits and back (fp4_layout.cuh has the formats).
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (es
// summary, Resumen técnico §2.4) names NVFP4 beside MXFP8 as Blackwell's
// recipes for the expert GEMMs, and §2.3.A keeping activations in FP8/FP4.
//
// Both directions are one pass bounded by HBM. A warp takes the rows r, r + 32,
// r + 64, r + 96 of a 128-row slab, eight lanes to a row and one block to a
// lane: a row's eight blocks are consecutive (256 or 512 bytes of bf16), and the
// scale bytes of the four rows are whole 16-byte lines of two atoms, written
// without staging. A block's maximum and its codes need no other lane.
#include "fp4_layout.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQCols = 512;                      // columns of one turn of a CTA

// Rows of a 128-row slab that hold data, and where the slab lies. Dense
// tensors: groups x rows; ragged: the rows [offsets[g], offsets[g] + counts[g])
// of one tensor, whose segments start at multiples of 128.
struct Rows {
  int64_t rows, K, ldx;
  const int32_t* counts;
  const int32_t* offsets;
  int segments;
  int32_t* status;
};

// First row (in the tensor) and row count of slab `sl`; 0 rows when it is empty. All
// threads of the block call it (ragged form: each looks at some of the segments, one
// load deep where a search would be as deep as their number's logarithm).
__device__ __forceinline__ int slab_rows(const Rows& p, int64_t sl, int64_t& row0) {
  if (!p.counts) {
    const int64_t per = f4::slabs(p.rows), g = sl / per, r = (sl - g * per) * 128;
    row0 = g * p.rows + r;
    return (int)min((int64_t)128, p.rows - r);
  }
  __shared__ int found;
  row0 = sl * 128;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.segments; i += blockDim.x) {
    const int64_t off = p.offsets[i], cnt = p.counts[i];
    if (off < 0 || off % 128 || cnt < 0 || off + cnt > p.rows) {
      record_status(p.status, MOE_ERR_DEVICE_CHECK);
    } else if (off <= row0 && row0 < off + cnt) {
      found = (int)min((int64_t)128, off + cnt - row0);
    }
  }
  __syncthreads();
  return found;
}

template <int FMT, bool VALUES>
__global__ void __launch_bounds__(kQThreads)
fp4_quantize_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales, __nv_bfloat16* __restrict__ values, float up,
                    float down, int turns, const Rows p) {
  constexpr int BLK = f4::block_of(FMT);
  constexpr int V = BLK / 8;                     // 16-byte vectors of a block
  ptx::grid_launch_dependents();                 // a product may start fetching its weights
  const int64_t sl = blockIdx.x >> 2;
  int64_t row0;
  const int n = slab_rows(p, sl, row0);
  if (n == 0) return;
  const int lane = threadIdx.x & 31;
  const int line = (blockIdx.x & 3) * 8 + (threadIdx.x >> 5);   // r % 32 of the warp's rows
  if (line >= n && p.counts) return;
  const int r = line + 32 * (lane >> 3);
  const bool live = r < n;
  const int64_t ka = f4::atoms_k(FMT, p.K);
  const int64_t nblk = p.K / BLK;
  const __nv_bfloat16* xr = x + (row0 + r) * p.ldx;
  uint8_t* cr = codes + (row0 + r) * (p.K / 2);
  __nv_bfloat16* vr = VALUES ? values + (row0 + r) * p.K : nullptr;
  uint8_t* sf = scales + sl * ka * f4::kAtomBytes;
  constexpr int IT = kQCols / (8 * BLK);
#pragma unroll 1
  for (int turn = 0; turn < turns; ++turn) {
    const int64_t k0 = ((int64_t)blockIdx.y * turns + turn) * kQCols;
    if (k0 >= p.K) break;
    const int64_t b0 = k0 / BLK + (lane & 7);
    uint4 v[IT][V];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t b = b0 + 8 * it;
#pragma unroll
      for (int i = 0; i < V; ++i)
        v[it][i] = live && b < nblk ? ldg_nc_v4(xr + b * BLK + 8 * i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t b = b0 + 8 * it;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, amax_bits8(v[it][i]));
      const Fp4Scale s = fp4_scale<FMT>(__uint_as_float(m << 16), m < 0x7F80u, down);
      uint32_t c[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(v[it][i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fp4_quotient<FMT>(f[j], s.inv);
        c[i] = s.inv > 0.f ? e2m1x8(f) : 0u;
      }
      if (live && b < nblk) {
        if (V == 2) *reinterpret_cast<uint2*>(cr + b * 8) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<uint4*>(cr + b * 16) = make_uint4(c[0], c[1], c[V - 2], c[V - 1]);
        if (VALUES) {
          const float sv = fp4_scale_value<FMT>(s.byte) * up;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            uint32_t h[4];
            e2m1x8_to_half(c[i], h);
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
              f[2 * j] = t.x * sv;
              f[2 * j + 1] = t.y * sv;
            }
            stg_v4(vr + b * BLK + 8 * i, pack8(f));
          }
        }
      }
      // four blocks' bytes of a row in one word; the words of the four rows are
      // one line of the atom
      uint32_t word = (b < nblk && live ? s.byte : 0u) << (8 * (lane & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 1);
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      if ((lane & 3) == 0 && (b >> 2) < ka)
        *reinterpret_cast<uint32_t*>(sf + f4::sf_byte(r, b)) = word;
    }
  }
}

// Here a lane takes eight elements of a row and a warp 256 consecutive ones, so that
// a warp's store is 512 consecutive bytes (the stores are 78 % of the traffic; in the
// quantiser's arrangement, 32 bytes a lane in two stores, a layer's weights of 470 M
// elements took 218 us).
template <int FMT>
__global__ void __launch_bounds__(kQThreads)
fp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      __nv_bfloat16* __restrict__ out, float up, const Rows p) {
  constexpr int kPass = kQCols / 256;
  const int64_t sl = blockIdx.x >> 2;
  int64_t row0;
  const int n = slab_rows(p, sl, row0);
  const int lane = threadIdx.x & 31;
  const int line = (blockIdx.x & 3) * 8 + (threadIdx.x >> 5);
  const int64_t ka = f4::atoms_k(FMT, p.K);
  const uint8_t* sf = scales + sl * ka * f4::kAtomBytes;
  const int64_t k0 = (int64_t)blockIdx.y * kQCols + 8 * lane;
  uint32_t c[4][kPass], sb[4][kPass];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = line + 32 * i;
#pragma unroll
    for (int j = 0; j < kPass; ++j) {
      const int64_t k = k0 + 256 * j;
      const bool in = r < n && k < p.K;
      c[i][j] = in ? __ldg(reinterpret_cast<const uint32_t*>(codes + ((row0 + r) * p.K + k) / 2)) : 0u;
      sb[i][j] = in ? __ldg(sf + f4::sf_byte(r, k / f4::block_of(FMT))) : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = line + 32 * i;
#pragma unroll
    for (int j = 0; j < kPass; ++j) {
      const int64_t k = k0 + 256 * j;
      if (r >= n || k >= p.K) continue;
      const float sv = fp4_scale_value<FMT>(sb[i][j]) * up;
      uint32_t h[4];
      e2m1x8_to_half(c[i][j], h);
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        f[2 * e] = t.x * sv;
        f[2 * e + 1] = t.y * sv;
      }
      stg_v4(out + (row0 + r) * p.ldx + k, pack8(f));
    }
  }
}

float pow2f(int e) { return ldexpf(1.f, e); }

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, const void* x, int64_t ldx, int64_t groups, int64_t rows,
                                int64_t K, int scale_log2, const int32_t* counts,
                                const int32_t* offsets, int segments, uint8_t* codes,
                                uint8_t* scales, void* values, int32_t* status, cudaStream_t s) {
  const Rows p{rows, K, ldx, counts, offsets, segments, status};
  const int64_t sl = groups * f4::slabs(rows);
  if (sl == 0) return cudaSuccess;
  // Where there are many CTAs, four turns each: a CTA's start and the look for its
  // segment take longer than a turn's loads (32768 x 4096: 63.8 us
  // with one turn, 60.5 with four; 8192 x 14336: 57.0, 53.5); few rows keep a turn to a CTA, side by side.
  const int64_t chunks = (K + kQCols - 1) / kQCols;
  const int turns = 4 * sl * chunks > 16 * num_sms() ? 4 : 1;
  const dim3 grid((unsigned)(4 * sl), (unsigned)((chunks + turns - 1) / turns));
  const float up = pow2f(scale_log2), down = pow2f(-scale_log2);
  auto xb = static_cast<const __nv_bfloat16*>(x);
  auto vb = static_cast<__nv_bfloat16*>(values);
  if (fmt == MOE_FP4_NV) {
    if (values) fp4_quantize_kernel<MOE_FP4_NV, true><<<grid, kQThreads, 0, s>>>(xb, codes, scales, vb, up, down, turns, p);
    else fp4_quantize_kernel<MOE_FP4_NV, false><<<grid, kQThreads, 0, s>>>(xb, codes, scales, vb, up, down, turns, p);
  } else {
    if (values) fp4_quantize_kernel<MOE_FP4_MX, true><<<grid, kQThreads, 0, s>>>(xb, codes, scales, vb, up, down, turns, p);
    else fp4_quantize_kernel<MOE_FP4_MX, false><<<grid, kQThreads, 0, s>>>(xb, codes, scales, vb, up, down, turns, p);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(int fmt, const uint8_t* codes, const uint8_t* scales,
                                  int64_t groups, int64_t rows, int64_t K, int scale_log2,
                                  void* out, int64_t ldo, cudaStream_t s) {
  const Rows p{rows, K, ldo, nullptr, nullptr, 0, nullptr};
  const int64_t sl = groups * f4::slabs(rows);
  if (sl == 0) return cudaSuccess;
  const dim3 grid((unsigned)(4 * sl), (unsigned)((K + kQCols - 1) / kQCols));
  auto ob = static_cast<__nv_bfloat16*>(out);
  const float up = pow2f(scale_log2);
  if (fmt == MOE_FP4_NV)
    fp4_dequantize_kernel<MOE_FP4_NV><<<grid, kQThreads, 0, s>>>(codes, scales, ob, up, p);
  else
    fp4_dequantize_kernel<MOE_FP4_MX><<<grid, kQThreads, 0, s>>>(codes, scales, ob, up, p);
  return cudaGetLastError();
}

}  // namespace moe
