// The norm in front of a layer: residual's addition, root-mean-square norm and the 8-bit form
// of its output in one pass over the data, and its backward.
//
//   forward   h = bf16(x + residual), s = (mean(h^2) + eps)^-1/2, y = bf16(h s gamma), and
//             codes = E4M3(y / 2^c), c = ceil(log2(amax / 448)) of each 32 or 128 values;
//   backward  t = dy gamma, n = h s, dx = s (t - n mean(t n)) + dsum, dgamma = sum of dy n.
//
// HBM bounds both: a row is read once, stays in registers between the sum and its use, and is
// written once. A row belongs to a CTA (to a warp up to 1024 columns, eight rows to a CTA, so
// that short rows need no barrier); a thread holds 8 x V columns. Sums are fp32.
#include "common.cuh"
#include "fp8_layout.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRowWarps = 8;                    // rows of a CTA where a row is a warp's
constexpr int kWarpColumns = 1024;              // longest such row

// Eight consecutive elements of gamma, bf16 or fp32.
__device__ __forceinline__ void load_gamma(const void* gamma, bool f32, int v, float (&g)[8]) {
  if (f32) {
    const float4* p = static_cast<const float4*>(gamma) + 2 * v;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  } else {
    unpack8(__ldg(static_cast<const uint4*>(gamma) + v), g);
  }
}

// A row's tensors may be written where another is read (the sum in place of the residual):
// plain loads, as the read-only path may not see such a tensor.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Sum over the CTA's threads, the same bits in each; `red` is this row's own buffer.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : 1024)
rmsnorm_fwd_kernel(const RmsNormFwd p) {
  __shared__ float red[32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int64_t row = WARP ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.T) return;
  const int lane = threadIdx.x & 31;
  const int first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const int nvec = p.H >> 3;
  const __nv_bfloat16* x = p.x + row * p.ldx;
  const __nv_bfloat16* res = p.residual ? p.residual + row * p.ldr : nullptr;
  uint4 h[V], r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = first + i * step;
    h[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) {
      h[i] = load8(x + 8 * v);
      if (res) r[i] = load8(res + 8 * v);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    unpack8(h[i], f);
    if (res) {
      // the stream is held in bf16: rounded here, and normed as it is held
      float g[8];
      unpack8(r[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      h[i] = pack8(f);
      unpack8(h[i], f);
      const int v = first + i * step;
      if (p.sum && v < nvec) stg_v4(p.sum + row * p.lds + 8 * v, h[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
  }
  ss = WARP ? warp_sum(ss) : block_sum(ss, red);
  const float s = __frsqrt_rn(ss / (float)p.H + p.eps);
  if (first == 0 && p.rstd) p.rstd[row] = s;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = first + i * step;
    // (a warp's lanes stay together for the block maxima)
    if (v - lane >= nvec) break;
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) {
      float f[8], g[8];
      unpack8(h[i], f);
      load_gamma(p.gamma, p.gamma_f32, v, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * s * g[j];
      y = pack8(f);
      if (p.out) stg_v4(p.out + row * p.ldo + 8 * v, y);
    }
    if (p.codes) {
      // of the rounded output, as the dispatch quantises it; a block is 4 or 16 lanes' (a row
      // is whole blocks, so a block is in range or out)
      float f[8];
      unpack8(y, f);
      float m = amax8(f);
      const int lanes = p.block >> 3;
      for (int o = lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t code = ue8m0_code(m);
      if (v < nvec) {
        *reinterpret_cast<uint2*>(p.codes + row * p.H + 8 * v) = e4m3x8(f, ue8m0_inv(code));
        if ((lane & (lanes - 1)) == 0) p.scales[row * (p.H / p.block) + v / lanes] = (uint8_t)code;
      }
    }
  }
}

// Persistent: a thread keeps the same columns of every row that its CTA (its warp) takes, so
// their share of dgamma stays in registers; the CTAs' shares are added in order by
// dgamma_kernel. HOLD: a row stays in registers between the sum and its use, and the next
// one's loads are issued before this one's barrier (2), or not (1); long rows are read again,
// from L1 or L2 (0). What decides is the registers: 8 V of dgamma, 12 V a row held.
template <int V, int THREADS, bool WARP, int HOLD>
__global__ void __launch_bounds__(THREADS)
rmsnorm_bwd_kernel(const RmsNormBwd p) {
  __shared__ float red[2][32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const int nvec = p.H >> 3;
  const int64_t row0 = WARP ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t rows = WARP ? (int64_t)gridDim.x * kRowWarps : gridDim.x;
  const float inv_h = 1.f / (float)p.H;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float dg[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
  struct Row {
    uint4 dy[HOLD ? V : 1], h[HOLD ? V : 1], ds[HOLD ? V : 1];
    float s;
  };
  auto load = [&](Row& r, int64_t row) {
    if (row >= p.T) return;
    if constexpr (HOLD > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = first + i * step;
        if (v >= nvec) continue;
        r.dy[i] = load8(p.dy + row * p.lddy + 8 * v);
        r.h[i] = load8(p.h + row * p.ldh + 8 * v);
        r.ds[i] = p.dsum ? load8(p.dsum + row * p.ldds + 8 * v) : zero;
      }
    }
    r.s = __ldg(p.rstd + row);
  };
  Row next;
  if (HOLD == 2) load(next, row0);
  int turn = 0;
  for (int64_t row = row0; row < p.T; row += rows, turn ^= 1) {
    Row cur;
    if (HOLD == 2) cur = next;
    else load(cur, row);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      float a[8], b[8], g[8];
      unpack8(HOLD ? cur.dy[HOLD ? i : 0] : load8(p.dy + row * p.lddy + 8 * v), a);
      unpack8(HOLD ? cur.h[HOLD ? i : 0] : load8(p.h + row * p.ldh + 8 * v), b);
      load_gamma(p.gamma, p.gamma_f32, v, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = b[j] * cur.s;
        dot = fmaf(a[j] * g[j], n, dot);
        dg[i][j] = fmaf(a[j], n, dg[i][j]);
      }
    }
    if (HOLD == 2) load(next, row + rows);
    const float c = (WARP ? warp_sum(dot) : block_sum(dot, red[turn])) * inv_h;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      float a[8], b[8], d[8], g[8];
      unpack8(HOLD ? cur.dy[HOLD ? i : 0] : load8(p.dy + row * p.lddy + 8 * v), a);
      unpack8(HOLD ? cur.h[HOLD ? i : 0] : load8(p.h + row * p.ldh + 8 * v), b);
      unpack8(HOLD ? cur.ds[HOLD ? i : 0]
                   : p.dsum ? load8(p.dsum + row * p.ldds + 8 * v) : zero, d);
      load_gamma(p.gamma, p.gamma_f32, v, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(fmaf(-b[j] * cur.s, c, a[j] * g[j]), cur.s, d[j]);
      stg_v4(p.dx + row * p.lddx + 8 * v, pack8(d));
    }
  }
  if (!p.parts) return;
  float* part = p.parts + (int64_t)blockIdx.x * p.H;
  if (WARP) {
    __shared__ __align__(16) float s_dg[kRowWarps][kWarpColumns];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      float4* d = reinterpret_cast<float4*>(&s_dg[threadIdx.x >> 5][8 * v]);
      d[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
      d[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) a += s_dg[w][c];
      part[c] = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      float4* d = reinterpret_cast<float4*>(part + 8 * v);
      d[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
      d[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
  }
}

// dgamma[c] = the CTAs' shares in order: 16 threads a column, each every 16th share.
__global__ void __launch_bounds__(512)
dgamma_kernel(const float* __restrict__ parts, int n, int H, float* __restrict__ dgamma) {
  __shared__ float sum[16][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  float a = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int q = threadIdx.y; q < n; q += 16) a += __ldcg(parts + (int64_t)q * H + c);
  }
  sum[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < H) {
    a = sum[0][threadIdx.x];
#pragma unroll
    for (int y = 1; y < 16; ++y) a += sum[y][threadIdx.x];
    dgamma[c] = a;
  }
}

// Threads of a row that is a CTA's own, V vectors each.
int row_threads(int H, int V) { return ((H / 8 + V - 1) / V + 31) / 32 * 32; }

// CTAs of the backward, and with them the shares of dgamma: enough for the SMs' threads (two
// CTAs of 512, a CTA of 1024), at most kRmsNormParts.
int bwd_ctas(int64_t T, int H) {
  const bool warp = H <= kWarpColumns;
  const int64_t rows = warp ? (T + kRowWarps - 1) / kRowWarps : T;
  const int threads = warp ? 32 * kRowWarps : row_threads(H, H <= 8192 ? 2 : 4);
  int per_sm = threads >= 1024 ? 1 : 1024 / threads;
  if (per_sm > 3) per_sm = 3;
  int64_t n = (int64_t)num_sms() * per_sm;
  if (n > kRmsNormParts) n = kRmsNormParts;
  return (int)(rows < n ? rows : n);
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const RmsNormFwd& p, cudaStream_t s) {
  constexpr int W = 32 * kRowWarps;
  if (p.H <= kWarpColumns) {
    const unsigned grid = (unsigned)((p.T + kRowWarps - 1) / kRowWarps);
    return launch_early(p.H <= 512 ? rmsnorm_fwd_kernel<2, true> : rmsnorm_fwd_kernel<4, true>, grid,
                        dim3(W, 1, 1), 0, s, p);
  }
  const int V = p.H <= 16384 ? 2 : 4;
  return launch_early(V == 2 ? rmsnorm_fwd_kernel<2, false> : rmsnorm_fwd_kernel<4, false>,
                      (unsigned)p.T, dim3(row_threads(p.H, V), 1, 1), 0, s, p);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwd& p, float* dgamma, cudaStream_t s) {
  constexpr int W = 32 * kRowWarps;
  const int n = bwd_ctas(p.T, p.H);
  if (n > 0) {
    const int threads = p.H <= kWarpColumns ? W : row_threads(p.H, p.H <= 8192 ? 2 : 4);
    const cudaError_t e = launch_early(p.H <= 512            ? rmsnorm_bwd_kernel<2, W, true, 2>
                                       : p.H <= kWarpColumns ? rmsnorm_bwd_kernel<4, W, true, 1>
                                       : p.H <= 8192         ? rmsnorm_bwd_kernel<2, 512, false, 2>
                                       : p.H <= 16384        ? rmsnorm_bwd_kernel<4, 512, false, 1>
                                                             : rmsnorm_bwd_kernel<4, 1024, false, 0>,
                                       (unsigned)n, dim3(threads, 1, 1), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  if (!dgamma) return cudaSuccess;
  // (without rows there are no shares, and dgamma is zero)
  return launch_early(dgamma_kernel, (unsigned)((p.H + 31) / 32), dim3(32, 16, 1), 0, s, p.parts, n,
                      p.H, dgamma);
}

}  // namespace moe
