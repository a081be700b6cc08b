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
//
// 8192 rows of 7168 with residual, sum, bf16 output and MXFP8 codes: 80 us, 6.6 TB/s (a row a CTA with
// loads that wait for nothing but themselves: 101, with instructions in 73 % of the issue slots and
// HBM 63 % busy; the ring and packed arithmetic brought it here). 8192 rows of 4096 backward with
// dsum and dgamma: 45 us, 5.9 TB/s (67 before). One row of 4096 or 7168: 4.3 us, a launch.
#include "common.cuh"
#include "fp8_layout.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRowWarps = 8;                    // rows of a CTA where a row is a warp's
constexpr int kWarpColumns = 1024;              // longest such row
constexpr int kRingBytes = 196608;              // of the rows in flight at most

// Eight elements as four fp32 pairs: one instruction works on two (ptx::f2_*), and instructions
// are what these kernels run short of next to HBM.
struct Eight {
  uint64_t v[4];
};
__device__ __forceinline__ Eight eight_of(const uint4& b) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e.v[i] = ptx::f2_pack(bf16_lo(w[i]), bf16_hi(w[i]));
  return e;
}
__device__ __forceinline__ uint4 bf16_of(const Eight& e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    ptx::f2_unpack(e.v[i], a, b);
    w[i] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  ptx::f2_unpack(v, a, b);
  return a + b;
}

// Eight consecutive elements of gamma, bf16 or fp32.
__device__ __forceinline__ Eight load_gamma(const void* gamma, bool f32, int v) {
  if (!f32) return eight_of(__ldg(static_cast<const uint4*>(gamma) + v));
  const float4* p = static_cast<const float4*>(gamma) + 2 * v;
  const float4 a = __ldg(p), b = __ldg(p + 1);
  return Eight{{ptx::f2_pack(a.x, a.y), ptx::f2_pack(a.z, a.w), ptx::f2_pack(b.x, b.y),
                ptx::f2_pack(b.z, b.w)}};
}

// x + y of bf16 pairs, rounded once.
__device__ __forceinline__ uint4 add_bf16(const uint4& x, const uint4& y) {
  uint4 r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(x.x), "r"(y.x));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(x.y), "r"(y.y));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.z) : "r"(x.z), "r"(y.z));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.w) : "r"(x.w), "r"(y.w));
  return r;
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

// From the row's sum of squares to its outputs; h, g: this thread's columns of it and of gamma.
template <int V>
__device__ __forceinline__ void finish_row(const RmsNormFwd& p, int64_t row, const uint4 (&h)[V],
                                           const Eight (&g)[V], float ss, int first, int step,
                                           int lane) {
  const int nvec = p.H >> 3;
  const float s = __frsqrt_rn(ss / (float)p.H + p.eps);
  const uint64_t s2 = ptx::f2_pack(s, s);
  if (first == 0 && p.rstd) p.rstd[row] = s;
  __nv_bfloat16* out = p.out ? p.out + row * p.ldo : nullptr;
  uint8_t* codes = p.codes ? p.codes + row * p.H : nullptr;
  const int lanes = p.block >> 3, log2 = p.block == 32 ? 2 : 4;
  uint8_t* scales = p.codes ? p.scales + row * (nvec >> log2) : nullptr;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = first + i * step;
    // (a warp's lanes stay together for the block maxima)
    if (v - lane >= nvec) break;
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) {
      Eight e = eight_of(h[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) e.v[j] = ptx::f2_mul(ptx::f2_mul(e.v[j], s2), g[i].v[j]);
      y = bf16_of(e);
      if (out) stg_v4(out + 8 * v, y);
    }
    if (codes) {
      // of the rounded output, as the dispatch quantises it; a block is 4 or 16 lanes' (a row
      // is whole blocks, so a block is in range or out)
      float f[8];
      unpack8(y, f);
      float m = amax8(f);
      for (int o = lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t code = ue8m0_code(m);
      if (v < nvec) {
        *reinterpret_cast<uint2*>(codes + 8 * v) = e4m3x8(f, ue8m0_inv(code));
        if ((lane & (lanes - 1)) == 0) scales[v >> log2] = (uint8_t)code;
      }
    }
  }
}

// h = bf16(x + residual) of eight columns (x without one), written to the sum where it is
// wanted: the stream is held in bf16, rounded here and normed as it is held. Adds its squares.
__device__ __forceinline__ uint4 held(const RmsNormFwd& p, __nv_bfloat16* sum, int v, uint4 x,
                                      const uint4& r, uint64_t& ss) {
  if (p.residual) {
    x = add_bf16(x, r);
    if (sum) stg_v4(sum + 8 * v, x);
  }
  const Eight e = eight_of(x);
#pragma unroll
  for (int j = 0; j < 4; ++j) ss = ptx::f2_fma(e.v[j], e.v[j], ss);
  return x;
}

// A row a CTA (a warp): few rows, or short ones.
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
  __nv_bfloat16* sum = p.sum ? p.sum + row * p.lds : nullptr;
  uint4 h[V], r[V];
  Eight g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = first + i * step;
    h[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v >= nvec) continue;
    h[i] = load8(x + 8 * v);
    if (res) r[i] = load8(res + 8 * v);
    g[i] = load_gamma(p.gamma, p.gamma_f32, v);
  }
  uint64_t s2 = ptx::f2_pack(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = first + i * step;
    if (v < nvec) h[i] = held(p, sum, v, h[i], r[i], s2);
  }
  const float ss = WARP ? warp_sum(sum_of(s2)) : block_sum(sum_of(s2), red);
  finish_row<V>(p, row, h, g, ss, first, step, lane);
}

// Many long rows: a persistent CTA keeps the loads of S rows in flight. Each thread copies its own
// columns into its own places of shared memory (cp.async) and reads them back alone, so the
// ring needs no barrier, and the rows in flight take no registers.
template <int V, int S, int THREADS>
__global__ void __launch_bounds__(THREADS)
rmsnorm_fwd_ring_kernel(const RmsNormFwd p) {
  extern __shared__ uint4 ring[];                // [S][x, residual][V][threads]
  __shared__ float red[2][32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, step = blockDim.x, nvec = p.H >> 3;
  Eight g[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (tid + i * step < nvec) g[i] = load_gamma(p.gamma, p.gamma_f32, tid + i * step);
  auto place = [&](int s, int t, int i) { return ring + ((s * 2 + t) * V + i) * step + tid; };
  auto issue = [&](int64_t row, int s) {
    if (row < p.T) {
      const __nv_bfloat16* x = p.x + row * p.ldx;
      const __nv_bfloat16* r = p.residual + row * p.ldr;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v >= nvec) continue;
        ptx::cp_async16(place(s, 0, i), x + 8 * v);
        if (p.residual) ptx::cp_async16(place(s, 1, i), r + 8 * v);
      }
    }
    ptx::cp_async_commit();
  };
  int64_t ahead = blockIdx.x;
#pragma unroll
  for (int s = 0; s < S - 1; ++s, ahead += gridDim.x) issue(ahead, s);
  int s = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, ahead += gridDim.x, turn ^= 1) {
    issue(ahead, s == 0 ? S - 1 : s - 1);
    ptx::cp_async_wait<S - 1>();
    __nv_bfloat16* sum = p.sum ? p.sum + row * p.lds : nullptr;
    uint4 h[V];
    uint64_t s2 = ptx::f2_pack(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * step;
      h[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nvec) h[i] = held(p, sum, v, *place(s, 0, i), *place(s, 1, i), s2);
    }
    finish_row<V>(p, row, h, g, block_sum(sum_of(s2), red[turn]), tid, step, lane);
    if (++s == S) s = 0;
  }
  ptx::cp_async_wait<0>();
}

// The backward, persistent too: a thread keeps the same columns of every row that its CTA (its
// warp) takes, so their share of dgamma stays in registers; the CTAs' shares are added in order
// by dgamma_kernel. S: rows in flight (1: none ahead; a long row does not fit twice).
// KEEP: t and n stay in registers between the sum and their use; else they are made again.
template <int V, int S, int THREADS, bool WARP, bool KEEP>
__global__ void __launch_bounds__(THREADS)
rmsnorm_bwd_kernel(const RmsNormBwd p) {
  extern __shared__ uint4 ring[];                // [S][dy, h, dsum][V][threads]
  __shared__ float red[2][32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int first = WARP ? lane : tid, step = WARP ? 32 : blockDim.x;
  const int nvec = p.H >> 3;
  const int64_t row0 = WARP ? (int64_t)blockIdx.x * kRowWarps + (tid >> 5) : blockIdx.x;
  const int64_t rows = WARP ? (int64_t)gridDim.x * kRowWarps : gridDim.x;
  const float inv_h = 1.f / (float)p.H;
  const uint64_t zero2 = ptx::f2_pack(0.f, 0.f);
  Eight dg[V], g[KEEP ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i].v[j] = zero2;
    if (KEEP && first + i * step < nvec) g[KEEP ? i : 0] = load_gamma(p.gamma, p.gamma_f32, first + i * step);
  }
  auto place = [&](int s, int t, int i) {
    return ring + ((s * 3 + t) * V + i) * (int)blockDim.x + tid;
  };
  auto issue = [&](int64_t row, int s) {
    if (row < p.T) {
      const __nv_bfloat16* dy = p.dy + row * p.lddy;
      const __nv_bfloat16* h = p.h + row * p.ldh;
      const __nv_bfloat16* ds = p.dsum + row * p.ldds;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = first + i * step;
        if (v >= nvec) continue;
        ptx::cp_async16(place(s, 0, i), dy + 8 * v);
        ptx::cp_async16(place(s, 1, i), h + 8 * v);
        if (p.dsum) ptx::cp_async16(place(s, 2, i), ds + 8 * v);
      }
    }
    ptx::cp_async_commit();
  };
  int64_t ahead = row0;
#pragma unroll
  for (int s = 0; s < S - 1; ++s, ahead += rows) issue(ahead, s);
  int s = 0, turn = 0;
  float rs_next = row0 < p.T ? __ldg(p.rstd + row0) : 0.f;
  for (int64_t row = row0; row < p.T; row += rows, ahead += rows, turn ^= 1) {
    issue(ahead, s == 0 ? S - 1 : s - 1);
    const float rs = rs_next;
    if (row + rows < p.T) rs_next = __ldg(p.rstd + row + rows);
    ptx::cp_async_wait<S - 1>();
    const uint64_t rs2 = ptx::f2_pack(rs, rs);
    uint64_t dot = zero2;
    Eight t[KEEP ? V : 1], n[KEEP ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      const Eight dy = eight_of(*place(s, 0, i)), h = eight_of(*place(s, 1, i));
      const Eight gi = KEEP ? g[KEEP ? i : 0] : load_gamma(p.gamma, p.gamma_f32, v);
      Eight& ti = t[KEEP ? i : 0];
      Eight& ni = n[KEEP ? i : 0];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ni.v[j] = ptx::f2_mul(h.v[j], rs2);
        ti.v[j] = ptx::f2_mul(dy.v[j], gi.v[j]);
        dot = ptx::f2_fma(ti.v[j], ni.v[j], dot);
        dg[i].v[j] = ptx::f2_fma(dy.v[j], ni.v[j], dg[i].v[j]);
      }
    }
    const float c = -(WARP ? warp_sum(sum_of(dot)) : block_sum(sum_of(dot), red[turn])) * inv_h;
    const uint64_t c2 = ptx::f2_pack(c, c);
    __nv_bfloat16* dx = p.dx + row * p.lddx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      Eight d = eight_of(p.dsum ? *place(s, 2, i) : make_uint4(0u, 0u, 0u, 0u));
      Eight& ti = t[KEEP ? i : 0];
      Eight& ni = n[KEEP ? i : 0];
      if (!KEEP) {
        const Eight dy = eight_of(*place(s, 0, i)), h = eight_of(*place(s, 1, i));
        const Eight gi = load_gamma(p.gamma, p.gamma_f32, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ni.v[j] = ptx::f2_mul(h.v[j], rs2);
          ti.v[j] = ptx::f2_mul(dy.v[j], gi.v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d.v[j] = ptx::f2_fma(ptx::f2_fma(ni.v[j], c2, ti.v[j]), rs2, d.v[j]);
      stg_v4(dx + 8 * v, bf16_of(d));
    }
    if (++s == S) s = 0;
  }
  ptx::cp_async_wait<0>();
  if (!p.parts) return;
  float* part = p.parts + (int64_t)blockIdx.x * p.H;
  if (WARP) {
    __shared__ __align__(16) float s_dg[kRowWarps][kWarpColumns];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = first + i * step;
      if (v >= nvec) continue;
      uint64_t* d = reinterpret_cast<uint64_t*>(&s_dg[threadIdx.x >> 5][8 * v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = dg[i].v[j];
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
      ulonglong2* d = reinterpret_cast<ulonglong2*>(part + 8 * v);
      d[0] = make_ulonglong2(dg[i].v[0], dg[i].v[1]);
      d[1] = make_ulonglong2(dg[i].v[2], dg[i].v[3]);
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

// CTAs of a kernel that walks the rows: as many as are resident together, the same number on
// every SM, no more than one a row (a turn of the CTA) and `most`. set: of the kernel, by its warps
// (which decide its shared memory).
template <class Kernel>
cudaError_t resident(PerDevice (&set)[33], Kernel kern, int threads, int smem, int64_t turns, int most,
                     int* grid) {
  int per_sm = 0;
  const cudaError_t e = set[threads / 32].get(current_device(), &per_sm, [&](int* v) {
    cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (err != cudaSuccess) return err;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, threads, smem);
  });
  if (e != cudaSuccess) return e;
  const int sms = num_sms();
  if (per_sm > most / sms) per_sm = most / sms;
  const int64_t n = per_sm > 0 ? (int64_t)sms * per_sm : most;
  *grid = (int)(n < turns ? n : turns);
  return cudaSuccess;
}

template <int V, int S, int THREADS>
cudaError_t run_fwd_ring(const RmsNormFwd& p, cudaStream_t s) {
  auto kern = rmsnorm_fwd_ring_kernel<V, S, THREADS>;
  static PerDevice set[33];
  const int threads = row_threads(p.H, V), smem = S * 2 * V * threads * 16;
  int grid = 0;
  const cudaError_t e = resident(set, kern, threads, smem, p.T, 1 << 20, &grid);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)grid, dim3(threads, 1, 1), smem, s, p);
}

template <int V, int S, int THREADS, bool WARP, bool KEEP>
cudaError_t run_bwd(const RmsNormBwd& p, int* parts, cudaStream_t s) {
  auto kern = rmsnorm_bwd_kernel<V, S, THREADS, WARP, KEEP>;
  static PerDevice set[33];
  const int threads = WARP ? 32 * kRowWarps : row_threads(p.H, V);
  const int smem = S * 3 * V * threads * 16;
  const int64_t turns = WARP ? (p.T + kRowWarps - 1) / kRowWarps : p.T;
  const cudaError_t e = resident(set, kern, threads, smem, turns, kRmsNormParts, parts);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)*parts, dim3(threads, 1, 1), smem, s, p);
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const RmsNormFwd& p, cudaStream_t s) {
  constexpr int W = 32 * kRowWarps;
  // A warp a row up to kWarpColumns. (us with residual and sum, a row a warp's and a CTA's: 8192 x 256
  // 4.6 and 8.6, 8192 x 768 9.9 and 10.1, 65536 x 768 58 and 68, 65536 x 1024 78 and 77, 64 x 1024 2.6 and
  // 1.8; backward, 8192 x 1024, 14.8 and 19.4, 64 x 1024 4.8 and 3.7.)
  if (p.H <= kWarpColumns) {
    const unsigned grid = (unsigned)((p.T + kRowWarps - 1) / kRowWarps);
    return launch_early(p.H <= 512 ? rmsnorm_fwd_kernel<2, true> : rmsnorm_fwd_kernel<4, true>, grid,
                        dim3(W, 1, 1), 0, s, p);
  }
  // Long rows go through the ring where there are more than two an SM: with fewer there is nothing to
  // fetch ahead, and shorter ones have CTAs enough in flight. (us with residual and sum, through the
  // ring and a row a CTA's: 8192 x 4096 49.7 and 40.3, 8192 x 2048 24.8 and 21.2; 8192 x 7168 76.3 and 75.9,
  // with MXFP8 codes 79.1 and 87.3, without residual 51.1 and 61.9; 8192 x 8192 90.7 and 83.6, 93.2 and
  // 95.9, 55.8 and 67.5; 4096 x 16384 91.6 and 94.9, without residual 45.9 and 81.9. 304 rows of 7168 5.7
  // and 4.6, 608 8.4 and 8.1, 1216 12.9 and 14.1.)
  if (p.T > 2 * num_sms() && p.H > 4096) {
    if (p.H <= 8192) return run_fwd_ring<1, 3, 1024>(p, s);
    if (p.H <= 16384) return run_fwd_ring<2, 3, 1024>(p, s);
  }
  // (the widest rows' four vectors a thread spill 24 bytes: 2048 x 16384 47 us, x 16392 62, x 32768 100,
  // of 39, 39 and 79 that the bytes take; the backward's 48: 58, 72 and 116, of 30, 30 and 59)
  const int V = p.H <= 16384 ? 2 : 4;
  return launch_early(V == 2 ? rmsnorm_fwd_kernel<2, false> : rmsnorm_fwd_kernel<4, false>,
                      (unsigned)p.T, dim3(row_threads(p.H, V), 1, 1), 0, s, p);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwd& p, float* dgamma, cudaStream_t s) {
  int n = 0;
  if (p.T > 0) {
    const cudaError_t e = p.H <= 512            ? run_bwd<2, 3, 256, true, true>(p, &n, s)
                          : p.H <= kWarpColumns ? run_bwd<4, 2, 256, true, true>(p, &n, s)
                          : p.H <= 4096         ? run_bwd<1, 2, 512, false, true>(p, &n, s)
                          : p.H <= 8192         ? run_bwd<1, 2, 1024, false, true>(p, &n, s)
                          : p.H <= 16384        ? run_bwd<2, 2, 1024, false, false>(p, &n, s)
                                                : run_bwd<4, 1, 1024, false, false>(p, &n, s);
    if (e != cudaSuccess) return e;
  }
  if (!dgamma) return cudaSuccess;
  // (without rows there are no shares, and dgamma is zero)
  return launch_early(dgamma_kernel, (unsigned)((p.H + 31) / 32), dim3(32, 16, 1), 0, s, p.parts, n,
                      p.H, dgamma);
}

}  // namespace moe
