// Stage 2 of the MoE layer, dispatch, done locally: a stable counting sort of
// the (token, slot) assignments by (expert, token), then a copy of every token
// row into its experts' contiguous segments.
//
// Follows the dispatch stage of "Scalable Training of Mixture-of-Experts
// Models with Megatron Core" (es summary, Resumen técnico §2.1 step 2); with
// every expert on one GPU the all-to-all becomes this permutation. The maps
// are computed without atomics whose order matters, so they are
// deterministic and bit-identical from run to run.
//
// Three launches, two of them for up to 256 tokens (and one more with a paged stash):
//   hist    one block per chunk of 256 tokens, a thread per token: per-expert
//           counts of the chunk (not with a single chunk);
//   rank    one block per chunk: global counts, segment offsets, and the rank
//           of every assignment = (assignments of its expert in earlier
//           chunks) + (earlier tokens of this chunk that chose the same
//           expert, read from a per-expert bitmap of the chunk's tokens);
//           8192 tokens to 8 of 256 experts: 10.4 us, 61 to 8 of 128: 5.4 (three scans by the
//           whole CTA, one after the other, and one CTA for the padding rows: 9.5);
//   alloc   (paged stash) one block: the layer's stash pages and page table;
//   scatter one warp per token: reads the row once, writes it to each of its
//           rows with 16-byte stores; padding rows are zero-filled.
#include "common.cuh"
#include "fp8_layout.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

// The k experts of token t, in registers: -1 where an entry is out of range or names the same
// expert as an earlier slot of the token (possible only in a caller-given idx, e.g. a replayed
// one). Such entries are reported and dropped, so that every counted row of an expert segment
// is written exactly once.
__device__ __forceinline__ bool token_experts(const int32_t* __restrict__ idx, int t, int k, int E,
                                              int (&e)[kMaxK]) {
  int raw[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) raw[j] = j < k ? __ldg(idx + (size_t)t * k + j) : -1;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    bool ok = (unsigned)raw[j] < (unsigned)E;
#pragma unroll
    for (int i = 0; i < j; ++i) ok = ok && raw[i] != raw[j];
    e[j] = ok && j < k ? raw[j] : -1;
    bad = bad || (j < k && !ok);
  }
  return bad;
}

static_assert(kChunkTokens == 256, "a thread of the dispatch's kernels has one token");

__global__ void __launch_bounds__(256)
permute_hist_kernel(const int32_t* __restrict__ idx, int32_t* __restrict__ hist, int T, int k,
                    int E, int32_t* status) {
  __shared__ int cnt[kMaxExperts];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  cnt[threadIdx.x] = 0;
  __syncthreads();
  const int t = blockIdx.x * kChunkTokens + threadIdx.x;
  if (t < T) {
    int e[kMaxK];
    if (token_experts(idx, t, k, E, e)) record_status(status, MOE_ERR_DEVICE_CHECK);
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (e[j] >= 0) atomicAdd(&cnt[e[j]], 1);
  }
  __syncthreads();
  if ((int)threadIdx.x < E) hist[(size_t)blockIdx.x * E + threadIdx.x] = cnt[threadIdx.x];
}

// One chunk (T <= 256) needs no histogram: its own bitmap has the counts.
__global__ void __launch_bounds__(256)
permute_rank_kernel(const int32_t* __restrict__ idx, const int32_t* __restrict__ hist,
                    int n_chunk, int T, int k, int E, int S, int align, int C,
                    int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ row_of, int32_t* __restrict__ token_of,
                    int32_t* __restrict__ sel_offsets, int32_t* __restrict__ sel_tokens,
                    int32_t* __restrict__ pad_prefix, int32_t* status) {
  constexpr int W = kChunkTokens / 32;
  __shared__ int tot[kMaxExperts];
  __shared__ int before[kMaxExperts];
  __shared__ int seg[kMaxGroups + 1];
  __shared__ int kept[kMaxGroups];
  __shared__ int pad[kMaxGroups + 1];
  __shared__ int soff[kMaxExperts + 1];
  __shared__ __align__(16) uint32_t bm[kMaxExperts][W];        // tokens of the chunk, per expert
  __shared__ __align__(8) uint8_t pre[kMaxExperts][W];         // how many in the words before
  // (with a single chunk the CTAs behind the first share its padding rows alone)
  const int c = n_chunk > 1 ? blockIdx.x : 0, G = E + S, tid = threadIdx.x, nt = blockDim.x;
  const int t = c * kChunkTokens + tid;

  for (int i = tid; i < E * W; i += nt) (&bm[0][0])[i] = 0u;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  int e[kMaxK];
  const bool bad = t < T && token_experts(idx, t, k, E, e);
  if (bad && n_chunk == 1 && blockIdx.x == 0) record_status(status, MOE_ERR_DEVICE_CHECK);
  if (tid < E && n_chunk > 1) {
    int a = 0, b = 0;
#pragma unroll 8
    for (int cc = 0; cc < n_chunk; ++cc) {
      const int h = __ldcg(hist + (size_t)cc * E + tid);
      a += h;
      if (cc < c) b += h;
    }
    tot[tid] = a;
    before[tid] = b;
    soff[tid] = a;
  }
  __syncthreads();
  if (t < T) {
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (e[j] >= 0) atomicOr(&bm[e[j]][tid >> 5], 1u << (tid & 31));
  }
  __syncthreads();
  if (tid < E) {
    int n = 0;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      pre[tid][q] = (uint8_t)n;                  // (at most 224)
      n += __popc(bm[tid][q]);
    }
    if (n_chunk <= 1) {
      tot[tid] = soff[tid] = n;
      before[tid] = 0;
    }
  }
  __syncthreads();
  for (int g = tid; g < G; g += nt) {
    int kp, sl;
    if (g < E) {
      kp = C > 0 ? min(tot[g], C) : tot[g];
      sl = C > 0 ? C : (kp + align - 1) / align * align;
    } else {
      kp = T;
      sl = (T + align - 1) / align * align;
    }
    kept[g] = kp;
    seg[g] = sl;
    // padding rows that a GEMM reads: the rest of the segment's last 128-row
    // block (rows past it -- capacity segments, row_align > 128 -- are never read)
    pad[g] = min(sl, (kp + 127) / 128 * 128) - kp;
  }
  __syncthreads();
  // exclusive sums of the three side by side, by a warp each, a lane neighbouring groups
  if (tid < 96) {
    int* a = tid < 32 ? seg : tid < 64 ? pad : soff;
    const int n = tid < 64 ? G : E, lane = tid & 31, per = (n + 31) / 32, from = lane * per;
    int own = 0;
    for (int i = from; i < min(from + per, n); ++i) own += a[i];
    int run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) a[n] = run;
    run -= own;
    for (int i = from; i < min(from + per, n); ++i) {
      const int v = a[i];
      a[i] = run;
      run += v;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int g = tid; g < G; g += nt) counts[g] = kept[g];
    for (int g = tid; g <= G; g += nt) {
      offsets[g] = seg[g];
      pad_prefix[g] = pad[g];
    }
    for (int q = tid; q <= E; q += nt) sel_offsets[q] = soff[q];
  }
  if (t < T && (n_chunk > 1 || blockIdx.x == 0)) {
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      if (j >= k) break;
      int row = -1;
      if (e[j] >= 0) {
        const int rank = before[e[j]] + pre[e[j]][tid >> 5] +
                         __popc(bm[e[j]][tid >> 5] & ((1u << (tid & 31)) - 1u));
        sel_tokens[soff[e[j]] + rank] = t;
        if (C == 0 || rank < C) {
          row = seg[e[j]] + rank;
          token_of[row] = t;
        }
      }
      row_of[(size_t)t * k + j] = row;
    }
    for (int s = 0; s < S; ++s) token_of[seg[E + s] + t] = t;
  }
  // padding rows of groups g = blockIdx.x, + gridDim.x, .., a warp each (gridDim.x >= 1 even when T == 0)
  for (int g = blockIdx.x + (tid >> 5) * gridDim.x; g < G; g += gridDim.x * (nt >> 5))
    for (int r = seg[g] + kept[g] + (tid & 31); r < seg[g + 1]; r += 32) token_of[r] = -1;
}

// Paged stashing (es summary §2.3.C: the dynamic buffers are managed inside
// the CUDA graph instead of being reserved for the worst case). The rows a
// layer keeps for its backward live in a pool of 128-row pages shared by the
// layers of a step. Once the segment offsets are on the device, one block
// takes as many pages as the layer has live 128-row blocks -- the
// ceil(counts[g] / 128) blocks of group g from offsets[g] / 128 on, the ones
// the grouped GEMMs' row tiles cover -- from the pool's counter (a
// compare-and-swap, so layers on other streams can allocate too), numbers
// them in block order, and maps every other block, including the one past the
// last row (the odd half of a CTA-pair tile reads there), to the spill page P.
// A layer that does not fit takes no page: all of its blocks map to the spill
// page, MOE_ERR_STASH_FULL is recorded, and every access stays in the pool.
// Entry nblk + 1 keeps the first page taken (the counter's value before),
// which the release writes back.
__global__ void __launch_bounds__(256)
stash_alloc_kernel(const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                   int G, int nblk, int P, int32_t* __restrict__ top,
                   int32_t* __restrict__ table, int32_t* status) {
  __shared__ int pre[kMaxGroups + 1];
  __shared__ int blk0[kMaxGroups + 1];
  __shared__ int tmp[33];
  __shared__ int s_first, s_ok;
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int g = tid; g < G; g += nt) {
    pre[g] = (counts[g] + 127) >> 7;
    blk0[g] = offsets[g] >> 7;
  }
  if (tid == 0) blk0[G] = offsets[G] >> 7;
  __syncthreads();
  const int n = block_exclusive_scan(pre, G, tmp);
  if (tid == 0) {
    pre[G] = n;
    int old = atomicAdd(top, 0);
    int first = -1;
    while (old >= 0 && old <= P - n) {
      const int seen = atomicCAS(top, old, old + n);
      if (seen == old) {
        first = old;
        break;
      }
      old = seen;
    }
    s_ok = first >= 0;
    s_first = first >= 0 ? first : old;
    if (first < 0) record_status(status, MOE_ERR_STASH_FULL);
    table[nblk + 1] = s_first;
  }
  __syncthreads();
  for (int b = tid; b <= nblk; b += nt) {
    int page = P;
    if (s_ok) {
      // the group whose segment holds block b: the last g with blk0[g] <= b
      int lo = 0, hi = G - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (blk0[mid] <= b) lo = mid;
        else hi = mid - 1;
      }
      const int i = b - blk0[lo];
      if (G > 0 && i >= 0 && i < pre[lo + 1] - pre[lo]) page = s_first + pre[lo] + i;
    }
    table[b] = page;
  }
}

__global__ void stash_release_kernel(const int32_t* __restrict__ table, int nblk,
                                     int32_t* __restrict__ top) {
  if (threadIdx.x == 0) *top = table[nblk + 1];
}

// Finds the group whose padding range holds padding row number p.
__device__ __forceinline__ int find_group(const int* prefix, int G, int p) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Virtual rows v < T copy token v to its rows; v >= T zero one padding row
// (the padding rows inside each segment's last 128-row block, the ones a GEMM
// reads).
// With xq (the FP8 configurations) every row is also written in its 1-byte
// form -- E4M3 codes of its 1 x 128 slices (MXFP8: 1 x 32) and their UE8M0
// scales in the atoms of xsf (fp8_layout.cuh) -- for the FC1 GEMM: each slice
// is quantised once per token and written to each of the token's rows;
// padding rows get zero codes and scale 1.
template <bool MX>
__global__ void __launch_bounds__(256)
permute_scatter_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ row_of,
                       const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                       const int32_t* __restrict__ pad_prefix, __nv_bfloat16* __restrict__ x_perm,
                       int T, int H, int k, int E, int S, uint8_t* __restrict__ xq,
                       uint8_t* __restrict__ xsf, const int32_t* __restrict__ pages) {
  __shared__ int s_pp[kMaxGroups + 1];
  __shared__ int s_off[kMaxGroups + 1];
  __shared__ int s_cnt[kMaxGroups];
  const int G = E + S;
  for (int g = threadIdx.x; g <= G; g += blockDim.x) {
    s_pp[g] = pad_prefix[g];
    s_off[g] = offsets[g];
    if (g < G) s_cnt[g] = counts[g];
  }
  __syncthreads();
  const int P = s_pp[G];
  const int lane = threadIdx.x & 31;
  const int nvec = H >> 3;
  const int64_t kg = f8::sf_stride(H, MX);
  const unsigned half = (lane & 16) ? 0xffff0000u : 0x0000ffffu;
  constexpr int piece_lanes = MX ? 4 : 16;         // lanes per scale piece
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int v = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); v < T + P; v += warps) {
    if (v < T) {
      const int t = v;
      int myrow = (lane < k) ? row_of[(size_t)t * k + lane] : -1;
      if (lane >= k && lane < k + S) myrow = s_off[E + lane - k] + t;
      const int nr = k + S;
      int rows[kMaxK + 4];
#pragma unroll
      for (int j = 0; j < kMaxK + 4; ++j) rows[j] = __shfl_sync(0xffffffffu, myrow, j);
      const __nv_bfloat16* src = x + (size_t)t * H;
      for (int c0 = lane; c0 < nvec; c0 += 32 * 4) {
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + 32 * u < nvec) q[u] = ldg_nc_v4(src + (size_t)(c0 + 32 * u) * 8);
        // 1-byte form: a half-warp holds one 128-element slice per u, four
        // lanes one 32-element piece (nvec is a multiple of 16, so a half-warp
        // is wholly in range or out)
        uint2 qb[4];
        uint32_t code[4];
        if (xq) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (c0 + 32 * u >= nvec) continue;
            float f[8];
            unpack8(q[u], f);
            float m = amax8(f);
#pragma unroll
            for (int o = piece_lanes / 2; o > 0; o >>= 1)
              m = fmaxf(m, __shfl_xor_sync(half, m, o));
            code[u] = ue8m0_code(m);
            qb[u] = e4m3x8(f, ue8m0_inv(code[u]));
          }
        }
#pragma unroll
        for (int j = 0; j < kMaxK + 4; ++j) {
          if (j >= nr || rows[j] < 0) continue;
          __nv_bfloat16* dst = x_perm + (size_t)stash_row(pages, rows[j]) * H;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (c0 + 32 * u < nvec) stg_v4(dst + (size_t)(c0 + 32 * u) * 8, q[u]);
          if (xq) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int c = c0 + 32 * u;
              if (c >= nvec) continue;
              *reinterpret_cast<uint2*>(xq + (size_t)rows[j] * H + (size_t)c * 8) = qb[u];
              if ((lane & (piece_lanes - 1)) == 0)
                xsf[f8::row_sf_index(rows[j], c, kg, MX)] = (uint8_t)code[u];
            }
          }
        }
      }
    } else {
      const int p = v - T;
      const int g = find_group(s_pp, G, p);
      const int r = s_off[g] + s_cnt[g] + (p - s_pp[g]);
      __nv_bfloat16* dst = x_perm + (size_t)stash_row(pages, r) * H;
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      for (int c0 = lane; c0 < nvec; c0 += 32) {
        stg_v4(dst + (size_t)c0 * 8, z);
        if (xq) {
          *reinterpret_cast<uint2*>(xq + (size_t)r * H + (size_t)c0 * 8) = make_uint2(0u, 0u);
          if ((c0 & (piece_lanes - 1)) == 0) xsf[f8::row_sf_index(r, c0, kg, MX)] = 127u;
        }
      }
    }
  }
}

// Rows that are in 8 bits already (E4M3 codes with a scale byte per 32 or 128 values): a warp
// takes 2 KB of a token's row, reads them once and writes them to each of its rows, 16 bytes a
// lane; its scale bytes go into the atoms four at a time (fp8_layout.cuh: both layouts keep four
// consecutive blocks of a row in one word). Rows without a token are not written: a product's rows
// depend on their own row alone, and only the combine's rows are read behind it. HBM bounds it:
// 8192 tokens of 7168 to 8 of 256 experts 65 us (of 78 with the maps).
__global__ void __launch_bounds__(256)
permute_scatter8_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                        const int32_t* __restrict__ row_of, int T, int H, int k, int block,
                        uint8_t* __restrict__ xq, uint8_t* __restrict__ xsf) {
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nvec = H >> 4, n = H / block;
  const int words = (n + 3) >> 2;                  // atoms along the row, in either layout
  const int pieces = (nvec + 127) >> 7;
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int64_t item = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
       item < (int64_t)T * pieces; item += warps) {
    const int t = (int)(item / pieces), piece = (int)(item - (int64_t)t * pieces);
    const int myrow = lane < k ? __ldg(row_of + (size_t)t * k + lane) : -1;
    const int c0 = piece * 128 + lane;
    const uint8_t* src = codes + (size_t)t * H;
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c0 + 32 * u < nvec) q[u] = ldg_nc_v4(src + (size_t)(c0 + 32 * u) * 16);
    // the scales of the row's words in turn of the pieces
    const int w = piece + lane * pieces;
    uint32_t v = 0;
    if (w < words) {
      const uint8_t* ssrc = scales + (size_t)t * n + 4 * w;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (4 * w + b < n) v |= (uint32_t)__ldg(ssrc + b) << (8 * b);
    }
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      const int row = __shfl_sync(0xffffffffu, myrow, j);
      if (row < 0) continue;
      uint8_t* dst = xq + (size_t)row * H;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + 32 * u < nvec) stg_v4(dst + (size_t)(c0 + 32 * u) * 16, q[u]);
      if (w < words)
        *reinterpret_cast<uint32_t*>(xsf + ((size_t)(row >> 7) * words + w) * f8::kAtomBytes +
                                     f8::atom_byte(row, 0)) = v;
    }
  }
}

// The maps: counts, offsets, rows and tokens of every assignment.
static cudaError_t launch_permute_maps(const moe_config& c, const int32_t* idx, int32_t* counts,
                                       int32_t* offsets, int32_t* row_of, int32_t* token_of,
                                       int32_t* sel_offsets, int32_t* sel_tokens,
                                       uint8_t* scratch, cudaStream_t s) {
  int32_t* status = reinterpret_cast<int32_t*>(scratch + kScratchStatus);
  int32_t* pad_prefix = reinterpret_cast<int32_t*>(scratch + kScratchPadPrefix);
  int32_t* hist = reinterpret_cast<int32_t*>(scratch + kScratchHist);
  const int nc = n_chunks(c);
  if (nc > 1) {
    const cudaError_t err = launch_early(permute_hist_kernel, (unsigned)nc, dim3(256, 1, 1), 0, s,
                                         idx, hist, c.T, c.k, c.E, status);
    if (err != cudaSuccess) return err;
  }
  // (a single chunk: a warp a group for the padding rows)
  const unsigned ctas = nc > 1 ? nc : (c.E + c.n_shared + 7) / 8;
  return launch_early(permute_rank_kernel, ctas, dim3(256, 1, 1), 0, s, idx, hist, nc, c.T, c.k, c.E,
                      c.n_shared, c.row_align, (int)capacity_rows(c), counts, offsets, row_of,
                      token_of, sel_offsets, sel_tokens, pad_prefix, status);
}

cudaError_t launch_permute(const moe_config& c, const void* x, const int32_t* idx,
                           int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* token_of,
                           int32_t* sel_offsets, int32_t* sel_tokens, void* x_perm,
                           uint8_t* scratch, cudaStream_t s, const Fp8Scratch* fp8,
                           const StashAlloc* alloc) {
  int32_t* status = reinterpret_cast<int32_t*>(scratch + kScratchStatus);
  int32_t* pad_prefix = reinterpret_cast<int32_t*>(scratch + kScratchPadPrefix);
  cudaError_t err = launch_permute_maps(c, idx, counts, offsets, row_of, token_of, sel_offsets,
                                        sel_tokens, scratch, s);
  if (err != cudaSuccess) return err;
  const int32_t* pages = nullptr;
  if (alloc) {
    stash_alloc_kernel<<<1, 256, 0, s>>>(counts, offsets, c.E + c.n_shared,
                                         (int)(rows_max(c) / 128), alloc->pool_pages, alloc->top,
                                         alloc->table, status);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    pages = alloc->table;
  }
  uint8_t* xq = nullptr;
  uint8_t* xsf = nullptr;
  if (c.dtype != MOE_DTYPE_BF16 && fp8) {
    xq = fp8->xq;
    xsf = fp8->xsf;
  }
  // (the MX pieces of x_perm's 1-byte form are 32 elements, the block recipe's 128)
  auto kern = (c.dtype == MOE_DTYPE_MXFP8 && xq) ? permute_scatter_kernel<true>
                                                 : permute_scatter_kernel<false>;
  kern<<<num_sms() * 8, 256, 0, s>>>(
      static_cast<const __nv_bfloat16*>(x), row_of, counts, offsets, pad_prefix,
      static_cast<__nv_bfloat16*>(x_perm), c.T, c.H, c.k, c.E, c.n_shared, xq, xsf, pages);
  return cudaGetLastError();
}

cudaError_t launch_permute_fp8(const moe_config& c, const uint8_t* codes, const uint8_t* scales,
                               const int32_t* idx, int32_t* counts, int32_t* offsets,
                               int32_t* row_of, int32_t* token_of, int32_t* sel_offsets,
                               int32_t* sel_tokens, uint8_t* xq, uint8_t* xsf, uint8_t* scratch,
                               cudaStream_t s) {
  const cudaError_t err = launch_permute_maps(c, idx, counts, offsets, row_of, token_of,
                                              sel_offsets, sel_tokens, scratch, s);
  if (err != cudaSuccess || c.T == 0) return err;
  const int64_t blocks = ((int64_t)c.T * ((c.H + 2047) / 2048) + 7) / 8, most = num_sms() * 8;
  return launch_early(permute_scatter8_kernel, (unsigned)(blocks < most ? blocks : most),
                      dim3(256, 1, 1), 0, s, codes, scales, row_of, c.T, c.H, c.k,
                      c.dtype == MOE_DTYPE_MXFP8 ? 32 : 128, xq, xsf);
}

cudaError_t launch_stash_release(const moe_config& c, const int32_t* table, int32_t* top,
                                 cudaStream_t s) {
  stash_release_kernel<<<1, 32, 0, s>>>(table, (int)(rows_max(c) / 128), top);
  return cudaGetLastError();
}

}  // namespace moe

// ------------------------------------------------------------------------------
// Dispatch without a caller-provided scratch buffer.
//
// Some callers cannot hand this library a scratch allocation: code that runs
// inside a host framework which owns every byte of device memory (a caching
// allocator or plugin host with no way to request an extra workspace), or
// code on a path where calling cudaMalloc is not allowed. For them
// moe_permute_noalloc keeps its scratch -- the per-chunk expert histograms,
// the padding prefix and the status word -- in one file-scope device array of
// fixed size, which every GPU that loads this library holds until the process
// exits. It allocates nothing.
namespace moe {
namespace {

constexpr size_t kNoAllocScratchBytes = 512 * 1024;
static __device__ __align__(256) uint8_t g_permute_scratch[kNoAllocScratchBytes];

// Device address of g_permute_scratch in the current context, looked up on
// every call (cheap): a cached address would go stale after cudaDeviceReset or
// under another context on the same device.
cudaError_t noalloc_scratch(uint8_t** out) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_permute_scratch);
  if (e != cudaSuccess) return e;
  *out = static_cast<uint8_t*>(p);
  return cudaSuccess;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_permute_noalloc(const moe_config* cfg, const void* x,
                                          const int32_t* idx, int32_t* counts, int32_t* offsets,
                                          int32_t* row_of, int32_t* token_of,
                                          int32_t* sel_offsets, int32_t* sel_tokens,
                                          void* x_perm, void* stream) {
  using namespace moe;
  const moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  // an FP8 dispatch also writes x_perm's E4M3 form into the caller's scratch,
  // which this entry point does not take
  if (cfg->dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
  auto a16 = [](const void* p) { return p && ((uintptr_t)p & 15u) == 0; };
  auto a4 = [](const void* p) { return p && ((uintptr_t)p & 3u) == 0; };
  const bool empty = cfg->T == 0;
  if (!((empty && !x) || a16(x)) || !((empty && !idx) || a4(idx)) || !a4(counts) ||
      !a4(offsets) || !((empty && !row_of) || a4(row_of)) || !a4(token_of) ||
      !a4(sel_offsets) || !((empty && !sel_tokens) || a4(sel_tokens)) || !a16(x_perm))
    return MOE_ERR_INVALID_ARG;
  if ((size_t)permute_scratch_bytes(*cfg) > kNoAllocScratchBytes) return MOE_ERR_WORKSPACE;
  uint8_t* sc = nullptr;
  if (noalloc_scratch(&sc) != cudaSuccess) return MOE_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  // the status word is the only part that must start at zero; the histograms
  // and the padding prefix are fully rewritten by every call
  if (cudaMemsetAsync(sc + kScratchStatus, 0, sizeof(int32_t), s) != cudaSuccess)
    return MOE_ERR_CUDA;
  const cudaError_t e = launch_permute(*cfg, x, idx, counts, offsets, row_of, token_of,
                                       sel_offsets, sel_tokens, x_perm, sc, s, nullptr);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Reads back what the last moe_permute_noalloc call recorded in its status
// word (an index out of range or repeated): synchronises `stream`, then copies
// the word from the library's array on the current device.
extern "C" moe_status moe_permute_noalloc_status(int32_t* code, void* stream) {
  using namespace moe;
  if (!code) return MOE_ERR_INVALID_ARG;
  uint8_t* sc = nullptr;
  if (noalloc_scratch(&sc) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(code, sc + kScratchStatus, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}
