// Grouped products of a short reduction (64 at most), forward and data gradient: the products that
// lead out of an adapter's rank. y[r, f] = sum_k a[r, k] w[k, f] + add[r, f] with k a few numbers:
// what moves is y and add, and HBM bounds it.
//
// So no tile goes through shared or tensor memory. A warp takes 64 features of a group, holds their
// weights as B operands of mma.sync m16n8k16 in registers, and streams over the group's rows, 16 at
// a time. Both operands' orders are free as long as they are the same: lane t of four has elements
// 4 t .. 4 t + 3 of every 16 of the reduction (one 8-byte load of a row), and the eight MMAs' columns
// are dealt so that it ends up with eight consecutive features of each half, 16 bytes of add and y.
// (8192 rows of 16 ranks to 4096 features with add: 28 us, 4.8 TB/s; through 256-wide
// tensor tiles, whose epilogue loads, turns and stores in phases, 46.)
#include "gemm_common.cuh"

namespace moe {
namespace {

constexpr int kShortWarps = 8;

// Sixteens of rows on their way, each in a thread's own pieces of a ring: four of add (16 bytes), two
// of x for every 16 of the reduction (8 bytes). No thread reads another's, so nothing is waited for
// but a thread's own copies.
template <int KS>
struct Short {
  static constexpr int CTAS = KS == 1 ? 3 : 2;       // on an SM: 24 warps, 16 where weights take more
  static constexpr int DEPTH = KS == 2 ? 4 : 3;
  static constexpr int SLOT = 32 * kShortWarps * (64 + 16 * KS);
  static constexpr int SMEM = DEPTH * SLOT;
};

// KS: sixteens of the reduction. w: [G, feat, red], or (DGRAD) [G, red, feat].
template <int KS, bool DGRAD>
__global__ void __launch_bounds__(32 * kShortWarps, Short<KS>::CTAS)
product_short_kernel(const RaggedProduct p, const __nv_bfloat16* __restrict__ x, int64_t ldx,
                     const __nv_bfloat16* __restrict__ w, int chunk) {
  __shared__ int prefix[kMaxGroups + 1];
  __shared__ int s_off[kMaxGroups], s_cnt[kMaxGroups];
  __shared__ int tmp[33];
  extern __shared__ uint8_t ring[];
  const int tid = threadIdx.x, lane = tid & 31, g8 = lane >> 2, t = lane & 3;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  for (int g = tid; g < p.G; g += 32 * kShortWarps) {
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
    prefix[g] = (int)(((int64_t)c + chunk - 1) / chunk);
  }
  __syncthreads();
  const int chunks = block_exclusive_scan(prefix, p.G, tmp);
  if (tid == 0) prefix[p.G] = chunks;
  __syncthreads();

  constexpr int kPiece = 32 * kShortWarps * 16;
  const uint32_t own = ptx::smem_u32(ring) + tid * 16, own8 = ptx::smem_u32(ring) + 4 * kPiece + tid * 8;
  // features fastest: warps that run together read the same rows
  const unsigned blocks = (p.feat + 63) / 64, items = chunks * blocks;
  for (unsigned item = blockIdx.x * kShortWarps + (tid >> 5); item < items;
       item += gridDim.x * kShortWarps) {
    const int ch = item / blocks, fb = (item - ch * blocks) * 64;
    const int g = gg::find_group(prefix, p.G, ch);
    const int r0 = (ch - prefix[g]) * chunk, n = min(chunk, s_cnt[g] - r0);
    const int64_t row0 = (int64_t)s_off[g] + r0;

    // the 16 rows from row i on into the ring's next slot, zeros of x behind the last row
    auto fetch = [&](int i, int slot) {
      const uint32_t to = own + slot * Short<KS>::SLOT;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool in = i + g8 + 8 * r < n;
        const int64_t row = row0 + (in ? i + g8 + 8 * r : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int f = fb + 32 * h + 8 * t;
          if (p.add && in && f < p.feat)
            ptx::cp_async16(to + (2 * r + h) * kPiece, p.add + row * p.ldadd + f);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int k = 16 * s + 4 * t;
          const bool some = in && k < p.red;
          ptx::cp_async8_or_zero(own8 + slot * Short<KS>::SLOT + (2 * s + r) * (kPiece / 2),
                                 x + (some ? row * ldx + k : 0), some);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < Short<KS>::DEPTH - 1; ++i) {
      if (16 * i < n) fetch(16 * i, i);
      ptx::cp_async_commit();
    }
    // column n = g8 of MMA 4 h + q is feature 32 h + 8 (n / 2) + 2 q + n % 2
    uint2 wb[KS][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int f = fb + 32 * (j >> 2) + 8 * (g8 >> 1) + 2 * (j & 3) + (g8 & 1);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = 16 * s + 4 * t;
        wb[s][j] = make_uint2(0u, 0u);
        if (f >= p.feat || k >= p.red) continue;
        if constexpr (DGRAD) {
          const uint16_t* from = reinterpret_cast<const uint16_t*>(w) +
                                 ((int64_t)g * p.red + k) * p.feat + f;
          wb[s][j].x = __ldg(from) | (uint32_t)__ldg(from + p.feat) << 16;
          wb[s][j].y = __ldg(from + 2 * (int64_t)p.feat) |
                       (uint32_t)__ldg(from + 3 * (int64_t)p.feat) << 16;
        } else {
          wb[s][j] = __ldg(reinterpret_cast<const uint2*>(w + ((int64_t)g * p.feat + f) * p.red + k));
        }
      }
    }

    int slot = 0;
    for (int i = 0; i < n; i += 16) {
      const int ahead = 16 * (Short<KS>::DEPTH - 1);
      const int free = slot == 0 ? Short<KS>::DEPTH - 1 : slot - 1;
      if (i + ahead < n) fetch(i + ahead, free);
      ptx::cp_async_commit();
      ptx::cp_async_wait<Short<KS>::DEPTH - 1>();
      const uint8_t* from = ring + slot * Short<KS>::SLOT;
      uint2 a[2][KS];                  // of rows g8 and g8 + 8 of the sixteen
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int s = 0; s < KS; ++s)
          a[r][s] = *reinterpret_cast<const uint2*>(from + 4 * kPiece + tid * 8 + (2 * s + r) * (kPiece / 2));
      if (++slot == Short<KS>::DEPTH) slot = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = fb + 32 * h + 8 * t;
        float d[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int e = 0; e < 4; ++e) d[q][e] = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s)
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                "{%8,%9}, {%0,%1,%2,%3};"
                : "+f"(d[q][0]), "+f"(d[q][1]), "+f"(d[q][2]), "+f"(d[q][3])
                : "r"(a[0][s].x), "r"(a[1][s].x), "r"(a[0][s].y), "r"(a[1][s].y),
                  "r"(wb[s][4 * h + q].x), "r"(wb[s][4 * h + q].y));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (i + g8 + 8 * r >= n || f >= p.feat) continue;
          float e[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            e[2 * q] = d[q][2 * r];
            e[2 * q + 1] = d[q][2 * r + 1];
          }
          if (p.add) {
            float b[8];
            unpack8(*reinterpret_cast<const uint4*>(from + (2 * r + h) * kPiece + tid * 16), b);
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] += b[q];
          }
          stg_v4(p.out + (row0 + i + g8 + 8 * r) * p.ldo + f, pack8(e));
        }
      }
    }
  }
}

template <int KS>
cudaError_t run_short(const RaggedProduct& p, bool dgrad, const void* x, int64_t ldx, const void* w,
                      int chunk, unsigned grid, cudaStream_t s) {
  auto kern = dgrad ? product_short_kernel<KS, true> : product_short_kernel<KS, false>;
  static PerDevice set[2];
  const cudaError_t e = set_smem_once(set[dgrad], kern, Short<KS>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_early(kern, grid, dim3(32 * kShortWarps, 1, 1), Short<KS>::SMEM, s, p,
                      static_cast<const __nv_bfloat16*>(x), ldx,
                      static_cast<const __nv_bfloat16*>(w), chunk);
}

}  // namespace

// Whether a product goes this way: its reduction, and pieces of 16 rows and 64 features in 32 bits.
// (64 ranks, 8192 rows to 4096 features, us, this way and by tensor tiles: 35.4 and 45 with add;
// without it 30.8 and 29, 55.6 and 51 for 32768 rows of 64 experts to 2048; one row: 6.2 and 10.)
bool short_fits(int64_t rows, int G, int64_t feat, int64_t red, bool add) {
  return red <= (add ? 64 : 48) && (rows / 16 + G) * ((feat + 63) / 64) < (1LL << 31);
}

cudaError_t launch_product_short(RaggedProduct p, int dgrad, const void* x, int64_t ldx,
                                 const void* w, int N, int K, cudaStream_t s) {
  p.feat = dgrad ? K : N;
  p.red = dgrad ? N : K;
  // Rows of a piece: 96, 256 where the weights take longer to load, or fewer where that leaves warps
  // without one. (8192 rows to 4096 features with add, us, pieces of 16, 96 and 256 rows: 16 ranks
  // 29.6, 27.3, 33.2; 64 ranks 61.6, 39.1, 35.8; 32768 rows to 64 features: 8.3, 10.4, 18.6.)
  const int64_t warps = (int64_t)num_sms() * (p.red <= 16 ? 3 : 2) * kShortWarps;
  const int64_t blocks = (p.feat + 63) / 64, groups = p.rows < p.G ? p.rows : p.G;
  int chunk = p.red <= 16 ? 96 : 256;
  while (chunk > 16 && (p.rows / chunk + groups / 2) * blocks < warps * 7 / 8) chunk -= 16;
  const int64_t ctas = ((p.rows / chunk + groups) * blocks + kShortWarps - 1) / kShortWarps;
  const unsigned grid = (unsigned)(ctas < warps / kShortWarps ? ctas : warps / kShortWarps);
  switch ((p.red + 15) / 16) {
    case 1: return run_short<1>(p, dgrad, x, ldx, w, chunk, grid, s);
    case 2: return run_short<2>(p, dgrad, x, ldx, w, chunk, grid, s);
    case 3: return run_short<3>(p, dgrad, x, ldx, w, chunk, grid, s);
    default: return run_short<4>(p, dgrad, x, ldx, w, chunk, grid, s);
  }
}

}  // namespace moe
