// Grouped products of ragged rows on the fifth-generation tensor cores: for the rows r of every
// group g, which follow each other without padding at any offset,
//   forward          y[r] = x[r] W[g]^T
//   data gradient    dx[r] = dy[r] W[g]
//   weight gradient  dW[g] = sum of dy[r]^T x[r]
// by CTA pairs (tcgen05 cta_group::2, M = 256, accumulators of up to 256 columns, two of them in
// tensor memory so that one is drained while the next is summed).
//
// The first two take W's features as M and the rows as N: the instruction's N is any multiple
// of 16, so a group's rows are cut into equal tiles of at most 256 without padding (512 rows an
// expert on average: tiles of 128 rows as M multiplied an eighth of padding), and the features
// are the dimension that is a multiple of the tile. What that costs is a transposed epilogue:
// a thread holds one feature of 32 rows, and the tile is turned in shared memory on its way to
// plain 16-byte stores, which need no wait and are masked row by row.
//
// A TMA request costs its issuer some 200 clocks whatever its size, and a k-block of a 256 x 256
// tile lasts 512: each operand comes in one request a CTA (a map of its own for every height of
// the row tile, chunked maps for operands that lie along M or N), issued by a warp each.
//
// What the raggedness adds:
//   - the weights' maps have the expert as a dimension of their own, so that a box that passes
//     an expert's last row or column reads zeros and not the next expert's;
//   - a tile's rows past its group's end are the next group's; each makes its own row of the
//     product alone, which is not stored;
//   - the weight gradient reduces over the rows: a warp of each CTA zeroes the next group's rows
//     of the last block in both operands (zero times a NaN is one) before it hands the stage to
//     the pair's MMAs.
//
// 32768 rows of 64 experts, 4096 x 2040 (0.55 PFLOP), call after call: data gradient 470 us, 1.16
// PFLOP/s; weight gradient 552, 0.99. In runs too short for the power limit 408 and 499. The weight
// gradient's 4.9 GB from L2 to the SMs bound it (its loads alone take 424, all but its stores 452).
// 8192^3 in one group: 1.65 to 1.70 PFLOP/s in each of the three.
#include <math.h>

#include "gemm_common.cuh"
#include "ragged_shares.h"

namespace moe {
namespace {

using gg::BK;
using gg::kWaitBudget;

enum Mode : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kPairThreads = 384;               // A's loads, MMAs, fixer, B's loads, eight epilogue warps
constexpr int kM = 256;                         // features of a pair tile
constexpr int kStages = 6;
constexpr int kABytes = 128 * BK * 2;           // of each CTA
constexpr int kStageBytes = 2 * kABytes;
constexpr int kBox = 2048;                      // an epilogue warp's: 16 x 32 fp32 or 32 x 32 bf16
constexpr int kEpiWarps = 8;
constexpr int kCtrl = 4096;
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kBox + kCtrl + 1024;
static_assert(kSmem <= 232448, "shared memory");

// a, b: one request a k-block and CTA: 128 features; 16 (i + 1) rows (b[i]), or all of a weight
// gradient's columns (b[0]). a2, b2: 64 columns of an operand that lies along M or N, where the
// last ones are not a whole chunk of 64.
struct Maps {
  CUtensorMap a, a2, b2, b[8];
};

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
ragged_pair_kernel(const __grid_constant__ Maps maps, const RaggedProduct p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* boxes = smem_raw + (base - raw) + kStages * kStageBytes;
  uint8_t* ctrl = boxes + kEpiWarps * kBox;
  const uint32_t ctrl_u = base + kStages * kStageBytes + kEpiWarps * kBox;
  // per stage: loaded (what the MMAs wait for, in the even CTA), read, loaded for the fixer
  const uint32_t bar_full = ctrl_u, bar_empty = ctrl_u + 48, bar_tail = ctrl_u + 96;
  const uint32_t bar_tfull = ctrl_u + 144, bar_tempty = ctrl_u + 160, bar_drain = ctrl_u + 176;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 352);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 356);
  int* prefix = reinterpret_cast<int*>(ctrl + 384);        // [kMaxGroups + 1] pair tiles
  int* s_off = reinterpret_cast<int*>(ctrl + 1440);        // [kMaxGroups]
  int* s_cnt = reinterpret_cast<int*>(ctrl + 2496);        // [kMaxGroups]
  int* tmp = reinterpret_cast<int*>(ctrl + 3552);          // [33]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 2);                 // A's loader twice, or both fixers
      ptx::mbar_init(bar_empty + 8 * s, 1);
      ptx::mbar_init(bar_tail + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(bar_tfull + 8 * a, 1);
      ptx::mbar_init(bar_tempty + 8 * a, 2 * kEpiWarps);
    }
    ptx::mbar_init(bar_drain, 1);
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&maps.a);
    ptx::tma_prefetch_desc(&maps.b[MODE == kWgrad ? 0 : 7]);
  }
  // what needs no memory comes before the wait for the kernel in front
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  // features: M tiles; columns: what N runs over (rows of the group, or the gradient's columns)
  const int FT = (p.feat + kM - 1) / kM, CT = (p.cols + p.tile - 1) / p.tile;
  for (int g = tid; g < p.G; g += kPairThreads) {
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
    prefix[g] = FT * (MODE == kWgrad ? CT : (c + p.tile - 1) / p.tile);
  }
  __syncthreads();
  const int total = block_exclusive_scan(prefix, p.G, tmp);
  if (tid == 0) prefix[p.G] = total;
  __syncthreads();
  // Few tiles: the reduction of each is cut among several pairs. Every pair then has one unit, and
  // so has its part of the scratch for itself.
  int splits = 1;
  const int most = min(nclusters, kRaggedPairs);
  if (total > 0 && 2 * total <= most) {
    int nk = (p.red + BK - 1) / BK;
    if (MODE == kWgrad)
      for (int g = 0; g < p.G; ++g) nk = max(nk, (s_cnt[g] + BK - 1) / BK);
    splits = shares(most / total, nk, p.tile);
  }
  const int units = total * splits;
  if (cluster >= units) {                                  // both CTAs of the pair leave together
    ptx::cluster_sync();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem_base, 512);
    return;
  }

  struct Tile {
    int g, f0, n0, n, k0, nk;       // features from f0, columns (rows of the group) n0 .. n0 + n - 1,
    bool ends;                      // blocks k0 .. k0 + nk - 1 of the reduction, whether to its end
  };
  // A role's walk over its pair's tiles: the next one is found while the present one is worked on
  // (its group from the present one's on), so that no role stands still between tiles.
  auto tile_at = [&](int tile, int g) {
    Tile t;
    unsigned split = 0;
    if (splits > 1) {
      split = tile / total;
      tile -= split * total;
    }
    while (prefix[g + 1] <= tile) ++g;
    t.g = g;
    const unsigned local = tile - prefix[g];
    const int c = s_cnt[g];
    if constexpr (MODE == kWgrad) {
      // columns fastest: pairs that run together share A's columns
      const unsigned m = local / (unsigned)CT;
      t.f0 = m * kM;
      t.n0 = (local - m * CT) * p.tile;
      t.n = p.tile;
      t.nk = (c + BK - 1) / BK;
    } else {
      // rows fastest (they share the expert's weights), cut into equal tiles of whole 32s
      const unsigned nt = (unsigned)(prefix[g + 1] - prefix[g]) / (unsigned)FT;
      const int size = ((c + nt - 1) / nt + 31) & ~31u;
      const unsigned m = local / nt;
      t.f0 = m * kM;
      t.n0 = (local - m * nt) * size;
      t.n = min(size, ((c - t.n0) + 31) & ~31);
      t.nk = (p.red + BK - 1) / BK;
    }
    t.k0 = 0;
    t.ends = true;
    if (splits > 1) {
      const unsigned nk = t.nk;
      t.k0 = nk * split / splits;
      t.nk = nk * (split + 1) / splits - t.k0;
      t.ends = t.k0 + t.nk == (int)nk && t.nk > 0;
    }
    return t;
  };

  if (warp == 0 || warp == 3) {
    // A's loader, B's loader
    const bool is_a = warp == 0;
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      uint32_t leader_full[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) leader_full[s] = ptx::mapa_shared(bar_full + 8 * s, 0);
      Tile t = tile_at(cluster, 0), next = t;
      for (int pt = cluster; pt < units && ok; pt += nclusters, t = next) {
        const int half = t.n >> 1, r = s_off[t.g];
        const int f0 = t.f0 + (int)rank * 128, c0 = t.n0 + (int)rank * half;
        const uint32_t bytes = kABytes + half * BK * 2;
        // whole chunks of 64 columns come together (also where none of the 128 is the tensor's)
        const bool a_whole = MODE == kFwd || f0 + 128 <= (p.feat & ~63) || (f0 >= p.feat && p.feat >= 64);
        const bool b_whole = MODE != kWgrad || c0 + half <= (p.cols & ~63) || (c0 >= p.cols && p.cols >= 64);
        for (int kb = 0; kb < t.nk; ++kb) {
          if (!ptx::mbar_wait(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sA = base + stage * kStageBytes, sB = sA + kABytes;
          const int k0 = (t.k0 + kb) * BK;
          // both CTAs' loads count on the even CTA's barrier; a weight gradient's last block goes
          // to each CTA's own fixer first
          const bool tail = MODE == kWgrad && s_cnt[t.g] - k0 < BK;
          const uint32_t fb = tail ? bar_tail + 8 * stage : leader_full[stage];
          if (is_a) {
            if (tail) {
              ptx::mbar_arrive_expect_tx(fb, bytes);
            } else if (rank == 0) {
              ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * bytes);
              ptx::mbar_arrive(bar_full + 8 * stage);
            }
          }
          if constexpr (MODE == kWgrad) {
            const CUtensorMap* m = is_a ? &maps.a : &maps.b[0];
            const CUtensorMap* m2 = is_a ? &maps.a2 : &maps.b2;
            const uint32_t to = is_a ? sA : sB;
            const int col = is_a ? f0 : c0;
            if (is_a ? a_whole : b_whole) {
              if (tail) ptx::tma_load_3d(to, m, fb, 0, r + k0, col / 64);
              else ptx::tma_load_3d_pair(to, m, fb, 0, r + k0, col / 64);
            } else {
              for (int j = 0; j < (is_a ? 2 : half / 64); ++j)
                if (tail) ptx::tma_load_2d(to + j * 8192, m2, fb, col + 64 * j, r + k0);
                else ptx::tma_load_2d_pair(to + j * 8192, m2, fb, col + 64 * j, r + k0);
            }
          } else if (!is_a) {
            ptx::tma_load_2d_pair(sB, &maps.b[half / 16 - 1], fb, k0, r + c0);
          } else if (MODE == kFwd) {
            ptx::tma_load_3d_pair(sA, &maps.a, fb, k0, f0, t.g);
          } else if (a_whole) {
            ptx::tma_load_4d_pair(sA, &maps.a, fb, 0, k0, f0 / 64, t.g);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              ptx::tma_load_3d_pair(sA + j * 8192, &maps.a2, fb, f0 + 64 * j, k0, t.g);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (pt + nclusters < units) next = tile_at(pt + nclusters, t.g);
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        // loads already issued land within microseconds; give them time
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr int A_MN = MODE != kFwd, B_MN = MODE == kWgrad;
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true, issued = false;
      const uint32_t peer_tfull[2] = {ptx::mapa_shared(bar_tfull, 1),
                                      ptx::mapa_shared(bar_tfull + 8, 1)};
      Tile t = tile_at(cluster, 0), next = t;
      for (int pt = cluster; pt < units && ok; pt += nclusters, t = next) {
        const uint32_t idesc = ptx::idesc_bf16(kM, t.n, A_MN, B_MN);
        if (!ptx::mbar_wait_cluster(bar_tempty + 8 * acc, acc_phase ^ 1u, kWaitBudget, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + acc * 256;
        for (int kb = 0; kb < t.nk; ++kb) {
          ok = MODE == kWgrad
                   ? ptx::mbar_wait_cluster(bar_full + 8 * stage, phase, kWaitBudget, abort_flag)
                   : ptx::mbar_wait(bar_full + 8 * stage, phase, kWaitBudget, abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sA = base + stage * kStageBytes, sB = sA + kABytes;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = A_MN ? ptx::smem_desc_sw128(sA + kk * 2048, 8192, 1024)
                                     : ptx::smem_desc_sw128(sA + kk * 32, 16, 1024);
            const uint64_t bd = B_MN ? ptx::smem_desc_sw128(sB + kk * 2048, 8192, 1024)
                                     : ptx::smem_desc_sw128(sB + kk * 32, 16, 1024);
            ptx::mma_bf16_pair(d, ad, bd, idesc, (kb | kk) ? 1u : 0u);
          }
          issued = true;
          ptx::mma_commit_pair(bar_empty + 8 * stage, 3);
          if (kb == 0 && pt + nclusters < units) next = tile_at(pt + nclusters, t.g);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (t.nk > 0) {
          ptx::mma_commit_pair(bar_tfull + 8 * acc, 3);
        } else {                                           // an empty group: nothing to wait for
          ptx::mbar_arrive(bar_tfull + 8 * acc);
          ptx::mbar_arrive_cluster(peer_tfull[acc]);
          if (pt + nclusters < units) next = tile_at(pt + nclusters, t.g);
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every MMA issued by this thread is waited for before tensor memory is freed
      if (issued) {
        ptx::mma_commit_pair(bar_drain, 1);
        ptx::mbar_wait(bar_drain, 0, kWaitBudget, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    if constexpr (MODE == kWgrad) {
      uint32_t stage = 0, phases = 0;                      // phases: a bit per stage, of bar_tail
      bool ok = true;
      int g = 0;
      for (int pt = cluster; pt < units && ok; pt += nclusters) {
        const Tile t = tile_at(pt, g);
        g = t.g;
        const int valid = t.ends ? s_cnt[t.g] & (BK - 1) : 0;
        if (valid) {
          stage = (stage + t.nk - 1) % kStages;
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_tail + 8 * stage, (phases >> stage) & 1u,
                                                      kWaitBudget, abort_flag));
          if (!ok) break;
          phases ^= 1u << stage;
          // rows valid .. 63 of every 64-column chunk of A and B (128 bytes a row)
          const uint32_t sA = base + stage * kStageBytes;
          for (int j = 0; j < 2 + t.n / 128; ++j)
            for (int b = valid * 128 + lane * 16; b < 8192; b += 512)
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};"
                           :: "r"(sA + j * 8192 + b), "r"(0u) : "memory");
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(bar_full + 8 * stage, 0));
          stage = (stage + 1) % kStages;
        } else {
          stage = (stage + t.nk) % kStages;
        }
      }
      if (!ok && lane == 0) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    // lane = feature; warps 4-7 take the even boxes of columns, 8-11 the odd ones
    const int q = warp & 3, odd = (warp - 4) >> 2;
    uint8_t* box = boxes + (warp - 4) * kBox;
    const uint32_t leader_tempty[2] = {ptx::mapa_shared(bar_tempty, 0),
                                       ptx::mapa_shared(bar_tempty + 8, 0)};
    const int fq = (int)rank * 128 + q * 32;               // this warp's features in a tile
    const int lr = lane >> 2, lc = lane & 3, l8 = lane & 7;
    uint32_t acc = 0, acc_phase = 0;
    Tile next = tile_at(cluster, 0);
    for (int pt = cluster; pt < units; pt += nclusters) {
      const Tile t = next;
      if (pt + nclusters < units) next = tile_at(pt + nclusters, t.g);
      const int f = t.f0 + fq;
      const int64_t row0 = (int64_t)s_off[t.g] + t.n0;
      // rows of the tile that are this lane's to write, sixteen bytes (features fl .. fl + 7) each
      const int fl = f + 8 * lc;
      const int rows = MODE != kWgrad && fl < p.feat ? min(s_cnt[t.g] - t.n0, t.n) : 0;
      uint4 add[4][4];
      auto fetch_add = [&] {
        if (p.add) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int i = 64 * b + 32 * odd + 8 * v + lr;
              if (i < rows)
                add[b][v] = *reinterpret_cast<const uint4*>(p.add + (row0 + i) * p.ldadd + fl);
            }
        }
      };
      // every load of the tile is under way before its sums are waited for
      if (MODE != kWgrad && splits == 1) fetch_add();
      // hands the accumulator back (what this publishes is tensor memory alone: a release would
      // wait for the stores, 5000 clocks a tile)
      auto give = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_tmem(leader_tempty[acc]);
      };
      // Parts of a tile that several pairs share: 4096 sums of a warp behind each other, by pair;
      // the warp that arrives last of those with the same piece adds them, in K's order.
      const int piece = (int)rank * kEpiWarps + warp - 4;
      auto part = [&](int unit, int b) {
        return reinterpret_cast<float4*>(p.parts) +
               ((int64_t)(unit * 2 * kEpiWarps + piece) * 4 + b) * 256 + lane;
      };
      auto put = [&](int b, const uint32_t (&r)[32]) {
        float4* to = part(pt, b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          __stcg(to + 32 * i, make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                          __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
      };
      auto last = [&] {
        uint32_t n = 0;
        __threadfence();
        __syncwarp();
        if (lane == 0) {
          uint32_t* arrived = p.arrived + (pt % total) * 2 * kEpiWarps + piece;
          n = ptx::atom_add_acq_rel(arrived, 1u);
          if (n + 1 == splits) *arrived = 0u;              // as the next launch expects it
        }
        n = __shfl_sync(0xffffffffu, n, 0);
        __threadfence();
        return n + 1 == splits;
      };
      auto get = [&](int unit, int b, uint32_t (&r)[32]) {
        const float4* from = part(unit, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 d = __ldcg(from + 32 * i);
          r[4 * i] = __float_as_uint(d.x);
          r[4 * i + 1] = __float_as_uint(d.y);
          r[4 * i + 2] = __float_as_uint(d.z);
          r[4 * i + 3] = __float_as_uint(d.w);
        }
      };
      // the sum of box b's parts takes the place of this pair's
      auto join = [&](int b) {
        float sum[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i] = 0.f;
#pragma unroll 2
        for (int u = pt % total; u < units; u += total) {
          uint32_t d[32];
          get(u, b, d);
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[i] += __uint_as_float(d[i]);
        }
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(sum[i]);
        put(b, r);
      };
      const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_tfull + 8 * acc, acc_phase,
                                                             kWaitBudget, abort_flag));
      if (!ok) {
        if (splits > 1) last();                            // (the counters as after any launch)
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      ptx::tc_fence_after();
      const uint32_t tbase = tmem_base + acc * 256 + ((uint32_t)(q * 32) << 16);
      if constexpr (MODE == kWgrad) {
        // 32 features x 64 columns, a row a lane, 16 rows at a time: whole lines leave the SM (half
        // lines cost as much). 16-byte chunk j of row r at j ^ (r & 7). The next
        // columns leave tensor memory while these are on their way.
        const int end = f < p.feat ? min(t.n, p.cols - t.n0) : 0;
        uint32_t r0[32], r1[32];
        auto take = [&](int c, bool shared) {
          if (c >= end) return;
          if (shared) {
            get(pt, c >> 7 << 1, r0);
            get(pt, (c >> 7 << 1) + 1, r1);
          } else if (t.nk == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r0[i] = r1[i] = 0u;
          } else {
            ptx::tmem_ld32(tbase + c, r0);
            ptx::tmem_ld32(tbase + c + 32, r1);
          }
        };
        if (splits > 1) {
#pragma unroll 1
          for (int c = 64 * odd; c < end; c += 128) {
            take(c, false);
            ptx::tmem_ld_wait();
            put(c >> 7 << 1, r0);
            put((c >> 7 << 1) + 1, r1);
          }
          if (!last()) break;                              // (a pair has one unit)
#pragma unroll 1
          for (int b = 0; 128 * (b >> 1) + 64 * odd < end; ++b) join(b);
        }
        take(64 * odd, splits > 1);
        if (64 * odd >= end) give();
#pragma unroll 1
        for (int c = 64 * odd; c < end; c += 128) {
          const int col = t.n0 + c + 8 * l8;
          ptx::tmem_ld_wait();
          uint4 a[4], b[4];
          gg::pack_slice(r0, a);
          gg::pack_slice(r1, b);
          take(c + 128, splits > 1);
          if (c + 128 >= end) give();
          __nv_bfloat16* out = p.out + ((int64_t)t.g * p.feat + f) * p.cols + col;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();                                  // the box before has been read
            if ((lane >> 4) == h) {
              uint8_t* rowp = box + (lane & 15) * 128;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                *reinterpret_cast<uint4*>(rowp + ((j ^ l8) << 4)) = a[j];
                *reinterpret_cast<uint4*>(rowp + (((j + 4) ^ l8) << 4)) = b[j];
              }
            }
            __syncwarp();
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int i = (lane >> 3) + 4 * v;
              if (col < p.cols && f + 16 * h + i < p.feat)
                stg_v4(out + (int64_t)(16 * h + i) * p.cols,
                       *reinterpret_cast<const uint4*>(box + i * 128 + ((l8 ^ (i & 7)) << 4)));
            }
          }
        }
      } else {
        // 16 rows x 32 features in fp32 at a time, 128 bytes a row, 16-byte chunk c of row i at
        // c ^ (i & 1): a feature's stores and a row's eight-feature loads meet every bank once
        const int here = f < p.feat ? min(s_cnt[t.g] - t.n0, t.n) : 0;
        if (splits > 1) {
#pragma unroll 1
          for (int b = 0; 64 * b + 32 * odd < here; ++b) {
            uint32_t r[32];
            ptx::tmem_ld32(tbase + 64 * b + 32 * odd, r);
            ptx::tmem_ld_wait();
            put(b, r);
          }
          if (!last()) break;                              // (a pair has one unit)
#pragma unroll 1
          for (int b = 0; 64 * b + 32 * odd < here; ++b) join(b);
          fetch_add();
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = 64 * b + 32 * odd;                 // the box's first row
          if (j >= here) break;
          uint32_t r[32];
          if (splits > 1) {
            get(pt, b, r);
          } else {
            ptx::tmem_ld32(tbase + j, r);
            ptx::tmem_ld_wait();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();                                  // the box before has been read
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint32_t*>(box + i * 128 + (((lane >> 2) ^ (i & 1)) << 4) +
                                           (lane & 3) * 4) = r[16 * h + i];
            __syncwarp();
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint8_t* from = box + (lr + 8 * v) * 128;
              const float4 lo = *reinterpret_cast<const float4*>(from + (((2 * lc) ^ (lr & 1)) << 4));
              const float4 hi = *reinterpret_cast<const float4*>(from + (((2 * lc + 1) ^ (lr & 1)) << 4));
              float e[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
              const int i = j + 16 * h + 8 * v + lr;
              if (i >= rows) continue;
              if (p.add) {
                float d[8];
                unpack8(add[b][2 * h + v], d);
#pragma unroll
                for (int x = 0; x < 8; ++x) e[x] += d[x];
              }
              stg_v4(p.out + (row0 + i) * p.ldo + fl, pack8(e));
            }
          }
        }
        give();
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, 512);
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

// Columns of an operand that lies along M or N, 64 to a chunk, `chunks` of them and 64 rows to a
// box: {64 columns of a chunk, rows, chunk, group}. Columns past the last whole chunk are not in it.
bool chunk_map(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t ld,
               uint64_t groups, uint32_t chunks) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = gg::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, rows, cols / 64, groups};
  cuuint64_t strides[3] = {ld * 2, 128, ld * rows * 2};
  cuuint32_t box[4] = {64, 64, chunks, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 4 : 3, const_cast<void*>(ptr), dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t run_ragged(const Maps& m, const RaggedProduct& p, cudaStream_t s) {
  auto kern = ragged_pair_kernel<MODE>;
  static PerDevice set;
  int grid = 0;
  const cudaError_t e = pair_grid_once(set, kern, kPairThreads, kSmem, &grid);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)grid, dim3(kPairThreads, 1, 1), kSmem, s, m, p);
}

// Columns of a tile, from what it takes in clocks: steps of 450 + 1.75 a column, an epilogue of 1280
// + 20 a column beside the next tile's steps; in rounds over the pairs of SMs, or shared among them.
// `others`: tiles in the other dimension; `groups`: each cuts `columns` once more (half a tile on
// average), or 0; nk: steps. (Against the best of 64, 128, 192 and 256 columns, 24 shapes from 333 rows of
// 4096 x 4096 to 8192 of 8192 x 8192 in the three modes: the same or within 5 % for 21. 1000 rows of 8
// experts, 2048 x 1024: 13.2 and 11.6 us, as a data gradient, whose joins it takes too low, 22.1 and 15.0;
// 2801 rows of 4, 200 x 7776, as a data gradient 23.6 and 20.2.)
int tile_columns(int64_t columns, int64_t others, int64_t groups, int nk, int least) {
  const int pairs = num_sms() / 2 < kRaggedPairs ? num_sms() / 2 : kRaggedPairs;
  int best = 256;
  double cost = 0;
  for (int tile = 256; tile >= least; tile -= least) {
    const double tiles = others * (groups ? (double)columns / tile + 0.5 * groups
                                          : (double)((columns + tile - 1) / tile));
    const double step = 450 + 1.75 * tile, epilogue = 20 * (tile + 64);
    const int n = shares((int)(pairs / (tiles < 1 ? 1 : tiles)), nk, tile);
    const double c = 2 * tiles <= pairs && n > 1
                         ? nk * step / n + 12.0 * tile * n + 10000 + epilogue
                         : ceil(tiles / pairs) * fmax(nk * step, epilogue) + epilogue;
    if (tile == 256 || c < 0.95 * cost) {
      best = tile;
      cost = c;
    }
  }
  return best;
}

}  // namespace

// Tiles of 256 features and 64 columns at least, in 32 bits.
bool ragged_fits(int64_t rows, int G, int64_t feat, int64_t cols) {
  const int64_t n = cols ? (cols + 127) / 128 * G : rows / 64 + G;
  return n * ((feat + kM - 1) / kM) < (1LL << 31);
}

cudaError_t launch_ragged_gemm(RaggedProduct p, int dgrad, const void* x, int64_t ldx,
                               const void* w, int N, int K, cudaStream_t s) {
  p.feat = dgrad ? K : N;
  p.red = dgrad ? N : K;
  p.cols = 0;
  p.tile = tile_columns(p.rows, (p.feat + kM - 1) / kM, p.rows < p.G ? p.rows : p.G,
                        (p.red + BK - 1) / BK, 64);
  Maps m;
  for (int i = 0; i < 8; ++i)
    if (!map2(&m.b[i], x, p.red, p.rows, ldx, 64, 16 * (i + 1))) return cudaErrorInvalidValue;
  if (!map3(&m.a2, w, K, N, p.G, 64, dgrad ? 64 : 128)) return cudaErrorInvalidValue;
  m.a = m.b2 = m.a2;
  if (dgrad && K >= 64 && !chunk_map(&m.a, w, K, N, K, p.G, 2)) return cudaErrorInvalidValue;
  return dgrad ? run_ragged<kDgrad>(m, p, s) : run_ragged<kFwd>(m, p, s);
}

cudaError_t launch_ragged_wgrad(RaggedProduct p, const void* dy, int64_t lddy, const void* x,
                                int64_t ldx, int N, int K, cudaStream_t s) {
  p.feat = N;
  p.cols = K;
  p.red = 0;
  p.add = nullptr;
  p.tile = tile_columns(K, (int64_t)p.G * ((N + kM - 1) / kM), 0, (int)(p.rows / p.G / BK) + 1, 128);
  // (without rows nothing is loaded: the maps are then of any valid extent)
  const bool some = p.rows > 0;
  const void *pa = some ? dy : p.out, *pb = some ? x : p.out;
  const int64_t rows = some ? p.rows : 1, lda = some ? lddy : N, ldb = some ? ldx : K;
  Maps m;
  if (!map2(&m.a2, pa, N, rows, lda, 64, 64) || !map2(&m.b2, pb, K, rows, ldb, 64, 64))
    return cudaErrorInvalidValue;
  m.a = m.a2;
  for (int i = 0; i < 8; ++i) m.b[i] = m.b2;
  if ((N >= 64 && !chunk_map(&m.a, pa, N, rows, lda, 0, 2)) ||
      (K >= 64 && !chunk_map(&m.b[0], pb, K, rows, ldb, 0, p.tile / 128)))
    return cudaErrorInvalidValue;
  return run_ragged<kWgrad>(m, p, s);
}

}  // namespace moe
