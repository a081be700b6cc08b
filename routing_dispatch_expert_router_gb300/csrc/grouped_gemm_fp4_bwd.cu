// The data gradients of 4-bit experts: bf16 rows times the experts' 4-bit weights,
// reduced over the weights' rows.
//   FC2:  dh = dO W2^,  then the SwiGLU derivative with gate and up from the 8-bit
//         checkpoint -> dGU (bf16);
//   FC1:  dX = alpha (dGU W13^) + the router's term (bf16).
// (The W/D split and the recompute-friendly checkpoints of "Scalable Training of
// Mixture-of-Experts Models with Megatron Core", es summary §2.3.)
//
// The codes' scales lie along the weights' columns and this product reduces over
// their rows, which the FP4 tensor cores cannot do: their scales belong to the
// reduced dimension. A weight's value, E2M1 times E4M3 or a power of two, has at
// most 6 significant bits, so it is exact in bf16, and the product runs on the bf16
// tensor cores (tcgen05 kind::f16) with B made from the codes in shared memory. That
// keeps the weights' traffic at 0.53-0.56 bytes an element; writing them out as bf16
// first costs 4 more each way (one layer of 64 experts, 4096 x 2048: 0.70 of 1.88 ms).
//
// CTA pairs, 256 x 256 tiles, one persistent CTA pair per two SMs, 608 threads:
//   warp 0      TMA producer of A (one lane): per 64-deep k-block this CTA's 128 rows;
//   warp 18     TMA producer of the codes and scale atoms of 64 weight rows x 128
//               columns a k-block (one lane), in a ring of their own: a stage of A and
//               B is then not held while codes are on their way;
//   warp 1      MMA issuer (one lane of the even CTA): M=256 N=256 K=16;
//   warps 2-9   epilogue, two warps per tensor-memory lane quarter, 128 of the 256
//               columns each;
//   warps 10-17 the codes' values into B's stage (MN-major, 128-byte swizzle), 8192
//               elements a k-block; teams of two warps take k-blocks in turn, so that
//               one team's waits, loads and stores pass under the others' work.
// Both products of that layer (32768 rows) take 1373 to 1381 us again and again on the same
// inputs, 1457 to 1493 with three sets in turn: 0.43 us a k-block, of which the MMAs and
// A's loads alone take 0.34. What is left is shared memory's bandwidth:
// the MMAs' reads, A's arrival and the codes' way in and values' way out fill about 600
// of 780 cycles a k-block. On the way: all eight warps on one k-block 3306 us, teams of
// four warps 2608, of two 1820; without bank conflicts 1772; the odd CTA's
// arrivals at the even CTA's barrier with a release of shared memory alone 1375 (one of
// all memory takes a warp 1600 cycles; made by a thread of its own, one k-block after the
// other, 2888). Tiles of 512 x 128 (B made once for 512 rows) take 2057: MMAs of N=128 run
// at half rate. 512 x 256 with one set of accumulators: 1850 before the arrivals changed
// (1772 then).
#include "fp4_layout.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace gg {

constexpr int kD4Threads = 608;
constexpr int kD4BN = 256;
constexpr int kD4Stages = 5;
constexpr int kD4ABytes = BM * BK * 2;                 // 16 KB
constexpr int kD4BBytes = 128 * BK * 2;                // 16 KB: this CTA's 128 columns
constexpr int kD4CodeBytes = BK * 64;                  // 64 rows x 128 codes
constexpr int kD4EpiWarps = 8;
constexpr int kD4ConvWarp = 2 + kD4EpiWarps;           // the first of the eight
constexpr int kD4ConvWarps = 8;
constexpr int kD4CodeWarp = kD4ConvWarp + kD4ConvWarps;
constexpr int kD4CodeSlots = 4;
constexpr int kD4Teams = 4;                            // of two warps, each every fourth k-block
constexpr int kD4EpiBytes = 2 * kBoxBytes;             // staging per epilogue warp: dG and dU
constexpr uint32_t kD4TmemCols = 2 * kD4BN;
enum D4Epi : int { kD4Swiglu = 0, kD4Out = 1 };

struct Dgrad4Params {
  int G, N, K;                 // output columns; reduction length (the weights' rows)
  int64_t rows;
  const int32_t* counts;
  const int32_t* offsets;
  const uint8_t* sfb;          // weight scales, [G][K / 128 slabs][ka][512]
  int ka;
  const uint8_t* ckpt;         // swiglu: gate | up, [rows, 2N]
  const uint8_t* ckpt_sf;
  const float* alpha_a;        // out: the factor, alpha_a[g] alpha_b[g] unit
  const float* alpha_b;
  float unit;                  // 2^unit_log2
  int unit_log2;
  const int32_t* token_of;     // out: the router's term, where dlogits is given
  const float* dlogits;
  const float* W_r;
  int router_E, router_T;
  int32_t* status;
};

template <int FMT>
struct D4Cfg {
  static constexpr int SF_BYTES = 128 / (4 * f4::block_of(FMT)) * f4::kAtomBytes;
  static constexpr int STAGE = kD4ABytes + kD4BBytes;
  static constexpr int RAW = kD4CodeBytes + SF_BYTES;          // codes and atoms of a stage
  static constexpr int RAW_OFF = kD4Stages * STAGE;
  static constexpr int CTRL_OFF = RAW_OFF + kD4CodeSlots * RAW;
  static constexpr int EPI_OFF = (CTRL_OFF + kCtrlBytes + 1023) / 1024 * 1024;
  static constexpr int SMEM = EPI_OFF + kD4EpiWarps * kD4EpiBytes + 1024;
  static_assert(SMEM <= 232448, "4-bit data gradient shared memory");
  static_assert(4864 + 16 * kD4CodeSlots <= kCtrlBytes, "code barriers in the control block");
};

// Eight codes (32 bits) -> their values in bf16 times f (the block's scale in both
// halves), in element order; exact. A code's three magnitude bits pick the high and
// the low byte of its value from tables of eight bytes, four codes to a byte
// permutation (0, .5, 1, 1.5 = 0000 3F00 3F80 3FC0; 2, 3, 4, 6 = 4000 4040 4080
// 40C0); its sign bit makes a permutation repeat the sign of a picked byte.
__device__ __forceinline__ uint4 weight8(uint32_t w, uint32_t f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t c = i ? w >> 16 : w;                   // four codes; prmt reads 16 bits
    const uint32_t m = c & 0x7777u;
    uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, m);
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, m);
    uint32_t neg;                                         // FF where negative, else 80
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(neg) : "r"(0x80808080u), "r"(c));
    hi |= (neg << 1) & 0x80808080u;
    const uint32_t v0 = __byte_perm(lo, hi, 0x5140), v1 = __byte_perm(lo, hi, 0x7362);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[2 * i]) : "r"(v0), "r"(f));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[2 * i + 1]) : "r"(v1), "r"(f));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A scale byte's value as a bf16 pair, exact.
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
  if (FMT == MOE_FP4_NV) {
    // E4M3's bits at a bf16's exponent and upper fraction are its value times
    // 2^-120, subnormals included
    const uint32_t e = byte << 4 | byte << 20;
    uint32_t f;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(f) : "r"(e), "r"(0x7B807B80u));
    return byte == 127u ? 0x7FC07FC0u : f;
  }
  const uint32_t e = byte == 255u ? 0x7FC0u : byte ? byte << 7 : 0x0040u;
  return e | e << 16;
}

// 32 checkpoint codes times their block's scale.
__device__ __forceinline__ void checkpoint8(uint32_t w0, uint32_t w1, float s, float (&f)[8]) {
  const uint32_t w[2] = {w0, w1};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[k >> 1] >> (16 * (k & 1)))));
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    f[2 * k] = t.x * s;
    f[2 * k + 1] = t.y * s;
  }
}

// Gate and up of 32 columns of one row, as the checkpoint keeps them.
struct Kept {
  uint4 g[2], u[2];
  uint32_t gs, us;
};

template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kD4Threads, 1)
fp4_dgrad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const Dgrad4Params p) {
  using C = D4Cfg<FMT>;
  constexpr int kStages = kD4Stages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t ctrl_u = base + C::CTRL_OFF;
  uint8_t* ctrl = sbase + C::CTRL_OFF;
  const uint32_t bar_full = ctrl_u;                       // [kStages], the even CTA's
  const uint32_t bar_empty = ctrl_u + 64;                 // [kStages]
  const uint32_t bar_code = ctrl_u + 4864;                // [kD4CodeSlots]
  const uint32_t bar_code_empty = bar_code + 8 * kD4CodeSlots;
  const uint32_t bar_tfull = ctrl_u + 128;                // [2]
  const uint32_t bar_tempty = ctrl_u + 144;               // [2]
  const uint32_t bar_drain = ctrl_u + 160;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 196);
  int* prefix = reinterpret_cast<int*>(ctrl + 256);
  int* mtiles = reinterpret_cast<int*>(ctrl + 1344);
  int* s_off = reinterpret_cast<int*>(ctrl + 2432);
  int* s_cnt = reinterpret_cast<int*>(ctrl + 3520);
  int* tmp = reinterpret_cast<int*>(ctrl + 4608);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int G = p.G;
  const int NT = (p.N + kD4BN - 1) / kD4BN;
  const int nk = p.K / BK;
  for (int g = tid; g < G; g += kD4Threads) {
    int64_t c = p.counts[g], o = p.offsets[g];
    if (c < 0 || o < 0 || o % 128 || o + c > p.rows) {
      record_status(p.status, MOE_ERR_DEVICE_CHECK);
      c = o = 0;
    }
    s_cnt[g] = (int)c;
    s_off[g] = (int)o;
    mtiles[g] = (int)((c + BM - 1) / BM);
    prefix[g] = ((mtiles[g] + 1) >> 1) * NT;             // pair tiles of the group
  }
  if (tid == 0) *abort_flag = 0;
  __syncthreads();
  const int total = block_exclusive_scan(prefix, G, tmp);
  if (tid == 0) prefix[G] = total;
  __syncthreads();
  if (cluster >= total) {                                // both CTAs of the pair leave together
    ptx::grid_dependency_wait();                         // and after the kernel before this one
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      // the even CTA's: its producer's arrival with A's bytes of both CTAs, and
      // the converting warps of both
      ptx::mbar_init(bar_full + 8 * s, 1 + 2 * kD4ConvWarps / kD4Teams);
      ptx::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < kD4CodeSlots; ++s) {
      ptx::mbar_init(bar_code + 8 * s, 1);
      ptx::mbar_init(bar_code_empty + 8 * s, kD4ConvWarps / kD4Teams);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(bar_tfull + 8 * a, 1);
      ptx::mbar_init(bar_tempty + 8 * a, 2 * kD4EpiWarps);
    }
    ptx::mbar_init(bar_drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), kD4TmemCols);
    ptx::tmem_relinquish_pair();
  }
  if (tid == 0) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  ptx::grid_launch_dependents();     // the next kernel's CTAs may start as these leave
  // pair tile -> group, m-pair, n-tile; m-pairs fastest
  auto decode_pair = [&](int pt, int& g, int& mp, int& nt) {
    g = find_group(prefix, G, pt);
    const int local = pt - prefix[g];
    const int npairs = (mtiles[g] + 1) >> 1;
    mp = local % npairs;
    nt = local / npairs;
  };

  if (warp == 0) {
    // ------------------------------------------------------- producer of A
    if (lane == 0) {
      ptx::grid_dependency_wait();     // A is what the kernel before this one wrote
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        int g, mp, nt;
        decode_pair(pt, g, mp, nt);
        const int row0 = s_off[g] + (2 * mp + (int)rank) * BM;
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget,
                                      abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * kD4ABytes);
          ptx::tma_load_2d_pair(base + stage * C::STAGE, &tmA,
                                ptx::mapa_shared(bar_full + 8 * stage, 0), kb * BK, row0);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        // A's loads already issued land within microseconds; give them time
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {
        }
      }
    }
  } else if (warp == kD4CodeWarp) {
    // ------------------------------------- producer of the codes and scales
    if (lane == 0) {
      uint32_t slot = 0, phase = 0;
      uint32_t issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        int g, mp, nt;
        decode_pair(pt, g, mp, nt);
        const int n0 = nt * kD4BN + (int)rank * 128;
        const uint8_t* sf = p.sfb + (int64_t)g * (p.K / 128) * p.ka * f4::kAtomBytes +
                            (int64_t)(n0 / 128) * C::SF_BYTES;
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait(bar_code_empty + 8 * slot, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const int k0 = kb * BK;
          const uint32_t cb = bar_code + 8 * slot;
          const uint32_t rawb = base + C::RAW_OFF + slot * C::RAW;
          ptx::mbar_arrive_expect_tx(cb, C::RAW);
          ptx::tma_load_2d(rawb, &tmB, cb, n0 / 2, g * p.K + k0);
          ptx::bulk_load(rawb + kD4CodeBytes, sf + (int64_t)(k0 / 128) * p.ka * f4::kAtomBytes,
                         C::SF_BYTES, cb);
          issued_mask |= 1u << slot;
          issued_phase = (issued_phase & ~(1u << slot)) | (phase << slot);
          if (++slot == kD4CodeSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every load issued must land before the CTA may exit
      for (int s = 0; s < kD4CodeSlots; ++s)
        if (issued_mask & (1u << s))
          ptx::mbar_wait(bar_code + 8 * s, (issued_phase >> s) & 1u, kWaitBudget, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t IDESC = ptx::idesc_bf16(2 * BM, kD4BN, 0, 1);
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        if (!ptx::mbar_wait_cluster(bar_tempty + 8 * acc, acc_phase ^ 1u, kWaitBudget,
                                    abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + acc * kD4BN;
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster(bar_full + 8 * stage, phase, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sA = base + stage * C::STAGE;
          const uint32_t sB = sA + kD4ABytes;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            ptx::mma_bf16_pair(d, ptx::smem_desc_sw128(sA + kk * 32, 16, 1024),
                               ptx::smem_desc_sw128(sB + kk * 2048, 8192, 1024), IDESC,
                               (kb | kk) ? 1u : 0u);
          issued = true;
          ptx::mma_commit_pair(bar_empty + 8 * stage, 3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair(bar_tfull + 8 * acc, 3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (issued) {
        ptx::mma_commit_pair(bar_drain, 1);
        ptx::mbar_wait(bar_drain, 0, kWaitBudget, nullptr);
      }
    }
  } else if (warp >= kD4ConvWarp) {  // up to kD4CodeWarp - 1
    // ------------------------------------------------------ codes to values
    // Lane: row lane / 4 of eight rows, the 32 columns 32 (lane % 4) .., so that a warp
    // reads 512 consecutive bytes of codes. Its four 16-byte pieces of values go out
    // in the order 0 1 2 3, or 2 3 0 1 in the right 64 columns: eight lanes then store
    // to eight distinct 16-byte bank groups (piece ^ (row % 8), two rows, four lanes).
    constexpr int kRows = 32 * kD4ConvWarps / kD4Teams / 4;      // rows of a pass
    const int team = (warp - kD4ConvWarp) / (kD4ConvWarps / kD4Teams);
    const int t = (tid - kD4ConvWarp * 32) % (32 * kD4ConvWarps / kD4Teams);
    const int trow = t >> 2, sub = t & 3;
    const int half = sub >> 1;                                   // which 64 columns
    uint32_t stage = 0, phase = 0, slot = 0, cphase = 0;
    int turn = 0;
    bool ok = true;
    const uint32_t leader_full = ptx::mapa_shared(bar_full, 0);
    for (int pt = cluster; pt < total && ok; pt += nclusters) {
      for (int kb = 0; kb < nk; ++kb) {
        if (turn == team) {
          // A team comes back to a slot when all slots have turned once, and to a
          // stage after at most two turns, of which the first is over: its k-block
          // before this one waited for it. So parities are never two phases off.
          static_assert(kD4CodeSlots % kD4Teams == 0 && kD4Teams <= kD4Stages, "parity waits");
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_code + 8 * slot, cphase, kWaitBudget,
                                                      abort_flag));
          if (!ok) break;
          const uint8_t* rawp = sbase + C::RAW_OFF + slot * C::RAW;
          uint8_t* sB = sbase + stage * C::STAGE + kD4ABytes;
          // all loads before the first store (the compiler cannot tell them apart)
          constexpr int kPass = BK / kRows;
          uint4 c[kPass];
          uint32_t f[kPass];                                     // the columns' scale bytes
#pragma unroll
          for (int i = 0; i < kPass; ++i) {
            const int row = trow + kRows * i;
            const int r = (kb & 1) * 64 + row;                   // row of the 128-row slab
            const uint8_t* sf = rawp + kD4CodeBytes + (r & 31) * 16 + (r >> 5) * 4;
            c[i] = *reinterpret_cast<const uint4*>(rawp + row * 64 + sub * 16);
            f[i] = FMT == MOE_FP4_NV
                       ? *reinterpret_cast<const uint16_t*>(sf + half * f4::kAtomBytes + (sub & 1) * 2)
                       : sf[sub];
          }
          // the MMAs that read this stage's B are done
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar_empty + 8 * stage, phase ^ 1u,
                                                              kWaitBudget, abort_flag));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kPass; ++i) {
            const int row = trow + kRows * i;
            const uint32_t s0 = scale_pair<FMT>(f[i] & 255u);
            const uint32_t s1 = FMT == MOE_FP4_NV ? scale_pair<FMT>(f[i] >> 8) : s0;
            uint8_t* dst = sB + row * 128 + half * 8192;
            // pieces 0, 1 (the first 16 columns) and 2, 3, swapped in the right half
            const uint32_t wa = half ? c[i].z : c[i].x, wb = half ? c[i].w : c[i].y;
            const uint32_t wc = half ? c[i].x : c[i].z, wd = half ? c[i].y : c[i].w;
            const uint32_t sa = half ? s1 : s0, sc = half ? s0 : s1;
            const int first = 4 * (sub & 1) + 2 * half, x = row & 7;
            *reinterpret_cast<uint4*>(dst + ((first ^ x) << 4)) = weight8(wa, sa);
            *reinterpret_cast<uint4*>(dst + (((first + 1) ^ x) << 4)) = weight8(wb, sa);
            *reinterpret_cast<uint4*>(dst + (((first ^ 2) ^ x) << 4)) = weight8(wc, sc);
            *reinterpret_cast<uint4*>(dst + ((((first ^ 2) + 1) ^ x) << 4)) = weight8(wd, sc);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          // (the codes' slot too only now: right after its reads the arrival could pass
          // ones that had not returned, and the next codes landed under them)
          if (lane == 0) {
            ptx::mbar_arrive(bar_code_empty + 8 * slot);
            if (rank == 0) ptx::mbar_arrive(bar_full + 8 * stage);
            else ptx::mbar_arrive_cluster_smem(leader_full + 8 * stage);
          }
        }
        if (++turn == kD4Teams) turn = 0;
        if (++slot == kD4CodeSlots) {
          slot = 0;
          cphase ^= 1u;
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                                  // lane quarter
    const int ch = (warp - 2) >> 2;                          // which 128 of the 256 columns
    uint8_t* box = sbase + C::EPI_OFF + (warp - 2) * kD4EpiBytes;
    const uint32_t box_u32 = base + C::EPI_OFF + (warp - 2) * kD4EpiBytes;
    const uint32_t leader_tempty[2] = {ptx::mapa_shared(bar_tempty, 0),
                                       ptx::mapa_shared(bar_tempty + 8, 0)};
    uint32_t acc = 0, acc_phase = 0;
    ptx::grid_dependency_wait();       // nothing is written before that kernel is done
    for (int pt = cluster; pt < total; pt += nclusters) {
      int g, mp, nt;
      decode_pair(pt, g, mp, nt);
      const int mt = 2 * mp + (int)rank;
      const int row0 = s_off[g] + mt * BM + q * 32;
      const int rv = s_cnt[g] - mt * BM - q * 32;            // rows of this warp that hold data
      const int f0 = nt * kD4BN + 128 * ch;
      const int64_t row = row0 + lane;
      // what the row needs besides the accumulator: gate and up of its next 32
      // columns, or the router's term
      Kept k = {};
      float rd = 0.f;
      Fp4Factor alpha = {1.f, kFp4One};
      const float* rw = nullptr;
      auto fetch = [&](int col) {
        if (lane >= rv || col >= p.N) return;
        const uint8_t* at = p.ckpt + row * 2 * p.N + col;
        k.g[0] = ldg_nc_v4(at);
        k.g[1] = ldg_nc_v4(at + 16);
        k.u[0] = ldg_nc_v4(at + p.N);
        k.u[1] = ldg_nc_v4(at + p.N + 16);
        const uint8_t* sc = p.ckpt_sf + row * (2 * p.N / 32) + col / 32;
        k.gs = __ldg(sc);
        k.us = __ldg(sc + p.N / 32);
      };
      if (EPI == kD4Swiglu) {
        fetch(f0);
      } else {
        alpha = fp4_factor(p.alpha_a ? p.alpha_a[g] : 1.f, p.alpha_b ? p.alpha_b[g] : 1.f, p.unit,
                           p.unit_log2);
        if (p.dlogits && g < p.router_E) {
          const int tk = lane < rv ? p.token_of[row] : -1;
          // (a lane without a token has no term: zero times W_r would be NaN where W_r is
          // not finite)
          if (tk >= 0 && tk < p.router_T) {
            rd = p.dlogits[(int64_t)tk * p.router_E + g];
            rw = p.W_r + (int64_t)g * p.N + f0;
          }
        }
      }
      bool ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar_tfull + 8 * acc, acc_phase,
                                                               kWaitBudget, abort_flag));
      if (!ok) {
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      ptx::tc_fence_after();
      const uint32_t tbase = tmem_base + acc * kD4BN + 128 * ch + ((uint32_t)(q * 32) << 16);
      // swiglu: rows without data need no gradient. out: a group's 128-row blocks are
      // written whole, their rows without data as zeros
      if (EPI == kD4Swiglu ? rv > 0 : mt < mtiles[g]) {
#pragma unroll 1
        for (int c = 0; c < 128 && f0 + c < p.N; c += 32) {
          uint32_t r[32];
          ptx::tmem_ld32(tbase + c, r);
          ptx::tmem_ld_wait();
          uint4 o[2][4];                                     // dG and dU, or dX
          if (EPI == kD4Swiglu) {
            const Kept n = k;
            if (c < 96) fetch(f0 + c + 32);
            const float gs = fp4_scale_value<MOE_FP4_MX>(n.gs);
            const float us = fp4_scale_value<MOE_FP4_MX>(n.us);
            const uint32_t gw[8] = {n.g[0].x, n.g[0].y, n.g[0].z, n.g[0].w,
                                    n.g[1].x, n.g[1].y, n.g[1].z, n.g[1].w};
            const uint32_t uw[8] = {n.u[0].x, n.u[0].y, n.u[0].z, n.u[0].w,
                                    n.u[1].x, n.u[1].y, n.u[1].z, n.u[1].w};
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float gf[8], uf[8], dg[8], du[8];
              checkpoint8(gw[2 * v], gw[2 * v + 1], gs, gf);
              checkpoint8(uw[2 * v], uw[2 * v + 1], us, uf);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float dh = __uint_as_float(r[8 * v + i]);
                const float s = sigmoid_f(gf[i]);
                const float si = gf[i] * s;
                du[i] = dh * si;
                dg[i] = dh * uf[i] * fmaf(si, 1.f - s, s);
              }
              // rounded to bf16: the next product's A. (Two bf16 terms each would keep
              // 16 bits, for twice that product's MMAs and A traffic; with one the
              // result is off by 0.0023 of its norm, 0.0017 being its own rounding.)
              o[0][v] = pack8(dg);
              o[1][v] = pack8(du);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              r[i] = __float_as_uint(lane < rv ? __uint_as_float(r[i]) * alpha.by : 0.f);
            if (alpha.rest != kFp4One) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(__uint_as_float(r[i]) * __uint_as_float(alpha.rest << 16));
            }
            if (rw) {
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                const float4 w4 = __ldg(reinterpret_cast<const float4*>(rw + c) + v);
                r[4 * v] = __float_as_uint(fmaf(rd, w4.x, __uint_as_float(r[4 * v])));
                r[4 * v + 1] = __float_as_uint(fmaf(rd, w4.y, __uint_as_float(r[4 * v + 1])));
                r[4 * v + 2] = __float_as_uint(fmaf(rd, w4.z, __uint_as_float(r[4 * v + 2])));
                r[4 * v + 3] = __float_as_uint(fmaf(rd, w4.w, __uint_as_float(r[4 * v + 3])));
              }
            }
            pack_slice(r, o[0]);
          }
          // dG and dU in the staging's two boxes, or dX in one of them in turn
          if (lane == 0) {
            if (EPI == kD4Swiglu) ptx::tma_store_wait_read();
            else ptx::tma_store_wait_read_1();
          }
          __syncwarp();
          const int at = EPI == kD4Swiglu ? 0 : (c >> 5) & 1;
          stage_row(box, at, lane, o[0]);
          if (EPI == kD4Swiglu) stage_row(box, 1, lane, o[1]);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_2d(&tmC, box_u32 + at * kBoxBytes, f0 + c, row0);
            if (EPI == kD4Swiglu) ptx::tma_store_2d(&tmC, box_u32 + kBoxBytes, p.N + f0 + c, row0);
            ptx::tma_store_commit();
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(leader_tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) ptx::tma_store_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, kD4TmemCols);
  }
}

// 4-bit weights [rows, K / 2 bytes] in boxes of 64 bytes x 64 rows, not swizzled.
static bool make_map_codes(CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols / 2, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols / 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// As many pairs as can be resident at once.
template <int FMT, int EPI>
static cudaError_t run_dgrad4(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                              const Dgrad4Params& p, bool early, cudaStream_t s) {
  auto kern = fp4_dgrad_kernel<FMT, EPI>;
  constexpr int smem = D4Cfg<FMT>::SMEM;
  static PerDevice set;
  int grid = 0;
  const cudaError_t e = pair_grid_once(set, kern, kD4Threads, smem, &grid);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(kD4Threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, a, b, c, p);
}

static Dgrad4Params dgrad4_params(const Fp4Problem& q, int32_t* status) {
  Dgrad4Params p{};
  p.G = q.G;
  p.N = (int)q.N;
  p.K = (int)q.K;
  p.rows = q.rows;
  p.counts = q.counts;
  p.offsets = q.offsets;
  p.sfb = q.sfb;
  p.ka = (int)f4::atoms_k(q.fmt, q.N);
  p.status = status;
  return p;
}

}  // namespace gg

using namespace gg;

cudaError_t launch_fp4_dgrad_swiglu(const Fp4Problem& q, const uint8_t* ckpt,
                                    const uint8_t* ckpt_sf, void* dGU, int32_t* status,
                                    cudaStream_t s) {
  if (q.rows == 0) return cudaSuccess;
  CUtensorMap a, b, c;
  if (!make_map(&a, q.a, (uint64_t)q.K, (uint64_t)q.rows, 128) ||
      !make_map_codes(&b, q.b, q.N, (int64_t)q.G * q.K) ||
      !make_out_map(&c, dGU, 2 * (uint64_t)q.N, (uint64_t)q.rows))
    return cudaErrorInvalidValue;
  Dgrad4Params p = dgrad4_params(q, status);
  p.ckpt = ckpt;
  p.ckpt_sf = ckpt_sf;
  return q.fmt == MOE_FP4_NV ? run_dgrad4<MOE_FP4_NV, kD4Swiglu>(a, b, c, p, q.early, s)
                             : run_dgrad4<MOE_FP4_MX, kD4Swiglu>(a, b, c, p, q.early, s);
}

cudaError_t launch_fp4_dgrad_out(const Fp4Problem& q, const float* alpha_b, void* dX,
                                 const int32_t* token_of, const float* dlogits, const float* W_r,
                                 int router_E, int router_T, int32_t* status, cudaStream_t s) {
  if (q.rows == 0) return cudaSuccess;
  CUtensorMap a, b, c;
  if (!make_map(&a, q.a, (uint64_t)q.K, (uint64_t)q.rows, 128) ||
      !make_map_codes(&b, q.b, q.N, (int64_t)q.G * q.K) ||
      !make_out_map(&c, dX, (uint64_t)q.N, (uint64_t)q.rows))
    return cudaErrorInvalidValue;
  Dgrad4Params p = dgrad4_params(q, status);
  p.alpha_a = q.alpha;
  p.alpha_b = alpha_b;
  p.unit = ldexpf(1.f, q.unit_log2);
  p.unit_log2 = q.unit_log2;
  p.token_of = token_of;
  p.dlogits = dlogits;
  p.W_r = W_r;
  p.router_E = router_E;
  p.router_T = router_T;
  return q.fmt == MOE_FP4_NV ? run_dgrad4<MOE_FP4_NV, kD4Out>(a, b, c, p, q.early, s)
                             : run_dgrad4<MOE_FP4_MX, kD4Out>(a, b, c, p, q.early, s);
}

}  // namespace moe
