// Grouped products of few rows: y[r] = x[r] W[g]^T with W in bf16 or in 4-bit integers with
// group scales. Every byte that has to move is a weight's, so HBM bounds them, and the kernel
// is a stream: one persistent CTA per SM takes an even share of all (expert, 256 output
// columns, step of K) pieces in order, whatever their expert, and its weights come by TMA into
// a ring of stages that never drains between experts.
//
//   warp 0         TMA producer (one lane): 256 weight rows x 128 bytes of K a stage, the same
//                  step of the tokens' rows, and the group scales and zero points;
//   warps 1-3      (4-bit) the tokens' elements in the order in which codes unpack;
//   eight warps    mma.sync m16n8k16, the weights as A: a warp has 32 weight rows. Tokens are
//                  B, eight to a tile, at most 16 a pass: with few tokens tcgen05's 128-row
//                  tiles would multiply padding, and its operands would have to be written
//                  back to shared memory as bf16 first, four times the bytes of the codes;
//   four warps     join units that CTAs share and write results, beside the next unit's sums.
//
// 4-bit weights are s (q - z). The codes become bf16 numbers 128 + q by placing their bits in
// the mantissa (one logic operation for two), and one packed addition takes 128 + z off again:
// q - z is exact in bf16, so what is summed is (q - z) x itself, in fp32 per group of K, and s is
// applied to the group's sum. (Sums of (128 + q) x with (128 + z) sum x taken off behind them need no
// such addition, but their roundings are those of 128 x: a channel 1000 times the others whose
// code is its zero point left an error of 2e-3 of the group's result, and values above 2^120 a NaN.)
//
// A (expert, columns) unit that two or more CTAs share is joined through scratch: every CTA
// writes its fp32 part, the one that arrives last adds the parts in K's order. So results do
// not depend on timing.
//
// With many rows and few outputs (an adapter's products into its rank) the roles change: 256 rows are
// the operand that streams, the expert's weights the one of 16, turned by ldmatrix where the
// reduction runs over their rows. 8192 rows of 4096 to 16: 21.9 us.
//
// A row of each of two experts through 28672 x 4096 in 4 bits (121 MB): 31.5 us, 3.8 TB/s; loads alone
// take 27.6, the launch, the shares and the last joins the rest. 512 rows of 64 experts through
// 4096 x 2048 (287 MB): 75 us, 3.8 TB/s: a step whose unit has two tiles of tokens takes
// 1.24 us (2560 clocks), for whose bytes HBM takes 0.77. bf16, 8 rows of five experts through
// 4096 x 14336 (587 MB): 86 us, 6.8 TB/s.
#include "gemm_common.cuh"

namespace moe {
namespace {

using gg::encode_fn;
using gg::kWaitBudget;

constexpr int kSlab = 256;                     // weight rows of a unit
constexpr int kTok = 16;                       // tokens of a unit
constexpr int kConsumers = kSlab / 32;
constexpr int kJoiners = 4;                    // warps that write results
constexpr int kTileLd = kTok + 1;
constexpr int kTileBytes = kSlab * kTileLd * 4;

// What streams as the 256-row operand, and what is the other one, of 16 rows a pass.
enum Roles : int {
  kWeightsStream = 0,      // an expert's weights; its rows
  kRowsStream = 1,         // an expert's rows; its weights, of few outputs
  kRowsStreamT = 2,        // the same where the reduction runs over the weights' rows
};

template <bool W4>
struct Cfg {
  static constexpr int HELPERS = W4 ? 3 : 0;       // (four warps a scheduler: 128 registers)
  static constexpr int THREADS = 32 * (1 + HELPERS + kConsumers + kJoiners);
  static constexpr int STAGES = W4 ? 4 : 5;
  static constexpr int STEP = W4 ? 256 : 64;           // elements of K a stage
  // what a step of one and of two token tiles takes, as measured (codes in L2, groups of 128, 64 and
  // 32 with zero points: 2070 and 2560 clocks, 2260 and 2790, 2640 and 3280)
  static constexpr int W1 = W4 ? 4 : 1, W2 = W4 ? 5 : 1;
  static constexpr int XBOXES = STEP / 64;             // boxes of 64 elements x 8 tokens
  static constexpr int X_OFF = kSlab * 128;
  static constexpr int S_OFF = X_OFF + kTok / 8 * XBOXES * 1024;
  static constexpr int Z_OFF = S_OFF + (W4 ? 8 * kSlab * 2 : 0);   // eight groups at most
  static constexpr int STAGE = (Z_OFF + (W4 ? 8 * kSlab : 0) + 1023) / 1024 * 1024;
  static constexpr int CTRL = W4 ? 4096 : 5376;
  static constexpr int SMEM = STAGES * STAGE + 2 * kTileBytes + CTRL + 1024;
};
static_assert(Cfg<true>::SMEM <= 232448 && Cfg<false>::SMEM <= 232448, "shared memory");

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Loads of a stage: its address the same in all lanes, the lane's place and a constant beside it,
// which one load instruction takes.
template <class T>
__device__ __forceinline__ T at(const uint8_t* st, uint32_t place, int offset) {
  return *reinterpret_cast<const T*>(st + place + offset);
}

// Elements i and i + 4 of a word of eight codes as the bf16 pair q - z; z: the pair -(128 + z).
__device__ __forceinline__ uint32_t codes_pair(uint32_t w, int i, uint32_t z) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w >> (4 * i)));
  asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(z));
  return r;
}

// The weight row of a warp's eight that lane group g of the MMA has. With 16-byte loads the
// eight lanes that go together have rows four apart, whose swizzled places are in all banks.
template <bool W4, int GC>
__device__ __forceinline__ int weight_row(int g) {
  return W4 && GC == 4 ? ((g & 1) << 2) | (g >> 1) : g;
}
// Where the helpers put 16-byte piece `piece` of box `box` of a token's 256 elements, so that
// the pieces that eight lanes read together are in all banks.
template <int GC>
__device__ __forceinline__ int token_place(int tok, int box, int piece) {
  return GC == 4 ? piece ^ (box & 1) ^ ((tok & 1) << 1) : piece ^ ((tok & 1) << 2);
}

// A lane's places in a stage, without the stage's address: weights, tokens' pieces, scales, zero points.
// In an MMA a lane has any 16-bit pairs of K as long as A's and B's are the same and all lanes'
// are of one group: with groups of 128 elements lane t has elements 32 t .. 32 t + 31 of the group
// (16 bytes of codes), else 8 t .. 8 t + 7 of each 32 (a word).
struct Places {
  uint32_t w[8], x[2][4], s, z;                 // x: for one tile of eight tokens, for two
};

template <bool W4, bool SWIGLU, int GC>
__device__ __forceinline__ Places places(const FewProduct& p, int rg, int g, int t) {
  using C = Cfg<W4>;
  Places a;
  const int r = weight_row<W4, GC>(g);
  const int row0 = rg * 32 + r;                  // and 8, 16, 24 on: the same low three bits
  if constexpr (W4) {
    if constexpr (GC == 4) {
#pragma unroll
      for (int q = 0; q < 2; ++q) a.w[q] = row0 * 128 + (((4 * q + t) ^ r) << 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.x[0][j] = C::X_OFF + g * 128 + (token_place<GC>(g, t >> 1, 4 * (t & 1) + j) << 4) +
                    (t >> 1) * 1024;
        a.x[1][j] = a.x[0][j] + (t >> 1) * 1024;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a.w[i] = row0 * 128 + ((i ^ r) << 4) + t * 4;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        a.x[0][b] = C::X_OFF + g * 128 + (token_place<GC>(g, 0, b * 4 + t) << 4);
    }
    // (scales and zero points: gate's and up's rows apart, or 256 rows a group)
    const int at = SWIGLU ? (rg >> 2) * p.groups_per_step * 128 + (row0 & 127) : row0;
    a.s = C::S_OFF + at * 2;
    a.z = C::Z_OFF + at;
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      a.w[b] = row0 * 128 + (((4 * b + t) ^ r) << 4);
      a.x[0][b] = C::X_OFF + g * 128 + (((4 * b + t) ^ g) << 4);
    }
  }
  return a;
}

// What a step adds to a warp's 32 rows x 8 NTL tokens. GC: chunks of 32 elements in a group.
template <int NTL, bool SWIGLU, int GC>
__device__ __forceinline__ void step_int4(float (&tot)[2][2][4], const uint8_t* st, const Places& a,
                                          bool has_zeros) {
  using C = Cfg<true>;
  constexpr int GS = SWIGLU ? 128 : 256;         // from one group's scales to the next's
  constexpr int XB = NTL * 1024;                 // from one box of the tokens to the next
#pragma unroll
  for (int c0 = 0; c0 < 8; c0 += GC) {
    float acc[2][NTL][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NTL; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    // -(128 + z) of the group, made as the codes' bf16 numbers are
    const int q = c0 / GC;
    uint32_t z[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        z[m][h] = has_zeros ? (at<uint8_t>(st, a.z, q * GS + 16 * m + 8 * h) & 127u) * 0x10001u | 0xc300c300u
                            : 0xc308c308u;
    uint4 w4[2][2];
    if (GC == 4) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) w4[m][h] = at<uint4>(st, a.w[c0 / 4], m * 2048 + h * 1024);
    }
#pragma unroll
    for (int c = c0; c < c0 + GC; ++c) {
      uint32_t w[2][2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4& v = w4[m][h];
          w[m][h] = GC == 4 ? (c & 3) == 0   ? v.x
                              : (c & 3) == 1 ? v.y
                              : (c & 3) == 2 ? v.z
                                             : v.w
                            : at<uint32_t>(st, a.w[c], m * 2048 + h * 1024);
        }
      uint4 x[NTL];
#pragma unroll
      for (int n = 0; n < NTL; ++n)
        x[n] = GC == 4 ? at<uint4>(st, a.x[NTL - 1][c & 3], n * 1024 + (c >> 2) * 2 * XB)
                       : at<uint4>(st, a.x[0][c & 1], n * 1024 + (c >> 1) * XB);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t a0 = codes_pair(w[m][0], 0, z[m][0]), a1 = codes_pair(w[m][1], 0, z[m][1]);
        const uint32_t a2 = codes_pair(w[m][0], 1, z[m][0]), a3 = codes_pair(w[m][1], 1, z[m][1]);
        const uint32_t b0 = codes_pair(w[m][0], 2, z[m][0]), b1 = codes_pair(w[m][1], 2, z[m][1]);
        const uint32_t b2 = codes_pair(w[m][0], 3, z[m][0]), b3 = codes_pair(w[m][1], 3, z[m][1]);
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          mma16816(acc[m][n], a0, a1, a2, a3, x[n].x, x[n].y);
          mma16816(acc[m][n], b0, b1, b2, b3, x[n].z, x[n].w);
        }
      }
    }
    // the group's sums by its scales
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = __uint_as_float(
            (uint32_t)at<uint16_t>(st, a.s, (q * GS + 16 * m + 8 * h) * 2) << 16);
        const uint64_t s2 = ptx::f2_pack(s, s);
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          const uint64_t d = ptx::f2_pack(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
          float(&t)[4] = tot[m][n];
          ptx::f2_unpack(ptx::f2_fma(s2, d, ptx::f2_pack(t[2 * h], t[2 * h + 1])), t[2 * h], t[2 * h + 1]);
        }
      }
  }
}

// TR: the tokens' operand lies [64 of K][8 NTL columns], and is turned on its way to registers (row
// i of matrix j of a 32: element 8 (i / 2) + i % 2 + 2 j, as the lanes have the other operand's).
template <int NTL, bool TR>
__device__ __forceinline__ void step_bf16(float (&tot)[2][2][4], const uint8_t* st, const Places& a) {
  const int lane = threadIdx.x & 31;
  const uint32_t turned = ptx::smem_u32(st) + Cfg<false>::X_OFF +
                          (8 * ((lane & 7) >> 1) + (lane & 1) + 2 * (lane >> 3)) * (16 * NTL);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint4 w[2][2], x[NTL];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[m][h] = at<uint4>(st, a.w[c], m * 2048 + h * 1024);
#pragma unroll
    for (int n = 0; n < NTL; ++n) {
      if (TR)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[n].x), "=r"(x[n].y), "=r"(x[n].z), "=r"(x[n].w)
                     : "r"(turned + c * 32 * 16 * NTL + n * 16) : "memory");
      else
        x[n] = at<uint4>(st, a.x[0][c], n * 1024);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NTL; ++n) {
        mma16816(tot[m][n], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, x[n].x, x[n].y);
        mma16816(tot[m][n], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, x[n].z, x[n].w);
      }
  }
}

// A place in the stream: step `step` of the unit (group, slab of columns, tile of tokens). Token
// tiles are fastest, so that those of the same weights follow each other and find them in L2.
struct Place {
  int g, slab, tile, step;
};

// A TMA request costs its issuer some 200 clocks whatever its size, and a stage's bytes come in
// 1400: each operand is one request. w: 256 rows, or 128 of the gate and of the up half; x: 8 and
// 16 tokens, all of a stage's K (in boxes of 64 elements, where K is not whole boxes); s, z.
struct Maps {
  CUtensorMap w, x[2], s, z;
};

// GC: chunks of 32 elements of K in a scale's group (4-bit).
template <bool W4, bool SWIGLU, int GC, int ROLES>
__global__ void __launch_bounds__(Cfg<W4>::THREADS, 1)
product_few_kernel(const __grid_constant__ Maps maps, const FewProduct p) {
  using C = Cfg<W4>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* stages = smem_raw + (base - raw);
  float* tiles = reinterpret_cast<float*>(stages + C::STAGES * C::STAGE);
  uint8_t* ctrl = reinterpret_cast<uint8_t*>(tiles) + 2 * kTileBytes;
  const uint32_t ctrl_u = base + C::STAGES * C::STAGE + 2 * kTileBytes;
  const uint32_t bar_full = ctrl_u, bar_ready = ctrl_u + 40, bar_empty = ctrl_u + 80;
  const uint32_t bar_tile = ctrl_u + 120, bar_free = ctrl_u + 136;     // of the two tiles
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 192);
  volatile int* s_last = reinterpret_cast<volatile int*>(ctrl + 196);
  Place* s_ends = reinterpret_cast<Place*>(ctrl + 208);    // [2]
  int* prefix = reinterpret_cast<int*>(ctrl + 256);        // [kMaxGroups + 1] weights
  int* s_off = reinterpret_cast<int*>(ctrl + 1536);        // [kMaxGroups]
  int* s_cnt = reinterpret_cast<int*>(ctrl + 2688);        // [kMaxGroups]
  int* tmp = reinterpret_cast<int*>(ctrl + 3840);          // [33]
  int* s_rows = reinterpret_cast<int*>(ctrl + 4096);       // [kMaxGroups] (rows that stream)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // what the steps of a slab of columns weigh: two token tiles of eight cost more than one
  auto slab_weight = [](int c) {
    const int rest = c % kTok;
    return c / kTok * C::W2 + (rest == 0 ? 0 : rest <= 8 ? C::W1 : C::W2);
  };
  if (tid == 0) {
    ptx::tma_prefetch_desc(&maps.w);
    ptx::tma_prefetch_desc(&maps.x[0]);
    if (W4) ptx::tma_prefetch_desc(&maps.s);
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_ready + 8 * s, C::HELPERS > 0 ? C::HELPERS : 1);
      ptx::mbar_init(bar_empty + 8 * s, kConsumers);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar_tile + 8 * i, kConsumers);
      ptx::mbar_init(bar_free + 8 * i, kJoiners);
    }
    ptx::fence_mbar_init();
  }
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  for (int g = tid; g < p.G; g += C::THREADS) {
    int c = (int)p.rows, o = 0;
    if (p.counts) {
      c = p.counts[g];
      o = p.offsets[g];
      if (c < 0 || o < 0 || (int64_t)o + c > p.rows) {
        if (blockIdx.x == 0) record_status(p.status, MOE_ERR_DEVICE_CHECK);
        c = 0;
      }
    }
    s_off[g] = o;
    int slabs = p.slabs;
    if (ROLES != kWeightsStream) {
      s_rows[g] = c;
      slabs = (c + kSlab - 1) / kSlab;
      c = c > 0 ? p.N : 0;
    }
    s_cnt[g] = c;
    prefix[g] = slab_weight(c) * slabs;
  }
  __syncthreads();
  const int weight = block_exclusive_scan(prefix, p.G, tmp);
  if (tid == 0) prefix[p.G] = weight;
  __syncthreads();
  auto slabs_of = [&](int g) {
    return ROLES != kWeightsStream ? (s_rows[g] + kSlab - 1) / kSlab : p.slabs;
  };
  // An even share of the steps, weighed by what they take, for each CTA: not under kFewLeast steps
  // where there are few, nor under what makes a unit's steps in one CTA and the parts that the last
  // one joins the least together (a part costs half a step), and no unit shared where whole ones leave the fullest CTA kFewJoin steps
  // more at most, which is what a join costs. CTA b begins with the first step (the first unit) at
  // or behind its share's start.
  const int KC = p.steps;
  const int64_t total = (int64_t)weight * KC;
  const int least = max(kFewLeast, (int)sqrtf(0.5f * KC));
  int nb = (int)fminf(fmaxf((float)total / (least * C::W1), 1.f), (float)gridDim.x);
  const unsigned round = gridDim.x * C::W2;
  const int64_t most = (int64_t)((weight + round - 1) / round) * C::W2 * KC;
  const bool whole = (most - kFewJoin * C::W1) * nb <= total;
  if (whole) nb = gridDim.x;
  if (total == 0 || (int)blockIdx.x >= nb) return;
  auto first_of = [&](int b) {
    const int64_t at = total * b / nb;
    Place v{p.G, 0, 0, 0};
    if (at >= total) return v;
    v.g = gg::find_group(prefix, p.G, (int)(at / KC));
    const int c = s_cnt[v.g];
    int64_t rest = at - (int64_t)prefix[v.g] * KC;
    const int64_t slab = (int64_t)slab_weight(c) * KC;
    v.slab = (int)(rest / slab);
    rest -= v.slab * slab;
    v.tile = min((int)(rest / (C::W2 * KC)), (c - 1) / kTok);
    rest -= (int64_t)v.tile * C::W2 * KC;
    const int w = c - v.tile * kTok <= 8 ? C::W1 : C::W2;
    v.step = (int)((rest + w - 1) / w);
    return v;
  };
  // the CTA of a step: the last whose share starts at or before it
  auto cta_of = [&](const Place& v, int step) {
    const int c = s_cnt[v.g], w = c - v.tile * kTok <= 8 ? C::W1 : C::W2;
    const int64_t at =
        ((int64_t)prefix[v.g] + v.slab * slab_weight(c) + v.tile * C::W2) * KC + (int64_t)step * w;
    return (int)(((at + 1) * nb - 1) / total);
  };
  auto next_unit = [&](Place& v) {
    v.step = 0;
    if ((++v.tile) * kTok < s_cnt[v.g]) return;
    v.tile = 0;
    if (++v.slab < slabs_of(v.g)) return;
    v.slab = 0;
    do ++v.g;
    while (v.g < p.G && s_cnt[v.g] == 0);
  };
  if (tid < 64 && lane == 0) {
    Place v = first_of(blockIdx.x + warp);
    if (v.step == KC || (whole && v.step > 0)) next_unit(v);
    s_ends[warp] = v;
  }
  __syncthreads();
  const Place begin = s_ends[0], end = s_ends[1];
  // steps of the unit at v that are this CTA's, 0 at its end; and the way there
  auto at_end = [&](const Place& v) {
    return v.g == end.g && v.slab == end.slab && v.tile == end.tile;
  };
  auto steps_at = [&](const Place& v) { return (at_end(v) ? end.step : KC) - v.step; };
  auto advance = [&](Place& v) {
    if (at_end(v)) v.step = end.step;
    else next_unit(v);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (Place v = begin; ok; advance(v)) {
        const int n = steps_at(v), k0 = v.step;
        if (n <= 0) break;
        const int ntl = min(2, (s_cnt[v.g] - v.tile * kTok + 7) >> 3);
        const int row = (ROLES != kWeightsStream ? v.g * p.N : s_off[v.g]) + v.tile * kTok;
        const int n0 = v.slab * (SWIGLU ? 128 : 256) + (ROLES != kWeightsStream ? s_off[v.g] : 0);
        const CUtensorMap* x = &maps.x[ntl - 1];
        const uint32_t bytes = kSlab * 128 + ntl * C::XBOXES * 1024 +
                               (W4 ? p.groups_per_step * (p.has_zeros ? 768 : 512) : 0);
        for (int k = k0; k < k0 + n; ++k) {
          if (!ptx::mbar_wait(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * stage, st = base + stage * C::STAGE;
          ptx::mbar_arrive_expect_tx(fb, bytes);
          const int kw = k * (W4 ? 128 : 64);            // in elements of the weights' map
          if (SWIGLU) ptx::tma_load_4d(st, &maps.w, fb, kw, n0, 0, v.g);
          else if (ROLES != kWeightsStream) ptx::tma_load_2d(st, &maps.w, fb, kw, n0);
          else ptx::tma_load_3d(st, &maps.w, fb, kw, n0, v.g);
          if (ROLES == kRowsStreamT) {
            ptx::tma_load_3d(st + C::X_OFF, x, fb, v.tile * kTok, k * C::STEP, v.g);
          } else if (W4 && p.x_whole) {
            ptx::tma_load_3d(st + C::X_OFF, x, fb, 0, row, k * C::XBOXES);
          } else {
            for (int b = 0; b < C::XBOXES; ++b)
              ptx::tma_load_2d(st + C::X_OFF + b * ntl * 1024, x, fb, k * C::STEP + b * 64, row);
          }
          if (W4) {
            const int k1 = k * p.groups_per_step;
            if (SWIGLU) ptx::tma_load_4d(st + C::S_OFF, &maps.s, fb, n0, k1, 0, v.g);
            else ptx::tma_load_3d(st + C::S_OFF, &maps.s, fb, n0, k1, v.g);
            if (p.has_zeros) {
              if (SWIGLU) ptx::tma_load_4d(st + C::Z_OFF, &maps.z, fb, n0, k1, 0, v.g);
              else ptx::tma_load_3d(st + C::Z_OFF, &maps.z, fb, n0, k1, v.g);
            }
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == C::STAGES) {
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
      for (int s = 0; s < C::STAGES; ++s)
        if (issued & (1u << s))
          ptx::mbar_wait(bar_full + 8 * s, (issued_phase >> s) & 1u, kWaitBudget, nullptr);
    }
    return;
  }
  if (W4 && warp <= C::HELPERS) {
    // the tokens' elements in pairs (i, i + 4) of each eight, as the codes unpack, the 16-byte
    // pieces of odd tokens four places on (so that two tokens' pieces are in all banks)
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (Place v = begin; ok; advance(v)) {
      const int n = steps_at(v);
      if (n <= 0) break;
      const int ntok = (min(kTok, s_cnt[v.g] - v.tile * kTok) + 7) & ~7;
      for (int k = 0; k < n && ok; ++k) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * stage, phase, kWaitBudget,
                                                    abort_flag));
        if (!ok) break;
        uint8_t* st = stages + stage * C::STAGE;
        // three tokens at a time: what bounds these warps is the loads' latency
        for (int tok0 = warp - 1; tok0 < ntok; tok0 += 3 * C::HELPERS) {
          uint4 q[3];
          uint8_t* r[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int tok = min(tok0 + i * C::HELPERS, ntok - 1);
            r[i] = st + C::X_OFF + (lane >> 3) * (ntok * 128) + tok * 128;
            q[i] = *reinterpret_cast<const uint4*>(r[i] + (((lane & 7) ^ (tok & 7)) << 4));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int tok = tok0 + i * C::HELPERS;
            if (tok >= ntok) break;
            *reinterpret_cast<uint4*>(r[i] + (token_place<GC>(tok, lane >> 3, lane & 7) << 4)) =
                make_uint4(__byte_perm(q[i].x, q[i].z, 0x5410), __byte_perm(q[i].x, q[i].z, 0x7632),
                           __byte_perm(q[i].y, q[i].w, 0x5410), __byte_perm(q[i].y, q[i].w, 0x7632));
          }
        }
        ptx::fence_proxy_async_smem();           // TMA writes here next
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_ready + 8 * stage);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  uint32_t buf = 0, buf_phase = 0;
  if (warp <= C::HELPERS + kConsumers) {
    const int rg = warp - 1 - C::HELPERS;
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    const Places here = places<W4, SWIGLU, GC>(p, rg, g, t);
    for (Place v = begin; ok; advance(v)) {
      const int n = steps_at(v);
      if (n <= 0) break;
      const bool two = s_cnt[v.g] - v.tile * kTok > 8;
      float tot[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[m][j][i] = 0.f;
      for (int k = 0; k < n; ++k) {
        // (the helpers arrive after they have seen the stage's loads land)
        ok = __all_sync(0xffffffffu, ptx::mbar_wait((W4 ? bar_ready : bar_full) + 8 * stage, phase,
                                                    kWaitBudget, abort_flag));
        if (!ok) break;
        const uint8_t* st = stages + stage * C::STAGE;
        if constexpr (W4) {
          if (two) step_int4<2, SWIGLU, GC>(tot, st, here, p.has_zeros);
          else step_int4<1, SWIGLU, GC>(tot, st, here, p.has_zeros);
        } else {
          if (two) step_bf16<2, ROLES == kRowsStreamT>(tot, st, here);
          else step_bf16<1, ROLES == kRowsStreamT>(tot, st, here);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_empty + 8 * stage);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(bar_free + 8 * buf, buf_phase ^ 1u,
                                                        kWaitBudget, abort_flag));
      if (!ok) break;
      float* tile = tiles + buf * (kTileBytes / 4);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tile[(rg * 32 + 16 * m + 8 * (i >> 1) + weight_row<W4, GC>(g)) * kTileLd + 8 * j +
                 2 * t + (i & 1)] =
                tot[m][j][i];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_tile + 8 * buf);
      buf ^= 1u;
      buf_phase ^= buf ^ 1u;
    }
    if (!ok && lane == 0) {
      record_status(p.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    return;
  }

  // the results' warps, beside the consumers' next unit
  constexpr int CT = 32 * kJoiners;
  const int ctid = tid - (C::THREADS - CT);
  auto sync = [] { asm volatile("bar.sync 1, %0;" :: "n"(CT) : "memory"); };
  bool ok = true;
  for (Place v = begin;; advance(v)) {
    const int n = steps_at(v);
    if (n <= 0) break;
    const int ntok = min(kTok, s_cnt[v.g] - v.tile * kTok);
    float* tile = tiles + buf * (kTileBytes / 4);
    // (after a wait that ran out the pieces go on without their sums, so that the parts' counters
    // come out as in any other launch)
    if (ok && !ptx::mbar_wait(bar_tile + 8 * buf, buf_phase, kWaitBudget, abort_flag)) {
      ok = false;
      record_status(p.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    bool mine = true;                              // whether the results are this CTA's to write
    if (n < KC) {
      // CTAs lo .. hi share the unit, each with one part: the first the one that it leaves
      // unfinished, the others the one that they begin with
      const int lo = cta_of(v, 0), hi = cta_of(v, KC - 1);
      auto part = [&](int b) { return p.parts + ((int64_t)2 * b + (b == lo)) * (kSlab * kTok); };
      float* to = part(blockIdx.x);
      // four rows of a token a thread and turn, in the parts' order [token][row]
      auto tile4 = [&](int e) { return tile + (e & (kSlab - 1)) * kTileLd + e / kSlab; };
      const int all = kSlab * ntok;
#pragma unroll 2
      for (int e = 4 * ctid; e < all; e += 4 * CT) {
        const float* f = tile4(e);
        __stcg(reinterpret_cast<float4*>(to + e),
               make_float4(f[0], f[kTileLd], f[2 * kTileLd], f[3 * kTileLd]));
      }
      __threadfence();
      sync();
      if (ctid == 0) *s_last = ptx::atom_add_acq_rel(p.arrived + lo, 1u) == (uint32_t)(hi - lo);
      sync();
      mine = *s_last;
      if (mine) {
        // (two parts' loads in flight at once: they cost one way to L2; code for four costs small calls more)
        for (int e = 4 * ctid; e < all; e += 16 * CT) {
          float4 sum[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int b = lo; b <= hi; b += 2) {
            float4 d[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (b + j <= hi && e + 4 * i * CT < all)
                  d[j][i] = __ldcg(reinterpret_cast<const float4*>(part(b + j) + e + 4 * i * CT));
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (b + j > hi || e + 4 * i * CT >= all) continue;
                sum[i].x += d[j][i].x;
                sum[i].y += d[j][i].y;
                sum[i].z += d[j][i].z;
                sum[i].w += d[j][i].w;
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (e + 4 * i * CT >= all) continue;
            float* f = tile4(e + 4 * i * CT);
            f[0] = sum[i].x;
            f[kTileLd] = sum[i].y;
            f[2 * kTileLd] = sum[i].z;
            f[3 * kTileLd] = sum[i].w;
          }
        }
        if (ctid == 0) p.arrived[lo] = 0u;         // as the next launch expects it
      }
      sync();
    }
    if (mine && ROLES != kWeightsStream) {
      // two neighbouring outputs of a row a thread
      const int pairs = ntok >> 1, rows = min(kSlab, s_rows[v.g] - v.slab * kSlab);
      const int64_t row0 = (int64_t)s_off[v.g] + v.slab * kSlab;
      for (int e = ctid; e < rows * pairs; e += CT) {
        const int r = e / pairs, tok = (e - r * pairs) * 2, col = v.tile * kTok + tok;
        float a = tile[r * kTileLd + tok], b = tile[r * kTileLd + tok + 1];
        if (p.add) {
          const uint32_t d = *reinterpret_cast<const uint32_t*>(p.add + (row0 + r) * p.ldadd + col);
          a += bf16_lo(d);
          b += bf16_hi(d);
        }
        *reinterpret_cast<uint32_t*>(p.out + (row0 + r) * p.ldo + col) = pack_bf16x2(a, b);
      }
    } else if (mine) {
      // two neighbouring columns a thread
      constexpr int COLS = SWIGLU ? kSlab / 2 : kSlab;
      const int n0 = v.slab * COLS, N = SWIGLU ? p.F : p.N;
      for (int e = ctid; e < COLS / 2 * ntok; e += CT) {
        const int c = e % (COLS / 2) * 2, tok = e / (COLS / 2);
        if (n0 + c >= N) continue;
        const int64_t row = s_off[v.g] + v.tile * kTok + tok;
        float a = tile[c * kTileLd + tok], b = tile[(c + 1) * kTileLd + tok];
        if (SWIGLU) {
          a = gg::silu_f(a) * tile[(c + 128) * kTileLd + tok];
          b = gg::silu_f(b) * tile[(c + 129) * kTileLd + tok];
        }
        if (p.add) {
          const uint32_t d = *reinterpret_cast<const uint32_t*>(p.add + row * p.ldadd + n0 + c);
          a += bf16_lo(d);
          b += bf16_hi(d);
        }
        *reinterpret_cast<uint32_t*>(p.out + row * p.ldo + n0 + c) = pack_bf16x2(a, b);
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar_free + 8 * buf);
    buf ^= 1u;
    buf_phase ^= buf ^ 1u;
  }
}

// The bf16 weights that codes stand for: a warp takes a row, a lane eight consecutive codes at a
// time; the rows of a CTA follow each other, so a line of scales serves all of them. HBM bounds it: 8 x
// 28672 x 4096, groups of 128, zero points: 390 us, 6.1 TB/s; 64 x 4096 x 2048, groups of 32, 238 us, 5.9.
__global__ void __launch_bounds__(256)
int4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                       const uint8_t* __restrict__ zeros, int64_t rows, int N, int K, int group,
                       uint4* __restrict__ out) {
  const int lane = threadIdx.x & 31, words = K >> 3, kg = K / group;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows;
       row += (int64_t)gridDim.x * 8) {
    const int64_t e = row / N;
    const int64_t sbase = e * kg * N + (row - e * N);
    for (int w = lane; w < words; w += 32) {
      const uint32_t q = __ldg(codes + row * words + w);
      const int64_t at = sbase + (int64_t)(8 * w / group) * N;
      const float s = __uint_as_float((uint32_t)__ldg(scales + at) << 16);
      const int z = zeros ? (__ldg(zeros + at) & 127) : 8;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = (float)((int)((q >> (4 * i)) & 15u) - z) * s;
      out[row * words + w] = pack8(f);
    }
  }
}

// A tensor map of 2 to 4 dimensions: dims and box from the innermost on, strides in bytes.
bool make_tensor_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, int rank,
                     const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                     bool swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, type, rank, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix of d1 x d0 elements for every group; halves: its columns (scales) or rows (weights) cut
// into the gate's and the up half, so that a box has both.
bool make_group_map(CUtensorMap* m, CUtensorMapDataType type, uint64_t bytes, const void* ptr,
                    uint64_t d0, uint64_t d1, uint64_t groups, uint32_t b0, uint32_t b1,
                    int halved, bool swizzle) {
  const cuuint64_t row = d0 * bytes, group = d0 * d1 * bytes;
  if (halved < 0) {
    const cuuint64_t dims[3] = {d0, d1, groups}, strides[2] = {row, group};
    const cuuint32_t box[3] = {b0, b1, 1};
    return make_tensor_map(m, type, ptr, 3, dims, strides, box, swizzle);
  }
  const cuuint64_t dims[4] = {halved == 0 ? d0 / 2 : d0, halved == 1 ? d1 / 2 : d1, 2, groups};
  const cuuint64_t strides[3] = {row, halved == 0 ? row / 2 : group / 2, group};
  const cuuint32_t box[4] = {b0, b1, 2, 1};
  return make_tensor_map(m, type, ptr, 4, dims, strides, box, swizzle);
}

template <bool W4, bool SWIGLU, int GC, int ROLES = kWeightsStream>
cudaError_t run_few(const Maps& m, const FewProduct& p, cudaStream_t stream) {
  auto kern = product_few_kernel<W4, SWIGLU, GC, ROLES>;
  static PerDevice set;
  const cudaError_t e = set_smem_once(set, kern, Cfg<W4>::SMEM);
  if (e != cudaSuccess) return e;
  const int n = num_sms();
  return launch_early(kern, n < kFewCtas ? n : kFewCtas, dim3(Cfg<W4>::THREADS, 1, 1), Cfg<W4>::SMEM,
                      stream, m, p);
}

template <bool SWIGLU>
cudaError_t run_int4(const Maps& m, const FewProduct& p, cudaStream_t stream) {
  return p.group == 128  ? run_few<true, SWIGLU, 4>(m, p, stream)
         : p.group == 64 ? run_few<true, SWIGLU, 2>(m, p, stream)
                         : run_few<true, SWIGLU, 1>(m, p, stream);
}

}  // namespace

cudaError_t launch_int4_dequantize(const void* codes, const void* scales, const void* zeros, int G,
                                   int N, int K, int group, void* out, cudaStream_t s) {
  const int64_t rows = (int64_t)G * N, blocks = (rows + 7) / 8;
  const int64_t most = (int64_t)num_sms() * 8;
  int4_dequantize_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(
      static_cast<const uint32_t*>(codes), static_cast<const uint16_t*>(scales),
      static_cast<const uint8_t*>(zeros), rows, N, K, group, static_cast<uint4*>(out));
  return cudaGetLastError();
}

static_assert(kFewPart == kSlab * kTok, "parts as the kernel writes them");

// Units of 16 tokens and 256 weight rows, weighed, that the kernel's 32-bit numbers hold.
bool few_fits(int64_t rows, int G, int64_t N, int64_t K) {
  return (rows / kTok + G + 1) * ((N + 127) / 128) * Cfg<true>::W2 < (1LL << 31) && K < (1LL << 24);
}

// A pass of the stream has 16 tokens, a tile of the tensor cores' kernel up to 256. With more than
// 16 the stream reads the weights again. (us, stream and tiles: 4 rows for each of 64 experts,
// 512 x 512: 10.4 and 14.4; 24 for each of 8, 1024 x 1024: 16.6 and 14.4; 48 for each of 4,
// 1128 x 7776: 32.9 and 25.0; 60 for each of two, 4096 x 4096: 35.0 and 22.6.)
bool few_rows(int64_t most) { return most <= kTok; }

// Whether a product's rows stream: few outputs, six steps a CTA at least (fewer make many parts of
// 256 rows to join), and units in 32 bits. (us, this way and by tensor tiles, 16 outputs: 8192 rows
// of 4096 21.9 and 28.8, 4096 of them 20.6 and 22.7, 2048 25 and 20.6, 512 20.5 and 16.6.)
bool narrow_fits(int64_t rows, int G, int64_t outputs, int64_t reduction) {
  return outputs <= kTok && rows / kSlab + G < (1LL << 28) &&
         rows / kSlab * ((reduction + 63) / 64) >= 6 * num_sms();
}

cudaError_t launch_product_narrow(FewProduct p, int dgrad, const void* x, int64_t ldx, const void* w,
                                  int N, int K, cudaStream_t s) {
  // p.N: outputs, p.K: the reduction
  p.N = dgrad ? K : N;
  p.K = dgrad ? N : K;
  p.steps = (p.K + 63) / 64;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t row[1] = {(cuuint64_t)ldx * 2}, wide[2] = {(cuuint64_t)p.K, (cuuint64_t)p.rows};
  const cuuint32_t slab[2] = {64, kSlab};
  Maps m;
  if (!make_tensor_map(&m.w, bf16, x, 2, wide, row, slab, true)) return cudaErrorInvalidValue;
  m.s = m.z = m.w;
  for (int i = 0; i < 2; ++i) {
    const cuuint32_t n = 8 * (i + 1), box[2] = {64, n}, turned[3] = {n, 64, 1};
    const cuuint64_t flat[2] = {(cuuint64_t)K, (cuuint64_t)p.G * N}, ld[1] = {(cuuint64_t)K * 2};
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)p.G};
    const cuuint64_t strides[2] = {(cuuint64_t)K * 2, (cuuint64_t)K * N * 2};
    if (!(dgrad ? make_tensor_map(&m.x[i], bf16, w, 3, dims, strides, turned, false)
                : make_tensor_map(&m.x[i], bf16, w, 2, flat, ld, box, true)))
      return cudaErrorInvalidValue;
  }
  return dgrad ? run_few<false, false, 1, kRowsStreamT>(m, p, s) : run_few<false, false, 1, kRowsStream>(m, p, s);
}

cudaError_t launch_product_few(FewProduct p, const void* x, int64_t ldx, const void* w,
                               const void* scales, const void* zeros, bool swiglu,
                               cudaStream_t s) {
  const bool w4 = scales != nullptr;
  const int64_t cols = swiglu ? p.N / 2 : p.N;
  p.F = (int)(p.N / 2);
  p.slabs = (int)((cols + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256));
  p.steps = (p.K + (w4 ? 255 : 63)) / (w4 ? 256 : 64);
  p.has_zeros = zeros != nullptr;
  p.groups_per_step = w4 ? 256 / p.group : 0;
  p.x_whole = w4 && p.K % 64 == 0;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t N = p.N, K = p.K, ld = ldx;
  Maps m;
  for (int i = 0; i < 2; ++i) {
    const cuuint32_t rows = 8 * (i + 1);
    const cuuint64_t dims[3] = {64, (cuuint64_t)p.rows, K / 64}, strides[2] = {ld * 2, 128};
    const cuuint64_t flat[2] = {K, (cuuint64_t)p.rows};
    const cuuint32_t box[3] = {64, rows, 4};
    if (!make_tensor_map(&m.x[i], bf16, x, p.x_whole ? 3 : 2, p.x_whole ? dims : flat, strides, box,
                         true))
      return cudaErrorInvalidValue;
  }
  if (!w4) {
    if (!make_group_map(&m.w, bf16, 2, w, K, N, p.G, 64, 256, -1, true)) return cudaErrorInvalidValue;
    m.s = m.z = m.w;
    return run_few<false, false, 1>(m, p, s);
  }
  const uint64_t kg = K / p.group;
  const uint32_t rows = swiglu ? 128 : 256, gps = p.groups_per_step;
  if (!make_group_map(&m.w, u8, 1, w, K / 2, N, p.G, 128, rows, swiglu ? 1 : -1, true) ||
      !make_group_map(&m.s, bf16, 2, scales, N, kg, p.G, rows, gps, swiglu ? 0 : -1, false))
    return cudaErrorInvalidValue;
  m.z = m.s;
  if (zeros && !make_group_map(&m.z, u8, 1, zeros, N, kg, p.G, rows, gps, swiglu ? 0 : -1, false))
    return cudaErrorInvalidValue;
  return swiglu ? run_int4<true>(m, p, s) : run_int4<false>(m, p, s);
}

}  // namespace moe
