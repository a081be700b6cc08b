// The expert products of 4-bit operands on the block-scaled FP4 tensor cores:
// tcgen05.mma.kind::mxf4nvf4 (E2M1 with an E4M3 scale per 16 elements) and
// kind::mxf4 (a UE8M0 scale per 32), fp32 accumulation in tensor memory.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (es
// summary, Resumen técnico §2.4) names NVFP4 and MXFP8 as Blackwell's recipes
// for the expert GEMMs and §2.3.C the grouped GEMM that reads token counts on
// the device. y[r] = alpha[g] * sum_k x4[r, k] W4[g, n, k] for the rows r of
// group g: the scales travel with the operands (fp4_layout.cuh) and the tensor
// core applies them, so the kernel only moves bytes, 0.5625 (NV) or 0.53 (MX)
// of them per element.
//
// One persistent kernel, one CTA per SM, 480 threads:
//   warp 0       TMA producer of the weights (one lane): per 256-deep k-block (128
//                bytes of codes a row) 256 rows of B and their scale atoms;
//   warp 14      TMA producer of the rows (one lane): A's rows and atoms;
//   warp 1       MMA issuer (one lane) and tensor-memory owner: four M=128 N=256
//                K=64 MMAs a k-block;
//   warps 2-9    epilogue, two warps per tensor-memory lane quarter, 128 of the
//                256 accumulator columns each, held in registers while the next
//                tile's MMAs run;
//   warps 10-13  scales: each writes a k-block's atoms into its lane quarter of
//                tensor memory (tcgen05.st). tcgen05.cp would do it in one thread,
//                but runs in the tensor core's own queue: the 12 copies of an NV
//                k-block take as long as its MMAs (8192 x 8192 x 8192: 340 us with
//                the copies, 254 us so).
//
// A decode step has a few rows per expert: then the weights' bytes are all the
// work, and what counts is that every SM streams its share of them. Only the
// rows a tile has are fetched (boxes of 32), and where whole tiles would leave
// SMs idle (few tiles, or a last wave of few) the k-blocks of all tiles are laid
// end to end and every CTA takes the same length of them. A tile cut that way
// leaves its parts' fp32 sums in scratch, and the warp that arrives last at a
// slice of the tile adds them in order, so the result does not depend on the
// order of arrival. No part waits for another.
#include "fp4_layout.cuh"
#include "fp8_layout.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace gg {

constexpr int kF4Threads = 480;
constexpr int kF4ScaleWarp = 10;                       // the first of the four
constexpr int kF4RowWarp = 14;
constexpr int kF4BN = 256;
constexpr int kF4RowBytes = f4::kStep / 2;             // codes of a k-block's row: 128 bytes
constexpr int kF4BBytes = kF4BN * kF4RowBytes;         // 32 KB
constexpr int kF4EpiWarps = 8;
constexpr uint32_t kF4TmemCols = 512;
constexpr uint32_t kF4SfCol = kF4BN;                   // first scale-factor column

enum F4Epi : int { kF4Store = 0, kF4Swiglu = 1 };

struct Fp4Params {
  int G, N, K;                 // groups, output columns (swiglu: 2F), reduction length
  int64_t rows;                // rows of A and of the outputs
  const int32_t* counts;       // null: one group of `rows` rows
  const int32_t* offsets;
  const float* alpha;          // [G], or null: 1
  float unit;                  // times alpha: the operands' tensor scales, 2^unit_log2
  int unit_log2;
  const uint8_t* sfa;          // A's atoms, [slabs][ka][512]
  int ka;                      // atoms of a slab
  __nv_bfloat16* out;          // store: [rows, N]
  // swiglu: h in 4 bits for the next product (codes [rows, F / 2], atoms), and
  // the checkpoint of gate and up ([rows, 2F] E4M3, [rows, 2F / 32] UE8M0) or null
  uint8_t* hq;
  uint8_t* hsf;
  int hka;
  float hdown;                 // 2^-(h's scale_log2)
  uint8_t* ckpt;
  uint8_t* ckpt_sf;
  // split K: fp32 parts, their arrival counters, the CTAs' counts of launches
  float* part;
  int64_t part_floats;
  uint32_t* arrived;
  int arrived_n;
  uint32_t* launches;
  int32_t* status;
};

// AROWS: rows of A that a stage has room for. Where the caller knows that no group
// has more than 32 (64) rows, the room of the others holds more stages. The MMA
// still reads 128 rows; the ones past the room are the stage's own B bytes, finite
// codes whose results no one reads.
template <int FMT, int AROWS>
struct F4Cfg {
  static constexpr int ATOMS = f4::step_atoms(FMT);              // per slab and k-block
  static constexpr int SF_A = ATOMS * f4::kAtomBytes;
  static constexpr int SF_STAGE = 3 * SF_A;                      // A's, then B's two slabs
  static constexpr int A_BYTES = AROWS * kF4RowBytes;
  static constexpr int STAGE = A_BYTES + kF4BBytes;
  static constexpr int STAGES = AROWS == 32 ? 5 : AROWS == 64 ? 4 : 3;
  static constexpr bool BOXES = AROWS > 32;                      // whole 32-row boxes by TMA
  static constexpr int SF_OFF = STAGES * STAGE;
  static constexpr int CTRL_OFF = SF_OFF + STAGES * SF_STAGE;
  static constexpr int EPI_OFF = (CTRL_OFF + kCtrlBytes + 1023) / 1024 * 1024;
  static constexpr int SMEM = EPI_OFF + (BOXES ? kF4EpiWarps * kBoxBytes : 0) + 1024;
  // scale columns of a k-block: A's 4 per atom, then B's 8 per atom
  static constexpr int SLOT_COLS = 12 * ATOMS;
  static_assert(STAGES <= 8, "barrier arrays");
  static_assert(SMEM <= 232448, "FP4 grouped GEMM shared memory");
  static_assert(kF4SfCol + STAGES * SLOT_COLS <= kF4TmemCols, "FP4 tensor-memory columns");
};

// The work of one CTA: whole tiles blockIdx.x, + gridDim.x, .. (even = 0), or its
// share of the k-blocks of all tiles laid end to end (even = 1): the positions
// [pos, end), tile p / nk, k-block p % nk.
struct Work {
  int nk, tiles, even, ctas;      // ctas: how many share evenly, two k-blocks each at least
  int64_t pos, end;
  int tile, kb0, kb1;             // the current piece

  __device__ __forceinline__ Work(int tiles_, int nk_, int even_)
      : nk(nk_), tiles(tiles_), even(even_) {
    const int64_t all = (int64_t)tiles * nk;
    ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, all / 2));
    const int64_t b = blockIdx.x;
    pos = !even ? b * nk : b < ctas ? b * all / ctas : all;
    end = even && b < ctas ? (b + 1) * all / ctas : all;
  }
  __device__ __forceinline__ bool next() {
    if (pos >= end) return false;
    tile = (int)(pos / nk);
    kb0 = (int)(pos - (int64_t)tile * nk);
    kb1 = (int)min((int64_t)nk, end - (int64_t)tile * nk);
    pos += even ? kb1 - kb0 : (int64_t)gridDim.x * nk;
    return true;
  }
  // The CTAs that hold parts of the current tile: the one that has position p is
  // the largest b with floor(b all / ctas) <= p.
  __device__ __forceinline__ int owner(int64_t p) const {
    return (int)(((p + 1) * ctas - 1) / ((int64_t)tiles * nk));
  }
  __device__ __forceinline__ int first() const { return owner((int64_t)tile * nk); }
  __device__ __forceinline__ int last() const { return owner((int64_t)tile * nk + nk - 1); }
  __device__ __forceinline__ bool whole() const { return kb1 - kb0 == nk; }
};

// Whether to share the k-blocks evenly. Unit: a hundredth of a k-block's time while all
// SMs stream weights (0.98 us). Whole tiles cost their full waves, and a last wave of m
// tiles as much as the m SMs take on their own, at best kAlone of that time. Even shares
// cost the share and the joining of the last tile's parts, kJoin and kJoinRow a row.
// They need scratch for two parts per CTA. Measured whole / even, us, for two experts:
// K = 14336, N = 4096: 35.8 / 18.5 with 1 row, 36.3 / 22.9 with 8, 36.1 / 31.6 with 16,
// 36.5 / 41 with 32; K = 4096, N = 28672: 30.3 / 28.6 with 1 row, 31.7 / 40 with 32.
constexpr int kAlone = 65, kJoin = 200, kJoinRow = 80;
__device__ __forceinline__ int share_evenly(int tiles, int nk, int grid, int most_rows,
                                            int64_t part_floats, int counters) {
  const int slot_rows = min(BM, (most_rows + 31) / 32 * 32);
  if ((int64_t)2 * grid * slot_rows * kF4BN > part_floats || tiles * kF4EpiWarps > counters ||
      grid > kFp4SplitCtas)
    return 0;
  const int m = tiles % grid;
  const int64_t whole = (int64_t)nk * (tiles / grid * 100 + (m ? max(kAlone, 100 * m / grid) : 0));
  const int64_t share = (int64_t)tiles * nk * 100 / grid;
  return whole > share + kJoin + most_rows * kJoinRow;
}

// The launch's number on this scratch, from 1: every CTA of every launch counts itself once,
// behind the kernel before this one, whatever becomes of its waits.
__device__ __forceinline__ uint32_t count_launch(const Fp4Params& p) {
  return gridDim.x <= kFp4SplitCtas ? atomicAdd(p.launches + blockIdx.x, 1u) + 1u : 0u;
}

// An arrival counter holds the parts that have arrived in its low eight bits and above them
// the launch they arrived in (`tag`). Each part's warp opens the counter before it waits for
// its first MMAs: what an earlier launch has left there (one that gave up leaves some
// arrivals counted and others not) gives way to this launch's zero.
__device__ __forceinline__ void open_counter(uint32_t* a, uint32_t tag) {
  uint32_t v = 0;
  while (true) {
    const uint32_t old = atomicCAS(a, v, tag);
    if (old == v || (old ^ tag) <= 255u) return;
    v = old;
  }
}

// h of 32 columns (bf16 pairs) in 4 bits: codes to `dst` (16 bytes); returns the
// blocks' scale bytes.
template <int FMT>
__device__ __forceinline__ uint32_t quantize_h32(const uint4 (&h)[4], float down, uint8_t* dst) {
  constexpr int BLK = f4::block_of(FMT), V = BLK / 8;
  uint32_t c[4];
  uint32_t bytes = 0;
#pragma unroll
  for (int b = 0; b < 32 / BLK; ++b) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, amax_bits8(h[b * V + i]));
    const Fp4Scale s = fp4_scale<FMT>(__uint_as_float(m << 16), m < 0x7F80u, down);
    bytes |= s.byte << (8 * b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8(h[b * V + i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fp4_quotient<FMT>(f[j], s.inv);
      c[b * V + i] = s.inv > 0.f ? e2m1x8(f) : 0u;
    }
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
  return bytes;
}

// 32 bf16 values as the checkpoint keeps them: E4M3 codes of the values over
// 2^ceil(log2(amax / 448)), the scale's byte returned. Half the bytes of bf16;
// the backward's SwiGLU derivative is the only reader.
__device__ __forceinline__ uint32_t checkpoint32(const uint4 (&v)[4], uint8_t* dst) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, amax_bits8(v[i]));
  // an infinity or a NaN: the scale NaN marks the whole block
  const bool finite = m < 0x7F80u;
  const uint32_t code = finite ? ue8m0_code(__uint_as_float(m << 16)) : 255u;
  const float inv = finite ? ue8m0_inv(code) : 0.f;
  uint2 b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    unpack8(v[i], f);
    b[i] = e4m3x8(f, inv);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(b[0].x, b[0].y, b[1].x, b[1].y);
  *reinterpret_cast<uint4*>(dst + 16) = make_uint4(b[2].x, b[2].y, b[3].x, b[3].y);
  return code;
}

// 32 accumulator columns times alpha, as bf16.
__device__ __forceinline__ void scale_pack(const uint32_t (&r)[32], float alpha, uint4 (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[8 * v + i]) * alpha;
    o[v] = pack8(f);
  }
}

// First accumulator column of this warp's c-th 32-column slice: its 128 columns,
// or (swiglu) gate columns 64 half .. +63, then the matching up columns.
template <int EPI>
__device__ __forceinline__ int slice_col(int half, int c) {
  return EPI == kF4Swiglu ? (c >> 1) * 128 + 64 * half + 32 * (c & 1) : 128 * half + 32 * c;
}

// Stores one 32-column piece of a warp's 32 rows, of which rv hold data (the others are
// not written): c is the piece's number, 0-3 (store: o its bf16 values) or 0-1 (swiglu:
// o its gate and u its up values).
template <int FMT, int EPI, bool BOXES>
__device__ __forceinline__ void f4_epilogue(const Fp4Params& p, const CUtensorMap* tmC,
                                            uint8_t* stage, uint32_t stage_u32, int nt, int row0,
                                            int rv, int half, int lane, int c, const uint4 (&o)[4],
                                            const uint4 (&u)[4]) {
  if (EPI == kF4Swiglu) {
    if (lane >= rv) return;
    const int F = p.N / 2;
    const int f = nt * (kF4BN / 2) + 64 * half + 32 * c;
    const int64_t row = row0 + lane;
    if (p.ckpt) {
      uint8_t* ck = p.ckpt + row * 2 * F + f;
      uint8_t* cs = p.ckpt_sf + row * (2 * F / 32) + f / 32;
      cs[0] = (uint8_t)checkpoint32(o, ck);
      cs[F / 32] = (uint8_t)checkpoint32(u, ck + F);
    }
    uint4 h[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) h[v] = swiglu_h8<false>(o[v], u[v], 1.f);
    const uint32_t s = quantize_h32<FMT>(h, p.hdown, p.hq + row * (F / 2) + f / 2);
    uint8_t* sf = p.hsf + (row >> 7) * p.hka * (int64_t)f4::kAtomBytes +
                  f4::sf_byte((int)(row & 127), f / f4::block_of(FMT));
    if (FMT == MOE_FP4_NV) *reinterpret_cast<uint16_t*>(sf) = (uint16_t)s;
    else *sf = (uint8_t)s;
    return;
  }
  const int col = nt * kF4BN + 128 * half + 32 * c;
  if (col >= p.N) return;
  if (BOXES && rv >= 32) {
    // a full 32 x 32 box by TMA, which also clips the columns past N
    if (lane == 0) ptx::tma_store_wait_read();         // the slot's previous box has been read
    __syncwarp();
    stage_row(stage, 0, lane, o);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      ptx::tma_store_2d(tmC, stage_u32, col, row0);
      ptx::tma_store_commit();
    }
  } else if (lane < rv) {
    __nv_bfloat16* dst = p.out + (int64_t)(row0 + lane) * p.N + col;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (col + 8 * v < p.N) stg_v4(dst + 8 * v, o[v]);
  }
}

// (Not inlined: a decode step runs every instruction here once, from HBM -- the weights
// have swept L2 -- so that code costs by its length.)
// Four columns of one row of a joined tile per lane (v, times alpha already):
// columns 4 lane .. of the warp's 128 (the slices of slice_col end to end, so in
// the swiglu form lanes 0-15 hold gate and lanes 16-31 the matching up columns).
template <int FMT, int EPI>
__device__ __noinline__ void f4_epilogue_row(const Fp4Params& p, int nt, int64_t row, int half,
                                                int lane, const float4& v, uint32_t rest) {
  uint2 b = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b.x) : "r"(rest));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b.y) : "r"(rest));
  if (EPI == kF4Store) {
    const int col = nt * kF4BN + 128 * half + 4 * lane;
    if (col < p.N) *reinterpret_cast<uint2*>(p.out + row * p.N + col) = b;
    return;
  }
  const int F = p.N / 2;
  const int f = nt * (kF4BN / 2) + 64 * half + 4 * (lane & 15);
  if (p.ckpt) {
    // 32 values: the 8 lanes 8i .. 8i + 7
    uint32_t m = max(max(b.x & 0x7FFFu, b.x >> 16 & 0x7FFFu), max(b.y & 0x7FFFu, b.y >> 16 & 0x7FFFu));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < 0x7F80u;
    const uint32_t code = finite ? ue8m0_code(__uint_as_float(m << 16)) : 255u;
    const float inv = finite ? ue8m0_inv(code) : 0.f;
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo) : "f"(bf16_hi(b.x) * inv), "f"(bf16_lo(b.x) * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi) : "f"(bf16_hi(b.y) * inv), "f"(bf16_lo(b.y) * inv));
    const int c = (lane >> 4) * F + f;
    *reinterpret_cast<uint32_t*>(p.ckpt + row * 2 * F + c) = lo | (uint32_t)hi << 16;
    if ((lane & 7) == 0) p.ckpt_sf[row * (2 * F / 32) + c / 32] = (uint8_t)code;
  }
  const uint32_t ux = __shfl_down_sync(0xffffffffu, b.x, 16);
  const uint32_t uy = __shfl_down_sync(0xffffffffu, b.y, 16);
  const uint32_t hx = pack_bf16x2(silu_f(bf16_lo(b.x)) * bf16_lo(ux), silu_f(bf16_hi(b.x)) * bf16_hi(ux));
  const uint32_t hy = pack_bf16x2(silu_f(bf16_lo(b.y)) * bf16_lo(uy), silu_f(bf16_hi(b.y)) * bf16_hi(uy));
  constexpr int BLK = f4::block_of(FMT);
  uint32_t m = max(max(hx & 0x7FFFu, hx >> 16 & 0x7FFFu), max(hy & 0x7FFFu, hy >> 16 & 0x7FFFu));
#pragma unroll
  for (int o = 1; o < BLK / 4; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const Fp4Scale s = fp4_scale<FMT>(__uint_as_float(m << 16), m < 0x7F80u, p.hdown);
  const float q[8] = {fp4_quotient<FMT>(bf16_lo(hx), s.inv), fp4_quotient<FMT>(bf16_hi(hx), s.inv),
                      fp4_quotient<FMT>(bf16_lo(hy), s.inv), fp4_quotient<FMT>(bf16_hi(hy), s.inv),
                      0.f, 0.f, 0.f, 0.f};
  if (lane < 16) {
    *reinterpret_cast<uint16_t*>(p.hq + row * (F / 2) + f / 2) =
        s.inv > 0.f ? (uint16_t)e2m1x8(q) : (uint16_t)0;
    if (lane % (BLK / 4) == 0)
      p.hsf[(row >> 7) * p.hka * (int64_t)f4::kAtomBytes +
            f4::sf_byte((int)(row & 127), f / BLK)] = (uint8_t)s.byte;
  }
}

// A scale warp's part of a k-block: its lane's line of every atom into its lane quarter
// of tensor memory (A's atoms, then B's two slabs' by turns), complete on return.
template <int FMT>
__device__ __forceinline__ void write_scales(const uint8_t* src, uint32_t col) {
  constexpr int ATOMS = f4::step_atoms(FMT), SF_A = ATOMS * f4::kAtomBytes;
  uint32_t a[4 * ATOMS], b[8 * ATOMS];
#pragma unroll
  for (int i = 0; i < ATOMS; ++i) {
    *reinterpret_cast<uint4*>(a + 4 * i) = *reinterpret_cast<const uint4*>(src + 512 * i);
    *reinterpret_cast<uint4*>(b + 8 * i) = *reinterpret_cast<const uint4*>(src + SF_A + 512 * i);
    *reinterpret_cast<uint4*>(b + 8 * i + 4) =
        *reinterpret_cast<const uint4*>(src + 2 * SF_A + 512 * i);
  }
  ptx::tc_fence_after();                 // after the MMAs that read these columns before
  if (FMT == MOE_FP4_NV) {
    ptx::tmem_st16(col, a);
    ptx::tmem_st32(col + 16, b);
  } else {
    ptx::tmem_st8(col, a);
    ptx::tmem_st16(col + 8, b);
  }
  ptx::tmem_st_wait();
  ptx::tc_fence_before();
}

template <int FMT, int EPI, int AROWS>
__global__ void __launch_bounds__(kF4Threads, 1)
grouped_gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmA32,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSB,
                        const __grid_constant__ CUtensorMap tmC, const Fp4Params p) {
  using C = F4Cfg<FMT, AROWS>;
  constexpr bool NV = FMT == MOE_FP4_NV;
  constexpr int kStages = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t sf_u = base + C::SF_OFF;
  const uint32_t ctrl_u = base + C::CTRL_OFF;
  uint8_t* ctrl = sbase + C::CTRL_OFF;
  uint8_t* epi = sbase + C::EPI_OFF;
  const uint32_t epi_u = base + C::EPI_OFF;
  const uint32_t bar_full = ctrl_u;                       // [kStages]
  const uint32_t bar_empty = ctrl_u + 64;                 // [kStages]
  const uint32_t bar_scales = ctrl_u + 208;               // [kStages]
  const uint32_t bar_tfull = ctrl_u + 128;
  const uint32_t bar_tempty = bar_tfull + 8;
  const uint32_t bar_drain = bar_tfull + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 196);
  int* s_most = reinterpret_cast<int*>(ctrl + 200);
  uint32_t* s_launch = reinterpret_cast<uint32_t*>(ctrl + 204);
  int* prefix = reinterpret_cast<int*>(ctrl + 256);
  int* mtiles = reinterpret_cast<int*>(ctrl + 1344);
  int* s_off = reinterpret_cast<int*>(ctrl + 2432);
  int* s_cnt = reinterpret_cast<int*>(ctrl + 3520);
  int* tmp = reinterpret_cast<int*>(ctrl + 4608);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G;
  const int F = p.N / 2;
  const int NT = EPI == kF4Swiglu ? F / (kF4BN / 2) : (p.N + kF4BN - 1) / kF4BN;
  const int nk_all = (p.K + f4::kStep - 1) / f4::kStep;
  if (tid == 0) {
    *abort_flag = 0;
    *s_most = 0;
  }
  __syncthreads();
  for (int g = tid; g < G; g += kF4Threads) {
    int64_t c = p.counts ? p.counts[g] : p.rows, o = p.counts ? p.offsets[g] : 0;
    // rows outside the tensor, off the 128-row grid of the scale atoms, or more
    // than the caller said: the group is left out and reported
    if (c < 0 || o < 0 || o % 128 || o + c > p.rows || (AROWS < BM && c > AROWS)) {
      record_status(p.status, MOE_ERR_DEVICE_CHECK);
      c = o = 0;
    }
    s_cnt[g] = (int)c;
    s_off[g] = (int)o;
    mtiles[g] = (int)((c + BM - 1) / BM);
    prefix[g] = mtiles[g] * NT;
    atomicMax(s_most, (int)c);
  }
  __syncthreads();
  const int tiles = block_exclusive_scan(prefix, G, tmp);
  if (tid == 0) prefix[G] = tiles;
  const int slot_rows = min(BM, (*s_most + 31) / 32 * 32);
  const int even = share_evenly(tiles, nk_all, gridDim.x, *s_most, p.part_floats, p.arrived_n);
  __syncthreads();
  Work w(tiles, nk_all, even);
  if (w.pos >= w.end) {
    ptx::grid_dependency_wait();                 // this kernel ends after the one before it
    if (tid == 0) count_launch(p);
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 2);             // the two producers
      ptx::mbar_init(bar_empty + 8 * s, 1);
      ptx::mbar_init(bar_scales + 8 * s, 4);
    }
    ptx::mbar_init(bar_tfull, 1);
    ptx::mbar_init(bar_tempty, kF4EpiWarps);
    ptx::mbar_init(bar_drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kF4TmemCols);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmA32);
    ptx::tma_prefetch_desc(&tmB);
    ptx::tma_prefetch_desc(&tmSB);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  ptx::grid_launch_dependents();     // the next kernel's CTAs may start as these leave

  if (warp == 0) {
    // ------------------------------------- producer of the weights' stages
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      uint32_t issued_mask = 0, issued_phase = 0;
      bool ok = true;
      while (ok && w.next()) {
        const Tile t = decode(w.tile, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
        // rows of B and their slab: of group g, or (swiglu) of the gate and up parts
        // 2g, 2g + 1, both brought by one box
        const int b0 = t.nt * (EPI == kF4Swiglu ? kF4BN / 2 : kF4BN);
        const int part = EPI == kF4Swiglu ? 2 * t.g : t.g;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!ptx::mbar_wait(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * stage;
          ptx::mbar_arrive_expect_tx(fb, kF4BBytes + 2 * C::SF_A);
          ptx::tma_load_3d(base + stage * C::STAGE + C::A_BYTES, &tmB, fb, kb * kF4RowBytes, b0,
                           part);
          ptx::tma_load_3d(sf_u + stage * C::SF_STAGE + C::SF_A, &tmSB, fb, kb * (C::SF_A / 8),
                           b0 / 128, part);
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
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
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s))
          ptx::mbar_wait(bar_full + 8 * s, (issued_phase >> s) & 1u, kWaitBudget, nullptr);
    }
  } else if (warp == kF4RowWarp) {
    // ----------------------------------------- producer of the rows' stages
    // A thread of its own: one thread issues a load in about 0.15 us, four a k-block;
    // and an early start holds the rows (which the kernel before this one writes) back
    // while the weights are already on their way.
    if (lane == 0) {
      ptx::grid_dependency_wait();
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      const int64_t slab_bytes = (int64_t)p.ka * f4::kAtomBytes;
      while (ok && w.next()) {
        const Tile t = decode(w.tile, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
        const int row0 = s_off[t.g] + t.mt * BM;
        const int valid = min(BM, s_cnt[t.g] - t.mt * BM);
        const int boxes = (valid + 31) / 32;             // 4: one 128-row box
        const uint8_t* sfa = p.sfa + row0 / 128 * slab_bytes;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!ptx::mbar_wait(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * stage, sA = base + stage * C::STAGE;
          ptx::mbar_arrive_expect_tx(fb, boxes * 4096 + C::SF_A);
          if (AROWS == BM && boxes == 4) {
            ptx::tma_load_2d(sA, &tmA, fb, kb * kF4RowBytes, row0);
          } else {
            for (int i = 0; i < boxes; ++i)
              ptx::tma_load_2d(sA + 4096 * i, &tmA32, fb, kb * kF4RowBytes, row0 + 32 * i);
          }
          ptx::bulk_load(sf_u + stage * C::SF_STAGE, sfa + (int64_t)kb * C::SF_A, C::SF_A, fb);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_fp4(BM, kF4BN, NV ? 0 : 1);
      uint32_t stage = 0, phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      while (ok && w.next()) {
        if (!ptx::mbar_wait(bar_tempty, acc_phase ^ 1u, kWaitBudget, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!ptx::mbar_wait(bar_full + 8 * stage, phase, kWaitBudget, abort_flag) ||
              !ptx::mbar_wait(bar_scales + 8 * stage, phase, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sfa_t = tmem_base + kF4SfCol + C::SLOT_COLS * stage;
          const uint32_t sfb_t = sfa_t + 4 * C::ATOMS;
          const uint32_t sA = base + stage * C::STAGE;
          const uint32_t sB = sA + C::A_BYTES;
          // 64-wide slices of the k-block that K reaches into
          const int slices = min(4, (p.K - kb * f4::kStep + 63) / 64);
          for (int kk = 0; kk < slices; ++kk) {
            const uint64_t ad = ptx::smem_desc_sw128(sA + kk * 32, 16, 1024);
            const uint64_t bd = ptx::smem_desc_sw128(sB + kk * 32, 16, 1024);
            const int a = NV ? kk : kk >> 1;
            const uint32_t id = NV ? IDESC : ptx::idesc_with_sf_id(IDESC, (uint32_t)(kk & 1) * 2);
            ptx::mma_fp4<NV>(tmem_base, ad, bd, id, sfa_t + 4 * a, sfb_t + 8 * a,
                             (kb > w.kb0 || kk) ? 1u : 0u);
          }
          issued = true;
          ptx::mma_commit(bar_empty + 8 * stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit(bar_tfull);
        acc_phase ^= 1u;
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // wait for every MMA issued by this thread before tensor memory is freed
      if (issued) {
        ptx::mma_commit(bar_drain);
        ptx::mbar_wait(bar_drain, 0, kWaitBudget, nullptr);
      }
    }
  } else if (warp >= kF4ScaleWarp) {
    // -------------------------------------------------------------- scales
    // The stage's columns are free when its loads have landed again: the
    // producer waited for the MMAs that read them.
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + kF4SfCol;
    const uint8_t* sfl = sbase + C::SF_OFF + lane * 16;
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    while (ok && w.next()) {
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * stage, phase, kWaitBudget,
                                                    abort_flag));
        if (!ok) break;
        write_scales<FMT>(sfl + stage * C::SF_STAGE, tq + C::SLOT_COLS * stage);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_scales + 8 * stage);
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
    const int q = warp & 3;                       // tensor-memory lane quarter
    const int half = (warp - 2) >> 2;             // which 128 accumulator columns
    uint8_t* stage = epi + (warp - 2) * kBoxBytes;
    const uint32_t stage_u32 = epi_u + (warp - 2) * kBoxBytes;
    const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t acc_phase = 0;
    // nothing is written before the kernel before this one is done
    ptx::grid_dependency_wait();
    if (tid == 64) *s_launch = count_launch(p);
    asm volatile("bar.sync 1, %0;" :: "n"(32 * kF4EpiWarps) : "memory");
    if (even && lane < 2) {
      // the counters of the first and the last tile of this CTA's share: no other is cut
      const int tile = (int)(lane ? w.end - 1 : w.pos) / nk_all;
      open_counter(p.arrived + tile * kF4EpiWarps + (warp - 2), *s_launch << 8);
    }
    __syncwarp();
    while (w.next()) {
      const Tile t = decode(w.tile, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
      const int row0 = s_off[t.g] + t.mt * BM + q * 32;
      const int rv = s_cnt[t.g] - t.mt * BM - q * 32;    // rows of this warp that hold data
      const Fp4Factor f = fp4_factor(p.alpha ? p.alpha[t.g] : 1.f, 1.f, p.unit, p.unit_log2);
      const float alpha = f.by;
      const uint32_t rest = f.rest;
      const bool ok = __all_sync(
          0xffffffffu, ptx::mbar_wait(bar_tfull, acc_phase, kWaitBudget, abort_flag));
      if (!ok) {
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      ptx::tc_fence_after();
      // a cut tile: this warp's slice of a part, [slot_rows][128 columns] fp32;
      // CTA b's slots are 2b (a tile that began before its share) and 2b + 1
      const int64_t slice = (int64_t)slot_rows * 128;
      float* parts = p.part + half * slice + (int64_t)q * 32 * 128;
      auto release = [&]() {                      // the accumulator is free for the next piece
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_tempty);
      };
      acc_phase ^= 1u;
      if (rv <= 0) {
        release();
        continue;
      }
      if (w.whole()) {
        if constexpr (AROWS == BM) {
          // the tile's columns into registers first, so that the next one's MMAs start
          uint4 o[4][4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            ptx::tmem_ld32(tq + slice_col<EPI>(half, c), r);
            ptx::tmem_ld_wait();
            scale_pack(r, alpha, o[c]);
          }
          release();
          if (rest != kFp4One) {
#pragma unroll
            for (int i = 0; i < 16; ++i) fp4_times(o[i >> 2][i & 3], rest);
          }
#pragma unroll
          for (int c = 0; c < (EPI == kF4Swiglu ? 2 : 4); ++c)
            f4_epilogue<FMT, EPI, C::BOXES>(p, &tmC, stage, stage_u32, t.nt, row0, rv, half, lane,
                                            c, o[c], o[(c + 2) & 3]);
        } else {
          // few rows: the weights' arrival is what the kernel waits for, and short code
          // what it needs
#pragma unroll 1
          for (int c = 0; c < (EPI == kF4Swiglu ? 2 : 4); ++c) {
            uint32_t r[32];
            uint4 o[4], u[4];
            ptx::tmem_ld32(tq + slice_col<EPI>(half, c), r);
            ptx::tmem_ld_wait();
            scale_pack(r, alpha, o);
            if (EPI == kF4Swiglu) {
              ptx::tmem_ld32(tq + slice_col<EPI>(half, c + 2), r);
              ptx::tmem_ld_wait();
              scale_pack(r, alpha, u);
            }
            if (rest != kFp4One) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                fp4_times(o[i], rest);
                if (EPI == kF4Swiglu) fp4_times(u[i], rest);
              }
            }
            f4_epilogue<FMT, EPI, C::BOXES>(p, &tmC, stage, stage_u32, t.nt, row0, rv, half, lane,
                                            c, o, u);
            __syncwarp();
          }
          release();
        }
      } else {
        float* mine = parts + (2 * (int64_t)blockIdx.x + (w.kb0 == 0)) * 2 * slice + lane * 128;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          ptx::tmem_ld32(tq + slice_col<EPI>(half, c), r);
          ptx::tmem_ld_wait();
          if (lane < rv) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<uint4*>(mine + 32 * c + i),
                     make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]));
          }
          __syncwarp();
        }
        release();
        __syncwarp();
        const int b0 = w.first(), b1 = w.last();
        int last = 0;
        if (lane == 0) {
          uint32_t* counter = p.arrived + w.tile * kF4EpiWarps + (warp - 2);
          last = (int)(ptx::atom_add_acq_rel(counter, 1u) & 255u) == b1 - b0;
          if (last) *counter = 0;                 // so that a tag that comes round again meets none
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        if (!last) continue;
        // a shuffle orders no memory: what lane 0's atomic acquired (the other parts) the
        // other lanes may read only past this
        __syncwarp();
        const int rows = min(rv, 32);
        // the first part ends at its CTA's share (slot 2 b0 + 1), the others begin theirs
        const float* first = parts + (4 * (int64_t)b0 + 2) * slice + 4 * lane;
        const float* others = parts + 4 * (int64_t)(b0 + 1) * slice + 4 * lane;
#pragma unroll 1
        for (int r = 0; r < rows; ++r, first += 128, others += 128) {
          float4 v = __ldcg(reinterpret_cast<const float4*>(first));
          const float* at = others;
#pragma unroll 4
          for (int b = b0; b < b1; ++b, at += 4 * slice) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(at));
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          f4_epilogue_row<FMT, EPI>(
              p, t.nt, row0 + r, half, lane,
              make_float4(v.x * alpha, v.y * alpha, v.z * alpha, v.w * alpha), rest);
        }
      }
    }
    if (lane == 0) ptx::tma_store_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kF4TmemCols);
  }
}

// ------------------------------------------------------------ CTA pairs
// The same product for experts with many rows: tiles of 256 x 256, each CTA of a pair
// holding 128 rows of A and 128 of B (swiglu: the gate rows in the even CTA, the matching
// up rows in the odd one), its rows' scales and those of all 256 columns. A k-block is 38 KB
// a CTA instead of 54, so that five stages fit where three did (512 rows each, 64 experts,
// 4096 x 4096: 265 us with single CTAs, 233 so). What bounds either is not settled: tensor
// pipe 53 % active (single CTAs 40), L2 to the SMs 31 % (32) of its peak. Whole tiles only.
template <int FMT>
struct F4PairCfg {
  static constexpr int ATOMS = f4::step_atoms(FMT);
  static constexpr int SF_A = ATOMS * f4::kAtomBytes;
  static constexpr int SF_STAGE = 3 * SF_A;
  static constexpr int A_BYTES = BM * kF4RowBytes;               // 16 KB
  static constexpr int STAGE = 2 * A_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int SF_OFF = STAGES * STAGE;
  static constexpr int CTRL_OFF = SF_OFF + STAGES * SF_STAGE;
  static constexpr int EPI_OFF = (CTRL_OFF + kCtrlBytes + 1023) / 1024 * 1024;
  static constexpr int SMEM = EPI_OFF + kF4EpiWarps * kBoxBytes + 1024;
  static constexpr int SLOT_COLS = 12 * ATOMS;
  static_assert(SMEM <= 232448, "FP4 pair shared memory");
  static_assert(kF4SfCol + STAGES * SLOT_COLS <= kF4TmemCols, "FP4 pair tensor-memory columns");
};

template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF4Threads, 1)
grouped_gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                             const __grid_constant__ CUtensorMap tmB,
                             const __grid_constant__ CUtensorMap tmSB,
                             const __grid_constant__ CUtensorMap tmC, const Fp4Params p) {
  using C = F4PairCfg<FMT>;
  constexpr bool NV = FMT == MOE_FP4_NV;
  constexpr int kStages = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t sf_u = base + C::SF_OFF;
  const uint32_t ctrl_u = base + C::CTRL_OFF;
  uint8_t* ctrl = sbase + C::CTRL_OFF;
  const uint32_t bar_full = ctrl_u;                       // [kStages], the even CTA's
  const uint32_t bar_empty = ctrl_u + 40;                 // [kStages]
  const uint32_t bar_sf = ctrl_u + 80;                    // [kStages] this CTA's scale atoms
  const uint32_t bar_scales = ctrl_u + 120;               // [kStages], the even CTA's
  const uint32_t bar_tfull = ctrl_u + 160;
  const uint32_t bar_tempty = ctrl_u + 168;
  const uint32_t bar_drain = ctrl_u + 176;
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
  const int F = p.N / 2;
  const int NT = EPI == kF4Swiglu ? F / (kF4BN / 2) : (p.N + kF4BN - 1) / kF4BN;
  const int nk = (p.K + f4::kStep - 1) / f4::kStep;
  for (int g = tid; g < G; g += kF4Threads) {
    int64_t c = p.counts ? p.counts[g] : p.rows, o = p.counts ? p.offsets[g] : 0;
    if (c < 0 || o < 0 || o % 128 || o + c > p.rows) {    // as in the single-CTA kernel
      record_status(p.status, MOE_ERR_DEVICE_CHECK);
      c = o = 0;
    }
    s_cnt[g] = (int)c;
    s_off[g] = (int)o;
    mtiles[g] = (int)((c + 2 * BM - 1) / (2 * BM));       // 256-row tiles
    prefix[g] = mtiles[g] * NT;
  }
  if (tid == 0) *abort_flag = 0;
  __syncthreads();
  const int total = block_exclusive_scan(prefix, G, tmp);
  if (tid == 0) prefix[G] = total;
  __syncthreads();
  if (cluster >= total) {                                 // both CTAs of the pair leave together
    ptx::grid_dependency_wait();
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 2);                // the even CTA's two producers
      ptx::mbar_init(bar_empty + 8 * s, 1 + 4);           // the MMAs, and this CTA's scale warps
      ptx::mbar_init(bar_sf + 8 * s, 2);
      ptx::mbar_init(bar_scales + 8 * s, 8);              // four warps of both CTAs
    }
    ptx::mbar_init(bar_tfull, 1);
    ptx::mbar_init(bar_tempty, 2 * kF4EpiWarps);
    ptx::mbar_init(bar_drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), kF4TmemCols);
    ptx::tmem_relinquish_pair();
  }
  if (tid == 0) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
    ptx::tma_prefetch_desc(&tmSB);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  ptx::grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------- producer of the weights' stages
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        const Tile t = decode(pt, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
        const int b0 = t.nt * (EPI == kF4Swiglu ? kF4BN / 2 : kF4BN);
        const int part = EPI == kF4Swiglu ? 2 * t.g : t.g;
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget,
                                      abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t lf = ptx::mapa_shared(bar_full + 8 * stage, 0);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * C::A_BYTES);
          ptx::tma_load_3d_pair(base + stage * C::STAGE + C::A_BYTES, &tmB, lf, kb * kF4RowBytes,
                                EPI == kF4Swiglu ? b0 : b0 + 128 * (int)rank,
                                EPI == kF4Swiglu ? part + (int)rank : part);
          const uint32_t sb = bar_sf + 8 * stage;
          ptx::mbar_arrive_expect_tx(sb, 2 * C::SF_A);
          ptx::tma_load_3d(sf_u + stage * C::SF_STAGE + C::SF_A, &tmSB, sb, kb * (C::SF_A / 8),
                           b0 / 128, part);
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        // loads already issued land within microseconds; give them time
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {
        }
      }
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s))
          ptx::mbar_wait(bar_sf + 8 * s, (issued_phase >> s) & 1u, kWaitBudget, nullptr);
    }
  } else if (warp == kF4RowWarp) {
    // ----------------------------------------- producer of the rows' stages
    if (lane == 0) {
      ptx::grid_dependency_wait();
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      const int64_t slab_bytes = (int64_t)p.ka * f4::kAtomBytes;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        const Tile t = decode(pt, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
        const int row0 = s_off[t.g] + (2 * t.mt + (int)rank) * BM;
        // a tile's second half may hold no rows, and then may lie past the last slab
        const int64_t slab = min((int64_t)(row0 / 128), f4::slabs(p.rows) - 1);
        const uint8_t* sfa = p.sfa + slab * slab_bytes;
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster(bar_empty + 8 * stage, phase ^ 1u, kWaitBudget,
                                      abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t lf = ptx::mapa_shared(bar_full + 8 * stage, 0);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * C::A_BYTES);
          ptx::tma_load_2d_pair(base + stage * C::STAGE, &tmA, lf, kb * kF4RowBytes, row0);
          const uint32_t sb = bar_sf + 8 * stage;
          ptx::mbar_arrive_expect_tx(sb, C::SF_A);
          ptx::bulk_load(sf_u + stage * C::SF_STAGE, sfa + (int64_t)kb * C::SF_A, C::SF_A, sb);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t IDESC = ptx::idesc_fp4(2 * BM, kF4BN, NV ? 0 : 1);
      uint32_t stage = 0, phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int pt = cluster; pt < total && ok; pt += nclusters) {
        if (!ptx::mbar_wait_cluster(bar_tempty, acc_phase ^ 1u, kWaitBudget, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster(bar_full + 8 * stage, phase, kWaitBudget, abort_flag) ||
              !ptx::mbar_wait_cluster(bar_scales + 8 * stage, phase, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sfa_t = tmem_base + kF4SfCol + C::SLOT_COLS * stage;
          const uint32_t sfb_t = sfa_t + 4 * C::ATOMS;
          const uint32_t sA = base + stage * C::STAGE;
          const uint32_t sB = sA + C::A_BYTES;
          const int slices = min(4, (p.K - kb * f4::kStep + 63) / 64);
          for (int kk = 0; kk < slices; ++kk) {
            const int a = NV ? kk : kk >> 1;
            const uint32_t id = NV ? IDESC : ptx::idesc_with_sf_id(IDESC, (uint32_t)(kk & 1) * 2);
            ptx::mma_fp4_pair<NV>(tmem_base, ptx::smem_desc_sw128(sA + kk * 32, 16, 1024),
                                  ptx::smem_desc_sw128(sB + kk * 32, 16, 1024), id, sfa_t + 4 * a,
                                  sfb_t + 8 * a, (kb | kk) ? 1u : 0u);
          }
          issued = true;
          ptx::mma_commit_pair(bar_empty + 8 * stage, 3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair(bar_tfull, 3);
        acc_phase ^= 1u;
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
  } else if (warp >= kF4ScaleWarp) {
    // -------------------------------------------------------------- scales
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + kF4SfCol;
    const uint8_t* sfl = sbase + C::SF_OFF + lane * 16;
    const uint32_t leader_scales = ptx::mapa_shared(bar_scales, 0);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int pt = cluster; pt < total && ok; pt += nclusters) {
      for (int kb = 0; kb < nk; ++kb) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_sf + 8 * stage, phase, kWaitBudget,
                                                    abort_flag));
        if (!ok) break;
        write_scales<FMT>(sfl + stage * C::SF_STAGE, tq + C::SLOT_COLS * stage);
        __syncwarp();
        if (lane == 0) {
          // the even CTA's MMAs may read the columns, and the slot's bytes, read here, may
          // be overwritten once those MMAs are done (an order within this CTA)
          ptx::mbar_arrive_cluster_tmem(leader_scales + 8 * stage);
          ptx::mbar_arrive(bar_empty + 8 * stage);
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
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    uint8_t* stage = sbase + C::EPI_OFF + (warp - 2) * kBoxBytes;
    const uint32_t stage_u32 = base + C::EPI_OFF + (warp - 2) * kBoxBytes;
    const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
    const uint32_t leader_tempty = ptx::mapa_shared(bar_tempty, 0);
    uint32_t acc_phase = 0;
    ptx::grid_dependency_wait();
    for (int pt = cluster; pt < total; pt += nclusters) {
      const Tile t = decode(pt, prefix, mtiles, s_cnt, G, 0, p.K, NT, 0);
      const int m0 = (2 * t.mt + (int)rank) * BM + q * 32;
      const int row0 = s_off[t.g] + m0;
      const int rv = s_cnt[t.g] - m0;
      const Fp4Factor f = fp4_factor(p.alpha ? p.alpha[t.g] : 1.f, 1.f, p.unit, p.unit_log2);
      const float alpha = f.by;
      const uint32_t rest = f.rest;
      const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar_tfull, acc_phase,
                                                                     kWaitBudget, abort_flag));
      if (!ok) {
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      ptx::tc_fence_after();
      uint4 o[4][4];
      if (rv > 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          ptx::tmem_ld32(tq + slice_col<EPI>(half, c), r);
          ptx::tmem_ld_wait();
          scale_pack(r, alpha, o[c]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(leader_tempty);
      acc_phase ^= 1u;
      if (rv <= 0) continue;
      if (rest != kFp4One) {
#pragma unroll
        for (int i = 0; i < 16; ++i) fp4_times(o[i >> 2][i & 3], rest);
      }
#pragma unroll
      for (int c = 0; c < (EPI == kF4Swiglu ? 2 : 4); ++c)
        f4_epilogue<FMT, EPI, true>(p, &tmC, stage, stage_u32, t.nt, row0, rv, half, lane, c, o[c],
                                    o[(c + 2) & 3]);
    }
    if (lane == 0) ptx::tma_store_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, kF4TmemCols);
  }
}

template <int FMT, int EPI, int AROWS>
static cudaError_t run_fp4_rows(const CUtensorMap& a, const CUtensorMap& a32, const CUtensorMap& b,
                                const CUtensorMap& sb, const CUtensorMap& c, const Fp4Params& p,
                                bool early, cudaStream_t s) {
  auto kern = grouped_gemm_fp4_kernel<FMT, EPI, AROWS>;
  constexpr int smem = F4Cfg<FMT, AROWS>::SMEM;
  static PerDevice set;
  const cudaError_t e = set_smem_once(set, kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(num_sms(), 1, 1);
  lc.blockDim = dim3(kF4Threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, a, a32, b, sb, c, p);
}

template <int FMT, int EPI>
static cudaError_t run_fp4_pair(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sb,
                                const CUtensorMap& c, const Fp4Params& p, bool early,
                                cudaStream_t s) {
  auto kern = grouped_gemm_fp4_pair_kernel<FMT, EPI>;
  constexpr int smem = F4PairCfg<FMT>::SMEM;
  static PerDevice set;
  int grid = 0;
  const cudaError_t e = pair_grid_once(set, kern, kF4Threads, smem, &grid);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(kF4Threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, a, b, sb, c, p);
}

// Pairs where the experts expect at least kPairRows rows each: a 256-row tile whose second
// half is empty still takes its time. 512 rows each exactly (64 experts, 4096 x 4096): 265 us
// with single CTAs, 233 with pairs; 512 on average, 200 to 1200 (a whole FFN): 573 and 579;
// 1024 on average (eight experts, 4096 x 14336, with the quantiser): 299 and 287.
constexpr int64_t kPairRows = 768;
static bool fp4_pairs(const Fp4Problem& q) { return q.mean_rows >= kPairRows; }

template <int EPI>
static cudaError_t run_fp4(const Fp4Problem& q, const CUtensorMap& a, const CUtensorMap& a32,
                           const CUtensorMap& b, const CUtensorMap& sb, const CUtensorMap& c,
                           const Fp4Params& p, cudaStream_t s) {
  const bool nv = q.fmt == MOE_FP4_NV;
  if (fp4_pairs(q))
    return nv ? run_fp4_pair<MOE_FP4_NV, EPI>(a, b, sb, c, p, q.early, s)
              : run_fp4_pair<MOE_FP4_MX, EPI>(a, b, sb, c, p, q.early, s);
  if (q.most_rows <= 32)
    return nv ? run_fp4_rows<MOE_FP4_NV, EPI, 32>(a, a32, b, sb, c, p, q.early, s)
              : run_fp4_rows<MOE_FP4_MX, EPI, 32>(a, a32, b, sb, c, p, q.early, s);
  if (q.most_rows <= 64)
    return nv ? run_fp4_rows<MOE_FP4_NV, EPI, 64>(a, a32, b, sb, c, p, q.early, s)
              : run_fp4_rows<MOE_FP4_MX, EPI, 64>(a, a32, b, sb, c, p, q.early, s);
  return nv ? run_fp4_rows<MOE_FP4_NV, EPI, 128>(a, a32, b, sb, c, p, q.early, s)
            : run_fp4_rows<MOE_FP4_MX, EPI, 128>(a, a32, b, sb, c, p, q.early, s);
}

// 4-bit operand: [rows, K / 2] bytes, box of 128 bytes x box_rows.
static bool make_map_fp4(CUtensorMap* m, const void* ptr, int64_t K, int64_t rows,
                         uint32_t box_rows) {
  return make_map_u8(m, ptr, (uint64_t)K / 2, (uint64_t)rows, box_rows);
}

// Weights in 4 bits as `parts` blocks of `rows` rows, a box of 128 bytes x box_rows x
// box_parts (pair: one CTA's half of it), and their scale atoms, 8 bytes an element: one
// k-block's atoms of as many slabs. What lies past a block's rows reads as zero.
static bool make_map_weights(CUtensorMap* codes, CUtensorMap* scales, const Fp4Problem& q,
                             int64_t rows, int64_t parts, uint32_t box_rows, uint32_t box_parts,
                             bool pair) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t kb = (cuuint64_t)q.K / 2, sl = (cuuint64_t)f4::slabs(rows);
  const cuuint64_t sb = (cuuint64_t)f4::atoms_k(q.fmt, q.K) * f4::kAtomBytes;
  const cuuint32_t es[3] = {1, 1, 1};
  const cuuint64_t d[3] = {kb, (cuuint64_t)rows, (cuuint64_t)parts};
  const cuuint64_t st[2] = {kb, kb * (cuuint64_t)rows};
  const cuuint32_t box[3] = {kF4RowBytes, pair ? 128u : box_rows, pair ? 1u : box_parts};
  const cuuint64_t ds[3] = {sb / 8, sl, (cuuint64_t)parts};
  const cuuint64_t sts[2] = {sb, sb * sl};
  const cuuint32_t boxs[3] = {(cuuint32_t)f4::step_atoms(q.fmt) * f4::kAtomBytes / 8,
                              box_rows / 128, box_parts};
  return fn(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(q.b), d, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
             CUDA_SUCCESS &&
         fn(scales, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 3, const_cast<uint8_t*>(q.sfb), ds, sts, boxs,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
             CUDA_SUCCESS;
}

static Fp4Params fp4_params(const Fp4Problem& q, const Fp4Split& sp, int32_t* status) {
  Fp4Params p{};
  p.G = q.G;
  p.N = (int)q.N;
  p.K = (int)q.K;
  p.rows = q.rows;
  p.counts = q.counts;
  p.offsets = q.offsets;
  p.alpha = q.alpha;
  p.unit = ldexpf(1.f, q.unit_log2);
  p.unit_log2 = q.unit_log2;
  p.sfa = q.sfa;
  p.ka = (int)f4::atoms_k(q.fmt, q.K);
  p.part = sp.part;
  p.part_floats = sp.part_floats;
  p.arrived = sp.arrived;
  p.arrived_n = sp.arrived_n;
  p.launches = sp.launches;
  p.status = status;
  return p;
}

}  // namespace gg

using namespace gg;

cudaError_t launch_fp4_gemm(const Fp4Problem& q, void* out, const Fp4Split& sp, int32_t* status,
                            cudaStream_t s) {
  if (q.rows == 0 || q.N == 0) return cudaSuccess;
  CUtensorMap a, a32, b, sb, c;
  if (!make_map_fp4(&a, q.a, q.K, q.rows, 128) || !make_map_fp4(&a32, q.a, q.K, q.rows, 32) ||
      !make_map_weights(&b, &sb, q, q.N, q.G, 256, 1, fp4_pairs(q)) ||
      !make_out_map(&c, out, (uint64_t)q.N, (uint64_t)q.rows))
    return cudaErrorInvalidValue;
  Fp4Params p = fp4_params(q, sp, status);
  p.out = static_cast<__nv_bfloat16*>(out);
  return run_fp4<kF4Store>(q, a, a32, b, sb, c, p, s);
}

cudaError_t launch_fp4_swiglu(const Fp4Problem& q, uint8_t* hq, uint8_t* hsf, int h_scale_log2,
                              uint8_t* ckpt, uint8_t* ckpt_sf, const Fp4Split& sp, int32_t* status,
                              cudaStream_t s) {
  if (q.rows == 0) return cudaSuccess;
  CUtensorMap a, a32, b, sb;
  if (!make_map_fp4(&a, q.a, q.K, q.rows, 128) || !make_map_fp4(&a32, q.a, q.K, q.rows, 32) ||
      !make_map_weights(&b, &sb, q, q.N / 2, 2 * (int64_t)q.G, 128, 2, fp4_pairs(q)))
    return cudaErrorInvalidValue;
  Fp4Params p = fp4_params(q, sp, status);
  p.hq = hq;
  p.hsf = hsf;
  p.hka = (int)f4::atoms_k(q.fmt, q.N / 2);
  p.hdown = ldexpf(1.f, -h_scale_log2);
  p.ckpt = ckpt;
  p.ckpt_sf = ckpt_sf;
  return run_fp4<kF4Swiglu>(q, a, a32, b, sb, b, p, s);
}

}  // namespace moe
