// FP8 GEMM with float scales per 128 elements, on the sm_100 tensor cores:
//
//   D[m, n] = sum over K-blocks kb of  sa[m, kb] sb[n, kb] (A_kb B_kb^T)[m, n]
//
// A [M, K] in 1 x 128 tiles; B [N, K] in 1 x 128 tiles or 128 x 128 blocks;
// E4M3 or E5M2 each. The scales are arbitrary floats, which no MMA applies, so
// every K-block of 128 is accumulated by itself in tensor memory and added,
// scaled, to float sums in registers:
//   warp 0     TMA: one K-block of both operands per stage (128 bytes per row:
//              one 128-byte swizzle atom), S stages
//   warps 1-2  one thread each issues the four tcgen05.mma.kind::f8f6f4 (K = 32)
//              of its half of the columns, or of every other K-block, into the
//              next of NBUF accumulators
//   warp 3     the scales of four K-blocks at a time into shared memory
//   warps 4..  accumulator -> registers (tcgen05.ld, one row per thread),
//              acc += (s_row s_col) t with packed multiply-adds, accumulator
//              released; after the last K-block the tile is stored
// so the vector work of one K-block runs beside the MMAs of the next.
//
// Tiles, rows (MMA A) x columns (MMA B):
//   256 x 256  a pair of CTAs (cta_group::2), each with 128 of the rows and half
//              of the columns in its shared memory: large products
//   128 x 128, 128 x 64   one CTA
//   128 x 64, 32, 16 with the weights on the row side and the tokens on the
//              column side (SWAP): few tokens, no MMA row wasted, the weights
//              read once
// Where tiles are too few to fill the SMs a cluster of 2, 4 or 8 CTAs splits K,
// and each CTA adds up its share of the tile over the cluster's shared memory,
// in rank order (no atomics).
//
// What bounds it. One K-block of a pair's tile is 512 clocks of MMA; with
// nothing but the loads and MMAs it took 344 ns at the clock that the power
// limit left (3.6 PFLOP/s), as a whole 382 ns with block scales and 570 with
// column scales. There no pipe is full (4096 x 4096 x 16384: FMA pipe 52%, tensor
// pipe 49%, issue 53%): an accumulating warp waits, loads, multiplies row by
// column scale, adds and releases, and this chain overlaps only in part with the
// next K-block's MMAs. 8192^3 takes 443 us (2.48 PFLOP/s) in bursts and 501 to
// 529 us, by the card, in a steady loop at the power limit (1.37 GHz at 990 W); a
// library product of the same codes with one scale for the whole tensor, 418 us
// at 1.31 GHz. Few tokens are bound by the weights' bytes and 4 us of start and
// end: 1 x 8192 x 8192 14.1 us (4.8 TB/s), 16 x 1536 x 2048 4.7 us. What each step
// gave (8192^3, us): one CTA per tile 673; issuing and scale-loading warps of
// their own, packed sums 457; pairs in halves 443; a shorter loop 431; NaN for
// sums left unmade 443 (438 without it on the same card).
//
// Every wait is bounded in time (mbar_wait): one that runs out sets the
// caller's status word, and the CTA stores NaN for the sums that it could not
// make, in this tile and its further ones, drains its copies and MMAs, frees its
// TMEM and returns.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "mx_gemm128.h"
#include "mx_launch.h"
#include "mx_pdl.cuh"
#include "mx_tc.cuh"

namespace mxk {

namespace {

constexpr int kRows = 128;              // rows of a tile: the MMA's M
constexpr uint32_t kBlockK = 128;       // elements (bytes) of K per stage
constexpr uint32_t kTileP = kRows * kBlockK;

constexpr int kStatusProducer = 11, kStatusMma = 12, kStatusSums = 13, kStatusDrain = 14,
              kStatusScales = 15;

struct Gemm128Args {
  const float* p_scale;    // row side: tile scales [nk, p_ld] or block scales [., nk]
  const float* q_scale;    // column side, likewise
  int64_t p_ld, q_ld;      // tile scales: floats per K-block
  uint8_t* d;
  int* status;
  int64_t P, Q;            // rows and columns of the tile grid (SWAP: P = N, Q = M)
  int64_t ldd;             // elements per row of D
  int nk;                  // K-blocks
  int split;               // CTAs per tile (cluster size)
  uint32_t idesc;
  int p_block;             // the row side's scales are per 128 x 128 block
  int out_fp32;
  int vec;                 // rows of D start on 16-byte boundaries
};

// BN columns per tile; QCOL: a scale per column; SWAP: the weights on the row
// side; PAIR: two CTAs share a tile of 256 rows; S stages.
template <int BN_, bool QCOL_, bool SWAP_, bool PAIR_, int S_>
struct Cfg {
  static constexpr int BN = BN_, S = S_;
  static constexpr bool QCOL = QCOL_, SWAP = SWAP_, PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1;          // CTAs per tile (without a split)
  static constexpr int kTileRows = kRows * kCtas;
  // A pair's tile is multiplied in two halves of 128 columns, each with its own
  // two accumulators, issuer and warps: an accumulator is used again after two
  // K-blocks, and from its last MMA to its release takes longer than the other
  // accumulator's MMAs cover when each is a whole K-block of 256 columns.
  static constexpr int kHalves = PAIR ? 2 : 1;
  static constexpr int kUnitN = BN / kHalves;         // columns per MMA
  static constexpr int kBoxQ = kUnitN / kCtas;        // columns that a CTA loads at once
  static constexpr int kParts = BN >= 64 ? 2 : 1;     // of the columns
  static constexpr int kWork = 4 * kParts;            // accumulating warps
  // 256 threads with 128 sums each need more than the 168 registers that 384
  // threads can have: the first warpgroup (TMA, MMA, scales) gives of its share.
  // 128 x 56 + 256 x 224 = 384 x 168.
  static constexpr int kWork0 = 4;                    // first accumulating warp
  static constexpr bool kShift = BN / kParts == 128;
  static constexpr int kThreads = (kWork0 + kWork) * 32;
  static constexpr int kCols = BN / kParts;           // columns per thread
  static constexpr int NBUF = PAIR ? 2 : 4;           // accumulators (of each half)
  static constexpr uint32_t kTmemCols = NBUF * BN;
  static constexpr uint32_t kTileQ = kHalves * kBoxQ * kBlockK;
  static constexpr uint32_t kStage = kTileP + kTileQ;
  // Scales: a warp of its own puts four K-blocks at a time into one of two
  // slots: per row (for blocks, times the scale of each 128 columns), and per
  // column. The accumulating warps issue no loads: with the next scales' in
  // flight a K-block took 130 ns longer.
  static constexpr int kBatch = 4;
  static constexpr int kRowSets = QCOL ? 1 : (BN + 127) / 128;
  static constexpr uint32_t kSetBytes = kRows * 4;
  static constexpr uint32_t kRowSlot = kBatch * kRowSets * kSetBytes;
  static constexpr uint32_t kColSlot = QCOL ? kBatch * BN * 4 : 0;
  static constexpr uint32_t kSlot = kRowSlot + kColSlot;
  static constexpr uint32_t kStgRow = 64;             // store staging: 32 such rows per warp
  static constexpr uint32_t kStaging = SWAP ? 0 : kWork * 32 * kStgRow;
  static constexpr int kBars = S + kHalves * (S + NBUF) + 1 + 4;
  static constexpr uint32_t kSmem = S * kStage + kStaging + 2 * kSlot + 8 * kBars + 16 + 1024;
  static_assert((S & (S - 1)) == 0 && (NBUF & (NBUF - 1)) == 0, "counters");
  static_assert(kHalves == 1 || kParts == 2, "a half per part");
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(PAIR || S * kStage >= kRows * BN * 4, "the split's partial tile reuses the ring");
};

template <class C>
struct Smem {
  uint32_t raw, ring, stg, scl, bar;
  uint32_t* tmem_holder;
  volatile int* abort_flag;
  uint8_t* ring_ptr;
  uint8_t* stg_ptr;
  float* scl_ptr;
  __device__ explicit Smem(uint8_t* p) {
    raw = tc::smem_addr(p);
    ring = (raw + 1023u) & ~1023u;   // swizzle atoms need 1024-byte alignment
    stg = ring + C::S * C::kStage;
    scl = stg + C::kStaging;
    bar = scl + 2 * C::kSlot;
    ring_ptr = p + (ring - raw);
    stg_ptr = p + (stg - raw);
    scl_ptr = reinterpret_cast<float*>(p + (scl - raw));
    tmem_holder = reinterpret_cast<uint32_t*>(p + (bar + 8u * C::kBars - raw));
    abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  }
  __device__ uint32_t p_tile(int s) const { return ring + s * C::kStage; }
  __device__ uint32_t q_tile(int s) const { return ring + s * C::kStage + kTileP; }
  __device__ uint32_t full(int s) const { return bar + 8u * s; }
  // a stage's MMAs (of half h) are complete: its operands may go, its sums be read
  __device__ uint32_t done(int h, int s) const { return bar + 8u * (C::S * (1 + h) + s); }
  // accumulator b of half h may be overwritten
  __device__ uint32_t tempty(int h, int b) const {
    return bar + 8u * (C::S * (1 + C::kHalves) + C::NBUF * h + b);
  }
  __device__ uint32_t last() const { return bar + 8u * (C::kBars - 5); }
  __device__ uint32_t sfull(int s) const { return bar + 8u * (C::kBars - 4 + s); }
  __device__ uint32_t sempty(int s) const { return bar + 8u * (C::kBars - 2 + s); }
};

// A position in a ring of N slots: the slot and the parity of its phase.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      par ^= 1;
    }
  }
  __device__ __forceinline__ void prev() {
    if (--slot < 0) {
      slot = N - 1;
      par ^= 1;
    }
  }
};

// Tile t of the grid. Bands of 16 row tiles, within a band down the rows
// first: the tiles that run together then share few rows and columns, which
// stay in L2.
constexpr int64_t kBand = 16;
__device__ __forceinline__ void tile_at(int64_t t, int64_t tiles_p, int64_t tiles_q, int64_t& p,
                                        int64_t& q) {
  const int64_t band = t / (kBand * tiles_q);
  const int64_t left = tiles_p - band * kBand;
  const int64_t width = left < kBand ? left : kBand;
  const int64_t r = t - band * kBand * tiles_q;
  p = band * kBand + r % width;
  q = r / width;
}

// Two sums at once (packed multiply-add): a0 += f0 t0, a1 += f1 t1.
__device__ __forceinline__ void fma2(float& a0, float& a1, float f0, float f1, uint32_t t0,
                                     uint32_t t1) {
  const float2 v = __ffma2_rn(make_float2(f0, f1),
                              make_float2(__uint_as_float(t0), __uint_as_float(t1)),
                              make_float2(a0, a1));
  a0 = v.x;
  a1 = v.y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// Four consecutive values of a row of D (n of the row's N columns are left).
__device__ __forceinline__ void store4(const Gemm128Args& g, int64_t row, int64_t col, int64_t n,
                                       const float4& v) {
  const int64_t at = row * g.ldd + col;
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (g.out_fp32) {
    float* d = reinterpret_cast<float*>(g.d) + at;
    if (g.vec && n >= 4) {
      *reinterpret_cast<float4*>(d) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) d[i] = f[i];
    }
  } else {
    __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(g.d) + at;
    if (g.vec && n >= 4) {
      *reinterpret_cast<uint2*>(d) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) d[i] = __float2bfloat16_rn(f[i]);
    }
  }
}

// The split's partial tile in shared memory, in the order of D: `major` rows
// of L floats, 16-byte units permuted against bank conflicts.
template <int L>
__device__ __forceinline__ uint32_t part_at(int major, int minor) {
  return static_cast<uint32_t>(major * L + ((((minor >> 2) ^ (major & 7)) << 2) | (minor & 3))) * 4u;
}

// This CTA's share of the tile: the sum of the cluster's partial tiles in rank
// order, stored. Units of four floats along D's rows.
template <class C, int SPLIT>
__device__ __forceinline__ void add_split(const Smem<C>& sm, const Gemm128Args& g, int64_t p0,
                                          int64_t q0, uint32_t rank) {
  constexpr int L = C::SWAP ? kRows : C::BN;
  constexpr int kMajor = C::SWAP ? C::BN : kRows;
  constexpr int kUnits = kMajor * L / 4 / SPLIT;
  const int64_t rows = C::SWAP ? g.Q : g.P, cols = C::SWAP ? g.P : g.Q;
  const int64_t r0 = C::SWAP ? q0 : p0, c0 = C::SWAP ? p0 : q0;
  // several units' loads in flight: one after the other they took 3 us of a
  // 128-wide tile split in two
  constexpr int kThreads = C::kWork * 32;
  constexpr int kAtOnce = SPLIT == 8 ? 2 : 4;
  for (int u0 = threadIdx.x - C::kWork0 * 32; u0 < kUnits; u0 += kThreads * kAtOnce) {
    float4 v[kAtOnce][SPLIT];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int u = u0 + i * kThreads < kUnits ? u0 + i * kThreads : 0;
      const int at = static_cast<int>(rank) * kUnits + u;
      const uint32_t a = sm.ring + part_at<L>(at / (L / 4), at % (L / 4) * 4);
#pragma unroll
      for (int r = 0; r < SPLIT; ++r) v[i][r] = ld_cluster4(tc::mapa(a, r));
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int u = u0 + i * kThreads;
      const int at = static_cast<int>(rank) * kUnits + u;
      const int major = at / (L / 4), minor = at % (L / 4) * 4;
      if (u >= kUnits || r0 + major >= rows || c0 + minor >= cols) continue;
      float4 s = v[i][0];
#pragma unroll
      for (int r = 1; r < SPLIT; ++r) {
        s.x += v[i][r].x;
        s.y += v[i][r].y;
        s.z += v[i][r].z;
        s.w += v[i][r].w;
      }
      store4(g, r0 + major, c0 + minor, cols - c0 - minor, s);
    }
  }
}

// One tile of D from the sums in registers (rows on the row side): a warp
// stages 32 rows of kStgRow bytes in its own shared memory, so that a row
// leaves as full 16-byte lanes of one run.
template <class C, int ES, bool VEC>
__device__ __forceinline__ void store_tile(const Smem<C>& sm, const Gemm128Args& g,
                                           const float (&acc)[C::kCols], int64_t p0,
                                           int64_t q0, int warp, int lane) {
  constexpr int kChunk = (C::kStgRow / ES < C::kCols) ? C::kStgRow / ES : C::kCols;
  static_assert(kChunk <= 32, "a lane per column");
  constexpr int NJ = kChunk * ES / 16;          // 16-byte units per row
  constexpr int kPer = 16 / ES;                 // elements per unit
  constexpr int kRowsPer = 32 / NJ;             // rows per store instruction
  uint8_t* stg = sm.stg_ptr + (warp - C::kWork0) * 32 * C::kStgRow;
  const int64_t row0 = p0 + (warp & 3) * 32;
  const int64_t colh = q0 + ((warp - C::kWork0) / 4) * C::kCols;
#pragma unroll
  for (int c0 = 0; c0 < C::kCols; c0 += kChunk) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint4 v;
      uint32_t* w = &v.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = c0 + j * kPer + i * (4 / ES);
        if constexpr (ES == 2) w[i] = bf16x2(acc[at], acc[at + 1]);
        else w[i] = __float_as_uint(acc[at]);
      }
      *reinterpret_cast<uint4*>(stg + lane * (NJ * 16) + ((j ^ (lane & (NJ - 1))) * 16)) = v;
    }
    __syncwarp();
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        const int r = i * kRowsPer + lane / NJ, j = lane % NJ;
        const uint4 v =
            *reinterpret_cast<const uint4*>(stg + r * (NJ * 16) + ((j ^ (r & (NJ - 1))) * 16));
        const int64_t row = row0 + r, col = colh + c0 + j * kPer;
        // (N is then a multiple of kPer)
        if (row < g.P && col < g.Q)
          *reinterpret_cast<uint4*>(g.d + (row * g.ldd + col) * ES) = v;
      }
    } else {
      // rows at any alignment: neighbouring lanes write neighbouring elements
      // (a lane with 16 bytes of its own, element by element, took 30 us for
      // 7135 x 543 x 1557)
      const int c = lane % kChunk;
      const int64_t col = colh + c0 + c;
#pragma unroll 4
      for (int r = lane / kChunk; r < 32; r += 32 / kChunk) {
        const uint8_t* at = stg + r * (NJ * 16) + (((c / kPer) ^ (r & (NJ - 1))) * 16) + c % kPer * ES;
        const int64_t row = row0 + r;
        if (row < g.P && col < g.Q) {
          uint8_t* d = g.d + (row * g.ldd + col) * ES;
          if constexpr (ES == 2) *reinterpret_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(at);
          else *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(at);
        }
      }
    }
    __syncwarp();
  }
}

// The same with D's rows on the column side: lane = consecutive columns of D.
template <class C>
__device__ __forceinline__ void store_tile_swapped(const Gemm128Args& g,
                                                   const float (&acc)[C::kCols], int64_t p0,
                                                   int64_t q0, int warp, int lane) {
  const int64_t n = p0 + (warp & 3) * 32 + lane;
  const int64_t m0 = q0 + ((warp - C::kWork0) / 4) * C::kCols;
  if (n >= g.P) return;
#pragma unroll
  for (int i = 0; i < C::kCols; ++i) {
    const float v = acc[i];
    if (m0 + i < g.Q) {
      const int64_t at = (m0 + i) * g.ldd + n;
      if (g.out_fp32)
        reinterpret_cast<float*>(g.d)[at] = v;
      else
        reinterpret_cast<__nv_bfloat16*>(g.d)[at] = __float2bfloat16_rn(v);
    }
  }
}

// VEC: rows of D start on 16-byte boundaries (an instance of its own, since the
// other stores' code beside these made the K-blocks' loop 10% slower).
template <class C, bool VEC>
__global__ void __launch_bounds__(C::kThreads, 1)
    gemm128_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const Gemm128Args g) {
  extern __shared__ uint8_t smem_raw[];
  const Smem<C> sm(smem_raw);
  // (through a shuffle, so that the compiler keeps what follows from it in
  // uniform registers, where tcgen05 and TMA operands have to be)
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int64_t tiles_p = (g.P + C::kTileRows - 1) / C::kTileRows;
  const int64_t tiles_q = (g.Q + C::BN - 1) / C::BN;
  const int64_t ntiles = tiles_p * tiles_q;
  // a cluster shares a tile: its CTAs take the rows in turn (PAIR) or split K,
  // this one's K-blocks being [kb0, kb1)
  const int shared = C::PAIR ? 2 : g.split;
  const uint32_t rank = blockIdx.x % shared;
  const int64_t t_first = blockIdx.x / shared;
  const int64_t t_step = gridDim.x / shared;
  const int kb0 = C::PAIR ? 0 : static_cast<int>(static_cast<int64_t>(g.nk) * rank / g.split);
  const int kb1 = C::PAIR ? g.nk : static_cast<int>(static_cast<int64_t>(g.nk) * (rank + 1) / g.split);
  const uint32_t row_rank = C::PAIR ? rank : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) tc::mbar_init(sm.full(s), 1);
    for (int h = 0; h < C::kHalves; ++h) {
      for (int s = 0; s < C::S; ++s) tc::mbar_init(sm.done(h, s), 1);
      for (int b = 0; b < C::NBUF; ++b)
        tc::mbar_init(sm.tempty(h, b), C::kWork / C::kHalves * C::kCtas);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(sm.sfull(s), 1);
      tc::mbar_init(sm.sempty(s), C::kWork);
    }
    tc::mbar_init(sm.last(), 2);
    *sm.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (C::PAIR) tc::tmem_alloc_pair(tc::smem_addr(sm.tmem_holder), C::kTmemCols);
    else tc::tmem_alloc(tc::smem_addr(sm.tmem_holder), C::kTmemCols);
  }
  tc::tc_fence_before();
  __syncthreads();
  if constexpr (C::PAIR) tc::cluster_sync();   // the other CTA's barriers exist
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *sm.tmem_holder, 0);
  dependent_launch();
  dependent_wait();   // operands, scales and D from here on

  if (warp < C::kWork0) {
    if constexpr (C::kShift) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (tc::elect_one()) {
        tc::prefetch_tmap(&tmP);
        tc::prefetch_tmap(&tmQ);
        Ring<C::S> st;
        int issued = 0;   // this many of the last copies may be in flight
        bool ok = true;
        for (int64_t t = t_first; ok && t < ntiles; t += t_step) {
          int64_t p, q;
          tile_at(t, tiles_p, tiles_q, p, q);
          const int p0 = static_cast<int>(p * C::kTileRows + row_rank * kRows);
          const int q0 = static_cast<int>(q * C::BN);
          for (int kb = kb0; kb < kb1; ++kb) {
            ok = tc::mbar_pass(sm.done(0, st.slot), st.par ^ 1, sm.abort_flag, g.status,
                               kStatusProducer);
            if constexpr (C::kHalves == 2)
              ok = ok && tc::mbar_pass(sm.done(1, st.slot), st.par ^ 1, sm.abort_flag, g.status,
                                       kStatusProducer);
            if (!ok) break;
            const int k0 = kb * static_cast<int>(kBlockK);
            if constexpr (C::PAIR) {
              // both CTAs' copies count on the first CTA's barrier, where the MMAs are issued
              const uint32_t full = tc::mapa(sm.full(st.slot), 0);
              if (rank == 0) tc::mbar_arrive_expect_tx(sm.full(st.slot), 2 * C::kStage);
              tc::tma_load_2d_pair(sm.p_tile(st.slot), &tmP, k0, p0, full);
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
                tc::tma_load_2d_pair(sm.q_tile(st.slot) + h * C::kBoxQ * kBlockK, &tmQ, k0,
                                     q0 + h * C::kUnitN + static_cast<int>(rank) * C::kBoxQ, full);
            } else {
              tc::mbar_arrive_expect_tx(sm.full(st.slot), C::kStage);
              tc::tma_load_2d(sm.p_tile(st.slot), &tmP, k0, p0, sm.full(st.slot));
              tc::tma_load_2d(sm.q_tile(st.slot), &tmQ, k0, q0, sm.full(st.slot));
            }
            st.next();
            if (issued < C::S) ++issued;
          }
        }
        // every copy issued has landed before the CTA can exit (PAIR: the first
        // CTA sees to both CTAs' copies, and the other waits for it below)
        for (int j = 0; j < (rank == 0 || !C::PAIR ? issued : 0); ++j) {
          st.prev();
          tc::mbar_wait(sm.full(st.slot), st.par, sm.abort_flag, g.status, kStatusDrain, false);
        }
      }
      __syncwarp();
    } else if (warp < 3 && row_rank == 0) {
      // ------------------------------------------------------- MMA issuers
      // Two threads, since one's waits, issue and commit take longer than the
      // MMAs themselves: each has a half of the columns, or (one half) they
      // take turns K-block by K-block.
      if (tc::elect_one()) {
        constexpr bool kTurns = C::kHalves == 1;
        const int h = kTurns ? 0 : warp - 1;
        Ring<C::S> st;
        Ring<C::NBUF> tb;
        int64_t todo = ((ntiles - t_first + t_step - 1) / t_step) * (kb1 - kb0);
        if (kTurns && warp == 2) {
          st.next();
          tb.next();
          --todo;
        }
        const uint64_t pd0 = tc::kmajor_sw128_desc(sm.p_tile(0));
        const uint64_t qd0 = tc::kmajor_sw128_desc(sm.q_tile(0) + h * C::kBoxQ * kBlockK);
        for (; todo > 0; todo -= kTurns ? 2 : 1) {
          if (!tc::mbar_pass(sm.tempty(h, tb.slot), tb.par ^ 1, sm.abort_flag, g.status, kStatusMma) ||
              !tc::mbar_pass(sm.full(st.slot), st.par, sm.abort_flag, g.status, kStatusMma))
            break;
          tc::tc_fence_after();
          const uint64_t pd = pd0 + st.slot * (C::kStage >> 4);
          const uint64_t qd = qd0 + st.slot * (C::kStage >> 4);
          const uint32_t d = tmem + (h * C::NBUF + tb.slot) * C::kUnitN;
#pragma unroll
          for (int k = 0; k < 4; ++k) {   // K = 32: 32 bytes further along the rows
            if constexpr (C::PAIR) tc::mma_f8_pair(d, pd + 2 * k, qd + 2 * k, g.idesc, k != 0);
            else tc::mma_f8(d, pd + 2 * k, qd + 2 * k, g.idesc, k != 0);
          }
          if constexpr (C::PAIR) tc::tc_commit_pair(sm.done(h, st.slot), 3);
          else tc::tc_commit(sm.done(h, st.slot));
          st.next();
          tb.next();
          if constexpr (kTurns) {
            st.next();
            tb.next();
          }
        }
        // every MMA has finished before TMEM is freed, whatever ended the loop
        if constexpr (C::PAIR) tc::tc_commit_pair(sm.last(), 1);
        else tc::tc_commit(sm.last());
        tc::mbar_wait(sm.last(), 0, sm.abort_flag, g.status, kStatusDrain, false);
      }
      __syncwarp();
    }
    if (warp == 3) {
      // ------------------------------------------------------------ scales
      Ring<2> ss;
      int issued = 0;
      bool ok = true;
      for (int64_t t = t_first; ok && t < ntiles; t += t_step) {
        int64_t p, q;
        tile_at(t, tiles_p, tiles_q, p, q);
        const int64_t p0 = p * C::kTileRows + row_rank * kRows, q0 = q * C::BN;
        for (int kb = kb0; kb < kb1; kb += C::kBatch) {
          // four rows' scales per lane and K-block; block scales one per lane
          float a[C::kBatch][4], b = 1.0f;
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i) {
            const int k = kb + i < kb1 ? kb + i : kb1 - 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t row = p0 + j * 32 + lane;
              a[i][j] = g.p_block ? g.p_scale[p * g.nk + k]
                                  : g.p_scale[k * g.p_ld + (row < g.P ? row : g.P - 1)];
            }
          }
          if constexpr (!C::QCOL) {
            const int64_t col = q0 + (lane / C::kBatch) * kRows;
            const int k = kb + lane % C::kBatch < kb1 ? kb + lane % C::kBatch : kb1 - 1;
            if (lane < C::kBatch * C::kRowSets)
              b = g.q_scale[(col < g.Q ? col : g.Q - 1) / kRows * g.nk + k];
          }
          if (!__all_sync(~0u, tc::mbar_pass(sm.sempty(ss.slot), ss.par ^ 1, sm.abort_flag, g.status,
                                             kStatusScales))) {
            ok = false;
            break;
          }
          float* slot = sm.scl_ptr + ss.slot * (C::kSlot / 4);
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i)
#pragma unroll
            for (int n = 0; n < C::kRowSets; ++n) {
              const float f = C::QCOL ? 1.0f : __shfl_sync(~0u, b, n * C::kBatch + i);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                slot[(i * C::kRowSets + n) * kRows + j * 32 + lane] = C::QCOL ? a[i][j] : a[i][j] * f;
            }
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::QCOL) {
              // the columns' present: the rest of a slot belongs to columns past the edge
              const int64_t left = ((g.Q + 3) & ~int64_t(3)) - q0;
              const uint32_t bytes = static_cast<uint32_t>(left < C::BN ? left : C::BN) * 4;
              const int n = kb1 - kb < C::kBatch ? kb1 - kb : C::kBatch;
              tc::mbar_arrive_expect_tx(sm.sfull(ss.slot), n * bytes);
              for (int i = 0; i < n; ++i)
                tc::bulk_load(sm.scl + ss.slot * C::kSlot + C::kRowSlot + i * C::BN * 4,
                              g.q_scale + (kb + i) * g.q_ld + q0, bytes, sm.sfull(ss.slot));
            } else {
              tc::mbar_arrive(sm.sfull(ss.slot));
            }
          }
          ss.next();
          if (issued < 2) ++issued;
        }
      }
      if (C::QCOL && lane == 0)   // copies landed before the CTA can exit
        for (int j = 0; j < issued; ++j) {
          ss.prev();
          tc::mbar_wait(sm.sfull(ss.slot), ss.par, sm.abort_flag, g.status, kStatusDrain, false);
        }
      __syncwarp();
    }
    // (accumulators read, by the other branch's half of this barrier)
    tc::named_sync(1, C::kThreads);
    if constexpr (C::PAIR) tc::cluster_sync();   // and by the other CTA, whose copies have landed
    if (warp == 1) {
      tc::tc_fence_after();
      if constexpr (C::PAIR) tc::tmem_dealloc_pair(tmem, C::kTmemCols);
      else tc::tmem_dealloc(tmem, C::kTmemCols);
    }
    if (!C::PAIR && g.split > 1) {
      tc::cluster_sync();
      tc::cluster_sync();
    }
  } else {
    // ------------------------------------------------------ scaled sums
    if constexpr (C::kShift) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quarter = warp & 3, part = (warp - C::kWork0) / 4;
    const int h = C::kHalves == 2 ? part : 0;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                               (C::kHalves == 2 ? h * C::NBUF * C::kUnitN : part * C::kCols);
    // K-blocks and slots so far: stage, accumulator, slot and their parities are
    // its low bits (all powers of two)
    uint32_t n = 0, nslot = 0;
    // where accumulators are given back: to the CTA that issues the MMAs
    const uint32_t free0 = C::PAIR ? tc::mapa(sm.tempty(h, 0), 0) : sm.tempty(h, 0);
    // this thread's row scale and its part's column scales in a slot
    const int row_scale = (C::QCOL ? 0 : part * C::kCols / kRows) * kRows + quarter * 32 + lane;
    const int col_scale = C::kRowSlot / 4 + part * C::kCols;
    const uint32_t done0 = sm.done(h, 0);
    bool ok = true;
    const float none = __int_as_float(0x7fc00000);   // for sums left unmade
    for (int64_t t = t_first; t < ntiles; t += t_step) {
      int64_t p, q;
      tile_at(t, tiles_p, tiles_q, p, q);
      const int64_t p0 = p * C::kTileRows + row_rank * kRows, q0 = q * C::BN;
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = ok ? 0.0f : none;
      for (int kb = ok ? kb0 : kb1; kb < kb1; kb += C::kBatch, ++nslot) {
        ok &= tc::mbar_wait(sm.sfull(nslot & 1), (nslot >> 1) & 1, sm.abort_flag, g.status, kStatusSums);
        const float* slot = sm.scl_ptr + (nslot & 1) * (C::kSlot / 4);
        // (not unrolled: the loop's length in instructions is what the issuing
        // warps, which share the schedulers, have to be fetched past; unrolled
        // by four, 8192^3 took 595 us, 432 as it is)
#pragma unroll 1
        for (int at = 0; at < C::kBatch; ++at) {
          if (kb + at >= kb1) break;
          float s = slot[row_scale + at * C::kRowSets * kRows];
          // (after a wait that ran out the loop goes on to the tile's end and every
          // later wait returns at once, since tcgen05.ld needs the whole warp)
          ok &= tc::mbar_wait(done0 + 8 * (n & (C::S - 1)), (n / C::S) & 1, sm.abort_flag, g.status,
                              kStatusSums);
          if constexpr (!C::PAIR)   // (pairs: after the loop; here it cost them 2.5%, there others 4%)
            if (!ok) s = none;
          __syncwarp();
          tc::tc_fence_after();
          const uint32_t b = n & (C::NBUF - 1);
          ++n;
          // Columns per load, two loads in flight. Column scales come a load ahead
          // too (read where they are used, their latency took 280 ns per K-block).
          constexpr int kLd = C::QCOL || !C::PAIR ? 16 : 32;
          const uint32_t taddr = lane_base + b * C::kUnitN;
          uint32_t r[2][kLd];
          float4 f[2][C::QCOL ? kLd / 4 : 1];
          const float4* qv = reinterpret_cast<const float4*>(slot + col_scale + at * C::BN);
          tc::tmem_ld_start(taddr, r[0]);
          if constexpr (C::QCOL)
#pragma unroll
            for (int i = 0; i < kLd / 4; ++i) f[0][i] = qv[i];
          tc::tmem_ld_wait(r[0]);
#pragma unroll
          for (int c0 = 0; c0 < C::kCols; c0 += kLd) {
            constexpr int kMask = 1;
            uint32_t(&now)[kLd] = r[(c0 / kLd) & kMask];
            uint32_t(&next)[kLd] = r[(c0 / kLd + 1) & kMask];
            if (c0 + kLd < C::kCols) {
              tc::tmem_ld_start(taddr + c0 + kLd, next);
              if constexpr (C::QCOL)
#pragma unroll
                for (int i = 0; i < kLd / 4; ++i)
                  f[(c0 / kLd + 1) & kMask][i] = qv[(c0 + kLd) / 4 + i];
            } else {
              // the accumulator has been read
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (C::PAIR) tc::mbar_arrive_relaxed_cluster(free0 + 8 * b);
                else tc::mbar_arrive_relaxed(free0 + 8 * b);
              }
            }
#pragma unroll
            for (int i = 0; i < kLd; i += 4) {
              float4 q = make_float4(s, s, s, s);
              if constexpr (C::QCOL) {
                const float4 v = f[(c0 / kLd) & kMask][i / 4];
                const float2 lo = __fmul2_rn(make_float2(v.x, v.y), make_float2(s, s));
                const float2 hi = __fmul2_rn(make_float2(v.z, v.w), make_float2(s, s));
                q = make_float4(lo.x, lo.y, hi.x, hi.y);
              }
              fma2(acc[c0 + i], acc[c0 + i + 1], q.x, q.y, now[i], now[i + 1]);
              fma2(acc[c0 + i + 2], acc[c0 + i + 3], q.z, q.w, now[i + 2], now[i + 3]);
            }
            if (c0 + kLd < C::kCols) tc::tmem_ld_wait(next);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sm.sempty(nslot & 1));
      }
      if (!__all_sync(~0u, ok)) {
        ok = false;
        if constexpr (C::PAIR)
#pragma unroll
          for (int i = 0; i < C::kCols; ++i) acc[i] = none;
      }
      if (!C::PAIR && g.split > 1) {
        // the ring is idle: every K-block loaded has been multiplied. (The
        // generic writes below follow the MMAs' reads through `done`.) Where not,
        // see below.
#pragma unroll
        for (int i = 0; i < C::kCols; i += 4) {
          const float4 v = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          const int c = part * C::kCols + i, r = quarter * 32 + lane;
          if constexpr (C::SWAP) {
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float*>(sm.ring_ptr + part_at<kRows>(c + e, r)) = f[e];
          } else {
            *reinterpret_cast<float4*>(sm.ring_ptr + part_at<C::BN>(r, c)) = v;
          }
        }
      } else if constexpr (C::SWAP) {
        store_tile_swapped<C>(g, acc, p0, q0, warp, lane);
      } else {
        if (g.out_fp32) store_tile<C, 4, VEC>(sm, g, acc, p0, q0, warp, lane);
        else store_tile<C, 2, VEC>(sm, g, acc, p0, q0, warp, lane);
      }
    }
    tc::tc_fence_before();
    tc::named_sync(1, C::kThreads);
    if constexpr (C::PAIR) {
      tc::cluster_sync();
    } else if (g.split > 1) {
      int64_t p, q;
      tile_at(t_first, tiles_p, tiles_q, p, q);
      if (!ok)   // once more: copies may have landed on it since
#pragma unroll 1
        for (int c = part * C::kCols; c < (part + 1) * C::kCols; ++c)
          *reinterpret_cast<float*>(sm.ring_ptr + (C::SWAP ? part_at<kRows>(c, quarter * 32 + lane)
                                                           : part_at<C::BN>(quarter * 32 + lane, c))) = none;
      tc::cluster_sync();   // every partial tile is in shared memory
      if (g.split == 2) add_split<C, 2>(sm, g, p * kRows, q * C::BN, rank);
      else if (g.split == 4) add_split<C, 4>(sm, g, p * kRows, q * C::BN, rank);
      else add_split<C, 8>(sm, g, p * kRows, q * C::BN, rank);
      __syncwarp();
      tc::cluster_sync();   // no CTA leaves while another reads its share
    }
  }
}

// ------------------------------------------------------------------- host --

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Codes [rows, K], ld bytes per row, read in 128-byte x box_rows boxes with the
// 128-byte swizzle; past K and past the last row reads as zero.
bool codes_map(CUtensorMap* tm, const void* codes, int64_t rows, int64_t K, int64_t ld,
               int box_rows) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kBlockK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

cudaError_t device_sms(int* dev, int* sms) {
  static std::atomic<int> known[kMaxDevices];
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= kMaxDevices) return cudaErrorInvalidDevice;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms == 0) {
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess) known[*dev].store(*sms, std::memory_order_relaxed);
  }
  return e;
}

template <class C, bool VEC>
cudaError_t launch_vec(const Gemm128& u, Gemm128Args g, int dev, int sms, cudaStream_t st) {
  auto kern = gemm128_kernel<C, VEC>;
  // the kernel's shared-memory limit, set once per device
  static std::atomic<uint64_t> ready{0};
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  CUtensorMap tmP{}, tmQ{};
  const bool maps = C::SWAP ? codes_map(&tmP, u.b, u.N, u.K, u.ldb, kRows) &&
                                  codes_map(&tmQ, u.a, u.M, u.K, u.lda, C::BN)
                            : codes_map(&tmP, u.a, u.M, u.K, u.lda, kRows) &&
                                  codes_map(&tmQ, u.b, u.N, u.K, u.ldb, C::kBoxQ);
  if (!maps) return cudaErrorInvalidValue;
  const uint32_t fa = u.a_e5m2 ? 1 : 0, fb = u.b_e5m2 ? 1 : 0;
  g.idesc = tc::idesc_f8(C::kTileRows, C::kUnitN, C::SWAP ? fb : fa, C::SWAP ? fa : fb);
  g.P = C::SWAP ? u.N : u.M;
  g.Q = C::SWAP ? u.M : u.N;
  g.p_scale = C::SWAP ? u.b_scales : u.a_scales;
  g.q_scale = C::SWAP ? u.a_scales : u.b_scales;
  g.p_ld = C::SWAP ? u.ldsb : u.ldsa;
  g.q_ld = C::SWAP ? u.ldsa : u.ldsb;
  g.p_block = C::SWAP ? u.b_block : 0;
  const int64_t tiles = ((g.P + C::kTileRows - 1) / C::kTileRows) * ((g.Q + C::BN - 1) / C::BN);
  const int cluster = C::PAIR ? 2 : g.split;
  // one tile per cluster that splits K; else persistent CTAs, one per SM
  if (tiles > 0x7fffffff / 8) return cudaErrorInvalidValue;
  const int64_t most = g.split > 1 ? tiles : sms / cluster;
  const unsigned grid = static_cast<unsigned>((tiles < most ? tiles : most) * cluster);
  return launch_dependent(kern, dim3(grid), dim3(C::kThreads), C::kSmem, st, cluster, tmP, tmQ, g);
}

template <class C>
cudaError_t launch(const Gemm128& u, const Gemm128Args& g, int dev, int sms, cudaStream_t st) {
  if constexpr (!C::SWAP)   // (swapped tiles are stored element by element)
    if (!g.vec) return launch_vec<C, false>(u, g, dev, sms, st);
  return launch_vec<C, true>(u, g, dev, sms, st);
}

}  // namespace

// The cheapest cut by a model of the time: waves of clusters, each the K-blocks
// of a CTA times a K-block's time, a start and end, and what joining a split
// costs (more for wide tiles, whose partial sums cross the cluster). Its figures
// (us) are fitted to measurements of every cut at 120 sizes, of which it chose
// the best or one 1% slower on average, 15% at worst (2048 x 511 x 6000):
//   a tile that is finer than needed loses to its number of waves, one that is
//   coarser leaves SMs idle: 128 x 8192 x 4096 takes 10.6 us in 64-wide tiles,
//   13.1 in 128-wide ones on two CTAs each, 18 in pairs' tiles; 512 x 8192 x
//   8192 takes 66 us in 64-wide tiles, 50 in 128-wide ones, 34 in pairs'.
//   Clusters are not free to pack: 17 of 8 CTAs run as two waves (12.0 us, 7.6
//   with clusters of 4), since a cluster stays within one of the GPU's groups of
//   SMs, and the occupancy query counts one more than ever ran at once.
Plan128 plan_gemm128(int64_t M, int64_t N, int64_t K, bool b_block, int sms, int clusters4,
                     int clusters8, double* us) {
  struct Cut {
    int bn, swap;
    double kb_block, kb_tile, tail;   // per K-block with block / tile weights, per wave
  };
  static constexpr Cut kCuts[] = {
      {16, 1, 0.22, 0.215, 1.5}, {32, 1, 0.25, 0.26, 1.7}, {64, 1, 0.305, 0.31, 1.8},
      {64, 0, 0.21, 0.29, 1.9},  {128, 0, 0.31, 0.4, 1.5}, {256, 0, 0.37, 0.62, 3.75}};
  static constexpr double kJoin[] = {0.0, 0.7, 1.2, 1.6};
  const int64_t nk = (K + 127) / 128;
  Plan128 best{};
  double best_t = 0.0;
  for (const Cut& c : kCuts) {
    const int64_t P = c.swap ? N : M, Q = c.swap ? M : N;
    const int64_t rows = c.bn == 256 ? 256 : 128;
    const int64_t tiles = ((P + rows - 1) / rows) * ((Q + c.bn - 1) / c.bn);
    for (int i = 0; i < 4; ++i) {
      const int split = 1 << i;
      if (split > nk || (c.bn == 256 && split > 1)) break;
      const int64_t slots = c.bn == 256 ? sms / 2 : i == 0 ? sms : i == 1 ? sms / 2
                                                  : i == 2 ? clusters4 : clusters8;
      if (slots < 1) break;
      const int64_t waves = (tiles + slots - 1) / slots;
      const double t = static_cast<double>(waves) *
                           (static_cast<double>((nk + split - 1) / split) *
                                (b_block ? c.kb_block : c.kb_tile) +
                            c.tail + (i ? kJoin[i] + 0.022 * c.bn : 0.0));
      if (best_t == 0.0 || t < best_t) {
        best = {c.bn, c.swap, split};
        best_t = t;
      }
    }
  }
  *us = best_t;
  return best;
}

namespace {

// Clusters of 4 and of 8 CTAs (one per SM) that the device holds at once.
cudaError_t device_clusters(int dev, int* c4, int* c8) {
  static std::atomic<int> known[kMaxDevices];   // c4 | c8 << 16, 0 unknown
  int v = known[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    using C = Cfg<128, false, false, false, 4>;
    auto kern = gemm128_kernel<C, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(C::kSmem));
    int n[2] = {0, 0};
    for (int i = 0; e == cudaSuccess && i < 2; ++i) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = i ? 8 : 4;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(1024);
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n[i], kern, &cfg);
    }
    if (e != cudaSuccess) return e;
    // (8 groups of SMs hold two clusters of 8 each)
    v = n[0] | (n[1] < 16 ? n[1] : 16) << 16;
    known[dev].store(v, std::memory_order_relaxed);
  }
  *c4 = v & 0xffff;
  *c8 = v >> 16;
  return cudaSuccess;
}

}  // namespace

namespace {

cudaError_t launch_one(const Gemm128& u, const Plan128& p, int dev, int sms, cudaStream_t st) {
  Gemm128Args g{};
  g.d = static_cast<uint8_t*>(u.d);
  g.status = u.status;
  g.ldd = u.ldd;
  g.nk = static_cast<int>((u.K + 127) / 128);
  g.split = p.bn == 256 ? 1 : p.split;
  g.out_fp32 = u.out_fp32;
  g.vec = u.ldd * (u.out_fp32 ? 4 : 2) % 16 == 0;
  if (p.swap) {
    if (p.bn == 16) return launch<Cfg<16, true, true, false, 8>>(u, g, dev, sms, st);
    if (p.bn == 32) return launch<Cfg<32, true, true, false, 8>>(u, g, dev, sms, st);
    return launch<Cfg<64, true, true, false, 8>>(u, g, dev, sms, st);
  }
  if (u.b_block) {
    if (p.bn == 64) return launch<Cfg<64, false, false, false, 8>>(u, g, dev, sms, st);
    if (p.bn == 128) return launch<Cfg<128, false, false, false, 4>>(u, g, dev, sms, st);
    return launch<Cfg<256, false, false, true, 4>>(u, g, dev, sms, st);
  }
  if (p.bn == 64) return launch<Cfg<64, true, false, false, 8>>(u, g, dev, sms, st);
  if (p.bn == 128) return launch<Cfg<128, true, false, false, 4>>(u, g, dev, sms, st);
  return launch<Cfg<256, true, false, true, 4>>(u, g, dev, sms, st);
}

// Rows m0.. and columns n0.. of D (m0, n0 multiples of 256).
Gemm128 part_of(const Gemm128& u, int64_t m0, int64_t M, int64_t n0, int64_t N) {
  Gemm128 v = u;
  v.a = static_cast<const uint8_t*>(u.a) + m0 * u.lda;
  v.a_scales = u.a_scales + m0;
  v.b = static_cast<const uint8_t*>(u.b) + n0 * u.ldb;
  v.b_scales = u.b_scales + (u.b_block ? n0 / 128 * ((u.K + 127) / 128) : n0);
  v.d = static_cast<uint8_t*>(u.d) + (m0 * u.ldd + n0) * (u.out_fp32 ? 4 : 2);
  v.M = M;
  v.N = N;
  return v;
}

}  // namespace

// Sizes a little over a multiple of 256 cost whole tiles, at times a whole wave
// of them: rows and columns past the multiple are then products of their own,
// if by the model that is cheaper (4099 x 2056 x 8192: one wave of three, 84.5
// -> 72.2 us). A further launch on the stream costs 1.7 us beyond its own time.
cudaError_t launch_gemm128(const Gemm128& u, const Plan128* plan, cudaStream_t st) {
  constexpr double kLaunch = 1.7;
  int dev = 0, sms = 0, c4 = 0, c8 = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (plan) return launch_one(u, *plan, dev, sms, st);
  e = device_clusters(dev, &c4, &c8);
  if (e != cudaSuccess) return e;
  const auto cost = [&](const Gemm128& v, Plan128* p) {
    double us = 0.0;
    *p = plan_gemm128(v.M, v.N, v.K, v.b_block, sms, c4, c8, &us);
    return us;
  };
  Plan128 whole{};
  double best = cost(u, &whole);
  Gemm128 parts[3] = {u};
  Plan128 plans[3] = {whole};
  int n = 1;
  const int64_t m0 = u.M / 256 * 256, n0 = u.N / 256 * 256;
  for (int cut = 1; cut < 4; ++cut) {   // rows, columns, both
    const int64_t m = cut & 1 ? m0 : u.M, c = cut & 2 ? n0 : u.N;
    if (m == 0 || c == 0 || ((cut & 1) && m == u.M) || ((cut & 2) && c == u.N)) continue;
    Gemm128 q[3];
    Plan128 qp[3];
    int k = 0;
    q[k++] = part_of(u, 0, m, 0, c);
    if (c < u.N) q[k++] = part_of(u, 0, m, c, u.N - c);
    if (m < u.M) q[k++] = part_of(u, m, u.M - m, 0, u.N);
    double us = kLaunch * (k - 1);
    for (int i = 0; i < k; ++i) us += cost(q[i], &qp[i]);
    if (us < best) {
      best = us;
      n = k;
      for (int i = 0; i < k; ++i) {
        parts[i] = q[i];
        plans[i] = qp[i];
      }
    }
  }
  for (int i = 0; i < n && e == cudaSuccess; ++i) e = launch_one(parts[i], plans[i], dev, sms, st);
  return e;
}

}  // namespace mxk
