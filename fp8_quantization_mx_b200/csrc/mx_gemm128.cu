// FP8 GEMM with float scales per 128 elements, on the sm_100 tensor cores:
//
//   D[m, n] = sum over K-blocks kb of  sa[m, kb] sb[n, kb] (A_kb B_kb^T)[m, n]
//
// A [M, K] in 1 x 128 tiles; B [N, K] in 1 x 128 tiles or 128 x 128 blocks;
// E4M3 or E5M2 each. The scales are arbitrary floats, which no MMA applies, so
// every K-block of 128 is accumulated by itself in tensor memory and added,
// scaled, to float sums in registers:
//   warp 0     TMA: one K-block of both operands per stage (128 bytes per row:
//              one 128-byte swizzle atom), S stages; the column scales' ring
//   warp 1     one thread issues the four tcgen05.mma.kind::f8f6f4 (K = 32)
//              of a K-block into the next of NBUF accumulators
//   warps 4..  accumulator -> registers (tcgen05.ld, one row per thread),
//              acc += (s_row s_col) t with packed multiply-adds, accumulator
//              released; after the last K-block the tile is stored
// so the vector work of one K-block runs beside the MMAs of the next.
//
// A tile is 128 rows of one operand ("rows": MMA A) by BN of the other
// ("columns": MMA B). Few tokens: the weights take the row side (128 of N per
// tile) and the tokens the column side, BN = 16, 32 or 64, so that no MMA row
// is wasted and the weights are read once (SWAP). Too few tiles to fill the
// SMs: a cluster of 2, 4 or 8 CTAs splits K, and each CTA adds up its share of
// the tile over the cluster's shared memory, in rank order (no atomics).
//
// Every wait is bounded in time (mbar_wait): one that runs out sets the
// caller's status word, and the CTA drains its copies and MMAs, frees its TMEM
// and returns.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "mx_gemm128.h"
#include "mx_launch.h"
#include "mx_tc.cuh"

namespace mxk {

namespace {

constexpr int kRows = 128;              // rows of a tile: the MMA's M
constexpr uint32_t kBlockK = 128;       // elements (bytes) of K per stage
constexpr uint32_t kTileP = kRows * kBlockK;

constexpr int kStatusProducer = 11, kStatusMma = 12, kStatusSums = 13, kStatusDrain = 14;

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

template <int BN_, bool QCOL_, bool SWAP_, int S_>
struct Cfg {
  static constexpr int BN = BN_, S = S_;
  static constexpr bool QCOL = QCOL_, SWAP = SWAP_;   // QCOL: a scale per column
  static constexpr int kHalves = BN >= 64 ? 2 : 1;
  static constexpr int kWork = 4 * kHalves;           // accumulating warps
  // 256 threads with up to 128 sums each need more than the 168 registers that
  // 384 threads can have: the first warpgroup (TMA, MMA, two idle warps) gives
  // most of its share to the other two. 128 (40 + 2 x 232) = 384 x 168.
  static constexpr int kWork0 = 4;                    // first accumulating warp
  static constexpr bool kShift = kHalves == 2;
  static constexpr int kThreads = (kWork0 + kWork) * 32;
  static constexpr int kCols = BN / kHalves;          // columns per thread
  static constexpr int NBUF = BN == 256 ? 2 : 4;      // accumulators in TMEM
  static constexpr uint32_t kTmemCols = NBUF * BN;
  static constexpr uint32_t kTileQ = BN * kBlockK;
  static constexpr uint32_t kStage = kTileP + kTileQ;
  static constexpr int QS = QCOL ? 8 : 0;             // column-scale slots
  static constexpr uint32_t kQBytes = BN * 4;
  static constexpr uint32_t kStgRow = QCOL ? 64 : 128;   // store staging: 32 such rows per warp
  static constexpr uint32_t kStaging = SWAP ? 0 : kWork * 32 * kStgRow;
  static constexpr int kBars = 2 * S + 2 * NBUF + 2 * QS + 1;
  static constexpr uint32_t kSmem = S * kStage + kStaging + QS * kQBytes + 8 * kBars + 16 + 1024;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(S * kStage >= kRows * BN * 4, "the split's partial tile reuses the ring");
};

template <class C>
struct Smem {
  uint32_t raw, ring, stg, qv, bar;
  uint32_t* tmem_holder;
  volatile int* abort_flag;
  uint8_t* ring_ptr;
  uint8_t* stg_ptr;
  float* qv_ptr;
  __device__ explicit Smem(uint8_t* p) {
    raw = tc::smem_addr(p);
    ring = (raw + 1023u) & ~1023u;   // swizzle atoms need 1024-byte alignment
    stg = ring + C::S * C::kStage;
    qv = stg + C::kStaging;
    bar = qv + C::QS * C::kQBytes;
    ring_ptr = p + (ring - raw);
    stg_ptr = p + (stg - raw);
    qv_ptr = reinterpret_cast<float*>(p + (qv - raw));
    tmem_holder = reinterpret_cast<uint32_t*>(p + (bar + 8u * C::kBars - raw));
    abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  }
  __device__ uint32_t p_tile(int s) const { return ring + s * C::kStage; }
  __device__ uint32_t q_tile(int s) const { return ring + s * C::kStage + kTileP; }
  __device__ uint32_t full(int s) const { return bar + 8u * s; }
  __device__ uint32_t empty(int s) const { return bar + 8u * (C::S + s); }
  __device__ uint32_t tfull(int b) const { return bar + 8u * (2 * C::S + b); }
  __device__ uint32_t tempty(int b) const { return bar + 8u * (2 * C::S + C::NBUF + b); }
  __device__ uint32_t done() const { return bar + 8u * (2 * C::S + 2 * C::NBUF); }
  __device__ uint32_t qfull(int s) const { return bar + 8u * (2 * C::S + 2 * C::NBUF + 1 + s); }
  __device__ uint32_t qempty(int s) const {
    return bar + 8u * (2 * C::S + 2 * C::NBUF + 1 + C::QS + s);
  }
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

// ------------------------------------------------- packed float arithmetic --

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  for (int u = threadIdx.x - C::kWork0 * 32; u < kUnits; u += C::kWork * 32) {
    const int at = static_cast<int>(rank) * kUnits + u;
    const int major = at / (L / 4), minor = at % (L / 4) * 4;
    if (r0 + major >= rows || c0 + minor >= cols) continue;
    const uint32_t a = sm.ring + part_at<L>(major, minor);
    float4 v[SPLIT];
#pragma unroll
    for (int r = 0; r < SPLIT; ++r) v[r] = ld_cluster4(tc::mapa(a, r));
    float4 s = v[0];
#pragma unroll
    for (int r = 1; r < SPLIT; ++r) {
      s.x += v[r].x;
      s.y += v[r].y;
      s.z += v[r].z;
      s.w += v[r].w;
    }
    store4(g, r0 + major, c0 + minor, cols - c0 - minor, s);
  }
}

// One tile of D from the sums in registers (rows on the row side): a warp
// stages 32 rows of kStgRow bytes in its own shared memory, so that a row
// leaves as full 16-byte lanes of one run.
template <class C, int ES>
__device__ __forceinline__ void store_tile(const Smem<C>& sm, const Gemm128Args& g,
                                           const uint64_t (&acc)[C::kCols / 2], int64_t p0,
                                           int64_t q0, int warp, int lane) {
  constexpr int kChunk = (C::kStgRow / ES < C::kCols) ? C::kStgRow / ES : C::kCols;
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
        if constexpr (ES == 2) {
          float lo, hi;
          unpack2(acc[(c0 + j * kPer) / 2 + i], lo, hi);
          w[i] = bf16x2(lo, hi);
        } else {
          float lo, hi;
          unpack2(acc[(c0 + j * kPer) / 2 + i / 2], lo, hi);
          w[i] = __float_as_uint((i & 1) ? hi : lo);
        }
      }
      *reinterpret_cast<uint4*>(stg + lane * (NJ * 16) + ((j ^ (lane & (NJ - 1))) * 16)) = v;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NJ; ++i) {
      const int r = i * kRowsPer + lane / NJ, j = lane % NJ;
      const uint4 v =
          *reinterpret_cast<const uint4*>(stg + r * (NJ * 16) + ((j ^ (r & (NJ - 1))) * 16));
      const int64_t row = row0 + r, col = colh + c0 + j * kPer;
      if (row < g.P && col < g.Q) {
        uint8_t* d = g.d + (row * g.ldd + col) * ES;
        if (g.vec && col + kPer <= g.Q) {
          *reinterpret_cast<uint4*>(d) = v;
        } else {
          const uint32_t* w = &v.x;
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (col + e < g.Q) {
              if constexpr (ES == 2)
                reinterpret_cast<uint16_t*>(d)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
              else
                reinterpret_cast<uint32_t*>(d)[e] = w[e];
            }
        }
      }
    }
    __syncwarp();
  }
}

// The same with D's rows on the column side: lane = consecutive columns of D.
template <class C>
__device__ __forceinline__ void store_tile_swapped(const Gemm128Args& g,
                                                   const uint64_t (&acc)[C::kCols / 2], int64_t p0,
                                                   int64_t q0, int warp, int lane) {
  const int64_t n = p0 + (warp & 3) * 32 + lane;
  const int64_t m0 = q0 + ((warp - C::kWork0) / 4) * C::kCols;
  if (n >= g.P) return;
#pragma unroll
  for (int i = 0; i < C::kCols; ++i) {
    float lo, hi;
    unpack2(acc[i / 2], lo, hi);
    const float v = (i & 1) ? hi : lo;
    if (m0 + i < g.Q) {
      const int64_t at = (m0 + i) * g.ldd + n;
      if (g.out_fp32)
        reinterpret_cast<float*>(g.d)[at] = v;
      else
        reinterpret_cast<__nv_bfloat16*>(g.d)[at] = __float2bfloat16_rn(v);
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    gemm128_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const Gemm128Args g) {
  extern __shared__ uint8_t smem_raw[];
  const Smem<C> sm(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t tiles_p = (g.P + kRows - 1) / kRows;
  const int64_t tiles_q = (g.Q + C::BN - 1) / C::BN;
  const int64_t ntiles = tiles_p * tiles_q;
  // a cluster shares a tile: this CTA's K-blocks are [kb0, kb1)
  const uint32_t rank = g.split > 1 ? blockIdx.x % g.split : 0;
  const int64_t t_first = blockIdx.x / g.split;
  const int64_t t_step = gridDim.x / g.split;
  const int kb0 = static_cast<int>(static_cast<int64_t>(g.nk) * rank / g.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(g.nk) * (rank + 1) / g.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      tc::mbar_init(sm.full(s), 1);
      tc::mbar_init(sm.empty(s), 1);
    }
    for (int b = 0; b < C::NBUF; ++b) {
      tc::mbar_init(sm.tfull(b), 1);
      tc::mbar_init(sm.tempty(b), C::kWork);
    }
    for (int s = 0; s < C::QS; ++s) {
      tc::mbar_init(sm.qfull(s), 1);
      tc::mbar_init(sm.qempty(s), C::kWork);
    }
    tc::mbar_init(sm.done(), 1);
    *sm.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_addr(sm.tmem_holder), C::kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *sm.tmem_holder;

  if (warp < C::kWork0) {
    if constexpr (C::kShift) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        tc::prefetch_tmap(&tmP);
        tc::prefetch_tmap(&tmQ);
        Ring<C::S> st;
        Ring<C::QCOL ? C::QS : 1> qs;
        int64_t issued = 0, qissued = 0;
        bool ok = true;
        for (int64_t t = t_first; ok && t < ntiles; t += t_step) {
          int64_t p, q;
          tile_at(t, tiles_p, tiles_q, p, q);
          const int p0 = static_cast<int>(p * kRows), q0 = static_cast<int>(q * C::BN);
          // column scales present: the rest of the slot belongs to columns past the edge
          const int64_t left = ((g.Q + 3) & ~int64_t(3)) - q0;
          const uint32_t qbytes = static_cast<uint32_t>(left < C::BN ? left : C::BN) * 4;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!tc::mbar_wait(sm.empty(st.slot), st.par ^ 1, sm.abort_flag, g.status, kStatusProducer)) {
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(sm.full(st.slot), C::kStage);
            tc::tma_load_2d(sm.p_tile(st.slot), &tmP, kb * static_cast<int>(kBlockK), p0, sm.full(st.slot));
            tc::tma_load_2d(sm.q_tile(st.slot), &tmQ, kb * static_cast<int>(kBlockK), q0, sm.full(st.slot));
            st.next();
            ++issued;
            if constexpr (C::QCOL) {
              if (!tc::mbar_wait(sm.qempty(qs.slot), qs.par ^ 1, sm.abort_flag, g.status,
                                 kStatusProducer)) {
                ok = false;
                break;
              }
              tc::mbar_arrive_expect_tx(sm.qfull(qs.slot), qbytes);
              tc::bulk_load(sm.qv + qs.slot * C::kQBytes, g.q_scale + kb * g.q_ld + q0, qbytes,
                            sm.qfull(qs.slot));
              qs.next();
              ++qissued;
            }
          }
        }
        // every copy this thread issued has landed before the CTA can exit
        for (int64_t j = issued > C::S ? issued - C::S : 0; j < issued; ++j)
          tc::mbar_wait(sm.full(static_cast<int>(j % C::S)), static_cast<uint32_t>(j / C::S) & 1,
                        sm.abort_flag, g.status, kStatusDrain, false);
        if constexpr (C::QCOL)
          for (int64_t j = qissued > C::QS ? qissued - C::QS : 0; j < qissued; ++j)
            tc::mbar_wait(sm.qfull(static_cast<int>(j % C::QS)), static_cast<uint32_t>(j / C::QS) & 1,
                          sm.abort_flag, g.status, kStatusDrain, false);
      }
      __syncwarp();
    }
    if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      if (lane == 0) {
        Ring<C::S> st;
        Ring<C::NBUF> tb;
        bool ok = true;
        for (int64_t t = t_first; ok && t < ntiles; t += t_step)
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!tc::mbar_wait(sm.tempty(tb.slot), tb.par ^ 1, sm.abort_flag, g.status, kStatusMma) ||
                !tc::mbar_wait(sm.full(st.slot), st.par, sm.abort_flag, g.status, kStatusMma)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint64_t pd = tc::kmajor_sw128_desc(sm.p_tile(st.slot));
            const uint64_t qd = tc::kmajor_sw128_desc(sm.q_tile(st.slot));
#pragma unroll
            for (int k = 0; k < 4; ++k)   // K = 32: 32 bytes further along the rows
              tc::mma_f8(tmem + tb.slot * C::BN, pd + 2 * k, qd + 2 * k, g.idesc, k != 0);
            tc::tc_commit(sm.empty(st.slot));
            tc::tc_commit(sm.tfull(tb.slot));
            st.next();
            tb.next();
          }
        // every MMA has finished before TMEM is freed, whatever ended the loop
        tc::tc_commit(sm.done());
        tc::mbar_wait(sm.done(), 0, sm.abort_flag, g.status, kStatusDrain, false);
      }
      __syncwarp();
    }
    // (accumulators read, by the other branch's half of this barrier)
    tc::named_sync(1, C::kThreads);
    if (warp == 1) {
      tc::tc_fence_after();
      tc::tmem_dealloc(tmem, C::kTmemCols);
    }
    if (g.split > 1) {
      tc::cluster_sync();
      tc::cluster_sync();
    }
  } else {
    // ------------------------------------------------------ scaled sums
    if constexpr (C::kShift) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quarter = warp & 3, half = (warp - C::kWork0) / 4;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * C::kCols;
    Ring<C::NBUF> tb;
    Ring<C::QCOL ? C::QS : 1> qs;
    bool ok = true;
    for (int64_t t = t_first; ok && t < ntiles; t += t_step) {
      int64_t p, q;
      tile_at(t, tiles_p, tiles_q, p, q);
      const int64_t p0 = p * kRows, q0 = q * C::BN;
      // this row's scale, and (blocks on the column side) the columns'
      const int64_t row = p0 + quarter * 32 + lane;
      const int64_t prow = row < g.P ? row : g.P - 1;
      const float* ps = g.p_block ? g.p_scale + p * g.nk : g.p_scale + prow;
      const int64_t pstep = g.p_block ? 1 : g.p_ld;
      const int64_t qcol = q0 + half * C::kCols;
      const float* qb = C::QCOL ? nullptr
                                : g.q_scale + (qcol < g.Q ? qcol : g.Q - 1) / kRows * g.nk;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      float s_next = kb0 < kb1 ? ps[kb0 * pstep] : 0.0f;
      float b_next = !C::QCOL && kb0 < kb1 ? qb[kb0] : 1.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        const float s = C::QCOL ? s_next : s_next * b_next;
        if (kb + 1 < kb1) {
          s_next = ps[(kb + 1) * pstep];
          if (!C::QCOL) b_next = qb[kb + 1];
        }
        bool got = true;
        if constexpr (C::QCOL)
          got = tc::mbar_wait(sm.qfull(qs.slot), qs.par, sm.abort_flag, g.status, kStatusSums);
        got = got && tc::mbar_wait(sm.tfull(tb.slot), tb.par, sm.abort_flag, g.status, kStatusSums);
        // one decision for the warp: tcgen05.ld is a whole-warp instruction
        if (!__all_sync(~0u, got)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint64_t s2 = pack2(s, s);
        constexpr int kLd = C::kCols < 32 ? C::kCols : 32;
#pragma unroll
        for (int c0 = 0; c0 < C::kCols; c0 += kLd) {
          uint32_t r[kLd];
          const uint32_t taddr = lane_base + tb.slot * C::BN + c0;
          if constexpr (kLd == 32) tc::tmem_ld32(taddr, r);
          else tc::tmem_ld16(taddr, r);
          if constexpr (C::QCOL) {
            const float4* qv = reinterpret_cast<const float4*>(sm.qv_ptr + qs.slot * C::BN +
                                                               half * C::kCols + c0);
#pragma unroll
            for (int i = 0; i < kLd / 4; ++i) {
              const float4 f = qv[i];
              acc[(c0 + 4 * i) / 2] = fma2(mul2(pack2(f.x, f.y), s2), pack2u(r[4 * i], r[4 * i + 1]),
                                           acc[(c0 + 4 * i) / 2]);
              acc[(c0 + 4 * i) / 2 + 1] =
                  fma2(mul2(pack2(f.z, f.w), s2), pack2u(r[4 * i + 2], r[4 * i + 3]),
                       acc[(c0 + 4 * i) / 2 + 1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kLd / 2; ++i)
              acc[c0 / 2 + i] = fma2(s2, pack2u(r[2 * i], r[2 * i + 1]), acc[c0 / 2 + i]);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(sm.tempty(tb.slot));
          if constexpr (C::QCOL) tc::mbar_arrive(sm.qempty(qs.slot));
        }
        tb.next();
        if constexpr (C::QCOL) qs.next();
      }
      if (!ok) break;
      if (g.split > 1) {
        // the ring is idle: every K-block loaded has been multiplied. (The
        // generic writes below follow the MMAs' reads through tfull.)
#pragma unroll
        for (int i = 0; i < C::kCols; i += 4) {
          float4 v;
          unpack2(acc[i / 2], v.x, v.y);
          unpack2(acc[i / 2 + 1], v.z, v.w);
          const int c = half * C::kCols + i, r = quarter * 32 + lane;
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
        if (g.out_fp32) store_tile<C, 4>(sm, g, acc, p0, q0, warp, lane);
        else store_tile<C, 2>(sm, g, acc, p0, q0, warp, lane);
      }
    }
    tc::tc_fence_before();
    tc::named_sync(1, C::kThreads);
    if (g.split > 1) {
      int64_t p, q;
      tile_at(t_first, tiles_p, tiles_q, p, q);
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

template <class C>
cudaError_t launch(const Gemm128& u, Gemm128Args g, int dev, int sms, cudaStream_t st) {
  auto kern = gemm128_kernel<C>;
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
                                  codes_map(&tmQ, u.b, u.N, u.K, u.ldb, C::BN);
  if (!maps) return cudaErrorInvalidValue;
  const uint32_t fa = u.a_e5m2 ? 1 : 0, fb = u.b_e5m2 ? 1 : 0;
  g.idesc = tc::idesc_f8(kRows, C::BN, C::SWAP ? fb : fa, C::SWAP ? fa : fb);
  g.P = C::SWAP ? u.N : u.M;
  g.Q = C::SWAP ? u.M : u.N;
  g.p_scale = C::SWAP ? u.b_scales : u.a_scales;
  g.q_scale = C::SWAP ? u.a_scales : u.b_scales;
  g.p_ld = C::SWAP ? u.ldsb : u.ldsa;
  g.q_ld = C::SWAP ? u.ldsa : u.ldsb;
  g.p_block = C::SWAP ? u.b_block : 0;
  const int64_t tiles = ((g.P + kRows - 1) / kRows) * ((g.Q + C::BN - 1) / C::BN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(g.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = g.split > 1 ? 1 : 0;
  // one tile per cluster, or (no split) persistent CTAs, one per SM
  if (g.split > 1 && tiles * g.split > 0x7fffffff) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(static_cast<unsigned>(g.split > 1 ? tiles * g.split : tiles < sms ? tiles : sms));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmP, tmQ, g);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

Plan128 plan_gemm128(int64_t M, int64_t N, int64_t K, bool b_block, int sms) {
  (void)b_block;
  Plan128 p{};
  const int64_t nk = (K + 127) / 128;
  p.swap = M <= 64;
  p.bn = p.swap ? (M <= 16 ? 16 : M <= 32 ? 32 : 64) : N <= 64 ? 64 : N <= 128 ? 128 : 256;
  const auto tiles = [&]() {
    const int64_t P = p.swap ? N : M, Q = p.swap ? M : N;
    return ((P + 127) / 128) * ((Q + p.bn - 1) / p.bn);
  };
  if (!p.swap && p.bn == 256 && tiles() < sms) p.bn = 128;
  p.split = 1;
  while (p.split < 8 && tiles() * p.split * 2 <= sms && nk >= p.split * 4) p.split *= 2;
  return p;
}

cudaError_t launch_gemm128(const Gemm128& u, const Plan128* plan, cudaStream_t st) {
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const Plan128 p = plan ? *plan : plan_gemm128(u.M, u.N, u.K, u.b_block, sms);
  Gemm128Args g{};
  g.d = static_cast<uint8_t*>(u.d);
  g.status = u.status;
  g.ldd = u.N;
  g.nk = static_cast<int>((u.K + 127) / 128);
  g.split = p.split;
  g.out_fp32 = u.out_fp32;
  g.vec = u.N * (u.out_fp32 ? 4 : 2) % 16 == 0;
  if (p.swap) {
    if (p.bn == 16) return launch<Cfg<16, true, true, 10>>(u, g, dev, sms, st);
    if (p.bn == 32) return launch<Cfg<32, true, true, 10>>(u, g, dev, sms, st);
    return launch<Cfg<64, true, true, 8>>(u, g, dev, sms, st);
  }
  if (u.b_block) {
    if (p.bn == 64) return launch<Cfg<64, false, false, 8>>(u, g, dev, sms, st);
    if (p.bn == 128) return launch<Cfg<128, false, false, 6>>(u, g, dev, sms, st);
    return launch<Cfg<256, false, false, 4>>(u, g, dev, sms, st);
  }
  if (p.bn == 64) return launch<Cfg<64, true, false, 8>>(u, g, dev, sms, st);
  if (p.bn == 128) return launch<Cfg<128, true, false, 6>>(u, g, dev, sms, st);
  return launch<Cfg<256, true, false, 4>>(u, g, dev, sms, st);
}

}  // namespace mxk
