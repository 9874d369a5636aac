// RMSNorm with the residual's addition and FP8 output (float scales per 1 x 128
// tile), and its gradient.
//
//   h = x + residual (written in x's type; the norm uses the unrounded sum)
//   y = h r w,  r = 1 / sqrt(mean(h^2) + eps)
//   codes, scales: y's 1 x 128 tiles (mx_tile128.cuh), from the unrounded y
//
//   gradient, from gy = dL/dy (the quantizer passes gradients straight
//   through), the saved h and, optionally, the residual stream's own gradient:
//   gh = r (gy w - n mean(gy w n)) + gres,  n = h r;   gw = sum over rows of gy n
//
// Sums, r, y and the gradients are float; h, y (when asked for) and gh are
// rounded to x's type once, when stored. Both passes are bound by HBM: each
// row is read once into registers, 8 elements per lane, and written once. On a
// B200 with a copy bandwidth of 6.45 TB/s, bf16 with the residual: forward
// 16387 x 4096 76.9 us (95% of the bytes' time), 8192 x 8192 85 us (86%), 65536
// x 512 41.7 us (88%), one row of 2048 1.8 us; gradient 16384 x 4096 91.5 us
// (91%), 65536 x 512 47.2 us (88%), 1999 x 2048 9.5 us (40%: three or four
// rows per CTA, then the second kernel's sum of 592 shares of gw).

#include <cuda_runtime.h>

#include <type_traits>

#include "mx_launch.h"
#include "mx_pdl.cuh"
#include "mx_rowvec.h"
#include "mx_tile128.cuh"

namespace mxk {

namespace {

using namespace t128;

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;   // [rows, cols] or null
  const void* weight;     // [cols]
  void* h;                // [rows, cols] or null
  void* y;                // [rows, cols] or null
  uint8_t* codes;         // [rows, ldc]
  int64_t ldc;
  float* scales;          // [ceil(cols/128), lds]
  int64_t lds;
  int64_t rows, cols;
  float eps;
  int pow2;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The sum of N values over the CTA, the same in every thread (`red` holds 32
// N floats; the caller orders reuse of it).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < nw ? red[lane * N + i] : 0.0f);
}

// 1 / sqrt(sum / cols + eps)
__device__ __forceinline__ float row_rstd(float sum, int64_t cols, float eps) {
  return __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(cols)) + eps);
}

// Codes of -ny.
template <bool E5M2>
__device__ __forceinline__ uint2 encode8(const float2 (&ny)[4], const Divisor& d) {
  const float2 s = make_float2(d.s, d.s), ninv = make_float2(d.ninv, d.ninv);
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = ny[i];
    if (d.slow) x = __fmul2_rn(x, make_float2(kLift, kLift));
    q[i] = div2(x, s, ninv);
  }
  return make_uint2(enc4<E5M2>(q[0].x, q[0].y, q[1].x, q[1].y),
                    enc4<E5M2>(q[2].x, q[2].y, q[3].x, q[3].y));
}

// The threads of a row: a whole CTA, or (WARP, rows of up to 1024 elements) one
// of its eight warps, which needs no barrier. CTAs are as many as the SMs hold;
// each takes every gridDim-th row (or eight), and the next row's loads are
// issued before this row's sums, so that HBM is busy across them.
template <bool WARP>
struct RowThreads {
  int tid, nt;
  int64_t first, step;
  __device__ RowThreads()
      : tid(WARP ? threadIdx.x & 31 : threadIdx.x),
        nt(WARP ? 32 : blockDim.x),
        first(WARP ? blockIdx.x * int64_t(8) + (threadIdx.x >> 5) : blockIdx.x),
        step(WARP ? gridDim.x * int64_t(8) : gridDim.x) {}
  // Sums over the row's threads, the same in each (two buffers in turn: the
  // next row's sums may start while a warp reads these).
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N], float (&red)[2][32 * N], int par) const {
    if constexpr (WARP) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    } else {
      block_sum(v, red[par]);
    }
  }
};

// NV vectors of 8 elements per thread: the vectors of a tile are 16
// neighbouring lanes', each of which takes one of the NV tiles' scale.
// HALF: at most 256 threads with two vectors each, registers for three CTAs of
// 256 (floats two): 16387 x 4096 took 84.7 us with two of them, 78.2 with
// three, 92 with four (76.9 since the scales are shared out over the lanes).
template <int DT, bool E5M2, int NV, bool WARP, bool HALF = false>
__global__ void __launch_bounds__(WARP || NV == 1 || HALF ? 256 : 512,
                                  NV == 1 ? 4 : HALF ? (DT == kFP32 ? 2 : 3) : 1)
    norm128_kernel(const NormArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ float red[2][32];
  const RowThreads<WARP> rt;
  dependent_launch();
  dependent_wait();
  const int nvec = static_cast<int>(a.cols / 8);
  const int64_t pitch = (a.cols + 15) & ~int64_t(15);
  Vec<DT, 8> xv[NV], rv[NV], wv[NV];
  const auto load = [&](int64_t row, Vec<DT, 8>(&x)[NV], Vec<DT, 8>(&r)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = rt.tid + j * rt.nt;
      x[j].zero();
      r[j].zero();
      if (i < nvec && row < a.rows) {
        x[j].load(static_cast<const T*>(a.x) + row * a.ldx + 8 * i);
        if (a.residual) r[j].load(static_cast<const T*>(a.residual) + row * a.cols + 8 * i);
      }
    }
  };
  load(rt.first, xv, rv);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = rt.tid + j * rt.nt;
    wv[j].zero();
    if (i < nvec) wv[j].load(static_cast<const T*>(a.weight) + 8 * i);
  }
  int par = 0;
  for (int64_t row = rt.first; row < a.rows; row += rt.step, par ^= 1) {
    Vec<DT, 8> xn[NV], rn[NV];
    load(row + rt.step, xn, rn);
    float2 h[NV][4], sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = rt.tid + j * rt.nt;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[j][e] = __fadd2_rn(xv[j].get2(e), rv[j].get2(e));
        sq = __ffma2_rn(h[j][e], h[j][e], sq);
      }
      if (a.h && i < nvec) {
        Vec<DT, 8> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.set2(e, h[j][e].x, h[j][e].y);
        o.store(static_cast<T*>(a.h) + row * a.cols + 8 * i);
      }
    }
    float ss[1] = {sq.x + sq.y};
    rt.sum(ss, red, par);
    const float r = -row_rstd(ss[0], a.cols, a.eps);   // y negated, as div2 takes it
    float m[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      m[j] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[j][e] = __fmul2_rn(__fmul2_rn(h[j][e], make_float2(r, r)), wv[j].get2(e));
        m[j] = amax3(m[j], h[j][e].x, h[j][e].y);
      }
    }
    // each lane takes one of its NV tiles' scales
    float mm = spread_max(m, threadIdx.x & 31);
#pragma unroll
    for (int o = NV; o < 16; o <<= 1) mm = amax2(mm, __shfl_xor_sync(~0u, mm, o));
    const float s = tile_scale<E5M2>(mm, a.pow2);
    const Divisor mine = divisor(s, mm == 0.0f);
    {
      const int j = held_by<NV>(threadIdx.x & 31), i = rt.tid + j * rt.nt;
      if ((threadIdx.x & 15) < NV && (i & ~15) < nvec) a.scales[(i >> 4) * a.lds + row] = s;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = rt.tid + j * rt.nt;
      const uint2 c = encode8<E5M2>(h[j], divisor_of(mine, (threadIdx.x & 16) | lane_of<NV>(j)));
      // codes up to the row's padding to 16 bytes (the vector past the last is 0)
      if (8 * static_cast<int64_t>(i) < pitch)
        *reinterpret_cast<uint2*>(a.codes + row * a.ldc + 8 * i) = c;
      if (a.y && i < nvec) {
        Vec<DT, 8> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.set2(e, -h[j][e].x, -h[j][e].y);
        o.store(static_cast<T*>(a.y) + row * a.cols + 8 * i);
      }
      xv[j] = xn[j];
      rv[j] = rn[j];
    }
  }
}

// Any number of columns at any alignment: one CTA per row, element tid + 256 j
// in thread tid. Up to 256 NJ columns stay in registers; beyond, the row is
// read again (mostly from cache).
template <int DT, bool E5M2, int NJ>
__global__ void __launch_bounds__(256) norm128_any_kernel(const NormArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float red[32];
  __shared__ float sh_max[NJ][8];
  __shared__ Divisor sh_div[2 * NJ];
  dependent_launch();
  dependent_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  const auto h_at = [&](int64_t c) {
    return c < a.cols ? E::to_float(x[c]) + (res ? E::to_float(res[c]) : 0.0f) : 0.0f;
  };
  float h[NJ], ss[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    h[j] = h_at(tid + 256 * j);
    ss[0] = fmaf(h[j], h[j], ss[0]);
  }
  for (int64_t c = tid + 256 * NJ; c < a.cols; c += 256) {
    const float v = h_at(c);
    ss[0] = fmaf(v, v, ss[0]);
  }
  block_sum(ss, red);
  const float r = row_rstd(ss[0], a.cols, a.eps);
  const int64_t pitch = (a.cols + 15) & ~int64_t(15);
  for (int64_t c0 = 0; c0 < a.cols; c0 += 256 * NJ) {
    float y[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = c0 + tid + 256 * j;
      if (c0 > 0) h[j] = h_at(c);
      y[j] = c < a.cols ? h[j] * r * E::to_float(w[c]) : 0.0f;
      float m = fabsf(y[j]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) m = amax2(m, __shfl_xor_sync(~0u, m, o));
      if (lane == 0) sh_max[j][warp] = m;
    }
    __syncthreads();
    if (tid < 2 * NJ) {   // a tile is four warps' elements
      const float* p = &sh_max[tid >> 1][(tid & 1) * 4];
      const float m = amax2(amax2(p[0], p[1]), amax2(p[2], p[3]));
      const float s = tile_scale<E5M2>(m, a.pow2);
      sh_div[tid] = divisor(s, m == 0.0f);
      const int64_t t = c0 / 128 + tid;
      if (t * 128 < a.cols) a.scales[t * a.lds + row] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = c0 + tid + 256 * j;
      const Divisor d = sh_div[2 * j + (warp >> 2)];
      const float v = d.slow ? -y[j] * kLift : -y[j];
      const float2 q = div2(make_float2(v, 0.0f), make_float2(d.s, d.s), make_float2(d.ninv, d.ninv));
      if (c < pitch) a.codes[row * a.ldc + c] = static_cast<uint8_t>(enc2<E5M2>(q.x, 0.0f));
      if (c < a.cols) {
        if (a.h) static_cast<T*>(a.h)[row * a.cols + c] = E::from_float(h[j]);
        if (a.y) static_cast<T*>(a.y)[row * a.cols + c] = E::from_float(y[j]);
      }
    }
  }
}

// The same for rows of up to 32 NJ (at most 1024) columns: a warp per row, eight
// rows per CTA; four neighbouring elements of a lane are a tile's.
template <int DT, bool E5M2, int NJ>
__global__ void __launch_bounds__(256) norm128_any_warp_kernel(const NormArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  const int lane = threadIdx.x & 31;
  dependent_launch();
  dependent_wait();
  const int64_t row = blockIdx.x * int64_t(8) + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int cols = static_cast<int>(a.cols), pitch = (cols + 15) & ~15;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  float h[NJ], wv[NJ], ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int c = lane + 32 * j;
    h[j] = c < cols ? E::to_float(x[c]) + (res ? E::to_float(res[c]) : 0.0f) : 0.0f;
    wv[j] = c < cols ? E::to_float(w[c]) : 0.0f;
    ss = fmaf(h[j], h[j], ss);
  }
  const float r = row_rstd(warp_sum(ss), a.cols, a.eps);
#pragma unroll
  for (int t = 0; t < NJ / 4; ++t) {
    if (t * 128 >= cols) break;
    float y[4], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = lane + 32 * (4 * t + j);
      y[j] = c < cols ? h[4 * t + j] * r * wv[4 * t + j] : 0.0f;
      m = amax2(m, y[j]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = amax2(m, __shfl_xor_sync(~0u, m, o));
    const float s = tile_scale<E5M2>(m, a.pow2);
    const Divisor d = divisor(s, m == 0.0f);
    if (lane == 0) a.scales[t * a.lds + row] = s;
    const float k = d.slow ? -kLift : -1.0f;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 q = div2(make_float2(y[j] * k, y[j + 1] * k), make_float2(d.s, d.s),
                            make_float2(d.ninv, d.ninv));
      const uint32_t codes = enc2<E5M2>(q.x, q.y);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = lane + 32 * (4 * t + j + e);
        if (c < pitch) a.codes[row * a.ldc + c] = static_cast<uint8_t>(codes >> (8 * e));
        if (c < cols) {
          if (a.h) static_cast<T*>(a.h)[row * a.cols + c] = E::from_float(h[4 * t + j + e]);
          if (a.y) static_cast<T*>(a.y)[row * a.cols + c] = E::from_float(y[j + e]);
        }
      }
    }
  }
}

// --------------------------------------------------------------- gradient --

struct NormBwdArgs {
  const void* gy;         // [rows, cols]
  const void* h;          // [rows, cols]
  const void* weight;     // [cols]
  const void* gres;       // [rows, cols] or null
  void* gh;               // [rows, cols]
  float* part;            // [gridDim.x, pitch]: each CTA's share of gw
  int64_t pitch;
  int64_t rows, cols;
  float eps;
};

// The first n elements of the aligned vector at p (any n), the rest 0: by
// predicated words, so that no branch waits for its data.
template <int DT>
__device__ __forceinline__ void load_head(Vec<DT, 8>& v, const typename Elem<DT>::T* p, int n) {
#pragma unroll
  for (int k = 0; k < v.kWords; ++k) {
    const char* q = reinterpret_cast<const char*>(p) + 4 * k;
    if constexpr (DT == kFP32)
      asm volatile("{.reg .pred f; setp.gt.s32 f, %2, 0; mov.b32 %0, 0; @f ld.global.b32 %0, [%1];}"
                   : "=&r"(v.w[k]) : "l"(q), "r"(n - k));
    else
      asm volatile("{.reg .pred f, h; setp.gt.s32 f, %2, 1; setp.eq.s32 h, %2, 1; mov.b32 %0, 0;\n"
                   "@f ld.global.b32 %0, [%1]; @h ld.global.u16 %0, [%1];}"
                   : "=&r"(v.w[k]) : "l"(q), "r"(n - 2 * k));
  }
}

// Elements off..off + 7 (off 1 to 8) of the two vectors a, b.
template <int DT>
__device__ __forceinline__ Vec<DT, 8> between(const Vec<DT, 8>& a, const Vec<DT, 8>& b, int off) {
  constexpr int W = Vec<DT, 8>::kWords;
  uint32_t t[2 * W + 1];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    t[i] = a.w[i];
    t[W + i] = b.w[i];
  }
  t[2 * W] = 0;
#pragma unroll
  for (int e = 8; e * W >= 8; e /= 2)   // elements that are whole words
#pragma unroll
    for (int i = 0; i + e * W / 8 <= 2 * W; ++i) t[i] = off & e ? t[i + e * W / 8] : t[i];
  Vec<DT, 8> v;
#pragma unroll
  for (int i = 0; i < W; ++i)
    v.w[i] = DT == kFP32 ? t[i] : __funnelshift_r(t[i], t[i + 1], (off & 1) * 16);
  return v;
}

// Stores elements lo..hi - 1 of a vector.
template <int DT>
__device__ __forceinline__ void store_part(typename Elem<DT>::T* p, Vec<DT, 8> v, int lo, int hi) {
  using U = typename std::conditional<DT == kFP32, uint32_t, uint16_t>::type;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi)
      reinterpret_cast<U*>(p)[i] = DT == kFP32 ? v.w[i % v.kWords] : v.w[i / 2] >> (16 * (i & 1));
}

// A thread keeps its columns' share of gw in registers (shared memory with four
// vectors a thread in a CTA) over all its rows; WARP: the CTA's eight warps add
// theirs up at the end. (With four vectors a thread the next row's loads do not
// fit the registers and wait; they spill 120 to 192 bytes a thread in a CTA, the
// forward pass 16 and, of floats, 236; fewer vectors up to 88.)
//
// ODD: the columns are no multiple of 8, so that rows start at any element of a
// vector of the memory (mx_rowvec.h). A row's first and last vector hold elements
// of its neighbours, which are masked: in place, another CTA may be writing those
// meanwhile. Reads stop at the matrix's end. A thread takes rows a multiple of 8
// apart (the launch sees to that), whose shifts are the same, and so keeps its
// columns. (4097 x 3001: 26.2 us, 85 with an element at a time; 4 x 6940 5.6 us
// for 7.7; 5324 x 355 11.2 for 14.1. Loads that a branch had to wait for cost
// 0.7 us each.)
template <int DT, int NV, bool WARP, bool ODD>
__global__ void __launch_bounds__(WARP || NV == 1 ? 256 : 512, NV == 1 ? 3 : WARP && NV == 2 ? 2 : 1)
    norm_bwd_kernel(const NormBwdArgs a) {
  using T = typename Elem<DT>::T;
  constexpr bool kAhead = NV <= 2;
  constexpr bool kShared = NV > 2 && !WARP;    // gw: [NV][2][threads] of float4
  __shared__ float red[2][64];
  extern __shared__ __align__(16) float4 sh_gw[];
  const RowThreads<WARP> rt;
  const int tid = rt.tid, nt = rt.nt;
  dependent_launch();
  dependent_wait();
  const int cols = static_cast<int>(a.cols);
  const RowVectors<ODD> vecs(a.rows, a.cols, rt.first);
  const int nvec = vecs.count;
  const auto read = [&](Vec<DT, 8>& v, const void* p, int64_t row, int i) {
    const T* q = static_cast<const T*>(p) + vecs.at(row, i);
    if (vecs.cut(row, i)) load_head(v, q, vecs.held(row, i));
    else v.load(q);
  };
  // The elements of other rows, as 0: once they are there, so that no load waits.
  const auto mask = [&](Vec<DT, 8>& v, int i) {
    if (!vecs.whole(i)) v.keep(vecs.lo(i), vecs.hi(i));
  };
  float gw[kShared ? 1 : NV][8];
  Vec<DT, 8> wv[NV], gv[NV], hv[NV];
  const auto load = [&](int64_t row, Vec<DT, 8>(&g)[NV], Vec<DT, 8>(&h)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * nt;
      g[j].zero();
      h[j].zero();
      if (i < nvec && row < a.rows) {
        read(g[j], a.gy, row, i);
        read(h[j], a.h, row, i);
      }
    }
  };
  if (kAhead) load(rt.first, gv, hv);
  Vec<DT, 8> wn[ODD ? NV : 1];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    const T* p = static_cast<const T*>(a.weight) + 8 * i;
    wv[j].zero();
    if constexpr (ODD) wn[j].zero();
    if (i < nvec) {
      if constexpr (ODD) {
        if (i > 0) {
          if (8 * i <= cols) wv[j].load(p - 8);
          else load_head(wv[j], p - 8, cols - 8 * i + 8);
        }
        if (8 * i + 8 <= cols) wn[j].load(p);
        else load_head(wn[j], p, cols - 8 * i);
      } else {
        wv[j].load(p);
      }
    }
    if constexpr (kShared) {
      sh_gw[(2 * j) * nt + tid] = sh_gw[(2 * j + 1) * nt + tid] = make_float4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[j][e] = 0.0f;
    }
  }
  if constexpr (ODD)
#pragma unroll
    for (int j = 0; j < NV; ++j) wv[j] = between<DT>(wv[j], wn[j], 8 - vecs.shift);
  int par = 0;
  for (int64_t row = rt.first; row < a.rows; row += rt.step, par ^= 1) {
    Vec<DT, 8> gn[NV], hn[NV], rv[NV];
    if (kAhead) load(row + rt.step, gn, hn);
    else load(row, gv, hv);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * nt;
      rv[j].zero();
      if (a.gres && i < nvec) read(rv[j], a.gres, row, i);
    }
    if constexpr (ODD) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        mask(gv[j], tid + j * nt);
        mask(hv[j], tid + j * nt);
      }
    }
    float s[2] = {0.0f, 0.0f};   // sum h^2, sum gy w h
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = hv[j].get(e);
        s[0] = fmaf(h, h, s[0]);
        s[1] = fmaf(gv[j].get(e) * wv[j].get(e), h, s[1]);
      }
    rt.sum(s, red, par);
    const float r = row_rstd(s[0], a.cols, a.eps);
    const float c = __fdiv_rn(s[1] * r, static_cast<float>(a.cols));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * nt;
      float o[8];
      float* w = gw[kShared ? 0 : j];
      if constexpr (kShared) {
        const float4 lo = sh_gw[(2 * j) * nt + tid], hi = sh_gw[(2 * j + 1) * nt + tid];
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
        w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = hv[j].get(e) * r, g = gv[j].get(e);
        w[e] = fmaf(g, n, w[e]);
        o[e] = fmaf(r, fmaf(-n, c, g * wv[j].get(e)), rv[j].get(e));
      }
      if constexpr (kShared) {
        sh_gw[(2 * j) * nt + tid] = make_float4(w[0], w[1], w[2], w[3]);
        sh_gw[(2 * j + 1) * nt + tid] = make_float4(w[4], w[5], w[6], w[7]);
      }
      if (i < nvec) {
        T* out = static_cast<T*>(a.gh) + vecs.at(row, i);
        Vec<DT, 8> ov;
#pragma unroll
        for (int e = 0; e < 4; ++e) ov.set2(e, o[2 * e], o[2 * e + 1]);
        if (vecs.whole(i)) ov.store(out);
        else store_part<DT>(out, ov, vecs.lo(i), vecs.hi(i));
      }
      if (kAhead) {
        gv[j] = gn[j];
        hv[j] = hn[j];
      }
    }
  }
  float* part = a.part + blockIdx.x * a.pitch;
  if constexpr (WARP) {
    // the warps' shares (warp w's shifted by its rows'); ODD: all at once, else
    // vector by vector: [8 warps][32 lanes][8]
    constexpr int kAtOnce = ODD ? NV : 1;
    __shared__ __align__(16) float sh_part[8][kAtOnce * 256 + (ODD ? 8 : 0)];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int j0 = 0; j0 < NV; j0 += kAtOnce) {
      if (j0) __syncthreads();
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sh_part[warp][j * 256 + tid * 8 + e] = gw[j0 + j][e];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int at = j * 256 + threadIdx.x, c = j0 * 256 + at;
        if (c >= cols) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += sh_part[w][at + (ODD ? w * cols & 7 : 0)];
        part[c] = sum;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * nt;
      if (i < nvec) {
        float4* p = reinterpret_cast<float4*>(part + 8 * i);   // (ODD: shifted as the row is)
        if constexpr (kShared) {
          p[0] = sh_gw[(2 * j) * nt + tid];
          p[1] = sh_gw[(2 * j + 1) * nt + tid];
        } else {
          p[0] = make_float4(gw[j][0], gw[j][1], gw[j][2], gw[j][3]);
          p[1] = make_float4(gw[j][4], gw[j][5], gw[j][6], gw[j][7]);
        }
      }
    }
  }
}

// Any number of columns at any alignment, element tid + nt j in thread tid: up
// to 8 nt columns in registers (nt: 256 threads, 512 or 1024 for long rows);
// beyond, a row is read twice and a thread adds to its columns of the CTA's
// share of gw in memory.
template <int DT>
__global__ void __launch_bounds__(1024, 1) norm_bwd_any_kernel(const NormBwdArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int NJ = 8;
  __shared__ float red[2][64];
  dependent_launch();
  dependent_wait();
  const RowThreads<false> rt;
  const int tid = rt.tid, nt = rt.nt;
  const T* w = static_cast<const T*>(a.weight);
  float* part = a.part + blockIdx.x * a.pitch;
  float gw[NJ], wv[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    gw[j] = 0.0f;
    wv[j] = tid + nt * j < a.cols ? E::to_float(w[tid + nt * j]) : 0.0f;
  }
  int par = 0;
  for (int64_t row = rt.first; row < a.rows; row += rt.step, par ^= 1) {
    const T* gy = static_cast<const T*>(a.gy) + row * a.cols;
    const T* hh = static_cast<const T*>(a.h) + row * a.cols;
    const T* gres = a.gres ? static_cast<const T*>(a.gres) + row * a.cols : nullptr;
    T* gh = static_cast<T*>(a.gh) + row * a.cols;
    float g[NJ], h[NJ], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = tid + nt * j;
      g[j] = c < a.cols ? E::to_float(gy[c]) : 0.0f;
      h[j] = c < a.cols ? E::to_float(hh[c]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[0] = fmaf(h[j], h[j], s[0]);
      s[1] = fmaf(g[j] * wv[j], h[j], s[1]);
    }
    for (int64_t c = tid + nt * NJ; c < a.cols; c += nt) {
      const float v = E::to_float(hh[c]);
      s[0] = fmaf(v, v, s[0]);
      s[1] = fmaf(E::to_float(gy[c]) * E::to_float(w[c]), v, s[1]);
    }
    rt.sum(s, red, par);
    const float r = row_rstd(s[0], a.cols, a.eps);
    const float m = __fdiv_rn(s[1] * r, static_cast<float>(a.cols));
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = tid + nt * j;
      const float n = h[j] * r;
      gw[j] = fmaf(g[j], n, gw[j]);
      if (c < a.cols)
        gh[c] = E::from_float(fmaf(r, fmaf(-n, m, g[j] * wv[j]), gres ? E::to_float(gres[c]) : 0.0f));
    }
    for (int64_t c = tid + nt * NJ; c < a.cols; c += nt) {
      const float n = E::to_float(hh[c]) * r, v = E::to_float(gy[c]);
      part[c] = fmaf(v, n, row == blockIdx.x ? 0.0f : part[c]);
      gh[c] = E::from_float(
          fmaf(r, fmaf(-n, m, v * E::to_float(w[c])), gres ? E::to_float(gres[c]) : 0.0f));
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    if (tid + nt * j < a.cols) part[tid + nt * j] = gw[j];
}

// gw[c] = sum of the CTAs' shares, in an order that depends on their number
// alone: C threads side by side take C columns of every (1024 / C)th share, then
// a warp adds up each column. Bound by latency: C is the smallest (8, 16 or 32)
// that gives no SM a second CTA (1999 x 2048, 592 shares: 16 columns 9.5 us with
// the first kernel, 32 10.6; 700 x 8192: 16 columns 13.8 us, 32 12.4).
// `shifted`: share p starts at element p cols mod 8.
template <int C>
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int nparts, int64_t pitch,
                                                            int64_t cols, bool shifted, float* gw) {
  constexpr int kGroups = 1024 / C;
  __shared__ float red[C][kGroups + 1];
  const int col = threadIdx.x % C, group = threadIdx.x / C;
  dependent_launch();
  dependent_wait();
  const int64_t c = blockIdx.x * int64_t(C) + col;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = group; p < nparts; p += kGroups)
      s += part[p * pitch + c + (shifted ? p * static_cast<int>(cols) & 7 : 0)];
  }
  red[col][group] = s;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= C) return;
  s = red[warp][lane];
#pragma unroll
  for (int i = 32; i < kGroups; i += 32) s += red[warp][lane + i];
  s = warp_sum(s);
  const int64_t o = blockIdx.x * int64_t(C) + warp;
  if (lane == 0 && o < cols) gw[o] = s;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// How a row of nvec vectors is spread: up to 1024 elements one warp (one, two
// or four vectors a lane), up to 8192 a CTA with two vectors a thread, up to
// 16384 four (512 threads at most); beyond, the kernel for any size. A few rows
// of 256 to 2048 elements take a CTA each with one vector a thread: what counts
// is one row's time (forward 1 x 2048: 1.8 us, 2.06 with two vectors, but 16387 x
// 2048 44.3 us, 40.5 with two; gradient 1 x 1000: 2.7 us, 3.45 with one warp).
constexpr int64_t kMaxVecCols = 16384;
struct Shape {
  bool warp;
  int nv;
  unsigned nt;
};
Shape shape_of(int64_t nvec, int64_t rows, int sms) {
  const bool few = rows <= 4 * sms;
  if (nvec <= 32 || (nvec <= 128 && !few)) return {true, nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4, 256};
  const int nv = nvec <= 256 && few ? 1 : nvec <= 1024 ? 2 : 4;
  return {false, nv, static_cast<unsigned>(((nvec + nv - 1) / nv + 31) / 32 * 32)};
}

// CTAs for `rows` rows with at most `threads` threads on an SM: what the
// registers of the kernels' launch bounds allow. Some compiled kernels need more
// than that, and half of their CTAs run as a second wave: the forward pass of
// 4104 to 5632 columns (120 registers, two CTAs of 288 to 352 threads asked for,
// one fits), of 520 to 1024 (192) and of floats of 264 to 512 (136).
int64_t grid_for(const Shape& s, int64_t rows, int sms, int threads) {
  const int per_sm = threads / static_cast<int>(s.nt);
  const int64_t most = static_cast<int64_t>(sms) * (per_sm < 1 ? 1 : per_sm);
  const int64_t need = s.warp ? (rows + 7) / 8 : rows;
  return need < most ? need : most;
}

template <int DT, bool E5M2>
cudaError_t launch_norm(const NormArgs& a, bool vec, int sms, cudaStream_t st) {
  // (a few rows: a CTA each, since what counts is one row's time)
  if (!vec && a.cols <= 1024 && a.rows > 4 * sms) {
    const auto kern = a.cols <= 256   ? norm128_any_warp_kernel<DT, E5M2, 8>
                      : a.cols <= 512 ? norm128_any_warp_kernel<DT, E5M2, 16>
                                      : norm128_any_warp_kernel<DT, E5M2, 32>;
    return launch_dependent(kern, dim3(static_cast<unsigned>((a.rows + 7) / 8)), dim3(256), 0, st, 1, a);
  }
  if (!vec) {
    const auto kern = a.cols <= 1024   ? norm128_any_kernel<DT, E5M2, 4>
                      : a.cols <= 2048 ? norm128_any_kernel<DT, E5M2, 8>
                                       : norm128_any_kernel<DT, E5M2, 16>;
    return launch_dependent(kern, dim3(static_cast<unsigned>(a.rows)), dim3(256), 0, st, 1, a);
  }
  const Shape s = shape_of((a.cols + 15) / 16 * 2, a.rows, sms);   // with the codes' padding
  const bool half = !s.warp && s.nv == 2 && s.nt <= 256;
  const auto kern = s.warp ? (s.nv == 1   ? norm128_kernel<DT, E5M2, 1, true>
                              : s.nv == 2 ? norm128_kernel<DT, E5M2, 2, true>
                                          : norm128_kernel<DT, E5M2, 4, true>)
                           : (s.nv == 1   ? norm128_kernel<DT, E5M2, 1, false>
                              : half      ? norm128_kernel<DT, E5M2, 2, false, true>
                              : s.nv == 2 ? norm128_kernel<DT, E5M2, 2, false>
                                          : norm128_kernel<DT, E5M2, 4, false>);
  const int64_t grid = grid_for(s, a.rows, sms, s.nv == 1   ? 1024
                                                : half      ? (DT == kFP32 ? 512 : 768)
                                                : s.nv == 2 ? 704 : 512);
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(s.nt), 0, st, 1, a);
}

template <int DT, bool ODD>
cudaError_t launch_bwd_vec(const NormBwdArgs& a, const Shape& s, int64_t grid, cudaStream_t st) {
  const auto kern = s.warp ? (s.nv == 1   ? norm_bwd_kernel<DT, 1, true, ODD>
                              : s.nv == 2 ? norm_bwd_kernel<DT, 2, true, ODD>
                                          : norm_bwd_kernel<DT, 4, true, ODD>)
                           : (s.nv == 1   ? norm_bwd_kernel<DT, 1, false, ODD>
                              : s.nv == 2 ? norm_bwd_kernel<DT, 2, false, ODD>
                                          : norm_bwd_kernel<DT, 4, false, ODD>);
  const size_t smem = !s.warp && s.nv == 4 ? s.nt * size_t(4 * 8 * 4) : 0;   // up to 64 KiB
  if (smem) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 512 * 4 * 8 * 4);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(s.nt), smem, st, 1, a);
}

template <int DT>
cudaError_t launch_bwd(const NormBwdArgs& a, bool vec, int sms, float* gw, cudaStream_t st) {
  const bool odd = a.cols % 8 != 0;
  const Shape s = shape_of(odd ? (a.cols + 14) / 8 : a.cols / 8, a.rows, sms);
  int64_t grid;
  cudaError_t e;
  if (vec) {
    grid = grid_for(s, a.rows, sms, s.nv == 1 ? 768 : s.nv == 4 && s.warp ? 256 : 512);
    if (grid > kNormParts) grid = kNormParts;
    // rows a multiple of 8 apart to a CTA (a warp's are)
    if (odd && !s.warp && grid < a.rows) grid = grid / 8 * 8;
    e = odd ? launch_bwd_vec<DT, true>(a, s, grid, st) : launch_bwd_vec<DT, false>(a, s, grid, st);
  } else {
    const int nt = a.cols <= 2048 ? 256 : a.cols <= 4096 ? 512 : 1024;
    const int64_t most = static_cast<int64_t>(1024 / nt) * sms;
    grid = a.rows < most ? a.rows : most;
    if (grid > kNormParts) grid = kNormParts;
    e = launch_dependent(norm_bwd_any_kernel<DT>, dim3(static_cast<unsigned>(grid)), dim3(nt), 0, st, 1, a);
  }
  if (e != cudaSuccess) return e;
  const int c = a.cols <= 8 * sms ? 8 : a.cols <= 16 * sms ? 16 : 32;
  const auto kern = c == 8 ? norm_bwd_sum_kernel<8> : c == 16 ? norm_bwd_sum_kernel<16> : norm_bwd_sum_kernel<32>;
  return launch_dependent(kern, dim3(static_cast<unsigned>((a.cols + c - 1) / c)), dim3(1024), 0, st, 1,
                          static_cast<const float*>(a.part), static_cast<int>(grid), a.pitch, a.cols,
                          vec && odd && !s.warp, gw);
}

cudaError_t device_sms(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

cudaError_t launch_norm128(const void* x, int64_t ldx, const void* residual, const void* weight,
                           int dtype, int64_t rows, int64_t cols, float eps, bool e5m2, bool pow2,
                           void* h, void* y, uint8_t* codes, int64_t ldc, float* scales,
                           int64_t lds, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.weight = weight;
  a.h = h;
  a.y = y;
  a.codes = codes;
  a.ldc = ldc;
  a.scales = scales;
  a.lds = lds;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.pow2 = pow2;
  const int64_t bytes = dtype == kFP32 ? 4 : 2;
  const bool vec = cols % 8 == 0 && cols <= kMaxVecCols && aligned16(x) && aligned16(residual) &&
                   aligned16(weight) && aligned16(h) && aligned16(y) &&
                   (rows == 1 || ldx * bytes % 16 == 0);
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  switch (dtype * 2 + (e5m2 ? 1 : 0)) {
    case 0: return launch_norm<kBF16, false>(a, vec, sms, st);
    case 1: return launch_norm<kBF16, true>(a, vec, sms, st);
    case 2: return launch_norm<kFP16, false>(a, vec, sms, st);
    case 3: return launch_norm<kFP16, true>(a, vec, sms, st);
    case 4: return launch_norm<kFP32, false>(a, vec, sms, st);
    default: return launch_norm<kFP32, true>(a, vec, sms, st);
  }
}

cudaError_t launch_norm_bwd(const void* gy, const void* h, const void* weight, const void* gres,
                            int dtype, int64_t rows, int64_t cols, float eps, void* gh, float* gw,
                            float* part, cudaStream_t st) {
  NormBwdArgs a{};
  a.gy = gy;
  a.h = h;
  a.weight = weight;
  a.gres = gres;
  a.gh = gh;
  a.part = part;
  a.pitch = norm_part_pitch(cols);
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  const bool odd = cols % 8 != 0;
  const bool vec = cols <= kMaxVecCols - (odd ? 14 : 0) && aligned16(gy) && aligned16(h) &&
                   aligned16(weight) && aligned16(gres) && aligned16(gh) && aligned16(part);
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  switch (dtype) {
    case kBF16: return launch_bwd<kBF16>(a, vec, sms, gw, st);
    case kFP16: return launch_bwd<kFP16>(a, vec, sms, gw, st);
    default: return launch_bwd<kFP32>(a, vec, sms, gw, st);
  }
}

}  // namespace mxk
