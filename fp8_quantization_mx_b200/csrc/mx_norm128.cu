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
// row is read once into registers, 8 elements per lane, and written once.

#include <cuda_runtime.h>

#include "mx_launch.h"
#include "mx_pdl.cuh"
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

template <bool E5M2>
__device__ __forceinline__ uint2 encode8(const float (&y)[8], const Divisor& d) {
  const float2 s = make_float2(d.s, d.s), inv = make_float2(d.inv, d.inv);
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = make_float2(y[2 * i], y[2 * i + 1]);
    if (d.slow) x = __fmul2_rn(x, make_float2(kLift, kLift));
    q[i] = div2(x, s, inv);
  }
  return make_uint2(enc4<E5M2>(q[0].x, q[0].y, q[1].x, q[1].y),
                    enc4<E5M2>(q[2].x, q[2].y, q[3].x, q[3].y));
}

// One CTA per row, NV vectors of 8 elements per thread: the vectors of a tile
// are 16 neighbouring lanes' (four shuffles give its largest magnitude).
template <int DT, bool E5M2, int NV>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512) norm128_kernel(const NormArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ float red[32];
  const int tid = threadIdx.x, nt = blockDim.x;
  dependent_launch();
  dependent_wait();
  const int64_t row = blockIdx.x;
  const int nvec = static_cast<int>(a.cols / 8);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;

  Vec<DT, 8> xv[NV], rv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    xv[j].zero();
    rv[j].zero();
    if (i < nvec) {
      xv[j].load(x + 8 * i);
      if (res) rv[j].load(res + 8 * i);
    }
  }
  Vec<DT, 8> wv[NV];
  float h[NV][8];
  float ss[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    wv[j].zero();
    if (i < nvec) wv[j].load(static_cast<const T*>(a.weight) + 8 * i);
    float p = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[j][e] = xv[j].get(e) + rv[j].get(e);
      p = fmaf(h[j][e], h[j][e], p);
    }
    ss[0] += p;
    if (a.h && i < nvec) {
      Vec<DT, 8> o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o.set2(e, h[j][2 * e], h[j][2 * e + 1]);
      o.store(static_cast<T*>(a.h) + row * a.cols + 8 * i);
    }
  }
  block_sum(ss, red);
  const float r = row_rstd(ss[0], a.cols, a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    float y[8], m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = h[j][e] * r * wv[j].get(e);
      m = amax2(m, y[e]);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = amax2(m, __shfl_xor_sync(~0u, m, o));
    const float s = tile_scale<E5M2>(m, a.pow2);
    const uint2 c = encode8<E5M2>(y, divisor(s, m == 0.0f));
    // codes up to the row's padding to 16 bytes (the vector past the last is 0)
    if (8 * static_cast<int64_t>(i) < ((a.cols + 15) & ~int64_t(15)))
      *reinterpret_cast<uint2*>(a.codes + row * a.ldc + 8 * i) = c;
    if (i < nvec) {
      if ((i & 15) == 0) a.scales[(i >> 4) * a.lds + row] = s;
      if (a.y) {
        Vec<DT, 8> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.set2(e, y[2 * e], y[2 * e + 1]);
        o.store(static_cast<T*>(a.y) + row * a.cols + 8 * i);
      }
    }
  }
}

// Any number of columns at any alignment: the row is read twice (the second
// time mostly from cache); one warp per tile, 4 elements per lane.
template <int DT, bool E5M2>
__global__ void __launch_bounds__(256) norm128_any_kernel(const NormArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependent_launch();
  dependent_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  float ss[1] = {0.0f};
  for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
    const float v = E::to_float(x[c]) + (res ? E::to_float(res[c]) : 0.0f);
    ss[0] = fmaf(v, v, ss[0]);
  }
  block_sum(ss, red);
  const float r = row_rstd(ss[0], a.cols, a.eps);
  const int64_t pitch = (a.cols + 15) & ~int64_t(15);
  for (int64_t t = warp; t < (a.cols + 127) / 128; t += 8) {
    const int64_t c0 = t * 128 + 4 * lane;
    float h[4], y[4], m = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = y[e] = 0.0f;
      if (c0 + e < a.cols) {
        h[e] = E::to_float(x[c0 + e]) + (res ? E::to_float(res[c0 + e]) : 0.0f);
        y[e] = h[e] * r * E::to_float(w[c0 + e]);
      }
      m = amax2(m, y[e]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = amax2(m, __shfl_xor_sync(~0u, m, o));
    const float s = tile_scale<E5M2>(m, a.pow2);
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = __fdiv_rn(y[e], s);
    if (c0 < pitch)
      *reinterpret_cast<uint32_t*>(a.codes + row * a.ldc + c0) = enc4<E5M2>(q[0], q[1], q[2], q[3]);
    if (lane == 0) a.scales[t * a.lds + row] = s;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c0 + e < a.cols) {
        if (a.h) static_cast<T*>(a.h)[row * a.cols + c0 + e] = E::from_float(h[e]);
        if (a.y) static_cast<T*>(a.y)[row * a.cols + c0 + e] = E::from_float(y[e]);
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
  float* part;            // [gridDim.x, cols]: each CTA's share of gw
  int64_t rows, cols;
  float eps;
};

// CTA b takes rows b, b + gridDim.x, ...; a thread keeps its columns' share of
// gw in registers (shared memory with four vectors a thread) over all of them. The next row's loads are issued before
// this row's sums, so that HBM is busy across the barrier (not with four
// vectors a thread, whose registers the next row would not fit).
template <int DT, int NV>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512) norm_bwd_kernel(const NormBwdArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ float red[2][64];
  const int tid = threadIdx.x, nt = blockDim.x;
  dependent_launch();
  dependent_wait();
  const int nvec = static_cast<int>(a.cols / 8);
  const T* gy = static_cast<const T*>(a.gy);
  const T* hh = static_cast<const T*>(a.h);
  constexpr bool kAhead = NV <= 2;
  constexpr bool kShared = NV > 2;    // gw in shared memory: [NV][2][threads] of float4
  extern __shared__ __align__(16) float4 sh_gw[];
  float gw[kShared ? 1 : NV][8];
  Vec<DT, 8> wv[NV], gv[NV], hv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    wv[j].zero();
    gv[j].zero();
    hv[j].zero();
    if (i < nvec) {
      wv[j].load(static_cast<const T*>(a.weight) + 8 * i);
      if (kAhead) {
        gv[j].load(gy + blockIdx.x * a.cols + 8 * i);
        hv[j].load(hh + blockIdx.x * a.cols + 8 * i);
      }
    }
    if constexpr (kShared) {
      sh_gw[(2 * j) * nt + tid] = sh_gw[(2 * j + 1) * nt + tid] = make_float4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[j][e] = 0.0f;
    }
  }
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const int64_t next = row + gridDim.x;
    Vec<DT, 8> gn[NV], hn[NV], rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * nt;
      gn[j].zero();
      hn[j].zero();
      rv[j].zero();
      if (i < nvec) {
        if (a.gres) rv[j].load(static_cast<const T*>(a.gres) + row * a.cols + 8 * i);
        if (!kAhead) {
          gv[j].load(gy + row * a.cols + 8 * i);
          hv[j].load(hh + row * a.cols + 8 * i);
        } else if (next < a.rows) {
          gn[j].load(gy + next * a.cols + 8 * i);
          hn[j].load(hh + next * a.cols + 8 * i);
        }
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
    // (two buffers: the next row's sums may start while a warp reads these)
    block_sum(s, red[par]);
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
        Vec<DT, 8> ov;
#pragma unroll
        for (int e = 0; e < 4; ++e) ov.set2(e, o[2 * e], o[2 * e + 1]);
        ov.store(static_cast<T*>(a.gh) + row * a.cols + 8 * i);
      }
      if (kAhead) {
        gv[j] = gn[j];
        hv[j] = hn[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * nt;
    if (i < nvec) {
      float4* p = reinterpret_cast<float4*>(a.part + blockIdx.x * a.cols + 8 * i);
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

// Any number of columns at any alignment: each thread adds to its own columns
// of the CTA's share of gw in memory.
template <int DT>
__global__ void __launch_bounds__(256) norm_bwd_any_kernel(const NormBwdArgs a) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float red[2][64];
  dependent_launch();
  dependent_wait();
  const T* w = static_cast<const T*>(a.weight);
  float* part = a.part + blockIdx.x * a.cols;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const T* gy = static_cast<const T*>(a.gy) + row * a.cols;
    const T* hh = static_cast<const T*>(a.h) + row * a.cols;
    const T* gres = a.gres ? static_cast<const T*>(a.gres) + row * a.cols : nullptr;
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
      const float h = E::to_float(hh[c]);
      s[0] = fmaf(h, h, s[0]);
      s[1] = fmaf(E::to_float(gy[c]) * E::to_float(w[c]), h, s[1]);
    }
    block_sum(s, red[par]);
    const float r = row_rstd(s[0], a.cols, a.eps);
    const float m = __fdiv_rn(s[1] * r, static_cast<float>(a.cols));
    for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
      const float n = E::to_float(hh[c]) * r, g = E::to_float(gy[c]);
      part[c] = fmaf(g, n, row == blockIdx.x ? 0.0f : part[c]);
      static_cast<T*>(a.gh)[row * a.cols + c] = E::from_float(
          fmaf(r, fmaf(-n, m, g * E::to_float(w[c])), gres ? E::to_float(gres[c]) : 0.0f));
    }
  }
}

// gw[c] = sum of the CTAs' shares, in an order that depends on their number
// alone: 8 warps take every eighth share of 32 columns, then add up.
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const float* part, int nparts,
                                                           int64_t cols, float* gw) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependent_launch();
  dependent_wait();
  const int64_t c = blockIdx.x * int64_t(32) + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = warp; p < nparts; p += 8) s += part[p * cols + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    gw[c] = s;
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Vectors of 8 per thread and threads per row: one up to 2048 columns (256
// threads), two up to 8192 and four up to 16384 (512 threads; beyond, the
// kernel for any size).
constexpr int64_t kMaxVecCols = 16384;
int vectors(int64_t nvec) { return nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4; }
unsigned threads(int64_t nvec, int nv) {
  return static_cast<unsigned>(((nvec + nv - 1) / nv + 31) / 32 * 32);
}

template <int DT, bool E5M2>
cudaError_t launch_norm(const NormArgs& a, bool vec, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.rows));
  if (!vec) return launch_dependent(norm128_any_kernel<DT, E5M2>, grid, dim3(256), 0, st, 1, a);
  const int64_t nvec = (a.cols + 15) / 16 * 2;   // with the codes' padding
  const int nv = vectors(nvec);
  const auto kern = nv == 1   ? norm128_kernel<DT, E5M2, 1>
                    : nv == 2 ? norm128_kernel<DT, E5M2, 2>
                              : norm128_kernel<DT, E5M2, 4>;
  return launch_dependent(kern, grid, dim3(threads(nvec, nv)), 0, st, 1, a);
}

// CTAs: as many as the SMs hold at once (registers: 768 threads with one
// vector each, else 512), the general kernel's 256-thread CTAs two per SM;
// never more than rows or shares.
template <int DT>
cudaError_t launch_bwd(const NormBwdArgs& a, bool vec, int sms, float* gw, cudaStream_t st) {
  int64_t most = 2 * sms;
  if (vec) {
    const int nv = vectors(a.cols / 8);
    const int per_sm = (nv == 1 ? 768 : 512) / static_cast<int>(threads(a.cols / 8, nv));
    most = static_cast<int64_t>(sms) * (per_sm < 1 ? 1 : per_sm);
  }
  if (most > kNormParts) most = kNormParts;
  const int grid = static_cast<int>(a.rows < most ? a.rows : most);
  cudaError_t e;
  if (!vec) {
    e = launch_dependent(norm_bwd_any_kernel<DT>, dim3(grid), dim3(256), 0, st, 1, a);
  } else {
    const int64_t nvec = a.cols / 8;
    const int nv = vectors(nvec);
    const unsigned nt = threads(nvec, nv);
    const auto kern = nv == 1   ? norm_bwd_kernel<DT, 1>
                      : nv == 2 ? norm_bwd_kernel<DT, 2>
                                : norm_bwd_kernel<DT, 4>;
    const size_t smem = nv == 4 ? nt * size_t(4 * 8 * 4) : 0;   // up to 64 KiB
    if (smem) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 512 * 4 * 8 * 4);
      if (e != cudaSuccess) return e;
    }
    e = launch_dependent(kern, dim3(grid), dim3(nt), smem, st, 1, a);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_bwd_sum_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32)),
                          dim3(256), 0, st, 1, a.part, grid, a.cols, gw);
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
  switch (dtype * 2 + (e5m2 ? 1 : 0)) {
    case 0: return launch_norm<kBF16, false>(a, vec, st);
    case 1: return launch_norm<kBF16, true>(a, vec, st);
    case 2: return launch_norm<kFP16, false>(a, vec, st);
    case 3: return launch_norm<kFP16, true>(a, vec, st);
    case 4: return launch_norm<kFP32, false>(a, vec, st);
    default: return launch_norm<kFP32, true>(a, vec, st);
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
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  const bool vec = cols % 8 == 0 && cols <= kMaxVecCols && aligned16(gy) && aligned16(h) &&
                   aligned16(weight) && aligned16(gres) && aligned16(gh) && aligned16(part);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  switch (dtype) {
    case kBF16: return launch_bwd<kBF16>(a, vec, sms, gw, st);
    case kFP16: return launch_bwd<kFP16>(a, vec, sms, gw, st);
    default: return launch_bwd<kFP32>(a, vec, sms, gw, st);
  }
}

}  // namespace mxk
