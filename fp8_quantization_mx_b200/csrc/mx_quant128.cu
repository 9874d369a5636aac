// FP8 quantization with float scales per 1 x 128 tile or 128 x 128 block,
// along the rows, along the columns (codes of the transposed matrix), or both
// from one read of x.
//
// One CTA of 256 threads takes a 128 x 128 piece of x: thread t holds rows
// 4 (t / 8) .. + 3, columns 16 (t % 8) .. + 15, in registers.
//   rows     a tile is 8 neighbouring lanes, which hold four rows' tiles: each
//            takes one row's largest magnitude and scale (four shuffles), 16
//            codes are one 16-byte store
//   columns  the largest magnitudes of a column over the four rows of a
//            thread, over the warp's four lane groups (an exchange that halves
//            the columns held at each step: 12 shuffles where reducing all 16
//            in every lane takes 32) and, through shared memory, over the eight
//            warps; the four codes of a column are one word, transposed through
//            shared memory (words permuted so that both sides are free of bank
//            conflicts) into 128-byte runs of the transposed codes
//   block    one scale for the piece; its codes are made once, and the
//            transposed codes by byte permutes of four rows' words
// Bound by HBM: x is read once and every code written once. Of bf16, on a B200
// with a copy bandwidth of 6.45 TB/s: 32768 x 4096 along the rows 63.7 us (99% of
// the bytes' time), both ways 103 us (82%; 18.6 instructions per element),
// 49152 x 2048 in blocks both ways 66 us (95%), 4099 x 4096 both ways 17 us
// (62%: 1.8 waves of CTAs, and 3 us of start and end).

#include <cuda_runtime.h>

#include "mx_launch.h"
#include "mx_pdl.cuh"
#include "mx_tile128.cuh"

namespace mxk {

namespace {

using namespace t128;

struct Quant128Args {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t* codes;     // [rows, ldc]
  int64_t ldc;
  float* scales;      // tiles: [ceil(cols/128), lds]; blocks: [ceil(rows/128), ceil(cols/128)]
  int64_t lds;
  uint8_t* codes_t;   // [cols, ldct]
  int64_t ldct;
  float* scales_t;    // tiles: [ceil(rows/128), ldst]; blocks: [ceil(cols/128), ceil(rows/128)]
  int64_t ldst;
  int64_t nbr, nbc;   // pieces along the rows and the columns
  int pow2;
  int vec;            // x and ldx allow 16-byte loads
};

constexpr int kThreads = 256;

// The word of codes of column c (0..127), rows 4g .. 4g + 3, in the transposed
// piece: 32 words a column, permuted by the column's group of 16 so that the
// eight lanes that write a column of their own group hit eight bank quads.
__device__ __forceinline__ int word_at(int c, int g) { return c * 32 + (g ^ (((c >> 4) & 7) << 2)); }

// Where a column's scale sits in the shared arrays: two floats of padding after
// 16 columns, so that the eight groups' pairs are in different banks.
constexpr int kPadded = 128 + 16;
__device__ __forceinline__ int col_at(int c) { return c + (c >> 4) * 2; }

template <bool E5M2, bool SLOW, int DT>
__device__ __forceinline__ uint4 encode_row(const Vec<DT, 16>& v, const Divisor& d) {
  uint32_t o[4];
  const float2 s = make_float2(d.s, d.s), ninv = make_float2(d.ninv, d.ninv);
  const float2 lift = make_float2(kLift, kLift);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = div2(SLOW ? __fmul2_rn(v.neg2(2 * i), lift) : v.neg2(2 * i), s, ninv);
    const float2 b = div2(SLOW ? __fmul2_rn(v.neg2(2 * i + 1), lift) : v.neg2(2 * i + 1), s, ninv);
    o[i] = enc4<E5M2>(a.x, a.y, b.x, b.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// col_s, col_ninv: of the piece's columns, lifted where the scale is tiny (SLOW
// takes notice).
template <bool E5M2, bool SLOW, int DT>
__device__ __forceinline__ void encode_cols(const Vec<DT, 16> (&v)[4], const float* col_s,
                                            const float* col_ninv, const float* col_lift, int g,
                                            int sub, uint32_t* out) {
#pragma unroll
  for (int c2 = 0; c2 < 8; ++c2) {
    const int at = col_at(sub * 16 + 2 * c2);
    const float2 s = *reinterpret_cast<const float2*>(col_s + at);
    const float2 ninv = *reinterpret_cast<const float2*>(col_ninv + at);
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x = v[i].neg2(c2);
      if constexpr (SLOW) x = __fmul2_rn(x, *reinterpret_cast<const float2*>(col_lift + at));
      q[i] = div2(x, s, ninv);
    }
    out[word_at(sub * 16 + 2 * c2, g)] = enc4<E5M2>(q[0].x, q[1].x, q[2].x, q[3].x);
    out[word_at(sub * 16 + 2 * c2 + 1, g)] = enc4<E5M2>(q[0].y, q[1].y, q[2].y, q[3].y);
  }
}

// CTAs per SM that the registers are cut for. What hides a piece's load, sums
// and stores is other CTAs: 32768 x 4096 both ways took 148, 123, 110, 110 us
// with 2 to 5 of them (before the scales were shared out over the lanes: 103
// with 4). Floats, twice the registers of x, spill 8 to 32 bytes a thread with 3.
// One CTA that loads the next piece ahead, at 2
// per SM: 152 us.
template <int DT>
constexpr int ctas_per_sm() {
  return DT == kFP32 ? 3 : 4;
}

template <int DT, bool E5M2, bool ROWS, bool COLS, bool BLOCK>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<DT>()) quant128_kernel(const Quant128Args a) {
  using T = typename Elem<DT>::T;
  __shared__ __align__(16) uint32_t sh_codes[COLS ? 128 * 32 : 4];
  __shared__ __align__(16) float sh_red[8][BLOCK || !COLS ? 4 : 128];
  constexpr int kCols = COLS && !BLOCK ? kPadded : 2;
  __shared__ __align__(16) float sh_s[kCols], sh_ninv[kCols], sh_lift[kCols];
  __shared__ int sh_slow;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = tid >> 3, sub = tid & 7;
  dependent_launch();
  dependent_wait();
  const int64_t rb = blockIdx.x / a.nbc, cb = blockIdx.x % a.nbc;
  const int64_t row0 = rb * 128 + 4 * g, col0 = cb * 128 + 16 * sub;

  // a shifted load reads up to 15 bytes around its elements: within x only
  const T* first = static_cast<const T*>(a.x) + 16;
  const T* past = static_cast<const T*>(a.x) + (a.rows - 1) * a.ldx + a.cols;
  Vec<DT, 16> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T* p = static_cast<const T*>(a.x) + (row0 + i) * a.ldx + col0;
    if (row0 + i >= a.rows || col0 >= a.cols)
      v[i].zero();
    else if (a.vec && col0 + 16 <= a.cols)
      v[i].load(p);
    else if (col0 + 16 <= a.cols && p >= first && p + 32 <= past)
      v[i].load_shifted(p);
    else
      v[i].load_some(p, a.cols - col0);
  }

  uint4 rcodes[4];   // BLOCK: the four rows' codes
  if constexpr (BLOCK) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = amax2(m, v[i].amax());
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = amax2(m, __shfl_xor_sync(~0u, m, o));
    if (lane == 0) sh_red[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = amax2(m, sh_red[w][0]);
    const float s = tile_scale<E5M2>(m, a.pow2);
    const Divisor d = divisor(s, m == 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rcodes[i] = d.slow ? encode_row<E5M2, true, DT>(v[i], d) : encode_row<E5M2, false, DT>(v[i], d);
    if (tid == 0) {
      if (ROWS) a.scales[rb * a.nbc + cb] = s;
      if (COLS) a.scales_t[cb * a.nbr + rb] = s;
    }
  }

  if constexpr (ROWS) {
    Divisor mine{};
    if constexpr (!BLOCK) {
      // a tile is eight lanes; each of them takes one of the four rows' scale
      float m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = v[i].amax();
      float mm = spread_max(m, lane);
      mm = amax2(mm, __shfl_xor_sync(~0u, mm, 4));
      const float s = tile_scale<E5M2>(mm, a.pow2);
      mine = divisor(s, mm == 0.0f);
      // (lds >= rows rounded up to 4)
      if (sub < 4 && row0 < a.rows) a.scales[cb * a.lds + row0 + held_by<4>(lane)] = s;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 codes;
      if constexpr (BLOCK) {
        codes = rcodes[i];
      } else {
        const Divisor d = divisor_of(mine, (lane & 24) | lane_of<4>(i));
        codes = d.slow ? encode_row<E5M2, true, DT>(v[i], d) : encode_row<E5M2, false, DT>(v[i], d);
      }
      // (a row's 16-byte piece ends within the row's padding to 16 bytes)
      if (row0 + i < a.rows && col0 < a.cols)
        *reinterpret_cast<uint4*>(a.codes + (row0 + i) * a.ldc + col0) = codes;
    }
  }

  if constexpr (COLS) {
    if constexpr (BLOCK) {
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t r[4];   // four codes of each of the four rows
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r[i] = c4 == 0 ? rcodes[i].x : c4 == 1 ? rcodes[i].y : c4 == 2 ? rcodes[i].z : rcodes[i].w;
        const uint32_t ab = __byte_perm(r[0], r[1], 0x5140);   // a0 b0 a1 b1
        const uint32_t AB = __byte_perm(r[0], r[1], 0x7362);   // a2 b2 a3 b3
        const uint32_t cd = __byte_perm(r[2], r[3], 0x5140);
        const uint32_t CD = __byte_perm(r[2], r[3], 0x7362);
        const int c = sub * 16 + 4 * c4;
        sh_codes[word_at(c, g)] = __byte_perm(ab, cd, 0x5410);
        sh_codes[word_at(c + 1, g)] = __byte_perm(ab, cd, 0x7632);
        sh_codes[word_at(c + 2, g)] = __byte_perm(AB, CD, 0x5410);
        sh_codes[word_at(c + 3, g)] = __byte_perm(AB, CD, 0x7632);
      }
    } else {
      // each step keeps half of the columns held: lane bit 3 columns 8-15 of
      // the 16, then lane bit 4 the upper four of those eight
      const bool hi8 = lane & 8, hi4 = lane & 16;
      float q[4];
      if constexpr (DT == kFP32) {
        float m[16], h[8];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          m[c] = fabsf(v[0].get(c));
#pragma unroll
          for (int i = 1; i < 4; ++i) m[c] = amax2(m[c], v[i].get(c));
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          h[c] = amax2(hi8 ? m[c + 8] : m[c], __shfl_xor_sync(~0u, hi8 ? m[c] : m[c + 8], 8));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          q[c] = amax2(hi4 ? h[c + 4] : h[c], __shfl_xor_sync(~0u, hi4 ? h[c] : h[c + 4], 16));
      } else {
        uint32_t m[8], h[4];   // pairs of columns
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          m[c] = v[0].w[c];
#pragma unroll
          for (int i = 1; i < 4; ++i) m[c] = amax_pair<DT>(m[c], v[i].w[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          h[c] = amax_pair<DT>(hi8 ? m[c + 4] : m[c], __shfl_xor_sync(~0u, hi8 ? m[c] : m[c + 4], 8));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          Vec<DT, 8> t;
          t.w[0] = amax_pair<DT>(hi4 ? h[c + 2] : h[c],
                                 __shfl_xor_sync(~0u, hi4 ? h[c] : h[c + 2], 16)) & 0x7fff7fffu;
          q[2 * c] = t.get(0);
          q[2 * c + 1] = t.get(1);
        }
      }
      if (tid == 0) sh_slow = 0;
      const int c0 = sub * 16 + (hi8 ? 8 : 0) + (hi4 ? 4 : 0);
      *reinterpret_cast<float4*>(&sh_red[warp][c0]) = make_float4(q[0], q[1], q[2], q[3]);
      __syncthreads();
      if (tid < 128) {
        float mm = sh_red[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) mm = amax2(mm, sh_red[w][tid]);
        const float s = tile_scale<E5M2>(mm, a.pow2);
        const Divisor d = divisor(s, mm == 0.0f);
        sh_s[col_at(tid)] = d.s;
        sh_ninv[col_at(tid)] = d.ninv;
        sh_lift[col_at(tid)] = d.slow ? kLift : 1.0f;
        if (d.slow) sh_slow = 1;
        // (columns past the edge: zero tiles; ldst >= cols rounded up to 4)
        if (cb * 128 + tid < ((a.cols + 3) & ~int64_t(3))) a.scales_t[rb * a.ldst + cb * 128 + tid] = s;
      }
      __syncthreads();
      if (sh_slow)
        encode_cols<E5M2, true, DT>(v, sh_s, sh_ninv, sh_lift, g, sub, sh_codes);
      else
        encode_cols<E5M2, false, DT>(v, sh_s, sh_ninv, sh_lift, g, sub, sh_codes);
    }
    __syncthreads();
    // eight lanes write a column's 128 codes; 32 columns at a time
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (tid >> 3) + 32 * i, part = tid & 7;
      const int64_t col = cb * 128 + c, row = rb * 128 + 16 * part;
      const uint4 w = *reinterpret_cast<const uint4*>(&sh_codes[word_at(c, 4 * part)]);
      if (col < a.cols && row < a.rows)
        *reinterpret_cast<uint4*>(a.codes_t + col * a.ldct + row) = w;
    }
  }
}

template <int DT, bool E5M2>
cudaError_t launch_fmt(const Quant128Args& a, bool block, cudaStream_t st) {
  const int64_t pieces = a.nbr * a.nbc;
  if (pieces > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(pieces);
  const bool rows = a.codes != nullptr, cols = a.codes_t != nullptr;
  const auto kern =
      block ? (rows && cols ? quant128_kernel<DT, E5M2, true, true, true>
               : rows       ? quant128_kernel<DT, E5M2, true, false, true>
                            : quant128_kernel<DT, E5M2, false, true, true>)
            : (rows && cols ? quant128_kernel<DT, E5M2, true, true, false>
               : rows       ? quant128_kernel<DT, E5M2, true, false, false>
                            : quant128_kernel<DT, E5M2, false, true, false>);
  return launch_dependent(kern, dim3(grid), dim3(kThreads), 0, st, 1, a);
}

}  // namespace

cudaError_t launch_quant128(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                            bool e5m2, bool block, bool pow2, uint8_t* codes, int64_t ldc,
                            float* scales, int64_t lds, uint8_t* codes_t, int64_t ldct,
                            float* scales_t, int64_t ldst, cudaStream_t st) {
  Quant128Args a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.codes = codes;
  a.ldc = ldc;
  a.scales = scales;
  a.lds = lds;
  a.codes_t = codes_t;
  a.ldct = ldct;
  a.scales_t = scales_t;
  a.ldst = ldst;
  a.nbr = (rows + 127) / 128;
  a.nbc = (cols + 127) / 128;
  a.pow2 = pow2;
  const int64_t bytes = dtype == kFP32 ? 4 : 2;
  a.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || ldx * bytes % 16 == 0);
  switch (dtype * 2 + (e5m2 ? 1 : 0)) {
    case 0: return launch_fmt<kBF16, false>(a, block, st);
    case 1: return launch_fmt<kBF16, true>(a, block, st);
    case 2: return launch_fmt<kFP16, false>(a, block, st);
    case 3: return launch_fmt<kFP16, true>(a, block, st);
    case 4: return launch_fmt<kFP32, false>(a, block, st);
    default: return launch_fmt<kFP32, true>(a, block, st);
  }
}

}  // namespace mxk
