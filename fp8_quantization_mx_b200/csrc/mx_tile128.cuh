// FP8 codes with one float scale per 128 elements: what the quantizer and the
// norm share. A tile is 128 consecutive elements of a row (or of a column), a
// block 128 x 128 of them; both may be cut short by the matrix's edge.
//
//   s = max(amax / maxv, 2^-126), rounded to float (maxv 448 or 57344), or
//       the smallest power of two >= 2^-126 with amax <= maxv s;
//   code = RNE_sat(x / s), x / s rounded to float first;
//   NaN or Inf in the tile: s = NaN and every code NaN (0x7F).
//
// The floor of 2^-126 keeps s normal and nonzero, so that a zero tile needs no
// case of its own (its codes are +-0) and 1 / s never overflows.

#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace mxk {
namespace t128 {

constexpr float kTinyScale = 1.17549435e-38f;   // 2^-126
// Below this scale the remainder q s - x of div2 may be subnormal for an x that
// still rounds to a nonzero code; such tiles are divided 2^64 times larger.
constexpr float kSlowScale = 8.2718061e-25f;    // 2^-80
constexpr float kLift = 1.84467441e19f;         // 2^64

template <bool E5M2>
__device__ __forceinline__ constexpr float max_code() {
  return E5M2 ? 57344.0f : 448.0f;
}

// Largest magnitudes of two pairs of 16-bit floats, NaN kept (the sign bits of
// the result are to be ignored).
template <int DT>
__device__ __forceinline__ uint32_t amax_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (DT == 0)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// max(|a|, |b|) that keeps a NaN (a >= 0 or NaN).
__device__ __forceinline__ float amax2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// max(|a|, |b|, |c|), NaN kept.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// N (1, 2 or 4) maxima that each of a group of lanes holds a part of, one per
// lane: every step exchanges half of those held with a neighbour (N - 1
// shuffles where reducing all N in every lane takes N log N). Lane l then holds
// part of maximum held_by<N>(l); what is left is to take the maximum over lanes
// a multiple of N apart. lane_of<N>(j) is the lane of the first N that holds j.
template <int N>
__device__ __forceinline__ int held_by(int lane) {
  return N == 4 ? (lane & 1) << 1 | (lane >> 1 & 1) : N == 2 ? lane & 1 : 0;
}
template <int N>
__device__ __forceinline__ int lane_of(int j) {
  return N == 4 ? j >> 1 | (j & 1) << 1 : j;
}
template <int N>
__device__ __forceinline__ float spread_max(const float (&m)[N], int lane) {
  static_assert(N == 1 || N == 2 || N == 4, "maxima");
  if constexpr (N == 1) {
    return m[0];
  } else if constexpr (N == 2) {
    const bool odd = lane & 1;
    return amax2(odd ? m[1] : m[0], __shfl_xor_sync(~0u, odd ? m[0] : m[1], 1));
  } else {
    const bool odd = lane & 1, two = lane & 2;
    const float a = amax2(odd ? m[2] : m[0], __shfl_xor_sync(~0u, odd ? m[0] : m[2], 1));
    const float b = amax2(odd ? m[3] : m[1], __shfl_xor_sync(~0u, odd ? m[1] : m[3], 1));
    return amax2(two ? b : a, __shfl_xor_sync(~0u, two ? a : b, 2));
  }
}

// The scale of a tile from its largest magnitude.
template <bool E5M2>
__device__ __forceinline__ float tile_scale(float amax, bool pow2) {
  if (!(amax < __int_as_float(0x7f800000))) return __int_as_float(0x7fc00000);
  if (!pow2) {
    // amax / maxv correctly rounded, as div2 does it (below 2^-126, where the
    // remainder is not exact, the floor decides)
    constexpr float c = 1.0f / max_code<E5M2>();
    const float q = amax * c;
    return fmaxf(fmaf(fmaf(q, -max_code<E5M2>(), amax), c, q), kTinyScale);
  }
  // maxv = 1.75 2^top: the exponent of amax less `top`, one more where the
  // significand is above 1.75 (in biased exponents, at least 1)
  constexpr int kTop = E5M2 ? 15 : 8;
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - kTop + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return __int_as_float((e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ float recip(float s) { return __frcp_rn(s); }

// {x.x / s.x, x.y / s.y} correctly rounded, given nx = -x and ninv = -(1 / s)
// correctly rounded: a quotient within one unit in the last place, corrected by
// its exact remainder (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990). Ties of the codes are decided on the
// rounded quotient. Packed: 1.5 instructions per element where a division takes
// about ten. The negations are the caller's because packed operands have none
// (left to the compiler they took as long as the rest); with these signs
// -0 / s stays -0.
__device__ __forceinline__ float2 div2(float2 nx, float2 s, float2 ninv) {
  const float2 q = __fmul2_rn(nx, ninv);
  const float2 r = __ffma2_rn(q, s, nx);
  return __ffma2_rn(r, ninv, q);
}

// A tile's scale with what division by it needs.
struct Divisor {
  float s, ninv;   // as div2 takes them (both lifted for a tiny scale)
  bool slow;       // x is to be lifted too
};

__device__ __forceinline__ Divisor divisor(float s, bool zero) {
  Divisor d{s, -recip(s), s < kSlowScale && !zero};
  if (d.slow) {
    d.s *= kLift;
    d.ninv *= 1.0f / kLift;
  }
  return d;
}

// Lane src's divisor in every lane.
__device__ __forceinline__ Divisor divisor_of(const Divisor& d, int src) {
  const float s = __shfl_sync(~0u, d.slow ? -d.s : d.s, src);   // (s > 0 or NaN)
  return {fabsf(s), __shfl_sync(~0u, d.ninv, src), s < 0.0f};
}

// Two codes: lo in bits 0-7, hi in bits 8-15.
template <bool E5M2>
__device__ __forceinline__ uint32_t enc2(float lo, float hi) {
  uint16_t r;
  if constexpr (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t enc4(float a, float b, float c, float d) {
  return enc2<E5M2>(a, b) | (enc2<E5M2>(c, d) << 16);
}

// --------------------------------------------------- elements and vectors --

enum DType { kBF16 = 0, kFP16 = 1, kFP32 = 2 };

template <int DT>
struct Elem;
template <>
struct Elem<kBF16> {
  using T = __nv_bfloat16;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float to_float(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T from_float(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<kFP16> {
  using T = __half;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float to_float(T v) { return __half2float(v); }
  static __device__ __forceinline__ T from_float(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<kFP32> {
  using T = float;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float to_float(T v) { return v; }
  static __device__ __forceinline__ T from_float(float v) { return v; }
};

// N consecutive elements as they lie in memory (N * bytes a multiple of 16).
template <int DT, int N>
struct Vec {
  using E = Elem<DT>;
  static constexpr int kWords = N * E::kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // 16-byte aligned p, all N elements present; read once (no L1 allocation). Not the
  // read-only path: an output may be the input in place. (volatile, here and
  // below: stays behind the wait for the kernel before)
  __device__ __forceinline__ void load(const typename E::T* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
          : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
          : "l"(reinterpret_cast<const char*>(p) + 4 * i));
  }
  // All N elements at any alignment of an element, from aligned 16-byte loads:
  // the bytes from p rounded down to 16 up to p + N elements rounded up are read.
  __device__ __forceinline__ void load_shifted(const typename E::T* p) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = at & 15;
    const char* q = reinterpret_cast<const char*>(at - off);
    uint32_t t[kWords + 4];
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
          : "=r"(t[i]), "=r"(t[i + 1]), "=r"(t[i + 2]), "=r"(t[i + 3])
          : "l"(q + 4 * i));
#pragma unroll
    for (int i = kWords; i < kWords + 4; ++i) t[i] = 0;
    if (off)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
          : "=r"(t[kWords]), "=r"(t[kWords + 1]), "=r"(t[kWords + 2]), "=r"(t[kWords + 3])
          : "l"(q + 4 * kWords));
#pragma unroll
    for (int i = 0; i < kWords + 2; ++i) t[i] = (off & 8) ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < kWords + 1; ++i) t[i] = (off & 4) ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(t[i], t[i + 1], (off & 3) * 8);
  }
  // Elements other than lo..hi - 1 become 0.
  __device__ __forceinline__ void keep(int lo, int hi) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < lo || i >= hi) {
        if constexpr (DT == kFP32) w[i] = 0;
        else w[i / 2] &= (i & 1) ? 0xffffu : 0xffff0000u;
      }
  }
  // The first n elements, one at a time; the rest 0.
  __device__ __forceinline__ void load_some(const typename E::T* p, int64_t n) {
    zero();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        if constexpr (DT == kFP32) {
          w[i] = __float_as_uint(p[i]);
        } else {
          const uint32_t b = reinterpret_cast<const uint16_t*>(p)[i];
          w[i / 2] |= b << (16 * (i & 1));
        }
      }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == kBF16) {
      return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    } else if constexpr (DT == kFP16) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i / 2]);
      return (i & 1) ? __high2float(h) : __low2float(h);
    } else {
      return __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ float2 get2(int i) const { return make_float2(get(2 * i), get(2 * i + 1)); }
  // Elements 2i and 2i + 1, negated.
  __device__ __forceinline__ float2 neg2(int i) const {
    if constexpr (DT == kFP32) {
      return make_float2(__uint_as_float(w[2 * i] ^ 0x80000000u), __uint_as_float(w[2 * i + 1] ^ 0x80000000u));
    } else {
      Vec<DT, 8> t;
      t.w[0] = w[i] ^ 0x80008000u;
      return make_float2(t.get(0), t.get(1));
    }
  }
  // The largest magnitude, NaN kept.
  __device__ __forceinline__ float amax() const {
    if constexpr (DT == kFP32) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < N; i += 2) m = amax3(m, get(i), get(i + 1));
      return m;
    } else {
      uint32_t m = w[0];
#pragma unroll
      for (int i = 1; i < kWords; ++i) m = amax_pair<DT>(m, w[i]);
      Vec<DT, 8> t;   // (its first pair)
      t.w[0] = m & 0x7fff7fffu;
      return amax2(t.get(0), t.get(1));
    }
  }
  // Elements 2i and 2i + 1, each rounded to nearest even.
  __device__ __forceinline__ void set2(int i, float lo, float hi) {
    if constexpr (DT == kBF16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else if constexpr (DT == kFP16) {
      const __half2 v = __floats2half2_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w[2 * i] = __float_as_uint(lo);
      w[2 * i + 1] = __float_as_uint(hi);
    }
  }
  __device__ __forceinline__ void store(typename E::T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
};

}  // namespace t128
}  // namespace mxk
