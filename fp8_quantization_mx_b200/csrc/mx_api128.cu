// C entry points of the FP8 operators with float scales per 128 elements
// (declared in include/mx.h): argument checks on the host, then the launches
// on the caller's stream. Nothing is allocated and no state is kept.

#include <cstdint>

#include "mx.h"
#include "mx_gemm128.h"
#include "mx_launch.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxSide = int64_t(1) << 31;   // TMA coordinates and grids are 32-bit

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }

int check_matrix(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows >= kMaxSide || cols >= kMaxSide) return MX_ERR_INVALID_ARG;
  if (rows > 0 && cols > kMaxElems / rows) return MX_ERR_INVALID_ARG;
  return MX_OK;
}

bool fp8(int format) { return format == MX_FMT_E4M3 || format == MX_FMT_E5M2; }

bool known_dtype(int dtype) { return dtype >= MX_BF16 && dtype <= MX_FP32; }

uintptr_t elem_bytes(int dtype) { return dtype == MX_FP32 ? 4 : 2; }

// Codes [rows, ld] and, for tiles, block-major scales [., lds] of a side.
int check_codes(const void* codes, int64_t rows, int64_t cols, int64_t ld) {
  if (!codes) return MX_ERR_INVALID_ARG;
  if (ld < up(cols, 16) || ld % 16 != 0 || ld >= kMaxElems || rows > kMaxElems / ld)
    return MX_ERR_SHAPE;
  return aligned(codes, 16) ? MX_OK : MX_ERR_ALIGN;
}

int check_scales(const float* scales, int64_t rows, int64_t lds, bool block) {
  if (!scales) return MX_ERR_INVALID_ARG;
  if (block) return aligned(scales, 4) ? MX_OK : MX_ERR_ALIGN;
  if (lds < up(rows, 4) || lds % 4 != 0 || lds >= kMaxElems) return MX_ERR_SHAPE;
  return aligned(scales, 16) ? MX_OK : MX_ERR_ALIGN;
}

}  // namespace

extern "C" {

int mx_quantize128(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int format,
                   int flags, void* codes, int64_t ldc, float* scales, int64_t lds, void* codes_t,
                   int64_t ldct, float* scales_t, int64_t ldst, void* stream) {
  if (!fp8(format) || !known_dtype(dtype) || (flags & ~(MX_BLOCK128 | MX_POW2_SCALES)) != 0)
    return MX_ERR_UNSUPPORTED;
  int st = check_matrix(rows, cols);
  if (st != MX_OK || rows == 0 || cols == 0) return st;
  if ((rows + 127) / 128 > 0x7fffffff / ((cols + 127) / 128)) return MX_ERR_INVALID_ARG;
  const bool block = (flags & MX_BLOCK128) != 0;
  if (!x || (!codes && !codes_t)) return MX_ERR_INVALID_ARG;
  if (rows > 1 && (ldx < cols || ldx > kMaxElems || rows > kMaxElems / ldx)) return MX_ERR_SHAPE;
  if (!aligned(x, elem_bytes(dtype))) return MX_ERR_ALIGN;
  if (codes) {
    if ((st = check_codes(codes, rows, cols, ldc)) != MX_OK) return st;
    if ((st = check_scales(scales, rows, lds, block)) != MX_OK) return st;
  }
  if (codes_t) {
    if ((st = check_codes(codes_t, cols, rows, ldct)) != MX_OK) return st;
    if ((st = check_scales(scales_t, cols, ldst, block)) != MX_OK) return st;
  }
  return from_cuda(mxk::launch_quant128(
      x, dtype, rows, cols, rows > 1 ? ldx : cols, format == MX_FMT_E5M2, block,
      (flags & MX_POW2_SCALES) != 0, static_cast<uint8_t*>(codes), ldc, scales, lds,
      static_cast<uint8_t*>(codes_t), ldct, scales_t, ldst, static_cast<cudaStream_t>(stream)));
}

int mx_rms_norm_quant128(const void* x, int64_t ldx, const void* residual, const void* weight,
                         int dtype, int64_t rows, int64_t cols, float eps, int format, int flags,
                         void* h, void* y, void* codes, int64_t ldc, float* scales, int64_t lds,
                         void* stream) {
  if (!fp8(format) || !known_dtype(dtype) || (flags & ~MX_POW2_SCALES) != 0)
    return MX_ERR_UNSUPPORTED;
  int st = check_matrix(rows, cols);
  if (st != MX_OK || rows == 0 || cols == 0) return st;
  if (!x || !weight || !(eps >= 0.0f)) return MX_ERR_INVALID_ARG;
  if (rows > 1 && (ldx < cols || ldx > kMaxElems || rows > kMaxElems / ldx)) return MX_ERR_SHAPE;
  const uintptr_t es = elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, es) || !aligned(h, es) ||
      !aligned(y, es))
    return MX_ERR_ALIGN;
  if ((st = check_codes(codes, rows, cols, ldc)) != MX_OK) return st;
  if ((st = check_scales(scales, rows, lds, false)) != MX_OK) return st;
  return from_cuda(mxk::launch_norm128(x, rows > 1 ? ldx : cols, residual, weight, dtype, rows, cols,
                                       eps, format == MX_FMT_E5M2, (flags & MX_POW2_SCALES) != 0, h,
                                       y, static_cast<uint8_t*>(codes), ldc, scales, lds,
                                       static_cast<cudaStream_t>(stream)));
}

int64_t mx_rms_norm_bwd_workspace(int64_t rows, int64_t cols) {
  if (check_matrix(rows, cols) != MX_OK) return -1;
  return (rows < mxk::kNormParts ? rows : mxk::kNormParts) * mxk::norm_part_pitch(cols) * 4;
}

int mx_rms_norm_bwd(const void* grad_y, const void* h, const void* weight, const void* grad_residual,
                    int dtype, int64_t rows, int64_t cols, float eps, void* grad_h,
                    float* grad_weight, void* workspace, void* stream) {
  if (!known_dtype(dtype)) return MX_ERR_UNSUPPORTED;
  const int st = check_matrix(rows, cols);
  if (st != MX_OK || cols == 0) return st;
  if (!grad_weight) return MX_ERR_INVALID_ARG;
  if (!aligned(grad_weight, 4)) return MX_ERR_ALIGN;
  const auto cs = static_cast<cudaStream_t>(stream);
  if (rows == 0)   // an empty sum
    return from_cuda(cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(cols) * 4, cs));
  if (!grad_y || !h || !weight || !grad_h || !workspace || !(eps >= 0.0f)) return MX_ERR_INVALID_ARG;
  const uintptr_t es = elem_bytes(dtype);
  if (!aligned(grad_y, es) || !aligned(h, es) || !aligned(weight, es) || !aligned(grad_residual, es) ||
      !aligned(grad_h, es) || !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  return from_cuda(mxk::launch_norm_bwd(grad_y, h, weight, grad_residual, dtype, rows, cols, eps,
                                        grad_h, grad_weight, static_cast<float*>(workspace), cs));
}

int mx_gemm128(const void* a_codes, int64_t lda, const float* a_scales, int64_t ldsa, int a_format,
               const void* b_codes, int64_t ldb, const float* b_scales, int64_t ldsb, int b_format,
               int b_flags, int64_t M, int64_t N, int64_t K, int out_fp32, void* d, int* status,
               void* stream) {
  if (!fp8(a_format) || !fp8(b_format) || (b_flags & ~MX_BLOCK128) != 0) return MX_ERR_UNSUPPORTED;
  if (out_fp32 != 0 && out_fp32 != 1) return MX_ERR_INVALID_ARG;
  int st = check_matrix(M, K);
  if (st == MX_OK) st = check_matrix(N, K);
  if (st == MX_OK) st = check_matrix(M, N);
  if (st != MX_OK || M == 0 || N == 0) return st;
  if (!d) return MX_ERR_INVALID_ARG;
  if (!aligned(d, 16) || !aligned(status, 4)) return MX_ERR_ALIGN;
  const auto cs = static_cast<cudaStream_t>(stream);
  if (K == 0)   // an empty sum
    return from_cuda(cudaMemsetAsync(d, 0, static_cast<size_t>(M * N) * (out_fp32 ? 4 : 2), cs));
  const bool block = (b_flags & MX_BLOCK128) != 0;
  if ((st = check_codes(a_codes, M, K, lda)) != MX_OK) return st;
  if ((st = check_codes(b_codes, N, K, ldb)) != MX_OK) return st;
  if ((st = check_scales(a_scales, M, ldsa, false)) != MX_OK) return st;
  if ((st = check_scales(b_scales, N, ldsb, block)) != MX_OK) return st;
  mxk::Gemm128 u{};
  u.a = a_codes;
  u.a_scales = a_scales;
  u.lda = lda;
  u.ldsa = ldsa;
  u.a_e5m2 = a_format == MX_FMT_E5M2;
  u.b = b_codes;
  u.b_scales = b_scales;
  u.ldb = ldb;
  u.ldsb = ldsb;
  u.b_e5m2 = b_format == MX_FMT_E5M2;
  u.b_block = block;
  u.M = M;
  u.N = N;
  u.K = K;
  u.out_fp32 = out_fp32;
  u.d = d;
  u.ldd = N;
  u.status = status;
  return from_cuda(mxk::launch_gemm128(u, nullptr, cs));
}

}  // extern "C"
