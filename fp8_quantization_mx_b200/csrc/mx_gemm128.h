// The FP8 GEMM with 128-element scales: a problem, and how it is cut up.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mxk {

struct Gemm128 {
  const void* a;           // codes [M, lda]
  const float* a_scales;   // [ceil(K/128), ldsa]
  int64_t lda, ldsa;
  int a_e5m2;
  const void* b;           // codes [N, ldb]
  const float* b_scales;   // tiles: [ceil(K/128), ldsb]; blocks: [ceil(N/128), ceil(K/128)]
  int64_t ldb, ldsb;
  int b_e5m2, b_block;
  int64_t M, N, K;
  int out_fp32;
  void* d;                 // [M, ldd]
  int64_t ldd;
  int* status;             // nullable
};

// Tile width bn (16, 32 or 64 swapped, else 64, 128 or 256), whether the
// weights take the row side of the MMA, and the CTAs that split K (1, 2, 4, 8).
struct Plan128 {
  int bn, swap, split;
};

// sms, and how many clusters of 4 and of 8 one-per-SM CTAs run at once. *us: the
// model's time, without a launch's own.
Plan128 plan_gemm128(int64_t M, int64_t N, int64_t K, bool b_block, int sms, int clusters4,
                     int clusters8, double* us);

// plan: NULL for plan_gemm128's choice on the current device.
cudaError_t launch_gemm128(const Gemm128& u, const Plan128* plan, cudaStream_t st);

}  // namespace mxk
