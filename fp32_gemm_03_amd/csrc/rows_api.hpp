// rows_api.hpp -- products of rows.hip that other sources of the library call.
#pragma once

#include <hip/hip_runtime.h>

namespace rowk {

// rows of C from which on rows_product() answers SGEMM_ERR_TOO_LARGE
constexpr int kMostRows = 1 << 29;

// C (M x N) = A (M x K) B + beta C, B K x N or (trans_b) N x K, on the kernels of
// sgemm_grouped() as one group.
__attribute__((visibility("hidden"))) int rows_product(int M, int N, int K, const float *A, int lda, const float *B,
                                                       int ldb, bool trans_b, float beta, float *C, int ldc,
                                                       hipStream_t stream);

}  // namespace rowk
