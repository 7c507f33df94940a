// rows_api.hpp -- products of rows.hip that other sources of the library call.
#pragma once

#include <hip/hip_runtime.h>

namespace rowk {

// rows of C from which on rows_product_pair() answers SGEMM_ERR_TOO_LARGE
constexpr int kMostRows = 1 << 29;

// C (M x N) = A[0] B[0]^T + A[1] B[1]^T, A M x K and B N x K, on the kernels of
// sgemm_grouped() as one group.
__attribute__((visibility("hidden"))) int rows_product_pair(int M, int N, int K, const float *const A[2], int lda,
                                                            const float *const B[2], const int ldb[2], float *C,
                                                            int ldc, hipStream_t stream);

}  // namespace rowk
