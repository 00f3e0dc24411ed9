// Tensor-memory columns of S^T and P^T in the backward kernels (plain C++, so
// that a host program can check them).
//
// S^T is 128 fp32 columns, a query row each. Two warps share a lane quarter:
// the warp of query columns [c0, c0 + 64), c0 = 0 or 64, reads those columns of
// S^T and puts P^T (bf16, two query rows to a column) in their place. Nothing
// orders the two warps between S^T's arrival and the product that reads P^T, so
// each keeps its P^T within the columns that it has itself read: stored side by
// side over the first 64 columns, the second warp's P^T would overwrite scores
// that the first may not have read yet.
#pragma once

#ifdef __CUDACC__
#define FA_HOST_DEVICE __host__ __device__
#else
#define FA_HOST_DEVICE
#endif

namespace fa {

// first of the 32 columns of the P^T of query columns [c0, c0 + 64)
FA_HOST_DEVICE constexpr int p_store_col(int c0) { return c0; }

// first of the 8 columns of P^T of query rows [16 kk, 16 kk + 16), the product's K step
FA_HOST_DEVICE constexpr int p_operand_col(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

}  // namespace fa
