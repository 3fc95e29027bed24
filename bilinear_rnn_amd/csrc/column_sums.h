// Column sums of float32 partial results, in a fixed order: the last step of every parameter
// gradient. part is [rows, stride]; the first `cols` columns are summed over the rows and given to
// out(column, sum).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace comba {

constexpr int kSumCols = 64, kSumGroups = 16;  // columns and row groups per workgroup

// One workgroup's columns. A wavefront reads 64 neighbouring columns (256 bytes) of one row; the 16 row
// groups keep enough loads in flight for the few thousand columns that a layer's parameters have.
template <typename F>
__device__ __forceinline__ void column_sums_block(const float* __restrict__ part, int64_t rows, int64_t stride, int cols,
                                                  int block, const F& out) {
  __shared__ float sums[kSumGroups][kSumCols];
  const int l = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int c = block * kSumCols + l;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int64_t r = g; r < rows; r += kSumGroups) s += part[r * stride + c];
  }
  sums[g][l] = s;
  __syncthreads();
  if (g == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kSumGroups; ++i) s += sums[i][l];
    out(c, s);
  }
}

template <typename F>
__global__ __launch_bounds__(kSumCols* kSumGroups) void column_sums_kernel(const float* __restrict__ part, int64_t rows,
                                                                           int64_t stride, int cols, F out) {
  column_sums_block(part, rows, stride, cols, blockIdx.x, out);
}

template <typename F>
static hipError_t column_sums(const float* part, int64_t rows, int64_t stride, int cols, hipStream_t st, F out) {
  column_sums_kernel<<<(cols + kSumCols - 1) / kSumCols, kSumCols * kSumGroups, 0, st>>>(part, rows, stride, cols, out);
  return hipGetLastError();
}

}  // namespace comba
