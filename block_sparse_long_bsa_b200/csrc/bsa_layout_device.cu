// What a layout's arrays need of the device when it is built.  A file of its own,
// so that the first layout of a process loads this one kernel and no other.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bsa_internal.h"

namespace bsa {
namespace {

// Where each entry of the transposed layout stands in col_idx, found on the
// device when a layout is built, a thread per entry: its row by bisection of
// row_ptr, its place in its column, whose rows ascend, by another.  (Scattered
// by the host and uploaded, the array made a layout's building 7 to 18 %
// longer; a warp per row walked the 512 entries of a row of a whole 32K route in 50 us.)
constexpr int kFillThreads = 256;
__global__ void __launch_bounds__(kFillThreads)
    fill_csr_pos_kernel(const int32_t* row_ptr, const int32_t* col_idx, const int32_t* col_ptr, const int32_t* row_idx,
                        int nb, int rows, int nnz, int32_t* csr_pos) {
  for (int64_t e = int64_t(blockIdx.x) * kFillThreads + threadIdx.x; e < nnz; e += int64_t(gridDim.x) * kFillThreads) {
    int lo = 0, hi = rows - 1;                     // the last row that begins at or before e
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (row_ptr[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    const int i = lo % nb, col = lo - i + col_idx[e];
    lo = col_ptr[col];
    hi = col_ptr[col + 1] - 1;                     // row i's entry lies in lo .. hi
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (row_idx[mid] < i) lo = mid + 1;
      else hi = mid;
    }
    csr_pos[lo] = int(e);
  }
}

}  // namespace

cudaError_t fill_csr_pos(const int32_t* row_ptr, const int32_t* col_idx, const int32_t* col_ptr, const int32_t* row_idx,
                         int nb, int rows, int nnz, int32_t* csr_pos) {
  const int grid = int(std::min<int64_t>((int64_t(nnz) + kFillThreads - 1) / kFillThreads, 8 * 148));
  fill_csr_pos_kernel<<<grid, kFillThreads>>>(row_ptr, col_idx, col_ptr, row_idx, nb, rows, nnz, csr_pos);
  return cudaGetLastError();
}

}  // namespace bsa
