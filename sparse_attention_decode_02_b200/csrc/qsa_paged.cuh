// Row formats of the paged K/V cache (f16, e4m3 + row scale, 4-bit codes + group scales)
// and the addressing of rows in pages, shared by the paged kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qsa_device.cuh"

namespace qsa {

constexpr int kInt4Group = 32;  // dims that share one scale of a 4-bit row

template <int FMT>
__host__ __device__ constexpr int page_row_bytes_c(int d) {
  return FMT == QSA_PAGE_F16 ? 2 * d : FMT == QSA_PAGE_FP8 ? d : d / 2;
}
template <int FMT>
__host__ __device__ constexpr int page_scale_bytes_c(int d) {
  return FMT == QSA_PAGE_F16 ? 0 : FMT == QSA_PAGE_FP8 ? 4 : d / kInt4Group * 2;
}

// Index of a row in its page: a head's rows of a page are consecutive.
__device__ __forceinline__ int row_in_page(const PagedView& c, int head, int place) {
  return (head << c.page_shift) + place;
}

}  // namespace qsa
