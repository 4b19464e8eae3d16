// Row formats of the paged K/V cache (f16, e4m3 + row scale, 4-bit codes + group scales)
// and the addressing of rows in pages, shared by the paged kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qsa_device.cuh"

namespace qsa {

// Bytes of a row and of its scales, as constants.
template <int FMT>
__host__ __device__ constexpr int page_row_bytes_c(int d) {
  return page_row_bytes(FMT, d);
}
template <int FMT>
__host__ __device__ constexpr int page_scale_bytes_c(int d) {
  return page_scale_bytes(FMT, d);
}

// Index of a row in its page: a head's rows of a page are consecutive.
__device__ __forceinline__ int row_in_page(const PagedView& c, int head, int place) {
  return (head << c.page_shift) + place;
}

}  // namespace qsa
