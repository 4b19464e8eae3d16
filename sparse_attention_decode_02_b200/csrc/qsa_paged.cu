// Paged K/V cache: rows quantised into pages as they are written, and read back as f16.
//
// The 8-bit K/V cache the Qwen3.8-Flash-Next parameter-tuning post on EVO-X2 tried (section
// "KV cacheをQ8_0にしてみる") in its paged form, and a 4-bit one beside it. A row is the
// head_dim values of one (token, KV head).
//   e4m3: scale = amax * (1/448), code = e4m3(x * (448 * (1/amax)));
//   4 bits: per 32 dims s = f16(amax * (1/7)), code = rint(x * (1/s)) in [-7, 7].
// Both calls only move data: a row's 2 * head_dim f16 bytes and its stored bytes.
#include "qsa_paged.cuh"
#include "qsa_pool.cuh"

namespace qsa {

namespace {

constexpr int kRowThreads = 256;

// Where row `row` of a write or a read lives. False, after reporting it, if nowhere.
__device__ __forceinline__ bool find_row(const PagedView& c, const PagedRows& r, int row, int lane, int* page,
                                         int* place, bool* padding) {
  *padding = row >= r.row_start[r.n_seqs];
  if (*padding) return false;
  int lo = 0, hi = r.n_seqs;  // the last sequence with row_start <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (r.row_start[mid] <= row) lo = mid; else hi = mid;
  }
  const long long pos = (long long)r.first[lo] + (row - r.row_start[lo]);
  const long long at = pos >> c.page_shift;
  if (row < r.row_start[lo] || pos < 0 || at >= r.table_width) {
    if (lane == 0) record_status(r.status, pos < 0 || row < r.row_start[lo] ? QSA_ERR_BAD_INDEX : QSA_ERR_CAPACITY);
    return false;
  }
  *page = r.block_table[(long long)lo * r.table_width + at];
  *place = int(pos) & ((1 << c.page_shift) - 1);
  if (*page < 0 || *page >= c.n_pages) {
    if (lane == 0) record_status(r.status, QSA_ERR_BAD_INDEX);
    return false;
  }
  return true;
}

// One warp stores one row: lane l holds dims [l*D/32, (l+1)*D/32).
template <int FMT, int D>
__device__ __forceinline__ void store_row(const __half* src, char* pages, char* scales, int64_t page_base,
                                          int64_t scale_base, int row, int lane) {
  constexpr int P = D / 32;
  char* dst = pages + page_base + int64_t(row) * page_row_bytes_c<FMT>(D);
  if constexpr (FMT == QSA_PAGE_F16) {
    if constexpr (P == 4) reinterpret_cast<uint2*>(dst)[lane] = reinterpret_cast<const uint2*>(src)[lane];
    else reinterpret_cast<uint32_t*>(dst)[lane] = reinterpret_cast<const uint32_t*>(src)[lane];
  } else if constexpr (FMT == QSA_PAGE_FP8) {
    const Fp8Row x = fp8_row_load(src, D, lane);
    const float top = warp_max(fmaxf(fmaxf(fabsf(x.x[0]), fabsf(x.x[1])), fmaxf(fabsf(x.x[2]), fabsf(x.x[3]))));
    const float factor = top > 0.0f ? __fmul_rn(448.0f, 1.0f / top) : 0.0f;
    unsigned codes = 0;
#pragma unroll
    for (int i = 0; i < P; i += 2)
      codes |= unsigned(__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x.x[i], factor), __fmul_rn(x.x[i + 1], factor)),
                                                 __NV_SATFINITE, __NV_E4M3))
               << (8 * i);
    if constexpr (P == 4) reinterpret_cast<uint32_t*>(dst)[lane] = codes;
    else reinterpret_cast<uint16_t*>(dst)[lane] = (unsigned short)codes;
    if (lane == 0)
      reinterpret_cast<float*>(scales + scale_base)[row] = top > 0.0f ? __fmul_rn(top, 1.0f / 448.0f) : 1.0f;
  } else {
    constexpr int GL = kInt4Group / P;  // lanes of a group
    __half x[P];
    unsigned top = 0;  // the largest |x| as bits: NaN and infinity rank above every number
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = src[lane * P + i];
      top = max(top, unsigned(__half_as_ushort(x[i]) & 0x7fff));
    }
#pragma unroll
    for (int off = 1; off < GL; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const __half s = top >= 0x7c00u ? __ushort_as_half(0x7fff)
                                    : __float2half_rn(__fmul_rn(__half2float(__ushort_as_half((unsigned short)top)), 1.0f / 7.0f));
    const float sf = __half2float(s);
    const float inv = sf == 0.0f ? 0.0f : 1.0f / sf;
    unsigned codes = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float y = rintf(__fmul_rn(__half2float(x[i]), inv));
      codes |= unsigned(int(fminf(fmaxf(y, -7.0f), 7.0f)) + 8) << (8 * i);
    }
    codes |= __shfl_down_sync(0xffffffffu, codes, GL / 2) << 4;  // dims + 16 in the high halves
    if ((lane & (GL - 1)) < GL / 2) {
      unsigned char* d = reinterpret_cast<unsigned char*>(dst) + (lane / GL) * 16 + (lane & (GL - 1)) * P;
      if constexpr (P == 4) *reinterpret_cast<uint32_t*>(d) = codes;
      else *reinterpret_cast<uint16_t*>(d) = (unsigned short)codes;
    }
    if ((lane & (GL - 1)) == 0)
      (reinterpret_cast<__half*>(scales + scale_base) + int64_t(row) * (D / kInt4Group))[lane / GL] = s;
  }
}

template <int FMT, int D>
__device__ __forceinline__ void load_row(__half* out, const char* pages, const char* scales, int64_t page_base,
                                         int64_t scale_base, int row, int lane) {
  constexpr int P = D / 32;
  const char* src = pages + page_base + int64_t(row) * page_row_bytes_c<FMT>(D);
  __half x[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int d = lane * P + i;
    if constexpr (FMT == QSA_PAGE_F16) {
      x[i] = reinterpret_cast<const __half*>(src)[d];
    } else if constexpr (FMT == QSA_PAGE_FP8) {
      const float s = (reinterpret_cast<const float*>(scales + scale_base))[row];
      const __half c = __half(__nv_cvt_fp8_to_halfraw(reinterpret_cast<const unsigned char*>(src)[d], __NV_E4M3));
      x[i] = __float2half_rn(__half2float(c) * s);
    } else {
      const __half s = (reinterpret_cast<const __half*>(scales + scale_base) + int64_t(row) * (D / 32))[d / 32];
      const unsigned b = reinterpret_cast<const unsigned char*>(src)[d / 32 * 16 + d % 16];
      x[i] = __hmul(__int2half_rn(int((d & 16) ? b >> 4 : b & 15) - 8), s);
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) out[lane * P + i] = x[i];
}

// One warp per (row, KV head).
template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) paged_write_kernel(PagedView c, PagedRows r, const __half* __restrict__ k,
                                                                  const __half* __restrict__ v) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long n = (long long)r.n_rows * c.n_kv_heads;
  for (long long w = ((long long)blockIdx.x * kRowThreads + threadIdx.x) >> 5; w < n;
       w += (long long)gridDim.x * (kRowThreads / 32)) {
    const int row = int(w / c.n_kv_heads), head = int(w % c.n_kv_heads);
    int page, place;
    bool padding;
    if (!find_row(c, r, row, lane, &page, &place, &padding)) continue;
    const int at = row_in_page(c, head, place);
    const int64_t src = row * r.row_stride + head * D;
    store_row<FMT, D>(k + src, c.k, c.ks, page * c.page_stride, page * c.scale_stride, at, lane);
    store_row<FMT, D>(v + src, c.v, c.vs, page * c.page_stride, page * c.scale_stride, at, lane);
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) paged_read_kernel(PagedView c, PagedRows r, __half* __restrict__ k,
                                                                 __half* __restrict__ v) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long n = (long long)r.n_rows * c.n_kv_heads;
  for (long long w = ((long long)blockIdx.x * kRowThreads + threadIdx.x) >> 5; w < n;
       w += (long long)gridDim.x * (kRowThreads / 32)) {
    const int row = int(w / c.n_kv_heads), head = int(w % c.n_kv_heads);
    int page, place;
    bool padding;
    const bool found = find_row(c, r, row, lane, &page, &place, &padding);
    if (padding) continue;
    const int64_t dst = row * r.row_stride + head * D;
    if (!found) {
      for (int i = 0; i < D / 32; ++i) {
        if (k) k[dst + lane * (D / 32) + i] = __half(0.0f);
        if (v) v[dst + lane * (D / 32) + i] = __half(0.0f);
      }
      continue;
    }
    const int at = row_in_page(c, head, place);
    if (k) load_row<FMT, D>(k + dst, c.k, c.ks, page * c.page_stride, page * c.scale_stride, at, lane);
    if (v) load_row<FMT, D>(v + dst, c.v, c.vs, page * c.page_stride, page * c.scale_stride, at, lane);
  }
}

int row_grid(const PagedView& c, const PagedRows& r, int n_sms) {
  const long long warps = (long long)r.n_rows * c.n_kv_heads;
  const long long ctas = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  return int(ctas < n_sms * 8LL ? ctas : n_sms * 8LL);
}

}  // namespace

cudaError_t launch_paged_write(const PagedView& c, int format, const PagedRows& r, const void* k, const void* v,
                               int n_sms, cudaStream_t s) {
  const dim3 grid(row_grid(c, r, n_sms)), block(kRowThreads);
#define QSA_WRITE(F, D)                                                                                      \
  if (format == F && c.head_dim == D)                                                                        \
    return launch_pdl(paged_write_kernel<F, D>, grid, block, 0, s, 1, c, r, (const __half*)k, (const __half*)v)
  QSA_WRITE(QSA_PAGE_F16, 64);
  QSA_WRITE(QSA_PAGE_F16, 128);
  QSA_WRITE(QSA_PAGE_FP8, 64);
  QSA_WRITE(QSA_PAGE_FP8, 128);
  QSA_WRITE(QSA_PAGE_INT4, 64);
  QSA_WRITE(QSA_PAGE_INT4, 128);
#undef QSA_WRITE
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_read(const PagedView& c, int format, const PagedRows& r, void* k, void* v, int n_sms,
                              cudaStream_t s) {
  const dim3 grid(row_grid(c, r, n_sms)), block(kRowThreads);
#define QSA_READ(F, D)                                                                            \
  if (format == F && c.head_dim == D)                                                             \
    return launch_pdl(paged_read_kernel<F, D>, grid, block, 0, s, 1, c, r, (__half*)k, (__half*)v)
  QSA_READ(QSA_PAGE_F16, 64);
  QSA_READ(QSA_PAGE_F16, 128);
  QSA_READ(QSA_PAGE_FP8, 64);
  QSA_READ(QSA_PAGE_FP8, 128);
  QSA_READ(QSA_PAGE_INT4, 64);
  QSA_READ(QSA_PAGE_INT4, 128);
#undef QSA_READ
  return cudaErrorInvalidValue;
}

}  // namespace qsa
