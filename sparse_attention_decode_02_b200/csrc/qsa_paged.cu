// Paged K/V cache: rows quantised into pages as they are written, and read back as f16.
//
// The 8-bit K/V cache the Qwen3.8-Flash-Next parameter-tuning post on EVO-X2 tried (section
// "KV cacheをQ8_0にしてみる") in its paged form, and a 4-bit one beside it. A row is the
// head_dim values of one (token, KV head).
//   e4m3: scale = amax * (1/448), code = e4m3(x * (448 * (1/amax)));
//   4 bits: per 32 dims s = min(f16(amax * (1/7)), 9352), code = rint(x * (1/s)) in [-7, 7].
// Both calls only move data: a row's 2 * head_dim f16 bytes and its stored bytes. A CTA takes
// some tokens: it finds their places once (sequence, then page), then every thread moves pieces
// of K and V rows; a row's pieces sit in neighbouring lanes, which share its scale by shuffles.
// Measured on B200 (us; share of a copy's 6,568 GB/s): 61,789 tokens x 4 heads x 128 dims
// written to f16 pages 40 (95%), to e4m3 33 (89%); 126,253 read from e4m3 64 (93%); 58,096
// written in 4 bits and read back 67 (69%: the issue slots, in both); 64 tokens 2.5 (latency).
// Pieces of 16 values take fewer instructions a value than 8 (e4m3 writes 38 -> 33, 4-bit
// 45 -> 35), but a read's stores then leave every other 16 bytes to a second instruction
// (65 -> 73), so reads take 8. More pieces in flight cost CTAs an SM (registers). Codes are
// rounded by an addition instead of conversions (4-bit writes a third faster).
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 64;   // most tokens a CTA takes: the places it keeps in shared memory
// K and V pieces a thread has in flight: of 16 values in a write, of 8 in a read. Twice as many
// cost CTAs an SM (61,789 tokens written to e4m3 in pieces of 8: four 50 us, two 45).
constexpr int kRowBatch = 1;
constexpr int kReadBatch = 2;

// Where a token's rows are: byte offsets of head 0's row and of its scales; rows -1: nowhere,
// -2: padding.
struct TokenPlace {
  int64_t rows, scales;
};

// Finds the places of tokens [t0, t0 + n) (the whole CTA; s_at holds n of them). Two rounds of
// dependent loads: the sequences' starts and first positions, then the pages.
template <int FMT, int D>
__device__ __forceinline__ void find_tokens(const PagedView& c, const PagedRows& r, int t0, int n, TokenPlace* s_at) {
  __shared__ int s_start[kRowThreads], s_first[kRowThreads];
  const int i = threadIdx.x, row = t0 + i;
  const int end = r.row_start[r.n_seqs];
  TokenPlace at{i < n && row >= end ? -2 : -1, 0};
  int seq = -1, start = 0, first = 0;
  for (int b = 0; b < r.n_seqs; b += kRowThreads) {
    const int m = min(kRowThreads, r.n_seqs - b);
    if (b > 0) __syncthreads();
    if (i < m) {
      s_start[i] = r.row_start[b + i];
      s_first[i] = r.first[b + i];
    }
    __syncthreads();
    if (i < n && s_start[0] <= row) {  // the last sequence that starts at or before the token
      int lo = 0, hi = m - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= row) lo = mid; else hi = mid - 1;
      }
      seq = b + lo;
      start = s_start[lo];
      first = s_first[lo];
    }
  }
  if (i < n) {
    if (at.rows != -2) {
      const long long pos = (long long)first + row - start, entry = pos >> c.page_shift;
      if (seq < 0 || pos < 0) {
        record_status(r.status, QSA_ERR_BAD_INDEX);
      } else if (entry >= r.table_width) {
        record_status(r.status, QSA_ERR_CAPACITY);
      } else {
        const int page = r.block_table[(long long)seq * r.table_width + entry];
        if (page < 0 || page >= c.n_pages) record_status(r.status, QSA_ERR_BAD_INDEX);
        else {
          const int place = int(pos) & ((1 << c.page_shift) - 1);
          at = TokenPlace{page * c.page_stride + place * page_row_bytes_c<FMT>(D),
                          page * c.scale_stride + place * page_scale_bytes_c<FMT>(D)};
        }
      }
    }
    s_at[i] = at;
  }
  __syncthreads();
}

// 16 values of a row to write: consecutive ones (half a 4-bit group), or for f16 pages two 16-byte
// chunks half a row apart, so that the lanes' stores are consecutive.
struct Piece {
  uint4 v[2];
};

__device__ __forceinline__ uint32_t word_of(const Piece& x, int i) {
  const uint4& v = x.v[i >> 2];
  return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
}
__device__ __forceinline__ __half2 half2_at(const Piece& x, int i) {
  const uint32_t w = word_of(x, i);
  return *reinterpret_cast<const __half2*>(&w);
}

// Stores piece `ch` of the row at `dst` with its scale(s) at `scale`: all lanes take part in the
// shuffles, `ok` ones store.
template <int FMT, int D>
__device__ __forceinline__ void store_piece(const Piece& x, char* dst, char* scale, int ch, bool ok) {
  if constexpr (FMT == QSA_PAGE_F16) {
    if (ok) {
      reinterpret_cast<uint4*>(dst)[ch] = x.v[0];
      reinterpret_cast<uint4*>(dst)[ch + D / 16] = x.v[1];
    }
  } else if constexpr (FMT == QSA_PAGE_FP8) {
    __half2 h = __habs2(half2_at(x, 0));
#pragma unroll
    for (int i = 1; i < 8; ++i) h = __hmax2(h, __habs2(half2_at(x, i)));
#pragma unroll
    for (int off = D / 32; off >= 1; off >>= 1) h = __hmax2(h, __shfl_xor_sync(0xffffffffu, h, off));
    const float top = fmaxf(__low2float(h), __high2float(h));
    const float factor = top > 0.0f ? __fmul_rn(448.0f, 1.0f / top) : 0.0f;
    uint32_t codes[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = __half22float2(half2_at(x, i));
      codes[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v.x, factor), __fmul_rn(v.y, factor)), __NV_SATFINITE,
                                          __NV_E4M3);
    }
    if (ok) {
      reinterpret_cast<uint4*>(dst)[ch] =
          make_uint4(__byte_perm(codes[0], codes[1], 0x5410), __byte_perm(codes[2], codes[3], 0x5410),
                     __byte_perm(codes[4], codes[5], 0x5410), __byte_perm(codes[6], codes[7], 0x5410));
      if (ch == 0) *reinterpret_cast<float*>(scale) = top > 0.0f ? __fmul_rn(top, 1.0f / 448.0f) : 1.0f;
    }
  } else {
    // the largest |x| of the group (2 lanes): a NaN or an infinity comes through
    __half2 h = __habs2(half2_at(x, 0));
#pragma unroll
    for (int i = 1; i < 8; ++i) h = __hmax2_nan(h, __habs2(half2_at(x, i)));
    h = __hmax2_nan(h, __shfl_xor_sync(0xffffffffu, h, 1));
    const __half top = __hmax_nan(__low2half(h), __high2half(h));
    // (at most 9352, the largest f16 that 7 times is one: 65504 / 7 would round up to 9360)
    const __half s = __half_as_ushort(top) >= 0x7c00u
                         ? __ushort_as_half(0x7fff)
                         : __hmin(__float2half_rn(__fmul_rn(__half2float(top), 1.0f / 7.0f)), __float2half_rn(9352.0f));
    const float sf = __half2float(s), inv = sf == 0.0f ? 0.0f : 1.0f / sf;
    // rint(y) + 8 in the low bits of y + (1.5 * 2^23 + 8): the sum rounds to a whole number, to
    // even at ties. |y| is below 7.5 unless the scale lost bits (a subnormal f16): then clamped.
    const bool coarse = sf < 6.1e-5f;
    uint32_t y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = __half22float2(half2_at(x, i));
      float f0 = __fmul_rn(v.x, inv), f1 = __fmul_rn(v.y, inv);
      if (coarse) {
        f0 = fminf(fmaxf(f0, -7.0f), 7.0f);
        f1 = fminf(fmaxf(f1, -7.0f), 7.0f);
      }
      y[2 * i] = __float_as_uint(__fadd_rn(f0, 12582920.0f));
      y[2 * i + 1] = __float_as_uint(__fadd_rn(f1, 12582920.0f));
    }
    uint32_t codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes[i] = __byte_perm(__byte_perm(y[4 * i], y[4 * i + 1], 0x0040), __byte_perm(y[4 * i + 2], y[4 * i + 3], 0x0040), 0x5410);
      codes[i] &= 0x0f0f0f0fu;
      // dims + 16 of the group, the next lane's, into the high halves
      codes[i] |= __shfl_down_sync(0xffffffffu, codes[i], 1) << 4;
    }
    if (ok && (ch & 1) == 0) {
      reinterpret_cast<uint4*>(dst)[ch >> 1] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
      reinterpret_cast<__half*>(scale)[ch >> 1] = s;
    }
  }
}

// What piece `ch` (8 values) of a stored row is read from, and its values.
template <int FMT>
struct StoredPiece {
  uint4 codes;
  float scale;  // e4m3
  __half s;     // 4 bits
};

template <int FMT>
__device__ __forceinline__ StoredPiece<FMT> load_piece(const char* src, const char* scale, int ch) {
  StoredPiece<FMT> p{};
  if constexpr (FMT == QSA_PAGE_F16) {
    p.codes = reinterpret_cast<const uint4*>(src)[ch];
  } else {
    const uint2 w = FMT == QSA_PAGE_FP8 ? reinterpret_cast<const uint2*>(src)[ch]
                                        : reinterpret_cast<const uint2*>(src + (ch >> 2) * 16)[ch & 1];
    p.codes.x = w.x;
    p.codes.y = w.y;
    if constexpr (FMT == QSA_PAGE_FP8) p.scale = *reinterpret_cast<const float*>(scale);
    else p.s = reinterpret_cast<const __half*>(scale)[ch >> 2];
  }
  return p;
}

template <int FMT>
__device__ __forceinline__ uint4 values_of(const StoredPiece<FMT>& p, int ch) {
  uint32_t out[4] = {p.codes.x, p.codes.y, p.codes.z, p.codes.w};
#pragma unroll
  for (int i = 0; i < (FMT == QSA_PAGE_F16 ? 0 : 4); ++i) {
    const uint32_t w = i < 2 ? p.codes.x : p.codes.y;
    __half2 h;
    if constexpr (FMT == QSA_PAGE_FP8) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * (i & 1))) & 0xffffu), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      h = __floats2half2_rn(__fmul_rn(f.x, p.scale), __fmul_rn(f.y, p.scale));
    } else {
      // two codes as 1024 + n in f16 (0x6400 | n), minus 1032: exact
      const uint32_t b = (__byte_perm((ch & 2) ? w >> 4 : w, 0, (i & 1) ? 0x4342 : 0x4140) & 0x000f000fu) | 0x64006400u;
      h = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&b), __float2half2_rn(1032.0f)), __half2half2(p.s));
    }
    out[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Piece e of a CTA's tokens is piece e % per_token of token e / per_token: a thread's
// pieces are kRowThreads apart, so one division serves them all.
struct PieceCursor {
  int per_token, tok, in, step_tok, step_in;
  __device__ __forceinline__ PieceCursor(int per) : per_token(per) {
    tok = int(threadIdx.x) / per;
    in = int(threadIdx.x) - tok * per;
    step_tok = kRowThreads / per;
    step_in = kRowThreads - step_tok * per;
  }
  __device__ __forceinline__ void next() {
    tok += step_tok;
    in += step_in;
    if (in >= per_token) {
      in -= per_token;
      ++tok;
    }
  }
};

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) paged_write_kernel(PagedView c, PagedRows r, const __half* __restrict__ k,
                                                                  const __half* __restrict__ v, int tokens) {
  constexpr int CH = D / 16;
  __shared__ TokenPlace s_at[kRowTokens];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * tokens, n = min(tokens, r.n_rows - t0);
  PieceCursor p(c.n_kv_heads * CH);
  // bytes from a head's rows (scales) of a page to the next one's
  const int head_rows = page_row_bytes_c<FMT>(D) << c.page_shift, head_scales = page_scale_bytes_c<FMT>(D) << c.page_shift;
  bool found = false;
  do {  // (the same trips in every thread: all take part in the shuffles)
    // the rows come while the CTA finds their places
    Piece x[kRowBatch], y[kRowBatch];
    PieceCursor q = p;
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) {
      x[i] = y[i] = Piece{};
      if (q.tok < n) {
        const int head = q.in / CH, ch = q.in % CH;
        const int64_t off = (t0 + q.tok) * r.row_stride + head * D + ch * (FMT == QSA_PAGE_F16 ? 8 : 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[i].v[h] = reinterpret_cast<const uint4*>(k + off)[h * (FMT == QSA_PAGE_F16 ? CH : 1)];
          y[i].v[h] = reinterpret_cast<const uint4*>(v + off)[h * (FMT == QSA_PAGE_F16 ? CH : 1)];
        }
      }
      q.next();
    }
    if (!found) find_tokens<FMT, D>(c, r, t0, n, s_at);
    found = true;
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) {
      TokenPlace at{-1, 0};
      if (p.tok < n) at = s_at[p.tok];
      const bool ok = at.rows >= 0;
      const int head = p.in / CH, ch = p.in % CH;
      const int64_t row = at.rows + head * head_rows, scale = at.scales + head * head_scales;
      store_piece<FMT, D>(x[i], c.k + row, c.ks + scale, ch, ok);
      store_piece<FMT, D>(y[i], c.v + row, c.vs + scale, ch, ok);
      p.next();
    }
  } while (__syncthreads_or(p.tok < n));
}

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) paged_read_kernel(PagedView c, PagedRows r, __half* __restrict__ k,
                                                                 __half* __restrict__ v, int tokens) {
  constexpr int CH = D / 8;
  __shared__ TokenPlace s_at[kRowTokens];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * tokens, n = min(tokens, r.n_rows - t0);
  find_tokens<FMT, D>(c, r, t0, n, s_at);
  PieceCursor p(c.n_kv_heads * CH);
  // bytes from a head's rows (scales) of a page to the next one's
  const int head_rows = page_row_bytes_c<FMT>(D) << c.page_shift, head_scales = page_scale_bytes_c<FMT>(D) << c.page_shift;
  while (p.tok < n) {
    StoredPiece<FMT> x[kReadBatch], y[kReadBatch];
    PieceCursor q = p;
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      x[i] = y[i] = StoredPiece<FMT>{};
      if (q.tok < n) {
        const TokenPlace at = s_at[q.tok];
        if (at.rows >= 0) {
          const int head = q.in / CH, ch = q.in % CH;
          const int64_t row = at.rows + head * head_rows, scale = at.scales + head * head_scales;
          if (k) x[i] = load_piece<FMT>(c.k + row, c.ks + scale, ch);
          if (v) y[i] = load_piece<FMT>(c.v + row, c.vs + scale, ch);
        }
      }
      q.next();
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int64_t at = p.tok < n ? s_at[p.tok].rows : -2;
      if (at != -2) {  // (padding rows stay as they are)
        const int64_t off = (t0 + p.tok) * r.row_stride + p.in * 8;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if (k) *reinterpret_cast<uint4*>(k + off) = at < 0 ? zero : values_of<FMT>(x[i], p.in % CH);
        if (v) *reinterpret_cast<uint4*>(v + off) = at < 0 ? zero : values_of<FMT>(y[i], p.in % CH);
      }
      p.next();
    }
  }
}

// Tokens a CTA takes: few enough to give every SM a few CTAs, and no more than two batches of
// pieces a thread: finding places costs two rounds of loads, which the other CTAs hide.
int row_tokens(const PagedView& c, const PagedRows& r, int n_sms) {
  const int spread = (r.n_rows + 4 * n_sms - 1) / (4 * n_sms);
  const int full = 2 * kRowThreads / (c.n_kv_heads * (c.head_dim / 16));
  const int most = full < kRowTokens ? full : kRowTokens;
  const int t = spread < most ? spread : most;
  return t < 1 ? 1 : t;
}

}  // namespace

cudaError_t launch_paged_write(const PagedView& c, int format, const PagedRows& r, const void* k, const void* v,
                               int n_sms, cudaStream_t s) {
  const int tokens = row_tokens(c, r, n_sms);
  const dim3 grid((r.n_rows + tokens - 1) / tokens), block(kRowThreads);
#define QSA_WRITE(F, D)                                                                                      \
  if (format == F && c.head_dim == D)                                                                        \
    return launch_pdl(paged_write_kernel<F, D>, grid, block, 0, s, 1, c, r, (const __half*)k, (const __half*)v, tokens)
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
  const int tokens = row_tokens(c, r, n_sms);
  const dim3 grid((r.n_rows + tokens - 1) / tokens), block(kRowThreads);
#define QSA_READ(F, D)                                                                            \
  if (format == F && c.head_dim == D)                                                             \
    return launch_pdl(paged_read_kernel<F, D>, grid, block, 0, s, 1, c, r, (__half*)k, (__half*)v, tokens)
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
