// Dense GQA attention of every sequence's newest tokens over a paged K/V cache.
//
// Web page "Part 10", section "なぜFlash Attentionがcontext長に比例していたのか": dense
// attention reads the whole context for every token, which is what the sparse path avoids.
//   out = sum_c softmax_c(scale * q.K_c) V_c over the cells c < len - T + u + 1 of query u < T.
// One pass with a running maximum and sum; a sequence's cells are split over CTAs, whose
// partials (m, l, o) are merged as sum_s e^(m_s - M) o_s / sum_s e^(m_s - M) l_s.
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kPaThreads = 128;
constexpr int kPaRows = 8 * QSA_MAX_QUERIES;  // (query, head) rows of one KV head at most

template <int FMT, int D>
__device__ __forceinline__ void row_values(float (&x)[D / 32], const char* pages, const char* scales, int64_t page_base,
                                           int64_t scale_base, int row, int lane) {
  const char* src = pages + page_base + int64_t(row) * page_row_bytes_c<FMT>(D);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int d = lane * (D / 32) + i;
    if constexpr (FMT == QSA_PAGE_F16) {
      x[i] = __half2float(reinterpret_cast<const __half*>(src)[d]);
    } else if constexpr (FMT == QSA_PAGE_FP8) {
      const __half c = __half(__nv_cvt_fp8_to_halfraw(reinterpret_cast<const unsigned char*>(src)[d], __NV_E4M3));
      x[i] = __half2float(c) * (reinterpret_cast<const float*>(scales + scale_base))[row];
    } else {
      const __half s = (reinterpret_cast<const __half*>(scales + scale_base) + int64_t(row) * (D / 32))[d / 32];
      const unsigned b = reinterpret_cast<const unsigned char*>(src)[d / 32 * 16 + d % 16];
      x[i] = __half2float(__hmul(__int2half_rn(int((d & 16) ? b >> 4 : b & 15) - 8), s));
    }
  }
}

// CTA (split, sequence x KV head): its warps take the split's cells in turn.
template <int FMT, int D>
__global__ void __launch_bounds__(kPaThreads) paged_split_kernel(PagedView c, PagedAttendArgs a, float* __restrict__ part,
                                                                 int n_splits) {
  constexpr int P = D / 32, W = kPaThreads / 32;
  __shared__ float s_q[kPaRows][D];
  __shared__ float s_m[W][kPaRows], s_l[W][kPaRows];
  __shared__ float s_o[kPaRows][D];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.x / n_splits, split = blockIdx.x % n_splits;
  const int seq = pair / c.n_kv_heads, g = pair % c.n_kv_heads;
  const int G = a.n_q_heads / c.n_kv_heads, T = a.n_queries, R = G * T;
  const __half* q = static_cast<const __half*>(a.q);
  for (int e = threadIdx.x; e < R * D; e += kPaThreads) {
    const int r = e / D, u = r / G, h = r % G;
    s_q[r][e % D] = __half2float(q[(int64_t(seq) * T + u) * a.q_stride + (g * G + h) * D + e % D]);
  }
  for (int e = threadIdx.x; e < R * D; e += kPaThreads) s_o[e / D][e % D] = 0.0f;
  __syncthreads();
  int len = a.seq_lens[seq];
  if (len < 0) {
    if (threadIdx.x == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    len = 0;
  }
  if (len > ((long long)a.table_width << c.page_shift)) {
    if (threadIdx.x == 0) record_status(a.status, QSA_ERR_CAPACITY);
    len = a.table_width << c.page_shift;
  }
  const int per = (len + n_splits - 1) / n_splits;
  const int c0 = min(len, split * per), c1 = min(len, c0 + per);
  float m[kPaRows], l[kPaRows], o[kPaRows][P];
#pragma unroll
  for (int r = 0; r < kPaRows; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) o[r][i] = 0.0f;
  }
  for (int cell = c0 + warp; cell < c1; cell += W) {
    const int page = a.block_table[(long long)seq * a.table_width + (cell >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
      continue;
    }
    const int row = row_in_page(c, g, cell & ((1 << c.page_shift) - 1));
    float kx[P], vx[P];
    row_values<FMT, D>(kx, c.k, c.ks, page * c.page_stride, page * c.scale_stride, row, lane);
    row_values<FMT, D>(vx, c.v, c.vs, page * c.page_stride, page * c.scale_stride, row, lane);
#pragma unroll
    for (int r = 0; r < kPaRows; ++r) {
      if (r < R && cell < len - T + r / G + 1) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) z = fmaf(s_q[r][lane * P + i], kx[i], z);
        z = warp_sum(z) * a.sm_scale;
        // a -inf logit has no weight; a NaN one makes l and o NaN (the maximum skips it)
        const float mn = fmaxf(m[r], z), f = m[r] == mn ? 1.0f : expf(m[r] - mn), p = z == -INFINITY ? 0.0f : expf(z - mn);
        m[r] = mn;
        l[r] = l[r] * f + p;
#pragma unroll
        for (int i = 0; i < P; ++i) o[r][i] = o[r][i] * f + p * vx[i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kPaRows; ++r) {
    if (lane == 0) {
      s_m[warp][r] = m[r];
      s_l[warp][r] = l[r];
    }
  }
  __syncthreads();
  for (int w = 0; w < W; ++w) {  // the warps add their share in turn: a fixed order
    if (warp == w) {
#pragma unroll
      for (int r = 0; r < kPaRows; ++r) {
        if (r < R) {
          float M = -INFINITY;
          for (int x = 0; x < W; ++x) M = fmaxf(M, s_m[x][r]);
          const float f = l[r] == 0.0f ? 0.0f : expf(m[r] - M);
#pragma unroll
          for (int i = 0; i < P; ++i) s_o[r][lane * P + i] += f * o[r][i];
        }
      }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < R * (D + 1); e += kPaThreads) {
    const int r = e / (D + 1), d = e % (D + 1);
    float M = -INFINITY, L = 0.0f;
    for (int x = 0; x < W; ++x) M = fmaxf(M, s_m[x][r]);
    for (int x = 0; x < W; ++x)
      if (s_l[x][r] != 0.0f) L += expf(s_m[x][r] - M) * s_l[x][r];
    if (n_splits == 1) {
      const int64_t row = (int64_t(seq) * T + r / G) * a.n_q_heads + g * G + r % G;
      if (d < D) a.out[row * D + d] = L == 0.0f ? 0.0f : s_o[r][d] / L;
      else if (a.lse) a.lse[row] = L == 0.0f ? -INFINITY : M + logf(L);
    } else {  // partial of (sequence, head, split, row): o [D], m, l
      float* p = part + (int64_t(blockIdx.x) * R + r) * (D + 2);
      if (d < D) {
        p[d] = s_o[r][d];
      } else {
        p[D] = M;
        p[D + 1] = L;
      }
    }
  }
}

__global__ void __launch_bounds__(128) paged_merge_kernel(PagedAttendArgs a, const float* __restrict__ part, int n_kv_heads,
                                                          int D, int n_splits) {
  pdl_wait();
  const int G = a.n_q_heads / n_kv_heads, T = a.n_queries, R = G * T;
  const int seq = blockIdx.x / n_kv_heads, g = blockIdx.x % n_kv_heads, r = blockIdx.y, u = r / G, h = g * G + r % G;
  const float* p0 = part + (int64_t(blockIdx.x) * n_splits * R + r) * (D + 2);
  const int64_t step = int64_t(R) * (D + 2);
  float M = -INFINITY, L = 0.0f;
  for (int s = 0; s < n_splits; ++s) M = fmaxf(M, p0[s * step + D]);
  for (int s = 0; s < n_splits; ++s)
    if (p0[s * step + D + 1] != 0.0f) L += expf(p0[s * step + D] - M) * p0[s * step + D + 1];
  const int64_t row = (int64_t(seq) * T + u) * a.n_q_heads + h;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float acc = 0.0f;
    for (int s = 0; s < n_splits; ++s)
      if (p0[s * step + D + 1] != 0.0f) acc += expf(p0[s * step + D] - M) * p0[s * step + d];
    a.out[row * D + d] = L == 0.0f ? 0.0f : acc / L;
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.0f ? -INFINITY : M + logf(L);
}

}  // namespace

// Splits per (sequence, KV head): about four CTAs an SM over the whole batch. With one split
// the results are written directly, else there are fewer than 8 * n_sms partials.
static int paged_splits(int pairs, int n_sms) { return pairs >= 4 * n_sms ? 1 : (4 * n_sms + pairs - 1) / pairs; }

size_t paged_workspace_bytes(int head_dim, int n_q_heads, int n_kv_heads, int n_queries, int n_sms) {
  return align256(size_t(8) * n_sms * (n_q_heads / n_kv_heads * n_queries) * (head_dim + 2) * sizeof(float));
}

cudaError_t launch_paged_attend(const PagedView& c, int format, const PagedAttendArgs& a, int n_sms, cudaStream_t s) {
  const int pairs = a.n_seqs * c.n_kv_heads, R = a.n_q_heads / c.n_kv_heads * a.n_queries;
  const int n_splits = paged_splits(pairs, n_sms);
  float* part = static_cast<float*>(a.workspace);
  const dim3 grid(pairs * n_splits);
  cudaError_t e = cudaErrorInvalidValue;
#define QSA_PA(F, D)                      \
  if (format == F && c.head_dim == D)     \
  e = launch_pdl(paged_split_kernel<F, D>, grid, dim3(kPaThreads), 0, s, 1, c, a, part, n_splits)
  QSA_PA(QSA_PAGE_F16, 64);
  QSA_PA(QSA_PAGE_F16, 128);
  QSA_PA(QSA_PAGE_FP8, 64);
  QSA_PA(QSA_PAGE_FP8, 128);
  QSA_PA(QSA_PAGE_INT4, 64);
  QSA_PA(QSA_PAGE_INT4, 128);
#undef QSA_PA
  if (e != cudaSuccess || n_splits == 1) return e;
  return launch_pdl(paged_merge_kernel, dim3(pairs, R), dim3(128), 0, s, 1, a, (const float*)part, c.n_kv_heads,
                    c.head_dim, n_splits);
}

}  // namespace qsa
