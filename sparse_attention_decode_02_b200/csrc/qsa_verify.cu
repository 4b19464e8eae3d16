// Verification of drafted tokens against the target's probabilities from given random
// numbers (speculative decoding; "Part 10", section "incremental pooled-key cache
// （COMMON-004）", requires that its dirty writes stay out of the pooled cache).
//
//   draft i accepted iff u_i q_i(d_i) < p_i(d_i) and all before it are;
//   next token: the lowest j with sum_{i<=j} w_i > u sum_i w_i, w = max(p_m - q_m, 0) at the
//   first rejected draft m, or w = p_n after the last.
// Only row m is read (of target and draft), once for its sum, and the part of it that one warp
// summed again to find j: the bytes of one or two rows bound it, and for few sequences the
// chain token -> its probabilities -> row -> sums -> token. A cluster of CTAs shares a row, as
// many as fill the GPU; their sums meet in distributed shared memory, so that one launch does.
// Measured on B200 (us; share of a copy's 6,568 GB/s): 64 sequences x 151,936 tokens 19 (48%),
// 256 x 100,003 40 to 42 (70 to 72%), one x 32,000 4.3, one x 151,936 6.8. The small ones are that chain.
// Sums are f64: among 150,000 weights an f32 sum is off by more than the small weights, and
// the token would depend on the order.
#include <atomic>

#include <cooperative_groups.h>

#include "qsa_device.cuh"

namespace cg = cooperative_groups;

namespace qsa {

namespace {

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfPerSm = 4;                // CTAs an SM holds (60 registers a thread)
constexpr int kVfMaxCluster = 16;
constexpr int kVfBatch = 8;                // tokens a lane has in flight from each row
constexpr int kVfBlock = 32 * kVfBatch;    // tokens of a warp's batch

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The row the next token is drawn from: p, less q (null: nothing), without the token `drop`.
struct VerifyRow {
  const float *p, *q;
  int drop;
};

// Weights of the tokens first, first + STEP, ... below `end`: NaN counts as 0. All loads first.
template <int STEP>
__device__ __forceinline__ void weights(const VerifyRow& r, int first, int end, double (&w)[kVfBatch]) {
  float x[kVfBatch], y[kVfBatch];
#pragma unroll
  for (int i = 0; i < kVfBatch; ++i) {
    const int j = first + STEP * i;
    const bool in = i * STEP < end - first && j != r.drop;
    x[i] = in ? r.p[j] : 0.0f;
    y[i] = in && r.q ? r.q[j] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kVfBatch; ++i) {
    const bool more = x[i] > y[i];
    w[i] = (double)(more ? x[i] : 0.0f) - (double)(more ? y[i] : 0.0f);
  }
}

__global__ void __launch_bounds__(kVfThreads) verify_kernel(VerifyArgs a) {
  __shared__ double s_sum[kVfWarps], s_total[kVfMaxCluster];
  __shared__ float s_top[kVfWarps], s_ctop[kVfMaxCluster];
  __shared__ int s_at[kVfWarps], s_cat[kVfMaxCluster];
  const cg::cluster_group cluster = cg::this_cluster();
  const int size = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seq = blockIdx.x / size;
  cluster_arrive_relaxed();  // waited for before the first store into another CTA's shared memory
  pdl_launch_dependents();
  pdl_wait();

  // ---- accepted drafts: lane i looks at drafts i and i + 32 (every warp for itself) ----
  int n = a.n_drafts ? a.n_drafts[seq] : a.max_drafts;
  const float* const u = a.uniforms + (int64_t)seq * (a.max_drafts + 1);
  const float* const target = a.target + (int64_t)seq * (a.max_drafts + 1) * a.target_stride;
  const float* const draft = a.draft ? a.draft + (int64_t)seq * a.max_drafts * a.draft_stride : nullptr;
  const int32_t* const tokens = a.tokens + (int64_t)seq * a.max_drafts;
  const float u_last = u[a.max_drafts];
  if (n < 0 || n > a.max_drafts) {
    if (rank == 0 && threadIdx.x == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    n = n < 0 ? 0 : a.max_drafts;
  }
  int m = n, d_m = -1;
  for (int b = 0; b < n && m == n; b += 32) {
    const int i = b + lane;
    int d = -1;
    bool kept = true, odd = false;
    if (i < n) {
      d = tokens[i];
      odd = d < 0 || d >= a.vocab;
      kept = false;
      if (!odd) {
        const double q = draft ? (double)draft[i * a.draft_stride + d] : 1.0;
        const float x = u[i];  // (a NaN keeps nothing)
        kept = (double)(x < 0.0f ? 0.0f : x) * q < (double)target[i * a.target_stride + d];
      }
    }
    const unsigned stop = __ballot_sync(0xffffffffu, !kept), bad = __ballot_sync(0xffffffffu, odd);
    if (stop) {
      const int at = __ffs(stop) - 1;
      m = b + at;
      d_m = __shfl_sync(0xffffffffu, d, at);
      // (an id that is reported is one that was looked at: the first rejected)
      if (((bad >> at) & 1) && rank == 0 && threadIdx.x == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    }
  }
  // (a rejected draft without probabilities has weight 0)
  const VerifyRow row{target + m * a.target_stride, m < n && draft ? draft + m * a.draft_stride : nullptr,
                      m < n && !draft ? d_m : -1};

  // ---- sums: warp w of CTA r has the tokens [(r * 8 + w) * per, + per), in at most 32 chunks
  // of whole blocks; lane i keeps chunk i's ----
  const int per = (a.vocab + size * kVfWarps - 1) / (size * kVfWarps);
  const int j0 = int(min((long long)a.vocab, (long long)(rank * kVfWarps + warp) * per)), j1 = min(a.vocab, j0 + per);
  const int chunk = (per + 32 * kVfBlock - 1) / (32 * kVfBlock) * kVfBlock;
  double chunk_sum = 0.0;
  for (int i = 0, c0 = j0; c0 < j1; ++i, c0 += chunk) {
    const int c1 = min(j1, c0 + chunk);
    double sum = 0.0;
    for (int b = c0; b < c1; b += kVfBlock) {
      double w[kVfBatch];
      weights<32>(row, b + lane, c1, w);
#pragma unroll
      for (int k = kVfBatch / 2; k >= 1; k >>= 1)
#pragma unroll
        for (int e = 0; e < k; ++e) w[e] += w[e + k];
      sum += w[0];
    }
    sum = warp_sum_f64(sum);
    if (lane == i) chunk_sum = sum;
  }
  const double mine = warp_sum_f64(chunk_sum);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  cluster_wait();  // every CTA of the cluster has started: its shared memory may be written
  if (warp == 0 && lane < size) {  // this CTA's sum to every CTA of the cluster
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kVfWarps; ++w) all += s_sum[w];
    *cluster.map_shared_rank(&s_total[rank], lane) = all;
  }
  cluster.sync();
  double total = 0.0;
  for (int r = 0; r < size; ++r) total += s_total[r];

  if (total > 0.0) {
    // ---- the first CTA, and warp of it, whose tokens pass t (the last with a weight if none) ----
    double t = (double)fmaxf(u_last, 0.0f) * total, upto = 0.0, before = 0.0;
    int owner = -1, last = 0;
    for (int r = 0; r < size; ++r) {
      if (s_total[r] > 0.0) last = r;
      if (owner < 0 && upto + s_total[r] > t) {
        owner = r;
        before = upto;
      }
      upto += s_total[r];
    }
    if (owner < 0) {
      owner = last;
      t = INFINITY;
    }
    if (rank != owner) return;
    upto = before;
    owner = -1;
    last = 0;
    for (int w = 0; w < kVfWarps; ++w) {
      if (s_sum[w] > 0.0) last = w;
      if (owner < 0 && upto + s_sum[w] > t) {
        owner = w;
        before = upto;
      }
      upto += s_sum[w];
    }
    if (owner < 0) {  // (rounding: the warps' sums in turn fall short of the CTA's)
      owner = last;
      t = INFINITY;
    }
    if (warp != owner) return;
    // ---- the chunk, then its blocks in turn: lane i takes the i-th 8 tokens of a block ----
    const auto scan = [&](double v) {  // inclusive over the lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
      }
      return v;
    };
    const double upto_chunk = scan(chunk_sum);
    const unsigned pass = __ballot_sync(0xffffffffu, chunk_sum > 0.0 && before + upto_chunk > t);
    const unsigned some = __ballot_sync(0xffffffffu, chunk_sum > 0.0);
    const int in = pass ? __ffs(pass) - 1 : 31 - __clz(some);  // (no chunk passes t: the last with a weight)
    if (!pass) t = INFINITY;
    before += __shfl_sync(0xffffffffu, upto_chunk - chunk_sum, in);
    const int c0 = j0 + in * chunk, c1 = min(j1, c0 + chunk);
    int found = -1;      // the last token with a weight so far
    bool passed = false;
    for (int b = c0; b < c1 && !passed; b += kVfBlock) {
      double w[kVfBatch], have = 0.0;
      weights<1>(row, b + lane * kVfBatch, c1, w);
#pragma unroll
      for (int i = 0; i < kVfBatch; ++i) have += w[i];
      const double to = scan(have);
      double run = before + to - have;
      int at = -1;
      bool hit = false;
#pragma unroll
      for (int i = 0; i < kVfBatch; ++i) {
        run += w[i];
        if (w[i] > 0.0 && !hit) {
          at = b + lane * kVfBatch + i;
          hit = run > t;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit), any = __ballot_sync(0xffffffffu, at >= 0);
      passed = hits != 0;
      if (any) found = __shfl_sync(0xffffffffu, at, hits ? __ffs(hits) - 1 : 31 - __clz(any));
      before += __shfl_sync(0xffffffffu, to, 31);
    }
    if (lane == 0) {
      a.n_accepted[seq] = m;
      a.next_token[seq] = found;
    }
    return;
  }

  // ---- no weight is positive: the lowest token with the largest probability ----
  float top = -1.0f;
  int at = 0;
  for (int j = j0 + lane; j < j1; j += 32)
    if (row.p[j] > top) {
      top = row.p[j];
      at = j;
    }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, top, off);
    const int z = __shfl_xor_sync(0xffffffffu, at, off);
    if (y > top || (y == top && z < at)) {
      top = y;
      at = z;
    }
  }
  if (lane == 0) {
    s_top[warp] = top;
    s_at[warp] = at;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kVfWarps; ++w)
      if (s_top[w] > s_top[0]) {
        s_top[0] = s_top[w];
        s_at[0] = s_at[w];
      }
    *cluster.map_shared_rank(&s_ctop[rank], 0) = s_top[0];
    *cluster.map_shared_rank(&s_cat[rank], 0) = s_at[0];
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    for (int r = 1; r < size; ++r)
      if (s_ctop[r] > s_ctop[0]) {
        s_ctop[0] = s_ctop[r];
        s_cat[0] = s_cat[r];
      }
    a.n_accepted[seq] = m;
    a.next_token[seq] = s_cat[0];
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int n_sms, int device, cudaStream_t s) {
  // CTAs a sequence: as many (a power of two) as the GPU holds at once for the whole batch, with
  // a token for every thread. At 64 x 151,936 tokens 8 CTAs take 19 us (512-thread CTAs, of
  // which an SM holds two, 33); at 256 x 100,003 2 take 40 us and 4, in two waves, 47. Clusters
  // of 16, which fit fewer places, only up to half of that: 12 sequences 9.5 us against 10.4
  // with 8, one 6.8 against 9.7, but 36 sequences 19 against 17.6.
  int size = kVfMaxCluster;
  if (2LL * a.n_seqs * size > kVfPerSm * (long long)n_sms) size /= 2;
  while (size > 1 && ((long long)a.n_seqs * size > kVfPerSm * (long long)n_sms || a.vocab < size * kVfThreads)) size /= 2;
  if (size > 8) {  // more than the portable 8: allowed once a device
    static std::atomic<unsigned long long> ready{0};
    const unsigned long long bit = 1ull << (device & 63);
    if (device >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
      const cudaError_t e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (device < 64) ready.fetch_or(bit, std::memory_order_release);
    }
  }
  return launch_pdl(verify_kernel, dim3(a.n_seqs * size), dim3(kVfThreads), 0, s, size, a);
}

}  // namespace qsa
