// Verification of drafted tokens against the target's probabilities from given random
// numbers (speculative decoding; "Part 10", section "incremental pooled-key cache
// （COMMON-004）", requires that its dirty writes stay out of the pooled cache).
//
//   draft i accepted iff u_i q_i(d_i) < p_i(d_i) and all before it are;
//   next token: the lowest j with sum_{i<=j} w_i > u sum_i w_i, w = max(p_m - q_m, 0) at the
//   first rejected draft m, or w = p_n after the last.
// Only row m is read (of target and draft), twice: once for its sum, once (a warp's part of
// it) to find j. Sums are f64: among 150,000 weights an f32 sum is off by more than the
// small weights, and the token would depend on the order.
#include "qsa_device.cuh"

namespace qsa {

namespace {

constexpr int kVfThreads = 1024;
constexpr int kVfWarps = kVfThreads / 32;

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Row the next token is drawn from.
struct VerifyRow {
  const float* p;
  const float* q;  // null: no draft probabilities, or none to subtract
  int drop;        // token whose weight is 0 (a rejected draft without probabilities), -1: none
};

__device__ __forceinline__ double weight(const VerifyRow& w, int j) {
  double x = w.p[j];
  if (w.q) x -= (double)w.q[j];
  return j != w.drop && x > 0.0 ? x : 0.0;  // NaN counts as 0
}

// One CTA per sequence; warp w holds the tokens [w*per, (w+1)*per).
__global__ void __launch_bounds__(kVfThreads) verify_kernel(VerifyArgs a) {
  __shared__ double s_sum[kVfWarps];
  __shared__ float s_top[kVfWarps];
  __shared__ int s_at[kVfWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seq = blockIdx.x;
  int n = a.n_drafts ? a.n_drafts[seq] : a.max_drafts;
  if (n < 0 || n > a.max_drafts) {
    if (threadIdx.x == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    n = n < 0 ? 0 : a.max_drafts;
  }
  const float* u = a.uniforms + (int64_t)seq * (a.max_drafts + 1);
  const float* target = a.target + (int64_t)seq * (a.max_drafts + 1) * a.target_stride;
  const float* draft = a.draft ? a.draft + (int64_t)seq * a.max_drafts * a.draft_stride : nullptr;
  const int32_t* tokens = a.tokens + (int64_t)seq * a.max_drafts;
  int m = 0;
  for (; m < n; ++m) {
    const int d = tokens[m];
    if (d < 0 || d >= a.vocab) {
      if (threadIdx.x == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
      break;
    }
    const double q = draft ? (double)draft[m * a.draft_stride + d] : 1.0;
    if (!((double)u[m] * q < (double)target[m * a.target_stride + d])) break;
  }
  VerifyRow w{target + m * a.target_stride, m < n && draft ? draft + m * a.draft_stride : nullptr,
              m < n && !draft ? tokens[m] : -1};
  const int per = (a.vocab + kVfWarps - 1) / kVfWarps;
  const int j0 = min(a.vocab, warp * per), j1 = min(a.vocab, j0 + per);
  double mine = 0.0;
  for (int j = j0 + lane; j < j1; j += 32) mine += weight(w, j);
  mine = warp_sum_f64(mine);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  double total = 0.0;
  for (int x = 0; x < kVfWarps; ++x) total += s_sum[x];
  if (total > 0.0) {
    double t = (double)fmaxf(u[a.max_drafts], 0.0f) * total;
    // the first warp whose tokens pass t, or the last with a weight
    int owner = -1, last = 0;
    double before = 0.0, upto = 0.0;
    for (int x = 0; x < kVfWarps; ++x) {
      if (s_sum[x] > 0.0) last = x;
      if (owner < 0 && upto + s_sum[x] > t) {
        owner = x;
        before = upto;
      }
      upto += s_sum[x];
    }
    if (owner < 0) {
      owner = last;  // no token passes: take the last with a weight
      t = INFINITY;
    }
    if (warp != owner) return;
    int found = -1, positive = j0;
    for (int b = j0; b < j1 && found < 0; b += 32) {
      const int j = b + lane;
      const double x = j < j1 ? weight(w, j) : 0.0;
      double c = x;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && before + c > t);
      const unsigned pos = __ballot_sync(0xffffffffu, x > 0.0);
      if (pos) positive = b + 31 - __clz(pos);
      if (hit) found = b + __ffs(hit) - 1;
      before += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) {
      a.n_accepted[seq] = m;
      a.next_token[seq] = found >= 0 ? found : positive;
    }
    return;
  }
  // no weight is positive: the lowest token with the largest probability
  float top = -1.0f;
  int at = 0;
  for (int j = j0 + lane; j < j1; j += 32)
    if (w.p[j] > top) {
      top = w.p[j];
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
    for (int x = 1; x < kVfWarps; ++x)
      if (s_top[x] > s_top[0]) {
        s_top[0] = s_top[x];
        s_at[0] = s_at[x];
      }
    a.n_accepted[seq] = m;
    a.next_token[seq] = s_at[0];
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int n_sms, cudaStream_t s) {
  return launch_pdl(verify_kernel, dim3(a.n_seqs), dim3(kVfThreads), 0, s, 1, a);
}

}  // namespace qsa
