// Dense GQA attention of every sequence's newest tokens over a paged K/V cache.
//
// Web page "Part 10", section "なぜFlash Attentionがcontext長に比例していたのか": dense
// attention reads the whole context for every token, which is what the sparse path avoids.
//   out = sum_c softmax_c(scale * q.K_c) V_c over the cells c < len - T + u + 1 of query u < T.
// One pass over K and V with a running maximum and sum, split over the whole batch:
//  - The (sequence, KV head) segments of a batch, cut into tiles of cells (a segment's start
//    counts as two more), form one list; team i of N takes the i-th N-th of it (found from
//    seq_lens on the device), so ragged batches and single long sequences load every SM alike.
//    A segment cut by a border is written as partials (m, l, o), at most two a team, which
//    paged_merge_kernel joins: sum_s w_s o_s / sum_s w_s l_s, w_s = exp(scale (m_s - M)). Whole segments
//    are written directly.
//  - One CTA an SM: two or three teams of four warps, each with its own share of the list, and
//    a warpgroup whose warps load for one team each and leave their registers to the teams.
//    Tiles of 64 cells come into the team's ring in shared memory (TMA tiles of a head's rows
//    of a page, scales by 16-byte copies of the loading lanes) across the segments' borders, so that the loads do not
//    pause while a segment's results are joined. Each warp of the team takes 16 cells of a
//    tile, with no barrier between warps inside a segment. The products run on the tensor
//    cores, transposed: S^T = K q^T and O^T = V^T P^T, cells resp. dims as the 16 MMA rows
//    and the (query, head) rows of the KV head as columns, so that no MMA row is padding.
//    mma.sync rather than tcgen05: with one query the bytes bound the f16 and e4m3 forms, and
//    8- and 4-bit rows become f16 operands in registers, where mma.sync takes them and tcgen05
//    would want them written back. (Not so for 32 columns over 4-bit rows: there the products
//    alone take twice as long as the bytes.)
//  - Precision: codes are exact in f16 (e4m3 scales multiply logits and weights in f32; a 4-bit
//    value is an f16 product by definition). A weight enters the second product as two f16
//    terms of 2^7 p (22 bits, down to 2^-32 of the largest), which costs a second MMA and
//    keeps the result at f32 precision; an e4m3 weight, p times the row's scale, relative to
//    the largest scale of its 16 rows. The products of each 16 cells are added to the
//    running output in f32: the MMA's own sums truncate, and over a long chain that adds up.
//  - The newest T - 1 cells are not seen by every query, and an infinity or a NaN in them must
//    not reach the others (0 * NaN is NaN): such a V row stays out of the MMA and is added to
//    the queries that see it.
//  - Code that runs once a segment is kept short and rolled: instructions come cold from L2
//    at some 50 cycles each, so an unrolled copy of the tile's code for the segment's end, or
//    a result loop unrolled over the columns, cost 19 us a segment.
// Measured on B200 (us; share of a copy's 6,568 GB/s over the bytes that must be read): one
// sequence of 126,253 tokens in f16 47 (84%), 255,181 in e4m3 52 to 56 (73 to 79%, over several
// boards), 128 sequences of up to 8,192 in e4m3 109 to 124 (74 to 85%): bound by the loads, less
// some 5 us to start and 4 us to merge. 24 sequences of up to 32,768 with four queries each in 4
// bits 203 (17%), with one 87 (40%): bound by the instructions that turn codes into operands and
// weights into fragments, and their latency at 8 to 12 warps an SM (issue slots 51% busy, tensor
// pipe 38%). A lone sequence of 1,024 tokens 8.0, all latency.
#include <atomic>

#include "qsa_paged.cuh"
#include "qsa_sm100.cuh"

namespace qsa {

namespace {

constexpr int kPaWarps = 4;                  // of a team
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaTile = 16 * kPaWarps;       // cells of a tile, 16 a warp
constexpr int kPaMaxTeams = 1024;            // over the GPU
constexpr int kPaStart = 2;                  // a segment's start (queries, joining) costs about as much as two tiles
// The running maximum is renewed when a logit passes it by 8 (in log 2), so that weights are
// at most 2^8; times 2^7 they fill f16's range (below 2^16).
constexpr float kPaSlack = 8.0f;
constexpr float kPaTop = 128.0f;
constexpr float kPaNone = -3e38f;  // the running maximum before the first cell: finite, so that -inf - it is -inf
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

template <int FMT, int D, int NC>
struct PaCfg {
  static constexpr int ROW = page_row_bytes_c<FMT>(D);
  static constexpr int SROW = page_scale_bytes_c<FMT>(D);
  static constexpr int KB = kPaTile * ROW;                 // bytes of a tile's K (V) rows
  static constexpr int SB = kPaTile * SROW;                // and of their scales
  static constexpr int KS = D / 16;                        // MMA k-steps of q.K = m-tiles of P.V
  // Teams of a CTA (one CTA an SM): three where a thread's sums take up to 32 registers (e4m3
  // rows: 48, 4-bit rows: 64), two where they take more or 256-byte rows need the shared memory.
  // One more warpgroup loads. (100 sequences of up to 8,192, us: two column groups of 128 dims,
  // three teams 154 against 169 at 4 bits, but 280 against 143 at e4m3, whose rows added one by
  // one take registers too; three groups of 64-dim e4m3 rows 121 against 131.)
  static constexpr int TEAMS = KS * NC <= (FMT == QSA_PAGE_INT4 ? 16 : FMT == QSA_PAGE_FP8 ? 12 : 8) && ROW <= 128 ? 3 : 2;
  static constexpr int THREADS = kPaThreads * (TEAMS + 1);
  // registers a thread: at launch, and as the warpgroups split them
  static constexpr int REGS = TEAMS == 3 ? 128 : 168;
  static constexpr int REGS_TEAM = TEAMS == 3 ? 152 : 224, REGS_LOAD = 56;
  static_assert(kPaThreads * (TEAMS * REGS_TEAM + REGS_LOAD) <= THREADS * REGS, "the shares add up");
  // shared memory of a team: ring (K and V rows, then scales), joined results, queries, small things
  static constexpr int JOIN = 8 * (D + 4) * kPaWarps * 4;
  static constexpr int Q = NC > 1 ? KS * NC * 32 * 8 : 0;
  static constexpr int SMALL = 4096;
  static constexpr int BUDGET = (226 * 1024) / TEAMS - JOIN - Q - SMALL;
  static constexpr int FIT = BUDGET / (2 * (KB + SB));
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int RING = STAGES * 2 * KB;
  static constexpr int SRING = STAGES * 2 * SB;
  static constexpr int BYTES = TEAMS * (RING + SRING + JOIN + Q + SMALL);
  static_assert(STAGES >= 2, "the ring needs two tiles");
  static_assert(KB % 1024 == 0, "swizzled tiles start on their pattern's border");
};

// sm_scale for base-2 exponents, and kPaSlack in units of q.K (as arguments they take no registers).
struct PaExp {
  float c1, slack;
};

// What merge CTA i joins: if the batch has no more segments than teams, segment i (written by
// the team that ends it, or by the first one that continues it), else the segment that team i is
// the first to continue.
struct PaSplit {
  int seq, head;    // seq < 0: nothing
  int first, last;  // teams that hold a part
  int slot0;        // slot of the first one's part: 2 * first + (0 or 1); the others: 2 * team
  int pad[3];
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same into fresh sums.
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Two f16 values with the infinities (and NaN) as the largest numbers.
__device__ __forceinline__ uint32_t finite2(uint32_t a) {
  uint32_t d;
  asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0x7bff7bffu));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log sum exp from the largest q.K and the sum of the weights relative to it.
__device__ __forceinline__ float lse_of(float top, float sum, float sm_scale) {
  return sum == 0.0f ? -INFINITY : fmaf(top, sm_scale, log2f(sum) * kLn2);
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Two e4m3 codes (the low or high half of a word) as f16: exact.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w, int high) {
  uint32_t d;
  if (high)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
// Variant v of a word of eight 4-bit codes as two f16 values: bit 0 takes bytes 1 and 3 instead
// of 0 and 2, bit 1 the high halves. 0x6400 | n is 1024 + n in f16, and 1024 + 16 n where
// the code sits four bits higher, so one subtraction or one fused step gives code - 8 exactly.
__device__ __forceinline__ uint32_t int4x2(uint32_t w, int v, __half2 scale) {
  if (v & 1) w >>= 8;
  __half2 h;
  if (v & 2) {
    h = __hfma2(as_h2((w & 0x00f000f0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));
  } else {
    h = __hsub2(as_h2((w & 0x000f000fu) | 0x64006400u), __float2half2_rn(1032.0f));
  }
  return as_u32(__hmul2(h, scale));
}

// Where byte `off` of a tile of 128-byte lines is: TMA's 128-byte swizzle xors the index of a
// 16-byte chunk in its line with the line's. (A line is a row of 128 bytes, 2 or 4 shorter
// ones, or half a row of 256: the halves are tiles of their own.)
__device__ __forceinline__ uint32_t swizzled(uint32_t off) { return off ^ ((off >> 3) & 0x70); }

// Cell of a 16-cell tile that MMA row (S^T) resp. k-slot (P.V) r takes. Any order gives the
// same sums; these keep the fragment reads of 8- and 4-bit rows off each other's banks: with
// 128-byte rows, rows 2a and 2a + 1 of the order differ in bit 2 and every other row of it
// has its own bits 1 and 2; with 64-byte rows they differ in bit 0 and every other row has
// its own bits 0 and 2; with 32-byte rows four in turn are distinct mod 4.
template <int FMT, int D>
__device__ __forceinline__ int cell_of(int r) {
  constexpr int ROW = page_row_bytes_c<FMT>(D);
  constexpr uint32_t order = FMT == QSA_PAGE_F16 ? 0x76543210u : ROW == 128 ? 0x37156240u : ROW == 64 ? 0x65742130u : 0x53427160u;
  return (r & 8) | ((order >> (4 * (r & 7))) & 7);
}

// Dim of k-slot i of lane group member t (slots 2t, 2t+1, 2t+8, 2t+9) in k-step j of q.K.
template <int FMT, int D>
__device__ __forceinline__ int q_dim(int j, int t, int i) {
  if constexpr (FMT == QSA_PAGE_F16) return j * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
  else if constexpr (FMT == QSA_PAGE_FP8) return (j >> 2) * 64 + t * 16 + (j & 3) * 4 + i;
  else {
    const int byte = (j >> 1) * 4 + ((i & 1) << 1) + (i >> 1);  // slots take bytes 0, 2, 1, 3 of a word
    return D == 128 ? t * 32 + (j & 1) * 16 + byte : (t >> 1) * 32 + (j & 1) * 16 + (t & 1) * 8 + byte;
  }
}
// Dim of MMA row g + 8 * half of m-tile mt of P.V.
template <int FMT, int D>
__device__ __forceinline__ int v_dim(int mt, int g, int half) {
  if constexpr (FMT == QSA_PAGE_F16) return mt * 16 + g + 8 * half;
  else if constexpr (FMT == QSA_PAGE_FP8) return g * (D / 8) + 2 * mt + half;
  else {
    const int v = mt & 3, sub = (v & 1) + (v >> 1) * 16 + 2 * half;
    return D == 128 ? (g >> 1) * 32 + (g & 1) * 8 + (mt >> 2) * 4 + sub : (g >> 2) * 32 + (g & 3) * 4 + sub;
  }
}

// One V value of a stored row, without its e4m3 scale.
template <int FMT>
__device__ __forceinline__ float v_value(const char* row, const char* scales, int d) {
  if constexpr (FMT == QSA_PAGE_F16) return __half2float(reinterpret_cast<const __half*>(row)[d]);
  else if constexpr (FMT == QSA_PAGE_FP8)
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(reinterpret_cast<const unsigned char*>(row)[d], __NV_E4M3)));
  else {
    const unsigned b = reinterpret_cast<const unsigned char*>(row)[d / 32 * 16 + d % 16];
    return __half2float(__hmul(__int2half_rn(int((d & 16) ? b >> 4 : b & 15) - 8), reinterpret_cast<const __half*>(scales)[d / 32]));
  }
}

// Position in the list: sequence s has, for each KV head, kPaStart places for the segment's
// start and then its nt = ceil(len / 64) tiles. `left` places of the team's share are left,
// this tile among them.
struct PaCursor {
  int seq, head, tile, nt, len;
  long long left;
};

// Sum over the CTA in thread order: this thread's exclusive prefix, the total in *total.
template <int WARPS>
__device__ __forceinline__ long long cta_scan(long long v, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return before + x - v;
}

// Small shared data of a team (PaCfg::SMALL bytes).
struct PaSmall {
  uint64_t full[8], empty[8];
  long long base;
  int64_t q_off[32];  // elements from the sequence's first query row to column c's
  int64_t out_off[32];                 // output rows: from the sequence's first
  int sees[32];       // u of column c (it sees cells < seen + u); far below 0 past the last column
  int seq;
  unsigned lost[8];   // of each ring slot: bit w is set if warp w's cells have no page in the pool
  float m[kPaWarps][32], l[kPaWarps][32];  // statistics, then each warp's factor and 1 / l
};
static_assert(sizeof(PaSmall) <= 4096, "PaCfg::SMALL");

template <int FMT, int D, int NC>
__global__ void __launch_bounds__(PaCfg<FMT, D, NC>::THREADS, 1)
paged_attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, PagedView c,
                    PagedAttendArgs a, PaExp ex, float* __restrict__ part, PaSplit* __restrict__ splits) {
  using C = PaCfg<FMT, D, NC>;
  constexpr int KS = C::KS, STAGES = C::STAGES, ROW = C::ROW, SROW = C::SROW, TEAMS = C::TEAMS;
  constexpr int ALL = C::THREADS;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ long long s_scan[ALL / 32];

  const int lane = threadIdx.x & 31, group = threadIdx.x / kPaThreads;
  // the last warpgroup's warp i loads for team i (its warps beyond the teams have nothing to do)
  const bool loads = group == TEAMS;
  const int warp = (threadIdx.x >> 5) % kPaWarps, tid = threadIdx.x % kPaThreads;
  const int team = loads ? min(warp, TEAMS - 1) : group;
  const auto small = [&](int i) -> PaSmall& {
    return *reinterpret_cast<PaSmall*>(smem + TEAMS * (C::RING + C::SRING + C::JOIN + C::Q) + i * C::SMALL);
  };
  PaSmall& sm = small(team);
  float* const s_join = reinterpret_cast<float*>(smem + TEAMS * (C::RING + C::SRING) + team * C::JOIN);  // [warp][8 columns][D + 4]
  uint2* const s_q = reinterpret_cast<uint2*>(smem + TEAMS * (C::RING + C::SRING + C::JOIN) + team * C::Q);
  const uint32_t ring = sm100::smem_u32(smem) + team * C::RING;
  const uint32_t sring = sm100::smem_u32(smem) + TEAMS * C::RING + team * C::SRING;

  const int G = a.n_q_heads / c.n_kv_heads, T = a.n_queries, R = G * T, Hkv = c.n_kv_heads;
  const int n_teams = gridDim.x * TEAMS;
  const int cta = blockIdx.x * TEAMS + team;  // the team's index in the GPU
  // (cell numbers stay clear of 2^31)
  const long long table_cells = min((long long)a.table_width << c.page_shift, 0x7fffff00ll);

  if (loads && lane == 0 && warp < TEAMS) {
    sm100::tma_prefetch_desc(&kmap);
    sm100::tma_prefetch_desc(&vmap);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      sm100::mbar_init(&sm.full[i], SROW > 0 ? 33 : 1);  // (each lane's copies of scales)
      sm100::mbar_init(&sm.empty[i], kPaWarps);
    }
    sm100::fence_mbar_init();
  }
  if (!loads && tid < 32) {
    const int u = tid / G, h = tid % G;
    sm.q_off[tid] = u * a.q_stride + h * D;
    sm.out_off[tid] = int64_t(u) * a.n_q_heads + h;
    sm.sees[tid] = tid < R ? u : -(1 << 30);
  }
  pdl_wait();  // (the merge launches when this grid ends: its CTAs find no room beside these)

  const auto length = [&](int s) {
    const int n = a.seq_lens[s];
    return n < 0 ? 0 : n > table_cells ? int(table_cells) : n;
  };
  const auto tiles = [&](int len) { return int(((long long)len + kPaTile - 1) / kPaTile); };
  const auto places = [&](int s) {
    const int len = length(s);
    return len > 0 ? tiles(len) + kPaStart : 0;
  };

  // ---- the team's share of the list: places [lo, hi) ----
  long long total = 0, per = 0;
  int N = 0, extra = 0;  // teams with a share: at least one place each
  const auto share = [&] {
    total *= Hkv;
    N = int(min((long long)n_teams, total));
    if (N == 0) return;
    per = total >> 31 ? total / N : (long long)(unsigned(total) / unsigned(N));
    extra = int(total - per * N);  // the first `extra` teams take one more
  };
  const auto start_of = [&](int i) { return i < N ? i * per + min(i, extra) : total; };
  const auto find = [&](int s, long long mine, long long at) {
    if (mine == 0) return;
#pragma unroll
    for (int i = 0; i < TEAMS; ++i) {
      const long long first = start_of(blockIdx.x * TEAMS + i);
      if (at <= first && first < at + mine * Hkv) {
        small(i).seq = s;
        small(i).base = at;
      }
    }
  };
  if (a.n_seqs <= ALL) {
    const int mine = int(threadIdx.x) < a.n_seqs ? places(threadIdx.x) : 0;
    const long long at = cta_scan<ALL / 32>(mine, s_scan, &total) * Hkv;
    share();
    find(threadIdx.x, mine, at);
  } else {
    long long sum, before = 0;
    for (int b = 0; b < a.n_seqs; b += ALL) {
      const int s = b + threadIdx.x;
      cta_scan<ALL / 32>(s < a.n_seqs ? places(s) : 0, s_scan, &sum);
      total += sum;
    }
    share();
    for (int b = 0; b < a.n_seqs; b += ALL) {
      const int s = b + threadIdx.x, mine = s < a.n_seqs ? places(s) : 0;
      const long long at = (before + cta_scan<ALL / 32>(mine, s_scan, &sum)) * Hkv;
      find(s, mine, at);
      before += sum;
    }
  }
  const long long lo = start_of(cta), hi = start_of(cta + 1);
  __syncthreads();
  PaCursor cur;
  cur.seq = cur.head = cur.tile = cur.nt = cur.len = 0;
  cur.left = hi - lo;
  long long b0 = 0;  // where the segment that `lo` is in begins
  const auto start_segment = [&](PaCursor& p) {
    p.len = length(p.seq);
    p.nt = tiles(p.len);
  };
  if (lo < hi) {
    cur.seq = sm.seq;
    start_segment(cur);
    const long long in = lo - sm.base;
    const int all = cur.nt + kPaStart;
    cur.head = in >> 31 ? int(in / all) : int(unsigned(in) / unsigned(all));
    const int at = int(in - (long long)cur.head * all);
    b0 = lo - at;
    cur.tile = max(0, at - kPaStart);
    cur.left -= max(0, kPaStart - at);
  }
  const auto next_segment = [&](PaCursor& p) {  // (the list has one if left stays above 0)
    p.tile = 0;
    p.left -= kPaStart;
    if (p.left <= 0 || ++p.head < Hkv) return;
    p.head = 0;
    if (++p.seq < a.n_seqs && length(p.seq) == 0) {
      // empty slots of a batch, maybe many in a row: 256 a round of loads (8,192 of them between two
      // sequences cost 9 us, and 990 when they were looked at one by one)
      int found = -1;
#pragma unroll 1
      for (int s0 = p.seq + 1; found < 0 && s0 < a.n_seqs; s0 += 256) {
        int n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = s0 + 32 * i + lane < a.n_seqs ? a.seq_lens[s0 + 32 * i + lane] : 0;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const unsigned some = __ballot_sync(0xffffffffu, n[i] > 0);
          if (some) found = s0 + 32 * i + __ffs(some) - 1;
        }
      }
      p.seq = found < 0 ? a.n_seqs : found;
    }
    if (p.seq >= a.n_seqs) {  // (only if the lengths changed meanwhile)
      p.left = 0;
      return;
    }
    start_segment(p);
  };
  const auto next_tile = [&](PaCursor& p) {
    --p.left;
    if (++p.tile == p.nt && p.left > 0) next_segment(p);
  };

  // =============================== loading warps ===============================
  // Lane i < 4 looks after the tile's cells 16 i .. 16 i + 15. With pages of 32 tokens or more
  // the first lane of a page loads all of its rows in the tile.
  if (loads) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOAD));
    if (warp >= TEAMS) return;
    const int rows = min(kPaTile, 1 << c.page_shift);
    const bool leads = lane < kPaWarps && (lane * 16) % rows == 0;
    const auto entry = [&](const PaCursor& p) {
      const int cell = p.tile * kPaTile + (lane * 16) / rows * rows;
      return lane < kPaWarps && cell < p.len ? a.block_table[(long long)p.seq * a.table_width + (cell >> c.page_shift)] : 0;
    };
    // the pages of two tiles ahead are on their way
    PaCursor ld = cur;
    int page = 0, page1 = 0;
    if (ld.left > 0) {
      page = entry(ld);
      next_tile(cur);
      if (cur.left > 0) page1 = entry(cur);
    }
    int slot = 0;
    uint32_t parity = 1;
#pragma unroll 1
    while (ld.left > 0) {
      const PaCursor next = cur;
      int page2 = 0;
      if (cur.left > 0) {
        next_tile(cur);
        if (cur.left > 0) page2 = entry(cur);
      }
      if (!sm100::mbar_wait(&sm.empty[slot], parity)) {
        if (lane == 0) record_status(a.status, QSA_ERR_TIMEOUT);
        break;  // the computing warps' waits run out as well
      }
      const int cell = ld.tile * kPaTile + lane * 16;
      const bool wanted = lane < kPaWarps && cell < ld.len;
      const bool ok = wanted && page >= 0 && page < c.n_pages;
      const unsigned lost = __ballot_sync(0xffffffffu, wanted && !ok);
      const int n_loads = __popc(__ballot_sync(0xffffffffu, ok && leads));
      uint64_t* const bar = &sm.full[slot];
      if (lane == 0) {
        if (lost) record_status(a.status, QSA_ERR_BAD_INDEX);
        sm.lost[slot] = lost;
        if (n_loads == 0) sm100::mbar_arrive(bar);
        else sm100::mbar_arrive_expect_tx(bar, n_loads * rows * 2 * ROW);
      }
      __syncwarp();
      if (ok && leads) {
        const int row = row_in_page(c, ld.head, cell & ((1 << c.page_shift) - 1));
        constexpr int LINE = ROW < 128 ? ROW : 128;  // bytes of a row in a line
        const uint32_t dst = ring + slot * 2 * C::KB + lane * 16 * LINE;
#pragma unroll
        for (int x = 0; x < ROW / LINE; ++x) {
          sm100::tma_load_3d(dst + x * kPaTile * 128, &kmap, x * 64, row * LINE / 128, page, bar);
          sm100::tma_load_3d(dst + C::KB + x * kPaTile * 128, &vmap, x * 64, row * LINE / 128, page, bar);
        }
      }
      if constexpr (SROW > 0) {
        // scales in 16-byte pieces, one or two a lane (they are too small for bulk copies: 64 bytes a page)
        const unsigned there = __ballot_sync(0xffffffffu, ok);
#pragma unroll
        for (int i = 0; i < SROW / 4; ++i) {
          const int piece = i * 32 + lane, of_v = piece / (4 * SROW), in = piece % (4 * SROW), cells = in / SROW;
          const int at = __shfl_sync(0xffffffffu, page, cells);
          if ((there >> cells) & 1) {
            const int first = (ld.tile * kPaTile + cells * 16) & ((1 << c.page_shift) - 1);
            const char* const src = (of_v ? c.vs : c.ks) + at * c.scale_stride +
                                    (int64_t)row_in_page(c, ld.head, first) * SROW + in % SROW * 16;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sring + (slot * 2 + of_v) * C::SB + in * 16), "l"(src) : "memory");
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
      }
      ld = next;
      page = page1;
      page1 = page2;
      if (++slot == STAGES) {
        slot = 0;
        parity ^= 1;
      }
    }
    // The copies on their way land before the CTA's shared memory may become another's, even if
    // the computing warps have given up waiting: slots before `slot` were last filled in this
    // round of the ring, the others in the one before (or never, which counts as landed).
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i)
      if (!sm100::mbar_wait(&sm.full[i], i < slot ? parity ^ 1 : parity)) break;
    return;
  }

  // =============================== computing warps ===============================
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_TEAM));
  const int g = lane >> 2, t = lane & 3;
  // p = 2^((s - top) c1). The difference comes first: it is exact near the maximum, while in
  // s c1 - top c1 the rounding of one product is 2^-24 of a logit, which for large ones is
  // more than an exponent.
  const float c1 = ex.c1, slack = ex.slack;
  const bool by_segment = (long long)a.n_seqs * Hkv <= n_teams;
  if (tid == 0) {
    // the first team that continues a segment names the parts to merge
    PaSplit sp;
    sp.seq = -1;
    if (cur.left > 0 && cur.tile > 0) {
      const long long before = start_of(cta - 1), last = b0 + kPaStart + cur.nt - 1;
      if (before <= b0 + kPaStart) {  // the team before this one has the segment's first tile
        const long long border = extra * (per + 1);
        sp.seq = cur.seq;
        sp.head = cur.head;
        sp.first = cta - 1;
        sp.last = int(last < border ? last / (per + 1) : extra + (last - border) / per);
        sp.slot0 = 2 * (cta - 1) + (before < b0);
      }
    }
    if (!by_segment) splits[cta] = sp;
    else if (sp.seq >= 0) splits[sp.seq * Hkv + sp.head] = sp;
  }
  // bad lengths and the results of sequences without cells: a team looks after its share
  for (int s = cta; s < a.n_seqs; s += n_teams) {
    const int n = a.seq_lens[s];
    if (tid == 0 && n < 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    if (tid == 0 && n > table_cells) record_status(a.status, QSA_ERR_CAPACITY);
    if (n <= 0) {
      const int rows = T * a.n_q_heads;
      if (by_segment)
        for (int h = tid; h < Hkv; h += kPaThreads) splits[s * Hkv + h].seq = -1;
      for (int e = tid; e < rows * D; e += kPaThreads) a.out[(int64_t)s * rows * D + e] = 0.0f;
      if (a.lse)
        for (int e = tid; e < rows; e += kPaThreads) a.lse[(int64_t)s * rows + e] = -INFINITY;
    }
  }

  const int w16 = warp * 16;  // this warp's rows of a tile
  // weights [cell][column] of rows added one by one (the warp's part of s_join, unused between joins)
  float* const stash = s_join + warp * 8 * (D + 4);
  static_assert(16 * 32 <= 8 * (D + 4), "the warp's part holds a step's weights");
  const int pg = w16 + cell_of<FMT, D>(g);
  const int pv0 = w16 + cell_of<FMT, D>(2 * t), pv1 = w16 + cell_of<FMT, D>(2 * t + 1);
  int slot = 0;
  uint32_t parity = 0;
  bool timed_out = false;
  bool first_segment = true;
  while (cur.left > 0) {
    const int tile0 = cur.tile, tile1 = int(min((long long)cur.nt, tile0 + cur.left));
    const int len = cur.len, seen = len - T + 1;  // cells before `seen` are seen by every query

    // queries: B fragments, column = (query, head) row of this KV head
    const __half* const q0 = static_cast<const __half*>(a.q) + (int64_t)cur.seq * T * a.q_stride + cur.head * G * D;
    const auto q_frag = [&](int j, int col, int tt) {
      uint2 f = make_uint2(0u, 0u);
      if (col < R) {
        const __half* q = q0 + sm.q_off[col];
        if constexpr (FMT == QSA_PAGE_F16) {  // slots 2t, 2t + 1 and 2t + 8, 2t + 9
          f.x = *reinterpret_cast<const uint32_t*>(q + q_dim<FMT, D>(j, tt, 0));
          f.y = *reinterpret_cast<const uint32_t*>(q + q_dim<FMT, D>(j, tt, 2));
        } else {  // four dims in turn; 4-bit slots take them as 0, 2, 1, 3
          f = *reinterpret_cast<const uint2*>(q + q_dim<FMT, D>(j, tt, 0));
          if constexpr (FMT == QSA_PAGE_INT4)
            f = make_uint2(__byte_perm(f.x, f.y, 0x5410), __byte_perm(f.x, f.y, 0x7632));
        }
      }
      return f;
    };
    uint2 qf[NC == 1 ? KS : 1];
    if constexpr (NC == 1) {
#pragma unroll
      for (int j = 0; j < KS; ++j) qf[j] = q_frag(j, g, t);
    } else {
#pragma unroll
      for (int e = tid; e < KS * NC * 32; e += kPaThreads) s_q[e] = q_frag(e / (32 * NC), (e / 32 % NC) * 8 + g, t);
      sm100::named_bar_sync(1 + team, kPaThreads);
    }
    // Per column: exponents are taken from `top`, the running maximum of q.K, which is renewed
    // when one passes it by `slack`.
    float top[NC][2], l[NC][2], acc[KS][NC][4];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[n][i] = kPaNone;
        l[n][i] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][n][i] = 0.0f;
    }

#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      const int u0 = tile * kPaTile + w16;  // this warp's 16 cells
      const uint32_t uk = ring + slot * 2 * C::KB, uv = uk + C::KB, uks = sring + slot * 2 * C::SB, uvs = uks + C::SB;
      if (!timed_out && !sm100::mbar_wait(&sm.full[slot], parity)) {
        timed_out = true;
        if (lane == 0) record_status(a.status, QSA_ERR_TIMEOUT);
      }
      const bool gone = (sm.lost[slot] >> warp) & 1;
      if (u0 < len && !gone) {
        const bool whole = u0 + 16 <= seen;  // every query sees every cell
        unsigned zero = 0, apart = 0;        // rows whose V must stay out of the MMA; those to add one by one
        if (!whole) {
          // Rows past the end hold anything; so may the newest cells, which only some queries
          // see: if one holds an infinity or a NaN it is taken apart (0 * NaN is NaN).
#pragma unroll 1
          for (int r = max(0, seen - u0); r < 16; ++r) {
            bool out = u0 + r >= len;
            if (!out) {
              bool odd = false;
              for (int b = lane * 4; b < ROW; b += 128) {
                const uint32_t w = lds32(uv + b / 128 * kPaTile * 128 + swizzled((w16 + r) * (ROW < 128 ? ROW : 128) + b % 128));
                if (FMT == QSA_PAGE_F16) odd |= (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
                if (FMT == QSA_PAGE_FP8) odd |= __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
              }
              if (FMT == QSA_PAGE_FP8) odd |= (lds32(uvs + (w16 + r) * 4) & 0x7f800000u) == 0x7f800000u;
              if (FMT == QSA_PAGE_INT4 && lane * 4 < SROW) {
                const uint32_t w = lds32(uvs + (w16 + r) * SROW + lane * 4);
                odd |= (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
              }
              out = __any_sync(0xffffffffu, odd);
              if (out) apart |= 1u << r;
            }
            if (!out) continue;
            zero |= 1u << r;
            for (int b = lane * 4; b < ROW; b += 128)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(uv + b / 128 * kPaTile * 128 +
                  swizzled((w16 + r) * (ROW < 128 ? ROW : 128) + b % 128)), "r"(0) : "memory");
            if (FMT == QSA_PAGE_INT4 && lane * 4 < SROW)  // (a 4-bit zero stands for -8 scale)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(uvs + (w16 + r) * SROW + lane * 4), "r"(0) : "memory");
          }
          __syncwarp();
        }

        // S^T: cells cell_of(g) and cell_of(g + 8), columns 2t and 2t + 1
        float s[NC][4];
        {
          uint4 raw[2][2];
          __half2 ksc[2];
          if constexpr (FMT == QSA_PAGE_FP8) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                raw[r][h] = lds128(uk + swizzled((pg + 8 * r) * ROW + h * 64 + t * 16));
          } else if constexpr (FMT == QSA_PAGE_INT4) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (D == 128) {
                raw[r][0] = lds128(uk + swizzled((pg + 8 * r) * ROW + t * 16));
              } else {
                const uint2 w = lds64(uk + swizzled((pg + 8 * r) * ROW + t * 8));
                raw[r][0] = make_uint4(w.x, w.y, 0u, 0u);
              }
              const int grp = D == 128 ? t : t >> 1;
              const uint32_t w = lds32(uks + (pg + 8 * r) * SROW + (grp >> 1) * 4);
              ksc[r] = as_h2(__byte_perm(w, w, (grp & 1) ? 0x3232 : 0x1010));
            }
          }
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            uint32_t f[4];
            if constexpr (FMT == QSA_PAGE_F16) {
              ldsm4(f, uk + (j >> 2) * kPaTile * 128 +
                           swizzled((w16 + (lane & 15)) * 128 + (j & 3) * 32 + (lane >> 4) * 16));
            } else if constexpr (FMT == QSA_PAGE_FP8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = e4m3x2(word_of(raw[i & 1][j >> 2], j & 3), i >> 1);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                f[i] = int4x2(word_of(raw[i & 1][0], j >> 1), (i >> 1) + 2 * (j & 1), ksc[i & 1]);
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              uint2 b;
              if constexpr (NC == 1) b = qf[j];
              else b = s_q[(j * NC + n) * 32 + lane];
              if (j == 0) mma0(s[n], f[0], f[1], f[2], f[3], b.x, b.y);
              else mma(s[n], f[0], f[1], f[2], f[3], b.x, b.y);
            }
          }
        }

        // V's codes are on their way from shared memory during the softmax
        uint4 vraw[4];
        __half2 vsc[2];  // 4-bit scales of cells (0, 1) and (2, 3)
        if constexpr (FMT != QSA_PAGE_F16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = ((i & 1) ? pv1 : pv0) + (i >> 1) * 8;
            const uint32_t at_row = uv + swizzled(row * ROW + g * (ROW / 8));
            if constexpr (ROW == 128) {
              vraw[i] = lds128(at_row);
            } else if constexpr (ROW == 64) {
              const uint2 w = lds64(at_row);
              vraw[i] = make_uint4(w.x, w.y, 0u, 0u);
            } else {
              vraw[i] = make_uint4(lds32(at_row), 0u, 0u, 0u);
            }
          }
          if constexpr (FMT == QSA_PAGE_INT4) {
            const int grp = D == 128 ? g >> 1 : g >> 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = lds32(uvs + (pv0 + 8 * i) * SROW + (grp >> 1) * 4);
              const uint32_t y = lds32(uvs + (pv1 + 8 * i) * SROW + (grp >> 1) * 4);
              vsc[i] = as_h2(__byte_perm(x, y, (grp & 1) ? 0x7632 : 0x5410));
            }
          }
        }

        // logits: times the row's scale (e4m3), masked
        uint32_t vf[2] = {0u, 0u};  // the rows' V scales (e4m3), as bits
        if constexpr (FMT == QSA_PAGE_FP8) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = __uint_as_float(lds32(uks + (pg + 8 * r) * 4));
            vf[r] = lds32(uvs + (pg + 8 * r) * 4);
            if ((zero >> (pg - w16 + 8 * r)) & 1) vf[r] = 0u;
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) s[n][2 * r + i] *= f;
          }
        }
        if (!whole) {
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const int2 u = *reinterpret_cast<const int2*>(&sm.sees[n * 8 + 2 * t]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int late = u0 + pg - w16 + 8 * r - seen;
              if (late >= u.x) s[n][2 * r] = -INFINITY;
              if (late >= u.y) s[n][2 * r + 1] = -INFINITY;
            }
          }
        }

        // a logit far above the running maximum: renew it
        bool over = false;
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) over |= fmaxf(s[n][i], s[n][2 + i]) - top[n][i] > slack;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = fmaxf(s[n][i], s[n][2 + i]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
              const float to = fmaxf(top[n][i], x), corr = ex2((top[n][i] - to) * c1);
              top[n][i] = to;
              l[n][i] *= corr;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                acc[k][n][i] *= corr;
                acc[k][n][2 + i] *= corr;
              }
            }
        }
        // weights
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p = ex2((s[n][2 * r + i] - top[n][i]) * c1);
              l[n][i] += p;
              s[n][2 * r + i] = p;
            }

        // An e4m3 weight is p times the row's scale. So that its two terms keep their bits it enters
        // relative to a power of two next above the largest scale of the 16 rows, by which the
        // product is scaled back as it is added. All-zero rows (their scale is 1; one that is not
        // finite makes them NaN) are left out, and
        // where the others' scales lie more than 2^8 apart the rows outside a window of 2^8,
        // from the top down the first that no more rows lie below than in, are added one by one
        // in f32 (one such row in every 16 of 126,000: 80 us instead of 46).
        float w[2] = {kPaTop, kPaTop}, unit = 1.0f;
        if constexpr (FMT == QSA_PAGE_FP8) {
          bool low[2];
          const auto choose = [&] {  // true: the scales lie too far apart
            const uint32_t most = __reduce_max_sync(0xffffffffu, max(vf[0] & 0x7fffffffu, vf[1] & 0x7fffffffu));
            // the bits of the power of two, 2^-119 (then no row is too small) to 2^126
            const uint32_t e = max((min(most, 0x7e800000u) + 0x7fffffu) & 0x7f800000u, 0x04000000u);
            unit = __uint_as_float(e) * (1.0f / kPaTop);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              low[r] = vf[r] != 0u && (vf[r] & 0x7fffffffu) < e - 0x04000000u;
              w[r] = low[r] ? 0.0f : __uint_as_float(vf[r]) * __uint_as_float(0x7f000000u - e) * kPaTop;
            }
            return __any_sync(0xffffffffu, low[0] || low[1]);
          };
          if (choose()) {
            uint32_t codes = 0;  // of half a row a lane
#pragma unroll 1
            for (int b = 0; b < ROW / 2; b += 4)
              codes |= lds32(uv + swizzled((w16 + (lane >> 1)) * ROW + (lane & 1) * (ROW / 2) + b)) & 0x7f7f7f7fu;
            codes |= __shfl_xor_sync(0xffffffffu, codes, 1);
            const unsigned some = __ballot_sync(0xffffffffu, codes != 0);  // bits 2 c of cells c
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!((some >> (2 * (pg - w16 + 8 * r))) & 1) && (vf[r] & 0x7fffffffu) < 0x7f800000u) vf[r] = 0u;
            const unsigned row0 = 1u << (pg - w16), row1 = row0 << 8;
#pragma unroll 1
            for (;;) {  // (ends: a window holds at least the largest row that is left)
              choose();
              const unsigned below = __reduce_or_sync(0xffffffffu, (low[0] ? row0 : 0u) | (low[1] ? row1 : 0u));
              const bool in0 = vf[0] != 0u && !low[0], in1 = vf[1] != 0u && !low[1];
              const unsigned in = __reduce_or_sync(0xffffffffu, (in0 ? row0 : 0u) | (in1 ? row1 : 0u));
              if (__popc(below) <= __popc(in)) {
                apart |= below;
                break;
              }
              apart |= in;
              if (in0) vf[0] = 0u;
              if (in1) vf[1] = 0u;
            }
          }
        }
        // O^T += V^T P^T
        uint32_t ph[NC][2], pl[NC][2];  // B fragments of P^T: two f16 terms each
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = s[n][2 * r] * w[r], y = s[n][2 * r + 1] * w[r];
            const __half2 h = __floats2half2_rn(x, y);
            const float2 back = __half22float2(h);
            ph[n][r] = transpose8x8(as_u32(h));
            pl[n][r] = transpose8x8(as_u32(__floats2half2_rn(x - back.x, y - back.y)));
          }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float d[NC][4];
          uint32_t f[4];
          if constexpr (FMT == QSA_PAGE_F16) {
            ldsm4_trans(f, uv + (k >> 2) * kPaTile * 128 +
                               swizzled((w16 + (lane >> 4) * 8 + (lane & 7)) * 128 + (k & 3) * 32 + ((lane >> 3) & 1) * 16));
          } else {
            // codes of the same dim of two cells side by side, then as f16 pairs
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if constexpr (FMT == QSA_PAGE_FP8) {
                const uint32_t z = __byte_perm(word_of(vraw[2 * i], k >> 1), word_of(vraw[2 * i + 1], k >> 1),
                                               (k & 1) ? 0x7362 : 0x5140);
                f[2 * i] = e4m3x2(z, 0);
                f[2 * i + 1] = e4m3x2(z, 1);
              } else {
                const uint32_t x = word_of(vraw[2 * i], k >> 2), y = word_of(vraw[2 * i + 1], k >> 2);
                f[2 * i] = int4x2(__byte_perm(x, y, 0x5410), k & 3, vsc[i]);
                f[2 * i + 1] = int4x2(__byte_perm(x, y, 0x7632), k & 3, vsc[i]);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NC; ++n) mma0(d[n], f[0], f[1], f[2], f[3], ph[n][0], ph[n][1]);
          if constexpr (FMT == QSA_PAGE_F16) {  // an infinity times the second term, 0 or negative, would be NaN
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = finite2(f[i]);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n) mma(d[n], f[0], f[1], f[2], f[3], pl[n][0], pl[n][1]);
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[k][n][i] = FMT == QSA_PAGE_FP8 ? fmaf(d[n][i], unit, acc[k][n][i]) : acc[k][n][i] + d[n][i];
        }

        if (apart) {  // rows that hold no numbers, to the queries that see them; rows with far smaller scales
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                stash[(pg - w16 + 8 * r) * 32 + n * 8 + 2 * t + i] = FMT == QSA_PAGE_FP8 ? s[n][2 * r + i] : s[n][2 * r + i] * kPaTop;
          __syncwarp();
#pragma unroll 1
          for (int r = 0; r < 16; ++r) {
            if (!((apart >> r) & 1)) continue;
            const int cell = u0 + r, late = cell - seen;
            const int page = a.block_table[(long long)cur.seq * a.table_width + (cell >> c.page_shift)];
            const int row = row_in_page(c, cur.head, cell & ((1 << c.page_shift) - 1));
            const char* vr = c.v + page * c.page_stride + (int64_t)row * ROW;
            const char* vs = SROW ? c.vs + page * c.scale_stride + (int64_t)row * SROW : nullptr;
            const float scale = FMT == QSA_PAGE_FP8 ? *reinterpret_cast<const float*>(vs) : 1.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = v_value<FMT>(vr, vs, v_dim<FMT, D>(k, g, h)) * scale;
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (late < sm.sees[n * 8 + 2 * t + i])
                      acc[k][n][2 * h + i] = fmaf(stash[r * 32 + n * 8 + 2 * t + i], x, acc[k][n][2 * h + i]);
              }
          }
        }
        if (zero) sm100::fence_proxy_async_smem();  // the zeroed rows before the next copy into them
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sm.empty[slot]);
      if (++slot == STAGES) {
        slot = 0;
        parity ^= 1;
      }
    }

    // ---- the warps' results joined ----
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], off);
        if (g == 0) {
          sm.m[warp][n * 8 + 2 * t + i] = top[n][i];  // the maximum, where l > 0
          sm.l[warp][n * 8 + 2 * t + i] = l[n][i];
        }
      }
    sm100::named_bar_sync(1 + team, kPaThreads);
    const bool complete = tile0 == 0 && tile1 == cur.nt;
    float* const out_part = part + int64_t(2 * cta + (first_segment ? 0 : 1)) * R * (D + 4);
    const int64_t out_row = int64_t(cur.seq) * T * a.n_q_heads + cur.head * G;
    if (complete && by_segment && tid == 0) splits[cur.seq * Hkv + cur.head].seq = -1;
    if (tid < R) {
      // a warp that saw nothing has l = 0 (a NaN logit makes l, and then everything, NaN)
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w)
        if (sm.l[w][tid] != 0.0f) M = fmaxf(M, sm.m[w][tid]);
      float fw[kPaWarps];
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) {
        const float lw = sm.l[w][tid];
        fw[w] = lw == 0.0f ? 0.0f : ex2((sm.m[w][tid] - M) * c1);
        L += fw[w] * lw;
      }
      const float end = complete ? (L == 0.0f ? 0.0f : 1.0f / L) : 1.0f;
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) sm.m[w][tid] = FMT == QSA_PAGE_FP8 ? fw[w] : fw[w] * (1.0f / kPaTop);
      sm.l[0][tid] = end;
      if (!complete) {
        out_part[tid * (D + 4) + D] = M;
        out_part[tid * (D + 4) + D + 1] = L;
      } else if (a.lse) {
        a.lse[out_row + sm.out_off[tid]] = lse_of(M, L, a.sm_scale);
      }
    }
    sm100::named_bar_sync(1 + team, kPaThreads);
#pragma unroll 1
    for (int n = 0; n < NC; ++n) {
      if (n > 0) sm100::named_bar_sync(1 + team, kPaThreads);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = sm.m[warp][n * 8 + 2 * t + i];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            s_join[(warp * 8 + 2 * t + i) * (D + 4) + v_dim<FMT, D>(k, g, h)] = acc[k][0][2 * h + i] * f;
      }
      sm100::named_bar_sync(1 + team, kPaThreads);
#pragma unroll 1
      for (int e = tid; e < 8 * D / 4; e += kPaThreads) {
        const int cc = e / (D / 4), d = e % (D / 4) * 4, col = n * 8 + cc;
        if (col >= R) break;
        float4 o = *reinterpret_cast<const float4*>(&s_join[cc * (D + 4) + d]);
#pragma unroll
        for (int w = 1; w < kPaWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(&s_join[(w * 8 + cc) * (D + 4) + d]);
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
        const float end = sm.l[0][col];
        o.x *= end, o.y *= end, o.z *= end, o.w *= end;
        float* const to = complete ? a.out + (out_row + sm.out_off[col]) * D : out_part + col * (D + 4);
        *reinterpret_cast<float4*>(to + d) = o;
      }
      if constexpr (NC > 1) {  // the next column group's sums into the registers of the first (one copy of this code)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x + 1 < NC; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[k][x][i] = acc[k][x + 1][i];
      }
    }
    sm100::named_bar_sync(1 + team, kPaThreads);  // sm.m, sm.l, s_join and s_q are free

    first_segment = false;
    cur.left -= tile1 - tile0;
    if (cur.left > 0) next_segment(cur);
  }
}

// Joins the parts of the segments that were cut: CTA x those of splits[x], its warps one row each
// or, with many parts, 2 to 8 warps a row, every one with several parts in flight; gridDim.y
// CTAs share a segment's rows.
constexpr int kPmWarps = 8;
// Parts a warp has in flight. 8 take up to 5% longer where a segment is cut into most parts (one
// sequence of 60,000, one KV head: 16.4 us a call against 15.9), 16 are no faster and take registers.
constexpr int kPmBatch = 12;

template <int D>
__global__ void __launch_bounds__(32 * kPmWarps) paged_merge_kernel(PagedAttendArgs a, const float* __restrict__ part,
                                                                    const PaSplit* __restrict__ splits, int n_kv_heads,
                                                                    float c1) {
  constexpr int V = D / 32;
  __shared__ float s_o[kPmWarps][D], s_ml[kPmWarps][2];
  pdl_launch_dependents();
  pdl_wait();
  const PaSplit sp = splits[blockIdx.x];
  if (sp.seq < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.n_q_heads / n_kv_heads, T = a.n_queries, R = G * T;
  const int n = sp.last - sp.first + 1;
  const int ways = n <= kPmBatch ? 1 : n <= 2 * kPmBatch ? 2 : n <= 4 * kPmBatch ? 4 : 8;  // warps a row
  const int way = warp % ways, rows = kPmWarps / ways;
  const int64_t step = int64_t(R) * (D + 4);
  for (int r0 = blockIdx.y * rows; r0 < R; r0 += gridDim.y * rows) {
    const int col = r0 + warp / ways;
    const auto row_of = [&](int p) { return part + (p == 0 ? sp.slot0 : 2 * (sp.first + p)) * step + col * (D + 4); };
    float M = -INFINITY, L = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    // adds m, l, x (a part that saw nothing has l = 0)
    const auto add = [&](float m, float l, const float* x) {
      if (l == 0.0f) return;
      const float to = fmaxf(M, m), keep = M == to ? 1.0f : ex2((M - to) * c1), w = m == to ? 1.0f : ex2((m - to) * c1);
      M = to;
      L = L * keep + w * l;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * keep + w * x[i];
    };
    for (int p0 = way; col < R && p0 < n; p0 += ways * kPmBatch) {
      float x[kPmBatch][V];
      float2 ml[kPmBatch];
#pragma unroll
      for (int b = 0; b < kPmBatch; ++b) {
        const int p = p0 + b * ways;
        ml[b] = make_float2(0.0f, 0.0f);
        if (p < n) {
          const float* const from = row_of(p);
          if constexpr (V == 4) *reinterpret_cast<float4*>(x[b]) = reinterpret_cast<const float4*>(from)[lane];
          else *reinterpret_cast<float2*>(x[b]) = reinterpret_cast<const float2*>(from)[lane];
          ml[b] = *reinterpret_cast<const float2*>(from + D);
        }
      }
#pragma unroll
      for (int b = 0; b < kPmBatch; ++b) add(ml[b].x, ml[b].y, x[b]);
    }
    if (ways > 1) {  // (the same in the whole CTA)
#pragma unroll
      for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = o[i];
      if (lane == 0) {
        s_ml[warp][0] = M;
        s_ml[warp][1] = L;
      }
      __syncthreads();
      if (way == 0)
        for (int w = 1; w < ways; ++w) add(s_ml[warp + w][0], s_ml[warp + w][1], &s_o[warp + w][lane * V]);
      __syncthreads();
    }
    if (way == 0 && col < R) {
      const int64_t row = (int64_t(sp.seq) * T + col / G) * a.n_q_heads + sp.head * G + col % G;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = L == 0.0f ? 0.0f : o[i] / L;
      float* const to = a.out + row * D + lane * V;
      if constexpr (V == 4) *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(o);
      else *reinterpret_cast<float2*>(to) = *reinterpret_cast<const float2*>(o);
      if (a.lse && lane == 0) a.lse[row] = lse_of(M, L, a.sm_scale);
    }
  }
}

int paged_ctas(int n_sms, int teams) { return min(n_sms, kPaMaxTeams / teams); }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// TMA descriptor of K or V pages as (128-byte lines, a page's lines, pages), or with 128-dim
// f16 rows (row, a page's rows, pages); a tile holds `rows` rows resp. halves of rows. The driver
// API asks for a base address and strides that are multiples of 16 bytes (32 only with
// interleaving) and, with the 128-byte swizzle, an inner extent of the tile of at most 128
// bytes; it is the tile in shared memory that lies on 1024 (the pattern), not the pages.
cudaError_t encode_pages(const PagedView& c, int format, void* pages, int rows, CUtensorMap* out) {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  if (!fn) return cudaErrorNotSupported;
  const bool f16 = format == QSA_PAGE_F16;
  const int bytes = page_row_bytes(format, c.head_dim), line = max(bytes, 128), per_line = line / bytes;
  const cuuint64_t dims[3] = {cuuint64_t(f16 ? line / 2 : line), (cuuint64_t(c.n_kv_heads) << c.page_shift) / per_line,
                              cuuint64_t(c.n_pages)};
  const cuuint64_t strides[2] = {cuuint64_t(line), cuuint64_t(c.page_stride)};
  const cuuint32_t box[3] = {f16 ? 64u : 128u, cuuint32_t(rows / per_line), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(out, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pages, dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Attributes of one kernel, set once per device. The warpgroups' shares of the registers come
// out of what the launch allocates (a larger sum would wait for registers for good): refused
// if the kernel was compiled for fewer.
template <typename C, typename K>  // C: one set of flags a kernel
cudaError_t prepare_kernel(K kernel, int smem, int regs, int device) {
  static std::atomic<unsigned long long> ready{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (device < 64 && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, kernel);
  if (e == cudaSuccess && f.numRegs < regs) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, kCarveoutMaxShared);
  if (e == cudaSuccess && device < 64) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int FMT, int D, int NC>
cudaError_t launch_pa(const PagedView& c, const PagedAttendArgs& a, int n_sms, int device, cudaStream_t s) {
  using C = PaCfg<FMT, D, NC>;
  const auto kernel = paged_attend_kernel<FMT, D, NC>;
  cudaError_t e = prepare_kernel<C>(kernel, C::BYTES, C::REGS, device);
  CUtensorMap kmap, vmap;
  const int rows = min(kPaTile, 1 << c.page_shift);  // of a TMA tile
  if (e == cudaSuccess) e = encode_pages(c, FMT, c.k, rows, &kmap);
  if (e == cudaSuccess) e = encode_pages(c, FMT, c.v, rows, &vmap);
  if (e != cudaSuccess) return e;
  const int ctas = paged_ctas(n_sms, C::TEAMS), n = ctas * C::TEAMS, R = a.n_q_heads / c.n_kv_heads * a.n_queries;
  const float c1 = a.sm_scale * kLog2e;
  const PaExp x{c1, kPaSlack / c1};
  PaSplit* splits = static_cast<PaSplit*>(a.workspace);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + align256(n * sizeof(PaSplit)));
  e = launch_pdl(kernel, dim3(ctas), dim3(C::THREADS), C::BYTES, s, 1, kmap, vmap, c, a, x, part, splits);
  if (e != cudaSuccess) return e;
  // one merge CTA for each segment that may be cut, or several where they are few
  const long long segments = (long long)a.n_seqs * c.n_kv_heads;
  const int nx = segments < n ? int(segments) : n, ny = min(R, max(1, 2 * n_sms / nx));
  return launch_pdl(paged_merge_kernel<D>, dim3(nx, ny), dim3(32 * kPmWarps), 0, s, 1, a, (const float*)part,
                    (const PaSplit*)splits, c.n_kv_heads, x.c1);
}

template <int FMT, int D>
cudaError_t launch_pa_cols(const PagedView& c, const PagedAttendArgs& a, int n_sms, int device, cudaStream_t s) {
  switch ((a.n_q_heads / c.n_kv_heads * a.n_queries + 7) / 8) {
    case 1: return launch_pa<FMT, D, 1>(c, a, n_sms, device, s);
    case 2: return launch_pa<FMT, D, 2>(c, a, n_sms, device, s);
    case 3: return launch_pa<FMT, D, 3>(c, a, n_sms, device, s);
    case 4: return launch_pa<FMT, D, 4>(c, a, n_sms, device, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

constexpr int kPaMostTeams = 3;  // the largest PaCfg::TEAMS

size_t paged_workspace_bytes(int head_dim, int n_q_heads, int n_kv_heads, int n_queries, int n_sms) {
  const size_t n = min(n_sms * kPaMostTeams, kPaMaxTeams), R = size_t(n_q_heads) / n_kv_heads * n_queries;
  return align256(n * sizeof(PaSplit)) + align256(2 * n * R * (head_dim + 4) * sizeof(float));
}

cudaError_t launch_paged_attend(const PagedView& c, int format, const PagedAttendArgs& a, int n_sms, int device,
                                cudaStream_t s) {
  const bool wide = c.head_dim == 128;
  switch (format) {
    case QSA_PAGE_F16:
      return wide ? launch_pa_cols<QSA_PAGE_F16, 128>(c, a, n_sms, device, s) : launch_pa_cols<QSA_PAGE_F16, 64>(c, a, n_sms, device, s);
    case QSA_PAGE_FP8:
      return wide ? launch_pa_cols<QSA_PAGE_FP8, 128>(c, a, n_sms, device, s) : launch_pa_cols<QSA_PAGE_FP8, 64>(c, a, n_sms, device, s);
    case QSA_PAGE_INT4:
      return wide ? launch_pa_cols<QSA_PAGE_INT4, 128>(c, a, n_sms, device, s) : launch_pa_cols<QSA_PAGE_INT4, 64>(c, a, n_sms, device, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
