// Dense GQA attention of every sequence's newest tokens over a paged K/V cache.
//
// Web page "Part 10", section "なぜFlash Attentionがcontext長に比例していたのか": dense
// attention reads the whole context for every token, which is what the sparse path avoids.
//   out = sum_c softmax_c(scale * q.K_c) V_c over the cells c < len - T + u + 1 of query u < T.
// One pass over K and V with a running maximum and sum, split over the whole batch:
//  - The (sequence, KV head) segments of a batch, cut into tiles of cells, form one list; CTA i
//    of N takes the i-th N-th of it (found from seq_lens on the device), so ragged batches
//    and single long sequences load every SM alike. A segment cut by a CTA border is written
//    as partials (m, l, o), at most two a CTA, which paged_merge_kernel joins:
//    sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s. Whole segments are written directly.
//  - A warp takes 16 or 32 cells at a time from its own ring of asynchronous 16-byte copies in
//    shared memory (no barrier between warps inside a segment). The products run on the tensor
//    cores, transposed: S^T = K q^T and O^T = V^T P^T, cells resp. dims as the 16 MMA rows
//    and the (query, head) rows of the KV head as columns, so that no MMA row is padding.
//    mma.sync rather than tcgen05: 8 to 32 columns leave the products far from any tensor
//    bound (the bytes bound this kernel), and 8- and 4-bit rows become f16 operands in
//    registers, where mma.sync takes them and tcgen05 would want them written back.
//  - Precision: codes are exact in f16 (e4m3 scales multiply logits and weights in f32; a 4-bit
//    value is an f16 product by definition). A weight enters the second product as two f16
//    terms of 2^15 p (22 bits, down to 2^-40 of the largest), which costs a second MMA and
//    keeps the result at f32 precision. The products of each 16 or 32 cells are added to the
//    running output in f32: the MMA's own sums truncate, and over a long chain that adds up.
//  - The newest T - 1 cells are not seen by every query, and whatever they hold must not reach
//    the others (0 * NaN is NaN): their V rows stay out of the MMA and are added one by one.
#include "qsa_paged.cuh"
#include "qsa_sm100.cuh"

namespace qsa {

namespace {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaCtasPerSm = 2;
constexpr int kPaTop = 32768;  // weights are scaled to f16's range: 2^15 p

template <int FMT, int D>
struct PaCfg {
  static constexpr int U = FMT == QSA_PAGE_F16 ? 16 : 32;  // cells a warp takes at a time
  static constexpr int SUBS = U / 16;
  static constexpr int TILE = U * kPaWarps;                // cells of a CTA's tile
  static constexpr int ROW = page_row_bytes_c<FMT>(D);
  static constexpr int SROW = page_scale_bytes_c<FMT>(D);
  static constexpr int KB = U * ROW;                       // bytes of a unit's K (V) rows
  static constexpr int SB = U * SROW;                      // and of their scales
  static constexpr int UNIT = 2 * KB + 2 * SB;
  // ring depth: about 100 KB a CTA, two CTAs an SM
  static constexpr int STAGES = 26112 / UNIT < 6 ? 26112 / UNIT : 6;
  static constexpr int KS = D / 16;                        // MMA k-steps of q.K = m-tiles of P.V
  static_assert(STAGES >= 2, "the ring needs two units");
};

// What merge CTA i joins: the segment that CTA i is the first to continue.
struct PaSplit {
  int seq, head;    // seq < 0: nothing
  int first, last;  // CTAs that hold a part
  int slot0;        // slot of the first one's part: 2 * first + (0 or 1); the others: 2 * cta
  int pad[3];
};

__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes16) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(high ? w >> 16 : w & 0xffffu), __NV_E4M3);
  return uint32_t(h.x) | (uint32_t(h.y) << 16);
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

// Where a 16-byte chunk of a unit's rows goes in shared memory: 128-byte lines whose chunks
// are permuted so that the fragment reads below fall on different banks.
template <int FMT, int D, bool IS_V>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
  constexpr int ROW = page_row_bytes_c<FMT>(D);
  if constexpr (FMT == QSA_PAGE_F16) {
    return off ^ (((off / ROW) & 7) << 4);
  } else if constexpr (!IS_V) {
    return ROW == 128 ? off ^ (((off >> 7) & 1) << 6) : off;
  } else if constexpr (ROW == 128) {
    return off ^ (((off >> 7) & 6) << 4);
  } else if constexpr (ROW == 64) {
    return off ^ (((off >> 7) & 3) << 5);
  } else {
    return off ^ (((off >> 7) & 1) << 5);
  }
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

// The work list: sequence s has tiles(s) = ceil(len / TILE) tiles for each KV head.
struct PaPlace {
  int seq;
  long long base;  // index of the sequence's first tile
};

// Sum over the CTA in thread order: this thread's exclusive prefix, the total in *total.
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
  for (int w = 0; w < kPaWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return before + x - v;
}

template <int FMT, int D, int NC>
struct PaSmem {
  using C = PaCfg<FMT, D>;
  static constexpr int RING = kPaWarps * C::STAGES * C::UNIT;
  static constexpr int OPAD = D + 4;  // floats a row of the warps' outputs, merged in the ring's memory
  static constexpr int MERGE = kPaWarps * 8 * OPAD * 4;
  static constexpr int Q = NC > 1 ? C::KS * NC * 32 * 8 : 0;
  static constexpr int BYTES = (RING > MERGE ? RING : MERGE) + Q;
  static_assert(BYTES <= 110 * 1024, "two CTAs an SM");
};

template <int FMT, int D, int NC>
__global__ void __launch_bounds__(kPaThreads, kPaCtasPerSm)
paged_attend_kernel(PagedView c, PagedAttendArgs a, float* __restrict__ part, PaSplit* __restrict__ splits) {
  using C = PaCfg<FMT, D>;
  using SM = PaSmem<FMT, D, NC>;
  constexpr int U = C::U, SUBS = C::SUBS, KS = C::KS, STAGES = C::STAGES;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kPaWarps], s_base;
  __shared__ int s_seq;
  __shared__ float s_m[kPaWarps][8 * NC], s_l[kPaWarps][8 * NC];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = a.n_q_heads / c.n_kv_heads, T = a.n_queries, R = G * T, Hkv = c.n_kv_heads;
  const int cta = blockIdx.x;
  const long long table_cells = (long long)a.table_width << c.page_shift;
  const uint32_t ring = sm100::smem_u32(smem) + warp * STAGES * C::UNIT;
  unsigned char* const s_q = smem + (SM::BYTES - SM::Q);
  const float c1 = a.sm_scale * 1.44269504088896341f;  // logits in units of log 2

  pdl_wait();
  pdl_launch_dependents();

  const auto length = [&](int s) {
    const int n = a.seq_lens[s];
    return n < 0 ? 0 : n > table_cells ? int(table_cells) : n;
  };
  const auto tiles = [&](int s) { return (length(s) + C::TILE - 1) / C::TILE; };

  // ---- this CTA's part of the list ----
  long long total = 0;
  for (int b = 0; b < a.n_seqs; b += kPaThreads) {
    long long sum;
    cta_scan(b + tid < a.n_seqs ? tiles(b + tid) : 0, s_scan, &sum);
    total += sum;
  }
  total *= Hkv;
  // at least one tile each: CTAs beyond the tiles have nothing to do
  const int N = int(min((long long)gridDim.x, total));
  const long long lo = cta < N ? cta * total / N : 0, hi = cta < N ? (cta + 1) * total / N : 0;
  {
    long long before = 0;
    for (int b = 0; b < a.n_seqs; b += kPaThreads) {
      const long long mine = b + tid < a.n_seqs ? tiles(b + tid) : 0;
      long long sum;
      const long long at = (before + cta_scan(mine, s_scan, &sum)) * Hkv;
      if (mine > 0 && at <= lo && lo < at + mine * Hkv) {
        s_seq = b + tid;
        s_base = at;
      }
      before += sum;
      if (before * Hkv > lo) break;
    }
  }
  // bad lengths and the results of sequences without cells: a CTA looks after its share
  for (int s = cta; s < a.n_seqs; s += gridDim.x) {
    const int n = a.seq_lens[s];
    if (tid == 0 && n < 0) record_status(a.status, QSA_ERR_BAD_INDEX);
    if (tid == 0 && n > table_cells) record_status(a.status, QSA_ERR_CAPACITY);
    if (n <= 0) {
      const int rows = T * a.n_q_heads;
      for (int e = tid; e < rows * D; e += kPaThreads) a.out[(int64_t)s * rows * D + e] = 0.0f;
      if (a.lse)
        for (int e = tid; e < rows; e += kPaThreads) a.lse[(int64_t)s * rows + e] = -INFINITY;
    }
  }
  __syncthreads();
  if (lo >= hi) {
    if (tid == 0) splits[cta].seq = -1;
    return;
  }

  int seq = s_seq, len = length(seq), nt = (len + C::TILE - 1) / C::TILE;
  int head = int((lo - s_base) / nt), tile0 = int((lo - s_base) % nt);
  if (tid == 0) {
    // the first CTA that continues a segment names the parts to merge
    PaSplit sp;
    sp.seq = -1;
    if (tile0 > 0) {
      const long long b = lo - tile0, e = b + nt;
      const long long first = ((b + 1) * N - 1) / total, last = (e * N - 1) / total;
      if (first == cta - 1) {
        sp.seq = seq;
        sp.head = head;
        sp.first = int(first);
        sp.last = int(last);
        sp.slot0 = int(2 * first + (first * total / N == b ? 0 : 1));
      }
    }
    splits[cta] = sp;
  }

  bool first_segment = true;
  for (long long at = lo; at < hi;) {
    const int tile1 = int(min((long long)nt, tile0 + (hi - at)));
    const int c0 = tile0 * C::TILE, c1_cell = min(len, tile1 * C::TILE);
    const int seen = len - T + 1;  // cells before this one are seen by every query

    // ---- copies ----
    const int my0 = c0 + warp * U;  // this warp's units: my0, my0 + TILE, ...
    const int units = my0 < c1_cell ? (c1_cell - my0 + C::TILE - 1) / C::TILE : 0;
    const int32_t* table = a.block_table + (long long)seq * a.table_width;
    const auto page_of = [&](int unit, int sub) {  // -1: past the end
      const int cell = my0 + unit * C::TILE + sub * 16;
      return unit < units && cell < c1_cell ? table[cell >> c.page_shift] : -1;
    };
    int next_page[SUBS];
    unsigned lost = 0;  // bit (ring slot, sub): its page is not in the pool
#pragma unroll
    for (int s = 0; s < SUBS; ++s) next_page[s] = page_of(0, s);
    const auto issue = [&](int unit) {
      if (unit < units) {
        const uint32_t dst = ring + (unit % STAGES) * C::UNIT;
        const int u0 = my0 + unit * C::TILE;
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
          const int cell0 = u0 + s * 16;
          int page = next_page[s];
          next_page[s] = page_of(unit + 1, s);
          int nk = min(16, len - cell0), nv = min(16, seen - cell0);  // rows to load (may be <= 0)
          const unsigned bit = 1u << ((unit % STAGES) * SUBS + s);
          lost &= ~bit;
          if (nk > 0 && (page < 0 || page >= c.n_pages)) {
            if (lane == 0) record_status(a.status, QSA_ERR_BAD_INDEX);
            lost |= bit;
            nk = 0;
          }
          if (nk <= 0) page = 0, nk = 0, nv = 0;
          const int row = row_in_page(c, head, cell0 & ((1 << c.page_shift) - 1));
          const char* ks = c.k + page * c.page_stride + (int64_t)row * C::ROW;
          const char* vs = c.v + page * c.page_stride + (int64_t)row * C::ROW;
#pragma unroll
          for (int i = 0; i < C::ROW / 32; ++i) {
            const uint32_t off = (i * 32 + lane) * 16;
            const int r = off / C::ROW;
            const uint32_t o = s * 16 * C::ROW + off;
            cp_async(dst + swizzled<FMT, D, false>(o), r < nk ? ks + off : c.k, r < nk ? 16 : 0);
            cp_async(dst + C::KB + swizzled<FMT, D, true>(o), r < nv ? vs + off : c.v, r < nv ? 16 : 0);
          }
          if constexpr (C::SROW > 0) {
            // (a 4-bit row of zeros stands for -8 scale: no scale where no V row is loaded)
            const bool ok = (lane & 15) < (FMT == QSA_PAGE_INT4 && lane >= 16 ? nv : nk);
            const char* base = lane < 16 ? c.ks : c.vs;
            const char* src = ok ? base + page * c.scale_stride + (int64_t)(row + (lane & 15)) * C::SROW : base;
            cp_async_small<C::SROW>(dst + 2 * C::KB + (lane < 16 ? 0 : C::SB) + (s * 16 + (lane & 15)) * C::SROW, src,
                                    ok ? C::SROW : 0);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(i);

    // ---- queries: B fragments, column = (query, head) row of this KV head ----
    const __half* q0 = static_cast<const __half*>(a.q) + (int64_t)seq * T * a.q_stride;
    const auto q_frag = [&](int j, int col, int tt) {
      uint2 f = make_uint2(0u, 0u);
      if (col < R) {
        const __half* q = q0 + (col / G) * a.q_stride + (head * G + col % G) * D;
        f.x = as_u32(__halves2half2(q[q_dim<FMT, D>(j, tt, 0)], q[q_dim<FMT, D>(j, tt, 1)]));
        f.y = as_u32(__halves2half2(q[q_dim<FMT, D>(j, tt, 2)], q[q_dim<FMT, D>(j, tt, 3)]));
      }
      return f;
    };
    uint2 qf[NC == 1 ? KS : 1];
    if constexpr (NC == 1) {
#pragma unroll
      for (int j = 0; j < KS; ++j) qf[j] = q_frag(j, g, t);
    } else {
      for (int e = tid; e < KS * NC * 32; e += kPaThreads)
        reinterpret_cast<uint2*>(s_q)[e] = q_frag(e / (32 * NC), (e / 32 % NC) * 8 + ((e & 31) >> 2), e & 3);
      __syncthreads();
    }
    int limit[NC][2];  // cells that column 2t + i sees
    float m[NC][2], l[NC][2], acc[KS][NC][4];
    float vtop = 0x1p-60f;  // power of two, at least the largest V scale so far (e4m3)
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * t + i;
        limit[n][i] = col < R ? seen + col / G : 0;
        m[n][i] = -INFINITY;
        l[n][i] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][n][i] = 0.0f;
    }

    // ---- this warp's units ----
    for (int unit = 0; unit < units; ++unit) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      const uint32_t uk = ring + (unit % STAGES) * C::UNIT, uv = uk + C::KB, uks = uv + C::KB, uvs = uks + C::SB;
      const int u0 = my0 + unit * C::TILE;

      // S^T: cells g and g + 8 of each 16, columns 2t and 2t + 1
      float s[SUBS][NC][4];
#pragma unroll
      for (int sb = 0; sb < SUBS; ++sb) {
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sb][n][i] = 0.0f;
        uint4 raw[2][2];
        __half2 ksc[2];
        if constexpr (FMT == QSA_PAGE_FP8) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              raw[r][h] = lds128(uk + swizzled<FMT, D, false>((sb * 16 + g + 8 * r) * D + h * 64 + t * 16));
        } else if constexpr (FMT == QSA_PAGE_INT4) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = sb * 16 + g + 8 * r;
            if constexpr (D == 128) {
              raw[r][0] = lds128(uk + row * 64 + t * 16);
            } else {
              const uint2 w = lds64(uk + row * 32 + t * 8);
              raw[r][0] = make_uint4(w.x, w.y, 0u, 0u);
            }
            const int grp = D == 128 ? t : t >> 1;
            const uint32_t w = lds32(uks + row * C::SROW + (grp >> 1) * 4);
            ksc[r] = (grp & 1) ? __high2half2(as_h2(w)) : __low2half2(as_h2(w));
          }
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          uint32_t f[4];
          if constexpr (FMT == QSA_PAGE_F16) {
            ldsm4(f, uk + swizzled<FMT, D, false>((lane & 15) * C::ROW + j * 32 + (lane >> 4) * 16));
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
            else b = reinterpret_cast<const uint2*>(s_q)[(j * NC + n) * 32 + lane];
            mma(s[sb][n], f[0], f[1], f[2], f[3], b.x, b.y);
          }
        }
      }

      // logits, running maximum, weights
      float vf[SUBS][2];
      float vmax = 0.0f;
#pragma unroll
      for (int sb = 0; sb < SUBS; ++sb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float f = c1;
          vf[sb][r] = 1.0f;
          if constexpr (FMT == QSA_PAGE_FP8) {
            const int row = sb * 16 + g + 8 * r;
            f *= __uint_as_float(lds32(uks + row * 4));
            if (u0 + row < seen) {  // (the newest cells' scales are applied with their rows)
              vf[sb][r] = __uint_as_float(lds32(uvs + row * 4));
              vmax = fmaxf(vmax, vf[sb][r]);
            }
          }
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) s[sb][n][2 * r + i] *= f;
        }
      // cells that some query does not see, or that are not there
#pragma unroll
      for (int sb = 0; sb < SUBS; ++sb) {
        const bool gone = (lost >> ((unit % STAGES) * SUBS + sb)) & 1;
        if (gone || u0 + sb * 16 + 16 > seen) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (gone || u0 + sb * 16 + g + 8 * r >= limit[n][i]) s[sb][n][2 * r + i] = -INFINITY;
        }
      }
      float fv = float(kPaTop), keep = 1.0f;
      if constexpr (FMT == QSA_PAGE_FP8) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
        const float top = fmaxf(vtop, __uint_as_float((__float_as_uint(vmax) + 0x7fffffu) & 0x7f800000u));
        keep = vtop / top;  // both powers of two
        vtop = top;
        fv = float(kPaTop) / top;
      }
      float corr[NC][2];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = -INFINITY;
#pragma unroll
          for (int sb = 0; sb < SUBS; ++sb) x = fmaxf(x, fmaxf(s[sb][n][i], s[sb][n][2 + i]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
          x = fmaxf(x, m[n][i]);
          const float base = x == -INFINITY ? 0.0f : x;  // nothing seen yet: all weights 2^-inf = 0
          corr[n][i] = ex2(m[n][i] - base);
          m[n][i] = x;
          float sum = 0.0f;
#pragma unroll
          for (int sb = 0; sb < SUBS; ++sb)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float p = ex2(s[sb][n][2 * r + i] - base);
              sum += p;
              s[sb][n][2 * r + i] = p * (vf[sb][r] * fv);
            }
          l[n][i] = l[n][i] * corr[n][i] + sum;
          corr[n][i] *= keep;
        }

      // P^T as B fragments: two f16 terms of each weight
      uint32_t ph[SUBS][NC][2], pl[SUBS][NC][2];
#pragma unroll
      for (int sb = 0; sb < SUBS; ++sb)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const bool in = u0 + sb * 16 + g + 8 * r < seen;
            const float x = in ? s[sb][n][2 * r] : 0.0f, y = in ? s[sb][n][2 * r + 1] : 0.0f;
            const __half2 h = __floats2half2_rn(x, y);
            const float2 back = __half22float2(h);
            ph[sb][n][r] = transpose8x8(as_u32(h));
            pl[sb][n][r] = transpose8x8(as_u32(__floats2half2_rn(x - back.x, y - back.y)));
          }

      // O^T += V^T P^T
      uint4 raw[SUBS][4];
      __half2 vsc[SUBS][4];
      if constexpr (FMT != QSA_PAGE_F16) {
#pragma unroll
        for (int sb = 0; sb < SUBS; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = sb * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
            const uint32_t at_row = uv + swizzled<FMT, D, true>(row * C::ROW + g * (C::ROW / 8));
            if constexpr (C::ROW == 128) {
              raw[sb][i] = lds128(at_row);
            } else if constexpr (C::ROW == 64) {
              const uint2 w = lds64(at_row);
              raw[sb][i] = make_uint4(w.x, w.y, 0u, 0u);
            } else {
              raw[sb][i] = make_uint4(lds32(at_row), 0u, 0u, 0u);
            }
            if constexpr (FMT == QSA_PAGE_INT4) {
              const int grp = D == 128 ? g >> 1 : g >> 2;
              const uint32_t w = lds32(uvs + row * C::SROW + (grp >> 1) * 4);
              vsc[sb][i] = (grp & 1) ? __high2half2(as_h2(w)) : __low2half2(as_h2(w));
            }
          }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        float d[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[n][i] = 0.0f;
#pragma unroll
        for (int sb = 0; sb < SUBS; ++sb) {
          uint32_t f[4];
          if constexpr (FMT == QSA_PAGE_F16) {
            ldsm4_trans(f, uv + swizzled<FMT, D, true>(((lane >> 4) * 8 + (lane & 7)) * C::ROW + k * 32 + ((lane >> 3) & 1) * 16));
          } else {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (FMT == QSA_PAGE_FP8) h[i] = e4m3x2(word_of(raw[sb][i], k >> 1), k & 1);
              else h[i] = int4x2(word_of(raw[sb][i], k >> 2), k & 3, vsc[sb][i]);
            }
            f[0] = __byte_perm(h[0], h[1], 0x5410);
            f[1] = __byte_perm(h[0], h[1], 0x7632);
            f[2] = __byte_perm(h[2], h[3], 0x5410);
            f[3] = __byte_perm(h[2], h[3], 0x7632);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            mma(d[n], f[0], f[1], f[2], f[3], ph[sb][n][0], ph[sb][n][1]);
            mma(d[n], f[0], f[1], f[2], f[3], pl[sb][n][0], pl[sb][n][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[k][n][i] = fmaf(acc[k][n][i], corr[n][i & 1], d[n][i]);
      }

      // the newest cells, which not every query sees: one by one
      if (u0 + U > seen && seen < len) {
#pragma unroll
        for (int sb = 0; sb < SUBS; ++sb)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            for (int cell = max(seen, u0 + sb * 16 + 8 * r); cell < min(len, u0 + sb * 16 + 8 * r + 8); ++cell) {
              const int page = cell >= 0 ? table[cell >> c.page_shift] : -1;
              const int src = ((cell - u0) & 7) * 4 + t;
              float w[NC][2];
#pragma unroll
              for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[n][i] = __shfl_sync(0xffffffffu, s[sb][n][2 * r + i], src);
              if (page < 0 || page >= c.n_pages) continue;
              const int row = row_in_page(c, head, cell & ((1 << c.page_shift) - 1));
              const char* vr = c.v + page * c.page_stride + (int64_t)row * C::ROW;
              const char* vs = C::SROW ? c.vs + page * c.scale_stride + (int64_t)row * C::SROW : nullptr;
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
                      if (cell < limit[n][i]) acc[k][n][2 * h + i] = fmaf(w[n][i], x, acc[k][n][2 * h + i]);
                }
            }
      }
      __syncwarp();
      issue(unit + STAGES - 1);
    }

    // ---- the warps' results joined in the ring's memory ----
    cp_async_wait<0>();
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], off);
        if (g == 0) {
          s_m[warp][n * 8 + 2 * t + i] = m[n][i];
          s_l[warp][n * 8 + 2 * t + i] = l[n][i];
        }
      }
    __syncthreads();
    const bool complete = tile0 == 0 && tile1 == nt;
    float* const out_part = part + int64_t(2 * cta + (first_segment ? 0 : 1)) * R * (D + 2);
    float* const s_o = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * t + i;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) M = fmaxf(M, s_m[w][col]);
        // a warp that saw nothing has l = 0 (a NaN logit makes l, and then everything, NaN)
        f[i] = s_l[warp][col] == 0.0f ? 0.0f : ex2(s_m[warp][col] - M) * (FMT == QSA_PAGE_FP8 ? vtop / kPaTop : 1.0f / kPaTop);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s_o[(warp * 8 + 2 * t + (i & 1)) * SM::OPAD + v_dim<FMT, D>(k, g, i >> 1)] = acc[k][n][i] * f[i & 1];
      __syncthreads();
      for (int e = tid; e < 8 * D; e += kPaThreads) {
        const int cc = e / D, d = e % D, col = n * 8 + cc;
        if (col >= R) break;
        float o = 0.0f, M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) {
          o += s_o[(w * 8 + cc) * SM::OPAD + d];
          M = fmaxf(M, s_m[w][col]);
        }
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w)
          if (s_l[w][col] != 0.0f) L += ex2(s_m[w][col] - M) * s_l[w][col];
        if (complete) {
          const int64_t row = (int64_t(seq) * T + col / G) * a.n_q_heads + head * G + col % G;
          a.out[row * D + d] = L == 0.0f ? 0.0f : o / L;
          if (a.lse && d == 0) a.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
        } else {
          out_part[col * (D + 2) + d] = o;
          if (d == 0) {
            out_part[col * (D + 2) + D] = M;
            out_part[col * (D + 2) + D + 1] = L;
          }
        }
      }
      __syncthreads();
    }

    // ---- next segment ----
    at += tile1 - tile0;
    tile0 = 0;
    first_segment = false;
    if (++head == Hkv && at < hi) {
      head = 0;
      do {
        ++seq;
        len = length(seq);
      } while (len == 0);
      nt = (len + C::TILE - 1) / C::TILE;
    }
  }
}

// CTA (i, row): joins row `row` of the parts of the segment that attend CTA i was the first
// to continue.
constexpr int kPmThreads = 128;

template <int D>
__global__ void __launch_bounds__(kPmThreads) paged_merge_kernel(PagedAttendArgs a, const float* __restrict__ part,
                                                                 const PaSplit* __restrict__ splits, int n_kv_heads) {
  __shared__ float s_w[2048];
  __shared__ float s_red[kPmThreads / 32];
  __shared__ float s_o[kPmThreads];
  pdl_launch_dependents();
  pdl_wait();
  const PaSplit sp = splits[blockIdx.x];
  if (sp.seq < 0) return;
  const int G = a.n_q_heads / n_kv_heads, T = a.n_queries, R = G * T, col = blockIdx.y;
  const int n = sp.last - sp.first + 1;
  const int64_t step = int64_t(R) * (D + 2);
  const auto row_of = [&](int p) { return part + (p == 0 ? sp.slot0 : 2 * (sp.first + p)) * step + col * (D + 2); };
  float M = -INFINITY;
  for (int p = threadIdx.x; p < n; p += kPmThreads) M = fmaxf(M, row_of(p)[D]);
  M = warp_max(M);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPmThreads / 32; ++w) M = fmaxf(M, s_red[w]);
  __syncthreads();
  float L = 0.0f;
  for (int p = threadIdx.x; p < n; p += kPmThreads) {
    const float l = row_of(p)[D + 1];
    const float w = l == 0.0f ? 0.0f : ex2(row_of(p)[D] - M);
    s_w[p] = w;
    L += w * l;
  }
  L = warp_sum(L);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = L;
  __syncthreads();
  L = 0.0f;
#pragma unroll
  for (int w = 0; w < kPmThreads / 32; ++w) L += s_red[w];
  // D = 64: two halves of the CTA take every other part
  constexpr int WAYS = kPmThreads / D;
  const int d = threadIdx.x % D, way = threadIdx.x / D;
  float o = 0.0f;
#pragma unroll 8
  for (int p = way; p < n; p += WAYS) o += s_w[p] * row_of(p)[d];
  if constexpr (WAYS == 2) {
    s_o[threadIdx.x] = o;
    __syncthreads();
    o += s_o[threadIdx.x ^ D];
    if (way) return;
  }
  const int64_t row = (int64_t(sp.seq) * T + col / G) * a.n_q_heads + sp.head * G + col % G;
  a.out[row * D + d] = L == 0.0f ? 0.0f : o / L;
  if (a.lse && d == 0) a.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
}

int paged_ctas(int n_sms) { return n_sms * kPaCtasPerSm < 2048 ? n_sms * kPaCtasPerSm : 2048; }

template <int FMT, int D, int NC>
cudaError_t launch_pa(const PagedView& c, const PagedAttendArgs& a, int n_sms, cudaStream_t s) {
  using SM = PaSmem<FMT, D, NC>;
  const auto kernel = paged_attend_kernel<FMT, D, NC>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::BYTES);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, kCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  const int n = paged_ctas(n_sms), R = a.n_q_heads / c.n_kv_heads * a.n_queries;
  PaSplit* splits = static_cast<PaSplit*>(a.workspace);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + align256(n * sizeof(PaSplit)));
  e = launch_pdl(kernel, dim3(n), dim3(kPaThreads), SM::BYTES, s, 1, c, a, part, splits);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_merge_kernel<D>, dim3(n, R), dim3(kPmThreads), 0, s, 1, a, (const float*)part,
                    (const PaSplit*)splits, c.n_kv_heads);
}

template <int FMT, int D>
cudaError_t launch_pa_cols(const PagedView& c, const PagedAttendArgs& a, int n_sms, cudaStream_t s) {
  switch ((a.n_q_heads / c.n_kv_heads * a.n_queries + 7) / 8) {
    case 1: return launch_pa<FMT, D, 1>(c, a, n_sms, s);
    case 2: return launch_pa<FMT, D, 2>(c, a, n_sms, s);
    case 3: return launch_pa<FMT, D, 3>(c, a, n_sms, s);
    case 4: return launch_pa<FMT, D, 4>(c, a, n_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t paged_workspace_bytes(int head_dim, int n_q_heads, int n_kv_heads, int n_queries, int n_sms) {
  const size_t n = paged_ctas(n_sms), R = size_t(n_q_heads) / n_kv_heads * n_queries;
  return align256(n * sizeof(PaSplit)) + align256(2 * n * R * (head_dim + 2) * sizeof(float));
}

cudaError_t launch_paged_attend(const PagedView& c, int format, const PagedAttendArgs& a, int n_sms, cudaStream_t s) {
  const bool wide = c.head_dim == 128;
  switch (format) {
    case QSA_PAGE_F16: return wide ? launch_pa_cols<QSA_PAGE_F16, 128>(c, a, n_sms, s) : launch_pa_cols<QSA_PAGE_F16, 64>(c, a, n_sms, s);
    case QSA_PAGE_FP8: return wide ? launch_pa_cols<QSA_PAGE_FP8, 128>(c, a, n_sms, s) : launch_pa_cols<QSA_PAGE_FP8, 64>(c, a, n_sms, s);
    case QSA_PAGE_INT4: return wide ? launch_pa_cols<QSA_PAGE_INT4, 128>(c, a, n_sms, s) : launch_pa_cols<QSA_PAGE_INT4, 64>(c, a, n_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
