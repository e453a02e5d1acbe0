// block_attn.cu -- decode attention over block rows (grouped-query heads; bf16 or 4-bit
// rows; sliding window with sinks; block tables or recalled selections).
//
// For the M = n_q * n_heads / n_kv_heads query rows that share KV head h of request b:
//   x_p = scale * q . k_p,   out = sum_p 2^(x_p log2 e - m) v_p / l,   one pass over p
// with the running maximum m and sum l of each row.  K and V are read once from HBM, which
// is the bound: 4 D bytes a token and KV head in bf16, 18 D / 16 in 4 bits, against
// 4 M D flops (M is 1 to 32, so the legacy-size matrix instructions below are never the
// limit; a 128-row tcgen05 tile would be 7/8 padding or more).
//
// sm_103a design.
//   Transposed products: S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16, tokens (then
//     dimensions) as the 16 rows and the query rows as the 8 columns, so a group of 8 query
//     heads fills the instruction exactly and each cache element is converted once for all
//     query rows.  P^T needs the transpose of S^T's fragment: one movmatrix per 8 tokens.
//   A warp is a worker of its own: it takes every kWarps-th chunk (16 or 32 tokens) of the
//     CTA's range, keeps its own m, l and O, and fills its own ring of shared-memory stages
//     with cp.async, ahead of the chunk it computes and across the borders of requests; no
//     barrier runs inside the stream.  The warps of a CTA merge at the end of each (b, h).
//   Lazy maximum: m moves only when some score exceeds it by 2^8, so the rescaling of O (and
//     the shuffles that find a column's maximum) run a few times per stream instead of once
//     per chunk; the result is the same softmax, its terms scaled by at most 2^8.
//   4-bit rows: a lane reads the 16 bytes of a token that it feeds to the tensor cores (the
//     contraction's dimensions are permuted so that they are contiguous; Q is laid out to
//     match), converts e2m1 pairs with cvt and multiplies by the e4m3 scales in fp16, where
//     every product is exact.  Queries are taken to fp16 scaled by a power of two per row.
//   Split: all chunks of the call form one line, cut into equal pieces, one per CTA, by
//     the lengths on the device (a ragged batch costs no idle SMs).  A piece that ends
//     inside a (b, h) leaves a partial result; a second kernel merges those in order (no
//     atomics: results do not depend on timing).  When the contexts are short or the
//     (b, h) pairs fill the GPU, a CTA takes a whole (b, h) and the second kernel is left out.
#include "block_rows.cuh"

namespace echo {

constexpr int kBaMaxGrid = 456;   // CTAs of a split call (workspace pieces: two per CTA)
constexpr float kBaLazy = 8.f;    // log2 of how far a score may exceed the running maximum
// fp16 softmax weights are kept 2^7 up: at most 2^(7 + 8), and the subnormals (a grid of
// 2^-24) begin 2^-21 below the running maximum instead of 2^-14
constexpr float kBaLift = 7.f;
constexpr int kBaNowhere = 0x7fffff00;  // position of a sub-block that is not there
constexpr int kBaMaxRows = 32;    // query rows of one CTA's (b, h) (4 columns of 8)

struct BlockAttnParams {
  const uint16_t *q, *rows;
  int64_t row_bytes;
  int32_t n_rows, bsub;              // bsub: 16-token sub-blocks of a row
  const int32_t *table, *sel;
  int32_t table_heads, max_blocks;
  const int32_t *ctx_len;
  int32_t B, n_q, n_heads, n_kv, group, mgroups;  // group: query heads per KV head
  int32_t sinks, window;
  float scale_log2;
  uint16_t *out;
  float *lse;
  int32_t whole;                     // one CTA per (b, h, row group), nothing split
  float *part_o;                     // [2 * grid][rows][D]
  float *part_ml;                    // [2 * grid][rows][2]
  int4 *tail;                        // [grid]: (b, h * mgroups + mg, pieces, 0)
  int32_t *status;
};

// What a request's context asks for: its visible sub-blocks as one list.
struct ReqView {
  int len, wlo;        // tokens of the last query; first window token of the first query
  int n_first, skip;   // list entries >= n_first are `skip` sub-blocks further on
  int nsub;
};

__device__ __forceinline__ ReqView req_view(const BlockAttnParams &P, int ctx) {
  ReqView v;
  v.len = min(max(ctx, 0), kBaNowhere - 256);
  v.wlo = 0;
  if (P.sel) {
    v.nsub = v.len > 0 ? P.max_blocks * P.bsub : 0;
    v.n_first = v.nsub;
    v.skip = 0;
    if (P.window) v.wlo = max(v.len - (P.n_q - 1) - P.window, 0);
    return v;
  }
  v.len = min(v.len, P.max_blocks * P.bsub * kSubTokens);
  const int all = (v.len + kSubTokens - 1) / kSubTokens;
  v.n_first = v.nsub = all;
  v.skip = 0;
  if (P.window) {
    v.wlo = max(v.len - (P.n_q - 1) - P.window, 0);
    const int first = (min(P.sinks, v.len) + kSubTokens - 1) / kSubTokens, from = v.wlo / kSubTokens;
    if (from > first) {
      v.n_first = first;
      v.skip = from - first;
      v.nsub = all - v.skip;
    }
  }
  return v;
}

__device__ __forceinline__ void check_context(const BlockAttnParams &P, int ctx) {
  if (!P.sel && ctx > P.max_blocks * P.bsub * kSubTokens) set_status(P.status, ECHO_DEV_BAD_INDEX);
}

template <int FMT, int D, int NT, int WARPS, int STAGES>
struct BaCfg {
  static constexpr bool kFp4 = FMT == ECHO_BLOCK_FP4;
  static constexpr int kSubBytes = kFp4 ? 18 * D : 64 * D;  // K and V of 16 tokens
  static constexpr int kSubs = kFp4 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 2);
  static constexpr int kTokens = kSubs * kSubTokens;
  static constexpr int kStageBytes = kSubs * kSubBytes;
  static constexpr int kThreads = WARPS * 32;
  static constexpr int kSteps = D / 16;                      // k-steps of S^T, dim tiles of O^T
  static constexpr int kRows = 8 * NT;
  static constexpr int kMergeRow = D + 4;                    // floats; + 4: no bank conflicts
  // shared memory: stages | merge buffers | q fragments | per-row values | scan
  static constexpr int kOffMerge = WARPS * STAGES * kStageBytes;
  static constexpr int kOffQ = kOffMerge + WARPS * 8 * kMergeRow * 4;
  static constexpr int kOffMl = kOffQ + kSteps * NT * 32 * 8;
  static constexpr int kOffQs = kOffMl + WARPS * kRows * 8;
  static constexpr int kOffMeta = kOffQs + kRows * 4;
  static constexpr int kOffScan = kOffMeta + WARPS * STAGES * kSubs * 4;
  static constexpr int kSmem = kOffScan + 64 * 8 + 64;
};

__device__ __forceinline__ void ba_cp16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void ba_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ba_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log of a row's sum of weights 2^(x - top + lift)
__device__ __forceinline__ float ba_lse(float top, float sum, float lift) {
  return top == -INFINITY ? -INFINITY : (top - lift + log2f(sum)) * 0.693147180559945309f;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A place on the line of chunks: chunk g of the call is chunk g - start of the row group hm
// (KV head * row groups + row group) of request b.
struct LinePos {
  int b, hm;
  int64_t start, end;  // the line's range of this (b, hm)
  ReqView v;
};

template <int kSubs>
__device__ __forceinline__ int chunks_of(const ReqView &v) {
  return (v.nsub + kSubs - 1) / kSubs;
}

// moves forward to the (b, hm) that holds chunk g (g < the line's length)
template <int kSubs>
__device__ __forceinline__ void seek(const BlockAttnParams &P, LinePos &L, int64_t g) {
  while (g >= L.end) {
    const int heads = P.n_kv * P.mgroups;
    const int n = chunks_of<kSubs>(L.v);
    if (n > 0 && L.hm + 1 < heads) {
      const int64_t step = (g - L.end) / n;  // whole heads of this request to pass over
      const int by = static_cast<int>(min(static_cast<int64_t>(heads - 1 - L.hm), step + 1));
      L.hm += by;
      L.start = L.end + static_cast<int64_t>(by - 1) * n;
    } else {
      ++L.b;
      L.hm = 0;
      L.start = L.end;
      L.v = req_view(P, __ldg(P.ctx_len + L.b));
    }
    L.end = L.start + chunks_of<kSubs>(L.v);
  }
}

template <int FMT, int D, int NT, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32, 1) block_attn_kernel(const BlockAttnParams P) {
  using C = BaCfg<FMT, D, NT, WARPS, STAGES>;
  constexpr bool F16 = C::kFp4;
  constexpr float kLift = F16 ? kBaLift : 0.f;
  extern __shared__ __align__(128) uint8_t ba_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, c4 = lane & 3;  // fragment row and column pair
  uint8_t *stage_base = ba_smem + warp * STAGES * C::kStageBytes;
  float *merge = reinterpret_cast<float *>(ba_smem + C::kOffMerge);
  uint2 *qfrag = reinterpret_cast<uint2 *>(ba_smem + C::kOffQ);
  float2 *ml = reinterpret_cast<float2 *>(ba_smem + C::kOffMl);       // [WARPS][kRows]
  float *qscale = reinterpret_cast<float *>(ba_smem + C::kOffQs);     // [kRows]
  int32_t *meta = reinterpret_cast<int32_t *>(ba_smem + C::kOffMeta) + warp * STAGES * C::kSubs;
  int64_t *scan = reinterpret_cast<int64_t *>(ba_smem + C::kOffScan);
  const int heads = P.n_kv * P.mgroups;

  // ===== this CTA's range of the line =====
  LinePos cur;
  int64_t g0, g1;
  if (P.whole) {
    cur.b = blockIdx.x / heads;
    cur.hm = blockIdx.x - cur.b * heads;
    cur.v = req_view(P, __ldg(P.ctx_len + cur.b));
    cur.start = 0;
    cur.end = chunks_of<C::kSubs>(cur.v);
    g0 = 0;
    g1 = cur.end;
    if (threadIdx.x == 0 && cur.hm == 0) check_context(P, __ldg(P.ctx_len + cur.b));
  } else {
    // lengths of all requests' parts of the line: a run of requests per thread, summed
    const int per_t = (P.B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per_t, P.B), b1 = min(b0 + per_t, P.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int ctx = __ldg(P.ctx_len + b);
      mine += chunks_of<C::kSubs>(req_view(P, ctx));
      if (blockIdx.x == 0) check_context(P, ctx);
    }
    mine *= heads;
    int64_t s = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s += x;
    }
    if (lane == 31) scan[warp] = s;
    __syncthreads();
    int64_t before = s - mine, total = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    __syncthreads();
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    per = per < WARPS ? WARPS : per;
    g0 = per * blockIdx.x;
    g1 = min(total, g0 + per);
    if (g0 >= total) {
      if (threadIdx.x == 0) P.tail[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    if (g0 >= before && g0 < before + mine) {  // one thread's run holds g0
      int b = b0;
      int64_t at = before;
      for (;; ++b) {
        const int64_t n = static_cast<int64_t>(chunks_of<C::kSubs>(req_view(P, __ldg(P.ctx_len + b)))) * heads;
        if (g0 < at + n) break;
        at += n;
      }
      scan[32] = b;
      scan[33] = at;
    }
    __syncthreads();
    cur.b = static_cast<int>(scan[32]);
    cur.hm = 0;
    cur.start = scan[33];
    cur.v = req_view(P, __ldg(P.ctx_len + cur.b));
    cur.end = cur.start + chunks_of<C::kSubs>(cur.v);
    seek<C::kSubs>(P, cur, g0);
    if (threadIdx.x == 0) {
      // where the range's last (b, hm) goes on, and whether it began here
      LinePos e = cur;
      seek<C::kSubs>(P, e, g1 - 1);
      int pieces = 0;
      if (e.end > g1 && e.start >= g0) pieces = 1 + static_cast<int>((e.end - g1 + per - 1) / per);
      P.tail[blockIdx.x] = make_int4(e.b, e.hm, pieces, 0);
    }
  }

  // ===== the loader: rows of the chunk after next are looked up one chunk ahead =====
  LinePos ld = cur;
  int64_t ld_g = g0 + warp;
  int32_t ld_row[C::kSubs], ld_pos[C::kSubs];
  int ld_in[C::kSubs];  // sub-block inside its row
  auto lookup = [&]() {
    if (ld_g >= g1) return;
    seek<C::kSubs>(P, ld, ld_g);
    const int h = ld.hm / P.mgroups;
    const int64_t tb = (static_cast<int64_t>(ld.b) * P.table_heads + (P.table_heads > 1 ? h : 0)) * P.max_blocks;
    const int first = static_cast<int>(ld_g - ld.start) * C::kSubs;
#pragma unroll
    for (int u = 0; u < C::kSubs; ++u) {
      int s = first + u;
      ld_row[u] = -1;
      ld_pos[u] = kBaNowhere;  // no token of a missing sub-block is below any length
      ld_in[u] = 0;
      if (s >= ld.v.nsub) continue;
      if (s >= ld.v.n_first) s += ld.v.skip;
      const int e = s / P.bsub, in = s - e * P.bsub;
      const int32_t id = __ldg(P.table + tb + e);
      const int32_t lb = P.sel ? __ldg(P.sel + tb + e) : e;
      const int64_t row = P.table_heads > 1 ? id : static_cast<int64_t>(id) * P.n_kv + h;
      // (a selected block past the 31-bit positions cannot be below any length)
      if (id < 0 || lb < 0 || static_cast<int64_t>(lb) * P.bsub + in >= kBaNowhere / kSubTokens) continue;
      if (row >= P.n_rows) {
        set_status(P.status, ECHO_DEV_BAD_INDEX);
        continue;
      }
      ld_row[u] = static_cast<int32_t>(row);
      ld_pos[u] = (lb * P.bsub + in) * kSubTokens;
      ld_in[u] = in;
    }
  };
  auto issue = [&](int st) {
    if (ld_g < g1) {
      uint32_t dst = smem_u32(stage_base + st * C::kStageBytes);
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u, dst += C::kSubBytes) {
        if (lane == 0) meta[st * C::kSubs + u] = ld_pos[u];
        const bool held = ld_row[u] >= 0;
        const uint8_t *row = reinterpret_cast<const uint8_t *>(P.rows) + (held ? ld_row[u] : 0) * P.row_bytes;
        if constexpr (C::kFp4) {
          const uint8_t *src = row + static_cast<int64_t>(ld_in[u]) * C::kSubBytes;
          constexpr int kPieces = C::kSubBytes / 16;
#pragma unroll
          for (int i = 0; i < (kPieces + 31) / 32; ++i) {
            const int x = i * 32 + lane;
            if ((i + 1) * 32 <= kPieces || x < kPieces) ba_cp16(dst + x * 16, src + x * 16, held);
          }
        } else {
          // rows of 2 D bytes, 16-byte pieces XORed with the token so that ldmatrix reads
          // 8 tokens from 8 different bank groups
          const uint8_t *src = row + static_cast<int64_t>(ld_in[u]) * (kSubTokens * D * 2);
          const int64_t vofs = static_cast<int64_t>(P.bsub) * kSubTokens * D * 2;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int x = i * 32 + lane, tk = x / (D / 8), pc = x % (D / 8);
            const int p = ld_pos[u] + tk;
            // a token no query sees is read as zeros: its bytes may be anything
            const bool on = held && p < ld.v.len && (p >= ld.v.wlo || p < P.sinks);
            const uint32_t o = tk * (2 * D) + ((pc ^ (tk & 7)) << 4);
            ba_cp16(dst + o, src + x * 16, on);
            ba_cp16(dst + kSubTokens * D * 2 + o, src + vofs + x * 16, on);
          }
        }
      }
    }
    ba_commit();
    ld_g += WARPS;
    lookup();
  };
  lookup();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);

  int st = 0;
  int64_t g = g0 + warp;
  for (;;) {  // the (b, hm) of this range, one after another
    const int64_t pend = min(cur.end, g1);
    const int h = cur.hm / P.mgroups, mg = cur.hm - h * P.mgroups;
    const int row0 = mg * kBaMaxRows, rows = min(P.n_q * P.group - row0, C::kRows);
    // ----- the queries of this (b, hm) as B fragments -----
    if constexpr (F16) {
      // a warp per row: the power of two that brings its largest entry to [1, 2)
      for (int rr = warp; rr < C::kRows; rr += WARPS) {
        float m = 0.f;
        if (rr < rows) {
          const int rq = row0 + rr, j = rq / P.group;
          const uint16_t *src = P.q + ((static_cast<int64_t>(cur.b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group) * D;
          for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(__uint_as_float(static_cast<uint32_t>(src[d]) << 16)));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        e = max(min(e, 126), -126);  // (zero rows, subnormal and infinite maxima)
        if (lane == 0) qscale[rr] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < C::kSteps * NT * 32; i += C::kThreads) {
      const int ln = i & 31, nt = (i >> 5) % NT, s = (i >> 5) / NT;
      const int rr = nt * 8 + (ln >> 2), c = ln & 3;
      uint2 f = make_uint2(0u, 0u);
      if (rr < rows) {
        const int rq = row0 + rr, j = rq / P.group;
        const uint16_t *src = P.q + ((static_cast<int64_t>(cur.b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group) * D;
        if constexpr (F16) {
          const int d = (D / 4) * c + 8 * (s >> 1) + 4 * (s & 1);
          const uint2 w = *reinterpret_cast<const uint2 *>(src + d);
          const float inv = __uint_as_float((254u << 23) - __float_as_uint(qscale[rr]));  // exact 1 / 2^e
          f.x = pack2<true>(__uint_as_float(w.x << 16) * inv, __uint_as_float(w.x & 0xffff0000u) * inv);
          f.y = pack2<true>(__uint_as_float(w.y << 16) * inv, __uint_as_float(w.y & 0xffff0000u) * inv);
        } else {
          f.x = *reinterpret_cast<const uint32_t *>(src + 16 * s + 2 * c);
          f.y = *reinterpret_cast<const uint32_t *>(src + 16 * s + 2 * c + 8);
        }
      }
      qfrag[i] = f;
    }
    __syncthreads();
    uint2 qreg[NT == 1 ? C::kSteps : 1];
    if constexpr (NT == 1) {
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) qreg[s] = qfrag[s * 32 + lane];
    }
    float cscale[NT][2];
    int clen[NT][2];  // tokens below which a column's query sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = nt * 8 + 2 * c4 + e;
        cscale[nt][e] = P.scale_log2 * (F16 ? qscale[rr] : 1.f);
        clen[nt][e] = cur.v.len - (P.n_q - 1 - min((row0 + rr) / P.group, P.n_q - 1));
      }
    const int len_first = cur.v.len - (P.n_q - 1), w_last = P.window ? cur.v.len - P.window : 0;

    float m[NT][2], l[NT][2], o[C::kSteps][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < C::kSteps; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
    }

    // ----- the stream -----
    for (; g < pend; g += WARPS) {
      ba_wait<STAGES - 2>();
      __syncwarp();
      issue(st == 0 ? STAGES - 1 : st - 1);
      const uint8_t *sp = stage_base + st * C::kStageBytes;
      int pos[C::kSubs];
      bool edge = false;
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u) {
        pos[u] = meta[st * C::kSubs + u];
        const int last = pos[u] + kSubTokens - 1;
        edge |= !(last < len_first && (pos[u] >= w_last || last < P.sinks));
      }

      float s[C::kSubs][NT][4];
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
        const uint8_t *kp = sp + u * C::kSubBytes;
        if constexpr (C::kFp4) {
          constexpr int kWords = D / 32;  // 32-bit words of codes a lane reads per token
          uint32_t wa[kWords], wb[kWords], sa, sb;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kp + lane * 16);
            const uint4 y = *reinterpret_cast<const uint4 *>(kp + 8 * (D / 2) + lane * 16);
            wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
            wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
            sa = *reinterpret_cast<const uint16_t *>(kp + Fp4Sub<D>::kKeyScales + lane * 2);
            sb = *reinterpret_cast<const uint16_t *>(kp + Fp4Sub<D>::kKeyScales + 8 * (D / 16) + lane * 2);
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(kp + lane * 8);
            const uint2 y = *reinterpret_cast<const uint2 *>(kp + 8 * (D / 2) + lane * 8);
            wa[0] = x.x, wa[1] = x.y, wb[0] = y.x, wb[1] = y.y;
            sa = kp[Fp4Sub<D>::kKeyScales + lane];
            sb = kp[Fp4Sub<D>::kKeyScales + 8 * (D / 16) + lane];
          }
          const uint32_t ha = e4m3x2_to_half2(sa), hb = e4m3x2_to_half2(sb);
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const bool hi = D == 128 && i >= kWords / 2;
            const uint32_t sca = __byte_perm(ha, 0, hi ? 0x3232 : 0x1010), scb = __byte_perm(hb, 0, hi ? 0x3232 : 0x1010);
            uint32_t fa[4], fb[4];
            e2m1x8_to_half2(wa[i], fa);
            e2m1x8_to_half2(wb[i], fb);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t a[4] = {hmul2(fa[2 * t], sca), hmul2(fb[2 * t], scb), hmul2(fa[2 * t + 1], sca),
                                     hmul2(fb[2 * t + 1], scb)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 q = NT == 1 ? qreg[NT == 1 ? 2 * i + t : 0] : qfrag[((2 * i + t) * NT + nt) * 32 + lane];
                mma16816<true>(s[u][nt], a, q.x, q.y);
              }
            }
          }
        } else {
          const int tk = (lane & 7) + (lane & 8);
          const uint32_t ka = smem_u32(kp) + tk * (2 * D);
#pragma unroll
          for (int i = 0; i < C::kSteps; ++i) {
            uint32_t a[4];
            ldsm4(a, ka + (((2 * i + (lane >> 4)) ^ (tk & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q = NT == 1 ? qreg[NT == 1 ? i : 0] : qfrag[(i * NT + nt) * 32 + lane];
              mma16816<false>(s[u][nt], a, q.x, q.y);
            }
          }
        }
      }

      // ----- softmax -----
      bool grow = false;
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[u][nt][e] * cscale[nt][e & 1];
            if (edge) {
              const int p = pos[u] + r8 + (e >> 1) * 8, n = clen[nt][e & 1];
              const bool see = p < n && (P.window == 0 || p >= n - P.window || p < P.sinks);
              x = see ? x : -INFINITY;
            }
            s[u][nt][e] = x;
            grow |= x > m[nt][e & 1] + kBaLazy;
          }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = m[nt][e];
#pragma unroll
            for (int u = 0; u < C::kSubs; ++u) x = fmaxf(x, fmaxf(s[u][nt][e], s[u][nt][e + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
            const float f = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - x);
            m[nt][e] = x;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < C::kSteps; ++j) o[j][nt][e] *= f, o[j][nt][e + 2] *= f;
          }
      }
      uint32_t pb[C::kSubs][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kLift, m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kLift;
#pragma unroll
        for (int u = 0; u < C::kSubs; ++u) {
          const float p0 = ex2(s[u][nt][0] - m0), p1 = ex2(s[u][nt][1] - m1);
          const float p2 = ex2(s[u][nt][2] - m0), p3 = ex2(s[u][nt][3] - m1);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          pb[u][nt][0] = movm_t(pack2<F16>(p0, p1));
          pb[u][nt][1] = movm_t(pack2<F16>(p2, p3));
        }
      }

      // ----- O^T += V^T P^T -----
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u) {
        const uint8_t *vp = sp + u * C::kSubBytes;
        if constexpr (C::kFp4) {
          constexpr int kWords = D / 64;  // 32-bit words of codes a lane reads per token
          uint32_t w[2][2][kWords], sc[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint8_t *src = vp + Fp4Sub<D>::kValues + p * (4 * D);
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4 *>(src + lane * 16);
              w[p][0][0] = x.x, w[p][0][1] = x.y, w[p][1][0] = x.z, w[p][1][1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2 *>(src + lane * 8);
              w[p][0][0] = x.x, w[p][1][0] = x.y;
            }
            const int grp = D == 128 ? r8 : r8 >> 1;
            sc[p] = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(vp + Fp4Sub<D>::kValueScales + p * (D / 2) + grp * 8 + 2 * c4));
            if (edge) {  // a token no query sees: its scale may be NaN
              const int t0 = pos[u] + 8 * p + 2 * c4;
              const bool on0 = t0 < cur.v.len && (t0 >= cur.v.wlo || t0 < P.sinks);
              const bool on1 = t0 + 1 < cur.v.len && (t0 + 1 >= cur.v.wlo || t0 + 1 < P.sinks);
              sc[p] &= (on0 ? 0xffffu : 0u) | (on1 ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            uint32_t f[2][2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int t = 0; t < 2; ++t) e2m1x8_to_half2(w[p][t][i], f[p][t]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              // dims (2j, 2j + 1) of tokens t, t + 1 -> (t, t + 1) of each dim
              const uint32_t a[4] = {hmul2(__byte_perm(f[0][0][b], f[0][1][b], 0x5410), sc[0]),
                                     hmul2(__byte_perm(f[0][0][b], f[0][1][b], 0x7632), sc[0]),
                                     hmul2(__byte_perm(f[1][0][b], f[1][1][b], 0x5410), sc[1]),
                                     hmul2(__byte_perm(f[1][0][b], f[1][1][b], 0x7632), sc[1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[4 * i + b][nt], a, pb[u][nt][0], pb[u][nt][1]);
            }
          }
        } else {
          const int tk = (lane & 7) + ((lane >> 4) << 3);
          const uint32_t va = smem_u32(vp) + kSubTokens * D * 2 + tk * (2 * D);
#pragma unroll
          for (int j = 0; j < C::kSteps; ++j) {
            uint32_t a[4];
            ldsm4_t(a, va + (((2 * j + ((lane >> 3) & 1)) ^ (tk & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[j][nt], a, pb[u][nt][0], pb[u][nt][1]);
          }
        }
      }
      st = st == STAGES - 1 ? 0 : st + 1;
    }

    // ----- merge the warps; the result, or this piece's part of it -----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
        if (r8 == 0) ml[warp * C::kRows + nt * 8 + 2 * c4 + e] = make_float2(m[nt][e], l[nt][e]);
      }
    __syncthreads();
    const bool split = !P.whole && (cur.start < g0 || cur.end > g1);
    const int slot = 2 * blockIdx.x + (cur.start < g0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * C::kRows + nt * 8 + 2 * c4 + e].x);
        const float f = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - top);
        float *dst = merge + (warp * 8 + 2 * c4 + e) * C::kMergeRow;
#pragma unroll
        for (int j = 0; j < C::kSteps; ++j) {
          // 4-bit rows: dim r8 * D/8 + 2j + i is kept at (2j + i) * 8 + r8, bf16 rows: dim
          // 16j + 8i + r8 at its own place (the same expression)
          dst[16 * j + r8] = o[j][nt][e] * f;
          dst[16 * j + 8 + r8] = o[j][nt][e + 2] * f;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 8 * D / 2; i += C::kThreads) {
        const int rr = i / (D / 2), d = 2 * (i % (D / 2)), row = nt * 8 + rr;
        int a0 = d, a1 = d + 1;
        if constexpr (C::kFp4) {
          a0 = (d % (D / 8)) * 8 + d / (D / 8);
          a1 = a0 + 8;
        }
        float top = -INFINITY, sum = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * C::kRows + row].x);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float2 v = ml[w * C::kRows + row];
          sum += v.x == -INFINITY ? 0.f : v.y * ex2(v.x - top);
          x0 += merge[(w * 8 + rr) * C::kMergeRow + a0];
          x1 += merge[(w * 8 + rr) * C::kMergeRow + a1];
        }
        if (split) {
          *reinterpret_cast<float2 *>(P.part_o + (static_cast<int64_t>(slot) * C::kRows + row) * D + d) = make_float2(x0, x1);
          if (d == 0) reinterpret_cast<float2 *>(P.part_ml)[slot * C::kRows + row] = make_float2(top, sum);
        } else if (row < rows) {
          const int rq = row0 + row, j = rq / P.group;
          const int64_t oh = (static_cast<int64_t>(cur.b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group;
          const float inv = sum > 0.f ? 1.f / sum : sum;  // (a NaN sum stays one)
          *reinterpret_cast<uint32_t *>(P.out + oh * D + d) = pack2<false>(x0 * inv, x1 * inv);
          if (d == 0 && P.lse) P.lse[oh] = ba_lse(top, sum, kLift);
        }
      }
      __syncthreads();
    }
    if (pend >= g1) break;
    seek<C::kSubs>(P, cur, pend);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Merge of the pieces of each (b, hm) that was cut: block (i, y) takes the one that begins
// in CTA i's range and goes on past it, rows y of it.  The pieces' weights 2^(m_s - max m)
// are formed once per row; D / 2 threads of each row then add the pieces in order.
constexpr int kBaCombThreads = 128;

template <int D>
__global__ void __launch_bounds__(kBaCombThreads) block_attn_combine_kernel(const BlockAttnParams P, int rows_pad,
                                                                                 float lift) {
  constexpr int kSlots = 2 * kBaMaxGrid;
  __shared__ float wgt[kSlots];
  __shared__ float red[2][kBaCombThreads / 32];
  const int cta = blockIdx.x, row = blockIdx.y, t = threadIdx.x;
  pdl_wait();
  // requests with nothing to see are not on the line (without a split, their own CTA, whose
  // stream is empty, writes the same)
  const int heads = P.n_kv * P.mgroups;
  for (int64_t i = cta; i < static_cast<int64_t>(P.B) * heads; i += gridDim.x) {
    const int b = static_cast<int>(i / heads);
    if (req_view(P, __ldg(P.ctx_len + b)).nsub > 0) continue;
    const int hm = static_cast<int>(i - static_cast<int64_t>(b) * heads), h = hm / P.mgroups;
    const int rq = (hm - h * P.mgroups) * kBaMaxRows + row;
    if (rq >= P.n_q * P.group) continue;
    const int j = rq / P.group;
    const int64_t oh = (static_cast<int64_t>(b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group;
    for (int d = t; d < D; d += kBaCombThreads) P.out[oh * D + d] = 0;
    if (t == 0 && P.lse) P.lse[oh] = -INFINITY;
  }
  const int4 tail = P.tail[cta];
  const int pieces = tail.z;
  if (pieces == 0) return;
  const int h = tail.y / P.mgroups;
  const int rq = (tail.y - h * P.mgroups) * kBaMaxRows + row;
  if (rq >= P.n_q * P.group) return;
  // piece 0 is CTA i's second slot, piece s > 0 the first slot of CTA i + s
  auto slot_of = [&](int s) { return s == 0 ? 2 * cta + 1 : 2 * (cta + s); };
  float top = -INFINITY;
  for (int s = t; s < pieces; s += kBaCombThreads) top = fmaxf(top, P.part_ml[2 * (static_cast<int64_t>(slot_of(s)) * rows_pad + row)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if ((t & 31) == 0) red[0][t >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBaCombThreads / 32; ++w) top = fmaxf(top, red[0][w]);
  float sum = 0.f;
  for (int s = t; s < pieces; s += kBaCombThreads) {
    const float2 v = *reinterpret_cast<const float2 *>(P.part_ml + 2 * (static_cast<int64_t>(slot_of(s)) * rows_pad + row));
    const float w = v.x == -INFINITY ? 0.f : ex2(v.x - top);
    wgt[s] = w;
    sum = fmaf(w, v.y, sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if ((t & 31) == 0) red[1][t >> 5] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kBaCombThreads / 32; ++w) sum += red[1][w];
  const int j = rq / P.group;
  const int64_t oh = (static_cast<int64_t>(tail.x) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group;
  const float inv = sum > 0.f ? 1.f / sum : sum;
  for (int d = t; d < D; d += kBaCombThreads) {
    float x = 0.f;
#pragma unroll 8
    for (int s = 0; s < pieces; ++s) x = fmaf(wgt[s], P.part_o[(static_cast<int64_t>(slot_of(s)) * rows_pad + row) * D + d], x);
    const __nv_bfloat16 y = __float2bfloat16_rn(x * inv);
    P.out[oh * D + d] = *reinterpret_cast<const uint16_t *>(&y);
  }
  if (t == 0 && P.lse) P.lse[oh] = ba_lse(top, sum, lift);
}

}  // namespace echo

namespace echo_host {

static int ba_row_pad(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

size_t block_attention_workspace_bytes(int32_t rows, int32_t head_dim) {
  const size_t pad = ba_row_pad(rows < echo::kBaMaxRows ? rows : echo::kBaMaxRows);
  return echo::kBaMaxGrid * sizeof(int4) + 2 * echo::kBaMaxGrid * pad * (2 + static_cast<size_t>(head_dim)) * sizeof(float);
}

template <int FMT, int D, int NT, int WARPS, int STAGES>
static int launch_ba(const echo::BlockAttnParams &P, int grid, cudaStream_t stream) {
  using C = echo::BaCfg<FMT, D, NT, WARPS, STAGES>;
  static_assert(C::kSmem <= 232448, "block attention: shared memory of one CTA");
  auto kernel = echo::block_attn_kernel<FMT, D, NT, WARPS, STAGES>;
  static std::atomic<bool> attr[kMaxDevices];
  if (int rr = smem_limit_once(attr, kernel, C::kSmem, "block attention smem attribute")) return rr;
  kernel<<<grid, C::kThreads, C::kSmem, stream>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "block attention launch");
  if (P.whole) return ECHO_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, C::kRows);
  cfg.blockDim = dim3(echo::kBaCombThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, echo::block_attn_combine_kernel<D>, P, static_cast<int>(C::kRows), C::kFp4 ? echo::kBaLift : 0.f);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block attention merge launch");
}

int launch_block_attention(const echo_block_attention_args *a, cudaStream_t stream) {
  echo::BlockAttnParams P{};
  P.q = a->q, P.rows = a->rows;
  P.row_bytes = 2 * echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.n_rows = a->n_rows;
  P.bsub = a->block_tokens / echo::kSubTokens;
  P.table = a->table, P.sel = a->sel;
  P.table_heads = a->table_heads, P.max_blocks = a->max_blocks;
  P.ctx_len = a->ctx_len;
  P.B = a->B, P.n_q = a->n_q, P.n_heads = a->n_heads, P.n_kv = a->n_kv_heads;
  P.group = a->n_heads / a->n_kv_heads;
  const int rows = P.n_q * P.group;
  P.mgroups = (rows + echo::kBaMaxRows - 1) / echo::kBaMaxRows;
  P.sinks = a->sinks, P.window = a->window;
  P.scale_log2 = a->scale * 1.4426950408889634f;
  P.out = a->out, P.lse = a->lse;
  P.status = a->dev_status;
  const int pad = ba_row_pad(rows < echo::kBaMaxRows ? rows : echo::kBaMaxRows);
  P.tail = reinterpret_cast<int4 *>(a->workspace);
  P.part_ml = reinterpret_cast<float *>(P.tail + echo::kBaMaxGrid);
  P.part_o = P.part_ml + 2 * static_cast<size_t>(echo::kBaMaxGrid) * pad * 2;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t pairs = static_cast<int64_t>(P.B) * P.n_kv * P.mgroups;
  // tokens a context can show at most
  int64_t most = static_cast<int64_t>(P.max_blocks) * a->block_tokens;
  if (!P.sel && P.window && most > P.sinks + static_cast<int64_t>(P.window) + P.n_q + 31) most = P.sinks + static_cast<int64_t>(P.window) + P.n_q + 31;
  P.whole = most <= 256;
  int grid = P.whole ? static_cast<int>(pairs) : sms;
  if (grid > echo::kBaMaxGrid && !P.whole) grid = echo::kBaMaxGrid;
#define BA_GO(FMT, D, W, S, S4)                              \
  (pad == 8    ? launch_ba<FMT, D, 1, W, S>(P, grid, stream) \
   : pad == 16 ? launch_ba<FMT, D, 2, W, S>(P, grid, stream) \
               : launch_ba<FMT, D, 4, W, S4>(P, grid, stream))
  if (a->format == ECHO_BLOCK_FP4) return a->head_dim == 128 ? BA_GO(ECHO_BLOCK_FP4, 128, 8, 4, 4) : BA_GO(ECHO_BLOCK_FP4, 64, 8, 4, 4);
  return a->head_dim == 128 ? BA_GO(ECHO_BLOCK_BF16, 128, 6, 4, 3) : BA_GO(ECHO_BLOCK_BF16, 64, 6, 4, 3);
#undef BA_GO
}

}  // namespace echo_host
