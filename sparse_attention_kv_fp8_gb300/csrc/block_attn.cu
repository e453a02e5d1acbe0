// block_attn.cu -- decode attention over block rows (grouped-query heads; bf16 or 4-bit
// rows; sliding window with sinks; block tables or recalled selections).
//
// For the M = n_q * n_heads / n_kv_heads query rows that share KV head h of request b:
//   x_p = scale * q . k_p,   out = sum_p 2^(x_p log2 e - m) v_p / l,   one pass over p
// with the running maximum m and sum l of each row.  K and V are read once for up to 32 rows
// (row groups of 32 beyond that read them once each), 4 D bytes a token and KV head in bf16,
// 18 D / 16 in 4 bits, against 4 M D flops.  In bf16 that is the bound.  4-bit rows are bound
// by instructions, and from 16 rows on by the registers that the output takes: a tcgen05.mma
// with tokens, then dims, as its 128 rows and the query rows as its columns would leave both
// to tensor memory; that kernel is not written.
//
// sm_103a design.
//   Transposed products: S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16, tokens (then
//     dimensions) as the 16 rows and the query rows as the 8 columns, so a group of 8 query
//     heads fills the instruction exactly and each cache element is converted once for all
//     query rows.  P^T needs the transpose of S^T's fragment: one movmatrix per 8 tokens.
//   A warp is a worker of its own: it takes every kWarps-th chunk (16 or 32 tokens) of the
//     CTA's range, keeps its own m, l and O, and fills its own ring of shared-memory stages
//     with cp.async, ahead of the chunk it computes and across the borders of requests; no
//     barrier runs inside the stream.  Where its next 32 sub-blocks lie is looked up by its
//     32 lanes at once (table, selection, window, request borders) into a small list.  The
//     warps of a CTA merge at the end of each (b, h).
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
//     (b, h) pairs fill the GPU, a CTA, or a cluster of up to 8 that merges over distributed
//     shared memory, takes a whole (b, h) and the second kernel is left out; with more pairs
//     than SMs two smaller CTAs share an SM, one streaming while the other starts or merges.
//
// Measured on a GB300 (8 KV heads of 128, 8 query heads each; HBM's measured copy rate is
// 6.67 TB/s): 16 requests of 16384 to 32768 tokens 236 us in bf16 (6.8 TB/s), 93 us in 4 bits
// (4.9 TB/s); of up to 131072 tokens 314 us in 4 bits (6.0 TB/s), 423 us with two query
// tokens; a window of 4096 and 4 sinks of 64 requests 162 us in bf16 (6.6 TB/s); one request
// of 1000 tokens 6 us.  bf16 is bound by HBM.  4-bit rows are bound by instructions, above
// all the conversions: some 600 per warp and 32 tokens, the integer pipe 64% and the issue
// slots 66% busy (without the scales' multiplies 277 us instead of 318); with two query
// tokens the registers leave 12 warps instead of 16 and the matrix pipe is 42% busy.  Short
// calls are bound by the launch, the look-ups and the merges (2.4 us before the first bytes,
// 0.8 us to merge the warps, 1.3 us a cluster, 4 us a second kernel).
#include <algorithm>
#include <cmath>

#include "block_rows.cuh"
#include "cluster_select.cuh"

namespace echo {

constexpr int kBaMaxGrid = 304;   // CTAs of a cut call: two on each of 152 SMs (workspace pieces: two per CTA)
constexpr float kBaLazy = 8.f;    // log2 of how far a score may exceed the running maximum
// fp16 softmax weights are kept 2^7 up: at most 2^(7 + 8), and the subnormals (a grid of
// 2^-24) begin 2^-21 below the running maximum instead of 2^-14
constexpr float kBaLift = 7.f;
constexpr float kBaNone = -3.4028234664e38f;  // (no score seen: finite, so that differences with it are too)
constexpr int kBaNowhere = 0x7fffff00;  // position of a sub-block that is not there
constexpr int kBaMaxCluster = 8;  // CTAs of a (b, h) that merge over distributed shared memory
constexpr int kBaList = 64;        // entries of a warp's list of sub-blocks (two batches of 32)
constexpr int kBaMaxRows = 32;    // query rows of one CTA's (b, h) (4 columns of 8)

struct BlockAttnParams {
  const uint16_t *q, *rows;
  int64_t row_bytes;
  int32_t n_rows, bsub;              // bsub: 16-token sub-blocks of a row
  const int32_t *table, *sel;
  int32_t table_heads, max_blocks;
  const int32_t *ctx_len;
  int32_t B, n_q, n_heads, n_kv, group;  // group: query heads per KV head
  int32_t mgroups;                   // row groups of a KV head (the kernel's kRows each)
  int32_t sinks, window;
  float scale_log2;                  // |scale| log2 e, over the keys' power of two
  float v_scale;                     // one over the values' power of two
  uint32_t q_sign;                   // 0x80008000 for a negative scale
  uint16_t *out;
  float *lse;
  int32_t cluster;                   // CTAs of a (b, h, row group), a cluster; 0: the line is cut
  float *part_o;                     // [2 * grid][rows][D]
  float *part_ml;                    // [2 * grid][rows][2]
  int4 *tail;                        // (b, h * mgroups + mg, pieces, first CTA) of each
  int32_t by_pair;                   // (b, h, row group), or of the last one of each CTA
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
  static constexpr int kSubs = kFp4 ? (D == 128 && NT == 4 ? 1 : D == 128 || NT >= 2 ? 2 : 4) : (D == 128 ? 1 : 2);  // of a chunk
  static constexpr int kTokens = kSubs * kSubTokens;
  static constexpr int kStageBytes = kSubs * kSubBytes;
  static constexpr int kThreads = WARPS * 32;
  static constexpr int kSteps = D / 16;                      // k-steps of S^T, dim tiles of O^T
  static constexpr int kRows = 8 * NT;
  static constexpr int kMergeRow = D / 2 + 4;                // floats; + 4: no bank conflicts
  // shared memory: stages | merge buffers | lists | q fragments | per-row values
  static constexpr int kOffMerge = WARPS * STAGES * kStageBytes;
  // parts of the output (8 rows, half of the dims) that the warps merge at a time: as many as
  // shared memory has room for beside the stages
  static constexpr int kParts = NT <= 2 ? 1 : kFp4 ? NT : 2;
  static constexpr int kPart = WARPS * 8 * kMergeRow;        // floats
  static constexpr int kOffList = kOffMerge + kParts * kPart * 4;
  static constexpr int kOffQ = kOffList + WARPS * kBaList * 16;
  static constexpr int kOffMl = kOffQ + kSteps * NT * 32 * 8;
  static constexpr int kOffQs = kOffMl + WARPS * kRows * 8;
  static constexpr int kOffFin = kOffQs + kRows * 4;
  static_assert(kOffFin % 8 == 0 && kOffList % 16 == 0 && kOffMerge % 16 == 0, "alignment");
  static constexpr int kSmem = kOffFin + kRows * 8;
  static constexpr int kQRows = (kRows + WARPS - 1) / WARPS;  // query rows a warp lays out
};

__device__ __forceinline__ void ba_cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ba_cp16_or_zeros(uint32_t dst, const void *src, bool on) {
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
// a shared-memory address of this CTA, in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// log of a row's sum of weights 2^(x - top)
__device__ __forceinline__ float ba_lse(float top, float sum) {
  return top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A place on the line of chunks, counted from the CTA's first chunk: the chunks start .. end
// belong to row group hm (KV head * row groups + row group) of request b.
struct LinePos {
  int b, hm;
  int start, end;
  ReqView v;
};

template <int kSubs>
__device__ __forceinline__ int chunks_of(const ReqView &v) {
  return (v.nsub + kSubs - 1) / kSubs;
}

// moves forward to the (b, hm) that holds chunk g (a chunk of the line; past the last request
// there is nothing, and the walk ends)
template <int kSubs>
__device__ __forceinline__ void seek(const BlockAttnParams &P, LinePos &L, int g) {
  while (g >= L.end) {
    const int heads = P.n_kv * P.mgroups;
    const int n = chunks_of<kSubs>(L.v);
    if (n > 0 && L.hm + 1 < heads) {
      const int by = min(heads - 1 - L.hm, (g - L.end) / n + 1);  // row groups to pass over
      L.hm += by;
      L.start = L.end + (by - 1) * n;
    } else if (L.b + 1 < P.B) {
      ++L.b;
      L.hm = 0;
      L.start = L.end;
      L.v = req_view(P, P.ctx_len[L.b]);
    } else {
      L.start = L.end;
      L.end = 0x7fffffff;
      L.v.nsub = 0;
      return;
    }
    L.end = L.start + chunks_of<kSubs>(L.v);
  }
}

// One sub-block of a warp's list: where it lies, its first token's position, which of its
// tokens some query sees (bits 0-15), and whether some query does not see all of them (edge).
struct __align__(16) SubEntry {
  const uint8_t *src;
  int pos;
  uint32_t flags;
};
constexpr uint32_t kBaEdge = 1u << 31;

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1; }

template <int FMT, int D>
__device__ __forceinline__ SubEntry sub_entry(const BlockAttnParams &P, const LinePos &L, int s) {
  SubEntry x{reinterpret_cast<const uint8_t *>(P.rows), kBaNowhere, kBaEdge};
  if (s >= L.v.nsub) return x;
  if (s >= L.v.n_first) s += L.v.skip;
  const int h = L.hm / P.mgroups, e = s / P.bsub, in = s - e * P.bsub;
  const int64_t at = (static_cast<int64_t>(L.b) * P.table_heads + (P.table_heads > 1 ? h : 0)) * P.max_blocks + e;
  const int32_t id = P.table[at];
  const int32_t lb = P.sel ? P.sel[at] : e;
  // (a selected block past the 31-bit positions cannot be below any length)
  if (id < 0 || lb < 0 || static_cast<int64_t>(lb) * P.bsub + in >= kBaNowhere / kSubTokens) return x;
  const int64_t row = P.table_heads > 1 ? id : static_cast<int64_t>(id) * P.n_kv + h;
  if (row >= P.n_rows) {
    set_status(P.status, ECHO_DEV_BAD_INDEX);
    return x;
  }
  const int pos = (lb * P.bsub + in) * kSubTokens, last = pos + kSubTokens - 1;
  x.src += row * P.row_bytes + static_cast<int64_t>(in) * (FMT == ECHO_BLOCK_FP4 ? Fp4Sub<D>::kBytes : kSubTokens * D * 2);
  x.pos = pos;
  // seen by some query: p < len and (p >= wlo or p < sinks)
  const uint32_t seen = low_bits(L.v.len - pos) & ((0xffffu & ~low_bits(L.v.wlo - pos)) | low_bits(P.sinks - pos));
  const int len_first = L.v.len - (P.n_q - 1), w_last = P.window ? L.v.len - P.window : 0;
  const bool all = last < len_first && (pos >= w_last || last < P.sinks);
  x.flags = seen | (all ? 0u : kBaEdge);
  return x;
}

template <int FMT, int D, int NT, int WARPS, int STAGES, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) block_attn_kernel(const BlockAttnParams P) {
  using C = BaCfg<FMT, D, NT, WARPS, STAGES>;
  constexpr bool F16 = C::kFp4;
  constexpr float kLift = F16 ? kBaLift : 0.f;
  extern __shared__ __align__(128) uint8_t ba_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, c4 = lane & 3;  // fragment row and column pair
  uint8_t *stage_base = ba_smem + warp * STAGES * C::kStageBytes;
  const uint32_t stage_u32 = smem_u32(stage_base) + lane * 16;
  float *merge = reinterpret_cast<float *>(ba_smem + C::kOffMerge);
  uint2 *qfrag = reinterpret_cast<uint2 *>(ba_smem + C::kOffQ);
  float2 *ml = reinterpret_cast<float2 *>(ba_smem + C::kOffMl);       // [WARPS][kRows]
  float *qscale = reinterpret_cast<float *>(ba_smem + C::kOffQs);     // [kRows]
  SubEntry *list = reinterpret_cast<SubEntry *>(ba_smem + C::kOffList) + warp * kBaList;
  float2 *fin = reinterpret_cast<float2 *>(ba_smem + C::kOffFin);     // [kRows]
  const int heads = P.n_kv * P.mgroups;
  pdl_launch_dependents();  // (what follows waits for this grid's end all the same)
  pdl_wait();

  // ===== this CTA's range of the line: chunks 0 .. n_chunks from its first =====
  LinePos cur;
  int n_chunks;
  // of a cut line: how many pieces a (b, hm) that begins here has (the next CTAs' ranges are as
  // long as this one's), or that it needs no merge here
  auto note_tail = [&](const LinePos &L) {
    if (threadIdx.x != 0 || !(P.by_pair ? L.start >= 0 : L.end >= n_chunks)) return;
    const int pieces = L.start >= 0 && L.end > n_chunks ? 1 + (L.end - 1) / n_chunks : 0;
    P.tail[P.by_pair ? L.b * heads + L.hm : blockIdx.x] = make_int4(L.b, L.hm, pieces, blockIdx.x);
  };
  if (P.cluster) {
    const int pair = blockIdx.x / P.cluster, rank = blockIdx.x - pair * P.cluster;
    cur.b = pair / heads;
    cur.hm = pair - cur.b * heads;
    const int ctx = P.ctx_len[cur.b];
    cur.v = req_view(P, ctx);
    const int n = chunks_of<C::kSubs>(cur.v);
    const int first = static_cast<int>(static_cast<int64_t>(n) * rank / P.cluster);
    cur.start = -first;
    cur.end = n - first;
    n_chunks = static_cast<int>(static_cast<int64_t>(n) * (rank + 1) / P.cluster) - first;
    if (threadIdx.x == 0 && rank == 0 && cur.hm == 0) check_context(P, ctx);
  } else {
    // lengths of all requests' parts of the line, by every warp for itself (no barrier): a
    // run of requests per lane, summed
    const int per_l = (P.B + 31) / 32;
    const int b0 = min(lane * per_l, P.B), b1 = min(b0 + per_l, P.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int ctx = P.ctx_len[b];
      mine += chunks_of<C::kSubs>(req_view(P, ctx));
      if (blockIdx.x == 0 && warp == 0) check_context(P, ctx);
    }
    mine *= heads;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    const int64_t total = __shfl_sync(~0u, upto, 31);
    int64_t per = total < (1ll << 31) ? (static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x
                                      : (total + gridDim.x - 1) / gridDim.x;
    per = per < WARPS ? WARPS : per;
    // requests with nothing to see are not on the line: their outputs are written here
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      if (req_view(P, P.ctx_len[b]).nsub > 0) continue;
      if (P.by_pair)
        for (int i = threadIdx.x; i < heads; i += C::kThreads) P.tail[b * heads + i] = make_int4(0, 0, 0, 0);
      const int64_t o0 = static_cast<int64_t>(b) * P.n_q * P.n_heads;
      for (int i = threadIdx.x; i < P.n_q * P.n_heads * (D / 8); i += C::kThreads)
        reinterpret_cast<uint4 *>(P.out + o0 * D)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (P.lse)
        for (int i = threadIdx.x; i < P.n_q * P.n_heads; i += C::kThreads) P.lse[o0 + i] = -INFINITY;
    }
    const int64_t g0 = per * blockIdx.x;
    if (g0 >= total) {
      if (threadIdx.x == 0 && !P.by_pair) P.tail[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    n_chunks = static_cast<int>(min(total - g0, per));
    int own_b = 0, own_hm = 0, own_start = 0;
    const bool own = g0 >= upto - mine && g0 < upto;  // one lane's run holds g0
    if (own) {
      int64_t at = upto - mine;
      int n = 1;
      for (own_b = b0; own_b < b1; ++own_b) {
        n = chunks_of<C::kSubs>(req_view(P, P.ctx_len[own_b]));
        if (g0 < at + static_cast<int64_t>(n) * heads) break;
        at += static_cast<int64_t>(n) * heads;
      }
      own_hm = static_cast<int>((g0 - at) / n);
      own_start = static_cast<int>(at + static_cast<int64_t>(own_hm) * n - g0);
    }
    const int src = __ffs(__ballot_sync(~0u, own)) - 1;
    cur.b = __shfl_sync(~0u, own_b, src);
    cur.hm = __shfl_sync(~0u, own_hm, src);
    cur.start = __shfl_sync(~0u, own_start, src);
    cur.v = req_view(P, P.ctx_len[cur.b]);
    cur.end = cur.start + chunks_of<C::kSubs>(cur.v);
    note_tail(cur);
  }

  // ===== the queries of a (b, hm), a row per warp: loaded early, laid out as B fragments later
  uint2 qrow[C::kQRows];
  const bool q_lane = lane < D / 4;  // lane (s, c) = (k-step, column pair) of the fragments
  auto row_index = [&](const LinePos &L, int rr) -> int64_t {  // (b, query token, head) of a row
    const int h = L.hm / P.mgroups, rq = (L.hm - h * P.mgroups) * C::kRows + rr, j = rq / P.group;
    return rq < P.n_q * P.group ? (static_cast<int64_t>(L.b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group : -1;
  };
  auto load_q = [&](const LinePos &L) {
#pragma unroll
    for (int i = 0; i < C::kQRows; ++i) {
      const int rr = warp + i * WARPS;
      qrow[i] = make_uint2(0u, 0u);
      const int64_t at = rr < C::kRows ? row_index(L, rr) : -1;
      if (at < 0 || !q_lane) continue;
      const uint16_t *src = P.q + at * D;
      if constexpr (F16) {
        qrow[i] = *reinterpret_cast<const uint2 *>(src + (D / 4) * c4 + 8 * (r8 >> 1) + 4 * (r8 & 1));
      } else {
        qrow[i].x = *reinterpret_cast<const uint32_t *>(src + 16 * r8 + 2 * c4);
        qrow[i].y = *reinterpret_cast<const uint32_t *>(src + 16 * r8 + 2 * c4 + 8);
      }
    }
  };
  auto store_q = [&]() {
#pragma unroll
    for (int i = 0; i < C::kQRows; ++i) {
      const int rr = warp + i * WARPS;
      if (rr >= C::kRows) break;
      uint2 f = qrow[i];
      if constexpr (F16) {
        // scaled by the power of two that brings the row's largest entry to [1, 2)
        const float x0 = __uint_as_float(f.x << 16), x1 = __uint_as_float(f.x & 0xffff0000u);
        const float x2 = __uint_as_float(f.y << 16), x3 = __uint_as_float(f.y & 0xffff0000u);
        float m = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        e = max(min(e, 126), -126);  // (zero rows, subnormal and infinite maxima)
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        f = make_uint2(pack2<true>(x0 * inv, x1 * inv), pack2<true>(x2 * inv, x3 * inv));
        if (lane == 0) qscale[rr] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      }
      f.x ^= P.q_sign, f.y ^= P.q_sign;
      if (q_lane) qfrag[(r8 * NT + (rr >> 3)) * 32 + (rr & 7) * 4 + c4] = f;
    }
  };
  load_q(cur);

  // ===== the loader =====
  // Entry i of the warp's list is sub-block i % kSubs of its chunk i / kSubs (chunk warp +
  // WARPS * (i / kSubs) of the range).  Entries are made 32 at a time; the loader is at
  // most (STAGES - 1) * kSubs < 32 entries ahead of the reader.
  static_assert((STAGES - 1) * C::kSubs <= kBaList - 32 && 32 % C::kSubs == 0, "list length");
  LinePos mine = cur;     // of the entry this lane makes
  int at = 0;             // entries loaded
  int to_load = (n_chunks - warp + WARPS - 1) / WARPS;  // chunks of this warp still to load
  auto issue = [&](int st) {
    if (to_load > 0) {    // (warp-uniform)
      --to_load;
      if ((at & 31) == 0) {
        const int i = at + lane, g = warp + WARPS * (i / C::kSubs);
        SubEntry x{reinterpret_cast<const uint8_t *>(P.rows), kBaNowhere, kBaEdge};
        if (g < n_chunks) {
          seek<C::kSubs>(P, mine, g);
          x = sub_entry<FMT, D>(P, mine, (g - mine.start) * C::kSubs + i % C::kSubs);
        }
        list[i % kBaList] = x;
        __syncwarp();
      }
      uint32_t dst = stage_u32 + st * C::kStageBytes;
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u, dst += C::kSubBytes) {
        const SubEntry x = list[at % kBaList + u];  // (kSubs divides kBaList)
        const uint8_t *src = x.src + lane * 16;
        if constexpr (C::kFp4) {
          // (what a sub-block that no query sees leaves here is never used: its scores are
          // masked and its value scales replaced by zeros)
          constexpr int kPieces = C::kSubBytes / 16;
          if (x.flags & 0xffffu) {
#pragma unroll
            for (int i = 0; i < (kPieces + 31) / 32; ++i)
              if ((i + 1) * 32 <= kPieces || lane < kPieces - i * 32) ba_cp16(dst + i * 512, src + i * 512);
          }
        } else {
          // rows of 2 D bytes, 16-byte pieces XORed with the token so that ldmatrix reads
          // 8 tokens from 8 different bank groups; a token no query sees is read as zeros
          // (its bytes may be anything)
          const int64_t vofs = static_cast<int64_t>(P.bsub) * kSubTokens * D * 2;
          constexpr int kPer = 256 / D;  // tokens of 32 pieces
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int tk = i * kPer + lane / (D / 8), pc = lane % (D / 8);
            const uint32_t o = tk * (2 * D) + ((pc ^ (tk & 7)) << 4) - lane * 16;
            const bool on = (x.flags >> tk) & 1;
            ba_cp16_or_zeros(dst + o, src + i * 512, on);
            ba_cp16_or_zeros(dst + kSubTokens * D * 2 + o, src + vofs + i * 512, on);
          }
        }
      }
      at += C::kSubs;
    }
    ba_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);
  store_q();
  __syncthreads();

  // the context of a row's query, and whether a query with context n sees position p
  auto len_at = [&](int rq) { return cur.v.len - (P.n_q - 1 - min(rq / P.group, P.n_q - 1)); };
  auto sees = [&](int n, int p) { return p < n && (P.window == 0 || p >= n - P.window || p < P.sinks); };

  int st = 0, g = warp, rd = 0;  // stage, chunk and list entry to compute
  for (;;) {  // the (b, hm) of this range, one after another
    const int pend = min(cur.end, n_chunks);
    const int row0 = (cur.hm % P.mgroups) * C::kRows;
    uint2 qreg[NT == 1 ? C::kSteps : 1];
    if constexpr (NT == 1) {
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) qreg[s] = qfrag[s * 32 + lane];
    }
    float cscale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) cscale[nt][e] = P.scale_log2 * (F16 ? qscale[nt * 8 + 2 * c4 + e] : 1.f);
    // what is taken off a column's scores (its running maximum less the lift), sum, output
    float m[NT][2], l[NT][2], o[C::kSteps][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kBaNone;
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
      uint32_t flags[C::kSubs], edge = 0;
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u) {
        const int2 x = *reinterpret_cast<const int2 *>(&list[rd % kBaList + u].pos);
        pos[u] = x.x;
        flags[u] = static_cast<uint32_t>(x.y);
        edge |= flags[u] & kBaEdge;
      }
      rd += C::kSubs;

      float s[C::kSubs][NT][4];
#pragma unroll
      for (int u = 0; u < C::kSubs; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
      if constexpr (C::kFp4) {
        constexpr int kWords = D / 32;  // 32-bit words of codes a lane reads per token
        uint32_t wa[C::kSubs][kWords], wb[C::kSubs][kWords], ha[C::kSubs], hb[C::kSubs];  // tokens r8, r8 + 8
#pragma unroll
        for (int u = 0; u < C::kSubs; ++u) {
          const uint8_t *kp = sp + u * C::kSubBytes;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kp + lane * 16);
            const uint4 y = *reinterpret_cast<const uint4 *>(kp + 8 * (D / 2) + lane * 16);
            wa[u][0] = x.x, wa[u][1] = x.y, wa[u][2] = x.z, wa[u][3] = x.w;
            wb[u][0] = y.x, wb[u][1] = y.y, wb[u][2] = y.z, wb[u][3] = y.w;
            ha[u] = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(kp + Fp4Sub<D>::kKeyScales + lane * 2));
            hb[u] = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(kp + Fp4Sub<D>::kKeyScales + 8 * (D / 16) + lane * 2));
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(kp + lane * 8);
            const uint2 y = *reinterpret_cast<const uint2 *>(kp + 8 * (D / 2) + lane * 8);
            wa[u][0] = x.x, wa[u][1] = x.y, wb[u][0] = y.x, wb[u][1] = y.y;
            ha[u] = e4m3x2_to_half2(kp[Fp4Sub<D>::kKeyScales + lane]);
            hb[u] = e4m3x2_to_half2(kp[Fp4Sub<D>::kKeyScales + 8 * (D / 16) + lane]);
          }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint2 q[2][NT];  // (read once for the chunk's sub-blocks)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) q[t][nt] = NT == 1 ? qreg[NT == 1 ? 2 * i + t : 0] : qfrag[((2 * i + t) * NT + nt) * 32 + lane];
#pragma unroll
          for (int u = 0; u < C::kSubs; ++u) {
            const bool hi = D == 128 && i >= kWords / 2;
            const uint32_t sa = __byte_perm(ha[u], 0, hi ? 0x3232 : 0x1010), sb = __byte_perm(hb[u], 0, hi ? 0x3232 : 0x1010);
            uint32_t fa[4], fb[4];
            e2m1x8_to_half2(wa[u][i], fa);
            e2m1x8_to_half2(wb[u][i], fb);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t a[4] = {hmul2(fa[2 * t], sa), hmul2(fb[2 * t], sb), hmul2(fa[2 * t + 1], sa),
                                     hmul2(fb[2 * t + 1], sb)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(s[u][nt], a, q[t][nt].x, q[t][nt].y);
            }
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < C::kSubs; ++u) {
          const int tk = (lane & 7) + (lane & 8);
          const uint32_t ka = smem_u32(sp + u * C::kSubBytes) + tk * (2 * D);
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
      if (edge) {
        // Tokens that some of the request's queries see and others do not (n_q > 1): a value that is
        // not finite would reach the others as 0 * infinity.  It becomes NaN here, in the rows that
        // see the token, and the product below finds a zero in its place.
        if (P.n_q > 1) {
#pragma unroll
          for (int u = 0; u < C::kSubs; ++u) {
            const int first = cur.v.len - (P.n_q - 1) - pos[u], from = P.window ? cur.v.len - P.window - pos[u] : 0;
            const uint32_t by_all = low_bits(first) & (~low_bits(from) | low_bits(P.sinks - pos[u]));
            for (uint32_t some = flags[u] & 0xffffu & ~by_all; some; some &= some - 1) {  // (the same in all lanes)
              const int t = __ffs(some) - 1;
              uint8_t *vp = stage_base + st * C::kStageBytes + u * C::kSubBytes;
              // what is not finite among the token's entries of this lane's output: bit 2 j + k of
              // tile j's row r8 + 8 k (in 4 bits a NaN scale, of all of them at once)
              uint32_t bad = 0;
              uint8_t *sc = vp + Fp4Sub<D>::kValueScales + (t >> 3) * (D / 2) + (D == 128 ? r8 : r8 >> 1) * 8 + (t & 7);
              auto entry = [&](int i) {  // row r8 + 8 (i % 2) of tile i / 2
                return reinterpret_cast<uint16_t *>(vp + kSubTokens * D * 2 + t * (2 * D) + ((i ^ (t & 7)) << 4) + 2 * r8);
              };
              if constexpr (C::kFp4) {
                bad = (*sc & 0x7f) == 0x7f ? ~0u : 0u;
              } else {
#pragma unroll
                for (int i = 0; i < 2 * C::kSteps; ++i) bad |= (*entry(i) & 0x7f80) == 0x7f80 ? 1u << i : 0u;
              }
              if (!__any_sync(~0u, bad != 0)) continue;
              __syncwarp();  // (read by every lane that shares it, then overwritten)
              if constexpr (C::kFp4) {
                if (bad) *sc = 0;
              } else {
#pragma unroll
                for (int i = 0; i < 2 * C::kSteps; ++i)
                  if (bad >> i & 1) *entry(i) = 0;
              }
              __syncwarp();
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (sees(len_at(row0 + nt * 8 + 2 * c4 + e), pos[u] + t))
#pragma unroll
                    for (int i = 0; i < 2 * C::kSteps; ++i)
                      if (bad >> i & 1) o[i / 2][nt][e + 2 * (i % 2)] = NAN;
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // tokens below which this column's query sees
            const int n = len_at(row0 + nt * 8 + 2 * c4 + e);
#pragma unroll
            for (int u = 0; u < C::kSubs; ++u)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                s[u][nt][e + 2 * k] = sees(n, pos[u] + r8 + 8 * k) ? s[u][nt][e + 2 * k] : -INFINITY;
          }
      }
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nt][e] = -INFINITY;
#pragma unroll
          for (int u = 0; u < C::kSubs; ++u) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[u][nt][e], s[u][nt][e + 2]));
          grow |= fmaf(top[nt][e], cscale[nt][e], -m[nt][e]) > kBaLazy + kLift;
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(m[nt][e], fmaf(top[nt][e], cscale[nt][e], -kLift));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
            const float f = ex2(m[nt][e] - x);
            m[nt][e] = x;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < C::kSteps; ++j) o[j][nt][e] *= f, o[j][nt][e + 2] *= f;
          }
      }
      // bf16 weights go in as two terms (a bf16 and the bf16 of what it leaves out): the cache's
      // own type then costs no precision, and the tensor cores have the time
      uint32_t pb[C::kSubs][NT][2], pr[C::kSubs][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int u = 0; u < C::kSubs; ++u) {
          float p0 = ex2(fmaf(s[u][nt][0], cscale[nt][0], -m[nt][0])), p1 = ex2(fmaf(s[u][nt][1], cscale[nt][1], -m[nt][1]));
          float p2 = ex2(fmaf(s[u][nt][2], cscale[nt][0], -m[nt][0])), p3 = ex2(fmaf(s[u][nt][3], cscale[nt][1], -m[nt][1]));
          if (edge) {  // (a zero scale leaves nothing of a masked score's infinity)
            p0 = s[u][nt][0] == -INFINITY ? 0.f : p0, p1 = s[u][nt][1] == -INFINITY ? 0.f : p1;
            p2 = s[u][nt][2] == -INFINITY ? 0.f : p2, p3 = s[u][nt][3] == -INFINITY ? 0.f : p3;
          }
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          // (4-bit rows: one fp16 term.  Its 2^-11 of a weight takes the outputs' distance to 64
          // bits from 1.661e-3, all of it their rounding to bf16, to 1.670e-3; a second term would
          // give that back for 8 registers and twice the value product: 16 x 32768 tokens 93 -> 100
          // us, 8 x 131072 with 16 rows 212 -> 257 us)
          const uint32_t a = pack2<F16>(p0, p1), b = pack2<F16>(p2, p3);
          pb[u][nt][0] = movm_t(a);
          pb[u][nt][1] = movm_t(b);
          if constexpr (!F16) {
            pr[u][nt][0] = movm_t(pack2<F16>(p0 - __uint_as_float(a << 16), p1 - __uint_as_float(a & 0xffff0000u)));
            pr[u][nt][1] = movm_t(pack2<F16>(p2 - __uint_as_float(b << 16), p3 - __uint_as_float(b & 0xffff0000u)));
          }
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
              const uint32_t on = flags[u] >> (8 * p + 2 * c4);
              sc[p] &= (on & 1 ? 0xffffu : 0u) | (on & 2 ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            // nibbles of tokens t, t + 1 side by side, even dims in one word, odd in another:
            // each byte then converts to the (t, t + 1) pair of one dim
            uint32_t f[2][2][4];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              constexpr uint32_t kLow = 0x0f0f0f0fu;
              const uint32_t t0 = w[p][0][i], t1 = w[p][1][i];
              e2m1x8_to_half2((t0 & kLow) | ((t1 << 4) & ~kLow), f[p][0]);
              e2m1x8_to_half2(((t0 >> 4) & kLow) | (t1 & ~kLow), f[p][1]);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t a[4] = {hmul2(f[0][0][b], sc[0]), hmul2(f[0][1][b], sc[0]), hmul2(f[1][0][b], sc[1]),
                                     hmul2(f[1][1][b], sc[1])};
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
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<false>(o[j][nt], a, pb[u][nt][0], pb[u][nt][1]);
              mma16816<false>(o[j][nt], a, pr[u][nt][0], pr[u][nt][1]);
            }
          }
        }
      }
      st = st == STAGES - 1 ? 0 : st + 1;
    }

    // ----- merge the warps; the result, or this piece's part of it -----
    const bool more = pend < n_chunks;
    LinePos nxt = cur;
    if (more) {  // the next queries are on their way while the warps merge
      seek<C::kSubs>(P, nxt, pend);
      load_q(nxt);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
        // no token seen (a sum that is NaN is a row's all the same: its maximum stays finite, so
        // that no merge takes it for an empty part)
        if (m[nt][e] == kBaNone && l[nt][e] == 0.f) m[nt][e] = -INFINITY;
        if (r8 == 0) ml[warp * C::kRows + nt * 8 + 2 * c4 + e] = make_float2(m[nt][e], l[nt][e]);
      }
    __syncthreads();
    if (more) store_q();
    if (warp == WARPS - 1 && lane < C::kRows) {  // maximum and sum of a row
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * C::kRows + lane].x);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 v = ml[w * C::kRows + lane];
        sum += v.x == -INFINITY ? 0.f : v.y * ex2(v.x - top);
      }
      fin[lane] = make_float2(top, sum);
    }
    const bool split = !P.cluster && (cur.start < 0 || cur.end > n_chunks);
    float *shared_o = reinterpret_cast<float *>(ba_smem);  // [kRows][D], where the stages were
    const int slot = 2 * blockIdx.x + (cur.start < 0 ? 0 : 1);
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * C::kRows + nt * 8 + 2 * c4 + e].x);
        f[nt][e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - top);
      }
#pragma unroll
    for (int p0 = 0; p0 < 2 * NT; p0 += C::kParts) {  // parts p: rows 8 (p / 2) and up, half p % 2 of the dims
#pragma unroll
      for (int p = p0; p < p0 + C::kParts; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float *dst = merge + (p - p0) * C::kPart + (warp * 8 + 2 * c4 + e) * C::kMergeRow + 2 * r8;
#pragma unroll
          for (int j = 0; j < C::kSteps / 2; ++j) {
            const float *x = o[(p % 2) * (C::kSteps / 2) + j][p / 2];
            *reinterpret_cast<float2 *>(dst + 16 * j) = make_float2(x[e] * f[p / 2][e], x[e + 2] * f[p / 2][e]);
          }
        }
      __syncthreads();
      // a thread adds four neighbouring values of a row: tile j of this half, fragment rows
      // r and r + 1, both halves of the tile
      for (int i = threadIdx.x; i < C::kParts * D; i += C::kThreads) {
        const int p = p0 + i / D, rr = i % D / (D / 8), k = i % (D / 8), hf = p % 2;
        const int j = hf * (C::kSteps / 2) + k / 4, r = 2 * (k % 4), row = (p / 2) * 8 + rr;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4 *>(merge + (p - p0) * C::kPart + (w * 8 + rr) * C::kMergeRow + 4 * k);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        // x.x, x.y: fragment row r (tile rows r, r + 8); x.z, x.w: row r + 1
        int d0, d1;
        float2 a, b;
        if constexpr (C::kFp4) {  // tile rows (r, r + 8) are dims r * D/8 + 2 j + (0, 1)
          d0 = r * (D / 8) + 2 * j, d1 = d0 + D / 8;
          a = make_float2(x.x, x.y), b = make_float2(x.z, x.w);
        } else {                  // dims 16 j + r and 16 j + 8 + r
          d0 = 16 * j + r, d1 = d0 + 8;
          a = make_float2(x.x, x.z), b = make_float2(x.y, x.w);
        }
        const float2 v = fin[row];
        if (P.cluster > 1) {
          *reinterpret_cast<float2 *>(shared_o + row * D + d0) = a;
          *reinterpret_cast<float2 *>(shared_o + row * D + d1) = b;
        } else if (split) {
          float *part = P.part_o + (static_cast<int64_t>(slot) * C::kRows + row) * D;
          *reinterpret_cast<float2 *>(part + d0) = a;
          *reinterpret_cast<float2 *>(part + d1) = b;
          if (k == 0 && hf == 0) reinterpret_cast<float2 *>(P.part_ml)[slot * C::kRows + row] = v;
        } else {
          const int64_t oh = row_index(cur, row);
          if (oh >= 0) {
            const float inv = v.y > 0.f ? P.v_scale / v.y : v.y;  // (a NaN sum stays one)
            *reinterpret_cast<uint32_t *>(P.out + oh * D + d0) = pack2<false>(a.x * inv, a.y * inv);
            *reinterpret_cast<uint32_t *>(P.out + oh * D + d1) = pack2<false>(b.x * inv, b.y * inv);
            if (k == 0 && hf == 0 && P.lse) P.lse[oh] = ba_lse(v.x, v.y);
          }
        }
      }
      __syncthreads();
    }
    if (!more) break;
    cur = nxt;
    note_tail(cur);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // ----- a cluster: each CTA joins every CS-th row over all CTAs' shared memory, in rank order
  if (P.cluster > 1) {
    cluster_arrive();
    cluster_wait();
    const int rank = blockIdx.x % P.cluster;
    for (int i = threadIdx.x;; i += C::kThreads) {
      const int row = rank + P.cluster * (i / (D / 4)), d = 4 * (i % (D / 4));
      if (row >= C::kRows) break;
      const int64_t oh = row_index(cur, row);
      if (oh < 0) continue;
      const uint32_t fin_at = smem_u32(fin + row), o_at = smem_u32(ba_smem) + (row * D + d) * 4;
      float2 v[kBaMaxCluster];
      float4 x[kBaMaxCluster];
#pragma unroll
      for (int r = 0; r < kBaMaxCluster; ++r) {
        v[r] = make_float2(-INFINITY, 0.f);
        x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < P.cluster) {
          const uint32_t fa = peer_smem(fin_at, r), oa = peer_smem(o_at, r);
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[r].x), "=f"(v[r].y) : "r"(fa) : "memory");
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[r].x), "=f"(x[r].y), "=f"(x[r].z), "=f"(x[r].w)
                       : "r"(oa)
                       : "memory");
        }
      }
      float top = -INFINITY, sum = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kBaMaxCluster; ++r) top = fmaxf(top, v[r].x);
#pragma unroll
      for (int r = 0; r < kBaMaxCluster; ++r) {
        const float f = v[r].x == -INFINITY ? 0.f : ex2(v[r].x - top);
        sum += v[r].y * f;
        y.x += x[r].x * f, y.y += x[r].y * f, y.z += x[r].z * f, y.w += x[r].w * f;
      }
      const float inv = sum > 0.f ? P.v_scale / sum : sum;
      *reinterpret_cast<uint2 *>(P.out + oh * D + d) =
          make_uint2(pack2<false>(y.x * inv, y.y * inv), pack2<false>(y.z * inv, y.w * inv));
      if (d == 0 && P.lse) P.lse[oh] = ba_lse(top, sum);
    }
    cluster_arrive();  // (no CTA's shared memory goes while another reads it)
    cluster_wait();
  }
}

// Merge of the pieces of each (b, hm) that was cut: block (i, y) takes row y of the i-th one
// (kPair), or of the one that begins in CTA i's range and goes on past it (its first loads then
// go out before it is known how many pieces there are: one round trip to L2 in the usual
// case).  D / 4 threads add a piece's row at a time, kGroups pieces side by side, then the
// groups in order.  Few (b, hm) have many pieces each and leave most CTAs none to begin: with 32
// rows 4864 blocks of 256 threads, nearly all without work, took 6.6 us.
template <int D, bool kPair>
struct BaComb {
  static constexpr int kGroups = kPair ? 16 : 512 / D, kThreads = kGroups * (D / 4);
};

template <int D, bool kPair>
__global__ void __launch_bounds__(BaComb<D, kPair>::kThreads) block_attn_combine_kernel(const BlockAttnParams P, int rows_pad) {
  constexpr int kLanes = D / 4, kGroups = BaComb<D, kPair>::kGroups;
  __shared__ float2 sml[kGroups];
  __shared__ __align__(16) float so[kGroups][D];
  const int row = blockIdx.y, grp = threadIdx.x / kLanes, d = 4 * (threadIdx.x % kLanes);
  pdl_launch_dependents();
  pdl_wait();
  const int4 tail = P.tail[blockIdx.x];
  const int cta = kPair ? tail.w : blockIdx.x, pieces = tail.z;
  if (kPair && pieces == 0) return;
  // piece 0 is the first CTA's second slot, piece s > 0 the first slot of the s-th CTA from there
  auto slot_row = [&](int s) {
    return static_cast<int64_t>(s == 0 ? 2 * cta + 1 : 2 * min(cta + s, kBaMaxGrid - 1)) * rows_pad + row;
  };
  float2 v = reinterpret_cast<const float2 *>(P.part_ml)[slot_row(grp)];
  float4 x = *reinterpret_cast<const float4 *>(P.part_o + slot_row(grp) * D + d);
  if (pieces == 0) return;
  const int h = tail.y / P.mgroups;
  const int rq = (tail.y - h * P.mgroups) * rows_pad + row;
  if (rq >= P.n_q * P.group) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = grp; s < pieces;) {
    const float top = fmaxf(m, v.x);
    const float fa = m == -INFINITY ? 0.f : ex2(m - top), fb = v.x == -INFINITY ? 0.f : ex2(v.x - top);
    m = top;
    l = l * fa + v.y * fb;
    acc.x = acc.x * fa + x.x * fb, acc.y = acc.y * fa + x.y * fb;
    acc.z = acc.z * fa + x.z * fb, acc.w = acc.w * fa + x.w * fb;
    s += kGroups;
    if (s < pieces) {
      v = reinterpret_cast<const float2 *>(P.part_ml)[slot_row(s)];
      x = *reinterpret_cast<const float4 *>(P.part_o + slot_row(s) * D + d);
    }
  }
  if (d == 0) sml[grp] = make_float2(m, l);
  *reinterpret_cast<float4 *>(&so[grp][d]) = acc;
  __syncthreads();
  if (grp != 0) return;
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) top = fmaxf(top, sml[k].x);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float2 w = sml[k];
    const float f = w.x == -INFINITY ? 0.f : ex2(w.x - top);
    const float4 a = *reinterpret_cast<const float4 *>(&so[k][d]);
    sum += w.y * f;
    y.x += a.x * f, y.y += a.y * f, y.z += a.z * f, y.w += a.w * f;
  }
  const int j = rq / P.group;
  const int64_t oh = (static_cast<int64_t>(tail.x) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group;
  const float inv = sum > 0.f ? P.v_scale / sum : sum;
  *reinterpret_cast<uint2 *>(P.out + oh * D + d) =
      make_uint2(pack2<false>(y.x * inv, y.y * inv), pack2<false>(y.z * inv, y.w * inv));
  if (d == 0 && P.lse) P.lse[oh] = ba_lse(top, sum);
}

}  // namespace echo

namespace echo_host {

static int ba_row_pad(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

size_t block_attention_workspace_bytes(int32_t rows, int32_t head_dim) {
  const size_t pad = ba_row_pad(rows < echo::kBaMaxRows ? rows : echo::kBaMaxRows);
  return echo::kBaMaxGrid * sizeof(int4) + 2 * echo::kBaMaxGrid * pad * (2 + static_cast<size_t>(head_dim)) * sizeof(float);
}

// One shape of the kernel: WARPS warps with STAGES stages each, CTAS CTAs to an SM.
template <int FMT, int D, int NT, int WARPS, int STAGES, int CTAS>
struct BaShape {
  using C = echo::BaCfg<FMT, D, NT, WARPS, STAGES>;
  static_assert(C::kSmem <= (CTAS == 1 ? 232448 : 115712), "block attention: shared memory of one CTA");

  static int prepare(int *dev) {
    static std::atomic<bool> attr[kMaxDevices];
    cudaGetDevice(dev);
    return smem_limit_once(attr, echo::block_attn_kernel<FMT, D, NT, WARPS, STAGES, CTAS>, C::kSmem, "block attention smem attribute");
  }

  // How many clusters of cs CTAs the device holds at once (a cluster sits in one group of SMs:
  // 76 of 2, 36 of 4 and 15 of 8 here, not 152 SMs' worth: 16 clusters of 8 take 14.4 us where
  // 15 take 8.4).  Asked once per shape and device.
  static int clusters_at_once(int cs, int dev) {
    static std::atomic<int> known[kMaxDevices][echo::kBaMaxCluster + 1];
    int n = known[dev][cs].load(std::memory_order_relaxed);
    if (n) return n - 1;
    cudaLaunchConfig_t cfg = config(cs, nullptr);
    cudaLaunchAttribute at = cluster(cs);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, echo::block_attn_kernel<FMT, D, NT, WARPS, STAGES, CTAS>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[dev][cs].store(n + 1, std::memory_order_relaxed);
    return n;
  }

  // P.cluster CTAs per (b, h), or (0) the line cut into a piece per CTA
  static int launch(echo::BlockAttnParams P, int cs, int64_t pairs, int sms, cudaStream_t stream) {
    P.cluster = cs;
    const int64_t grid = cs ? pairs * cs : std::min(sms * CTAS, echo::kBaMaxGrid);
    P.by_pair = !cs && 2 * pairs <= grid;
    cudaLaunchConfig_t cfg = config(grid, stream);
    cudaLaunchAttribute at[2] = {pdl(), cluster(cs)};
    cfg.attrs = at;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, echo::block_attn_kernel<FMT, D, NT, WARPS, STAGES, CTAS>, P);
    if (e != cudaSuccess) return cuda_fail(e, "block attention launch");
    if (cs) return ECHO_OK;
    e = P.by_pair ? combine<true>(cfg, pairs, P) : combine<false>(cfg, grid, P);
    return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block attention merge launch");
  }

 private:
  template <bool kPair>
  static cudaError_t combine(cudaLaunchConfig_t cfg, int64_t n, const echo::BlockAttnParams &P) {
    cfg.gridDim = dim3(static_cast<unsigned>(n), C::kRows);
    cfg.blockDim = dim3(echo::BaComb<D, kPair>::kThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, echo::block_attn_combine_kernel<D, kPair>, P, static_cast<int>(C::kRows));
  }
  static cudaLaunchConfig_t config(int64_t grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    return cfg;
  }
  static cudaLaunchAttribute pdl() {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
  }
  static cudaLaunchAttribute cluster(int cs) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    return at;
  }
};

// How the work of a call is laid over the CTAs: a cluster of them per (b, h), one CTA per (b,
// h) with two to an SM, or the line of all chunks cut into equal pieces.  Costs are counted
// in the tokens an SM works through.  Whole (b, h) cost their waves times the longest context;
// cutting costs an equal share, the second kernel (`extra`) and a piece border per (b, h)
// (`border`: the warps of an SM end together; overlapped by the other SMs where HBM is the
// bound), all for heads of 128: of half as many dims twice the tokens take as long (144 pairs of
// 8000 tokens of 64 dims 42.7 / 28.8 us cut, 38.2 / 23.4 a CTA each).  Measured, bf16 / 4-bit,
// us: 64 pairs of up to 1000 tokens 8.8 / 8.8 in clusters of 2 against 13.1 / 14.6 cut; 8 pairs
// of 8000 11.2 / 10.9 in clusters of 8, 12.4 / 13.5 cut, of 16000 16.9 / 14.5 and 19.9 / 15.2, with
// 32 rows 34.4 / 26.9 and 28.8 / 23.5; 128 pairs of 4000 35 / 21 a CTA each, 39 / 26 cut; 512 pairs
// of 512 20.7 / 18.6 with two CTAs an SM, 29 / 27 with one.  The host does not know the contexts,
// only how long they may be: past 4 `extra` tokens a CTA, what an uneven batch would cost is
// more than whole (b, h) save (152 pairs of 16384 to 32768 tokens in 4 bits: 125 us whole, 103 cut).
template <class Wide, class Narrow>
static int ba_go(const echo::BlockAttnParams &P, int64_t pairs, int64_t most, int sms, cudaStream_t stream) {
  using C = typename Wide::C;
  constexpr int64_t dims = 8 / C::kSteps, border = dims * (C::kFp4 ? 1000 : 200);
  constexpr int64_t extra = dims * (C::kRows > 16 ? 1024 : C::kFp4 ? 1536 : 1280);
  const int64_t cut = pairs * most / sms + extra;
  int dev = 0;
  const int64_t waves = (pairs + 2 * sms - 1) / (2 * sms);
  const bool whole = most <= 4 * extra && 2 * waves * most <= cut + pairs * border / sms;
  // (cutting with two CTAs an SM, one computes while the other merges: 512 pairs of 8192 tokens
  // in 4 bits 109 -> 103 us, 256 of 16384 101 -> 100, but 128 of 131072 318 -> 331)
  if (pairs > sms && (whole || (C::kFp4 && C::kRows == 8 && most <= 16384))) {
    if (int rr = Narrow::prepare(&dev)) return rr;
    return Narrow::launch(P, whole ? 1 : 0, pairs, sms, stream);
  }
  if (int rr = Wide::prepare(&dev)) return rr;
  // the largest cluster that the device holds for every pair at once and whose warps all get a
  // chunk (of any size: 16 pairs of 8000 tokens in 4 bits, 8 and 32 rows, 14.5 and 26.8 us in
  // fours, 12.3 and 21.0 in sixes)
  const int64_t fits = sms / pairs, useful = (most - 1) / (C::kThreads / 32 * C::kTokens) + 1;
  int cs = static_cast<int>(std::min<int64_t>({echo::kBaMaxCluster, fits, useful}));
  while (cs > 1 && pairs > Wide::clusters_at_once(cs, dev)) --cs;
  cs = cs < 1 ? 1 : cs;
  const int64_t share = (pairs * cs + sms - 1) / sms * most / cs;
  return Wide::launch(P, share <= cut && share <= 4 * extra ? cs : 0, pairs, sms, stream);
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
  // (48 rows as 24 + 24, not 32 + 16: 12 requests of up to 20000 tokens in 4 bits 200 -> 151 us)
  const int mrows = ((rows + P.mgroups - 1) / P.mgroups + 7) / 8 * 8;
  P.sinks = a->sinks, P.window = a->window;
  P.scale_log2 = std::ldexp(std::fabs(a->scale) * 1.4426950408889634f, -a->k_shift);
  P.v_scale = std::ldexp(1.f, -a->v_shift);
  P.q_sign = a->scale < 0.f ? 0x80008000u : 0u;
  P.out = a->out, P.lse = a->lse;
  P.status = a->dev_status;
  const int pad = ba_row_pad(rows < echo::kBaMaxRows ? rows : echo::kBaMaxRows);
  P.tail = reinterpret_cast<int4 *>(a->workspace);
  P.part_ml = reinterpret_cast<float *>(P.tail + echo::kBaMaxGrid);
  P.part_o = P.part_ml + 2 * static_cast<size_t>(echo::kBaMaxGrid) * pad * 2;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "block attention device");
  const int64_t pairs = static_cast<int64_t>(P.B) * P.n_kv * P.mgroups;
  // tokens a context can show at most
  int64_t most = static_cast<int64_t>(P.max_blocks) * a->block_tokens;
  if (!P.sel && P.window && most > P.sinks + static_cast<int64_t>(P.window) + P.n_q + 31) most = P.sinks + static_cast<int64_t>(P.window) + P.n_q + 31;
  // Warps and stages for 8, 16, 24 and 32 query rows, of a CTA with an SM to itself and of one of
  // two: as many warps as registers and shared memory allow in multiples of the 4 schedulers
  // (4-bit rows, bound by instructions: 12 warps of 3 stages 334 us, 16 of 2 318 us, 14 of 2 355
  // us for 16 x 131072 tokens x 8 KV heads), or enough bytes in flight (bf16 rows, bound by HBM).
  // 20 rows as 24 instead of 32: 12 requests of up to 38624 tokens in 4 bits 179 -> 143 us (3
  // stages; 4 take 148), 24 of 6479 in bf16 62 -> 52.5.  32 rows in chunks of 16 tokens: 183 ->
  // 186 us, but nothing spills, and one request of 1000 tokens takes 10.2 us instead of 12.4.
  // Two CTAs an SM for 512 pairs of up to 2000 tokens, 24 / 32 rows: 75 / 91 -> 61 / 77 us in 4
  // bits, 89 / 118 -> 78 / 94 in bf16.
#define BA_SHAPE(FMT, D, NT, W, S, CTAS) BaShape<FMT, D, NT, W, S, CTAS>
#define BA_GO(FMT, D, NT, W, S, W2, S2) ba_go<BA_SHAPE(FMT, D, NT, W, S, 1), BA_SHAPE(FMT, D, NT, W2, S2, 2)>(P, pairs, most, sms, stream)
#define BA_PICK(FMT, D, A1, A2, A3, A4) \
  (mrows == 8 ? BA_GO(FMT, D, 1, A1) : mrows == 16 ? BA_GO(FMT, D, 2, A2) : mrows == 24 ? BA_GO(FMT, D, 3, A3) : BA_GO(FMT, D, 4, A4))
  // (each: warps and stages of a CTA with an SM to itself, then of one of two)
#define X(...) __VA_ARGS__
  if (a->format == ECHO_BLOCK_FP4)
    return a->head_dim == 128 ? BA_PICK(ECHO_BLOCK_FP4, 128, X(16, 2, 8, 2), X(12, 3, 6, 3), X(8, 3, 4, 3), X(8, 3, 4, 3))
                              : BA_PICK(ECHO_BLOCK_FP4, 64, X(16, 2, 8, 2), X(16, 4, 8, 4), X(12, 3, 4, 3), X(8, 3, 4, 3));
  return a->head_dim == 128 ? BA_PICK(ECHO_BLOCK_BF16, 128, X(8, 3, 4, 3), X(7, 3, 4, 2), X(7, 3, 4, 2), X(7, 3, 4, 2))
                            : BA_PICK(ECHO_BLOCK_BF16, 64, X(8, 3, 4, 3), X(7, 3, 4, 2), X(8, 3, 4, 2), X(8, 3, 4, 2));
#undef X
#undef BA_PICK
#undef BA_SHAPE
#undef BA_GO
}

}  // namespace echo_host
