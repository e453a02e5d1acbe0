// block_select.cu -- which blocks a query attends to: the key range of each block, a bound on
// the scores a query can have in it, and the blocks of the best bounds.
//
// Summary of a cache row (a block of one KV head), over its tokens t:
//   lo_d = min_t k_td,  hi_d = max_t k_td
// Score of the block for query token j and KV head h, over the group's query heads g:
//   s = scale * max_g sum_d max(q_gd lo_d, q_gd hi_d)  >=  scale * q_g . k_t  for every t, g.
// max(q lo, q hi) is q hi for q >= 0 and q lo for q < 0, so with q+ = max(q, 0), q- = min(q, 0)
//   sum_d max(q_d lo_d, q_d hi_d) = [q-, q+] . [lo, hi],
// a product of length 2 D over the summary row as it lies in memory: tensor-core work that
// reads 4 D bytes for a block whose keys take 2 D bytes a token.
//
// sm_103a design.
//   Summary: a CTA of 128 threads per (block, KV head), 16-byte loads of its keys, packed
//     minima and maxima, joined over the lanes and then the warps.  The blocks that changed
//     are one line over the requests, found by every CTA from the lengths.
//   Scores: 16 blocks x 8 columns with mma.m16n8k16.  The order of a contraction's dims is free,
//     so a lane reads 16 contiguous bytes of "its" two blocks per 8 dims of a quarter and feeds them
//     as they are: a warp has the 16 summaries (8 KB) in registers after one round of loads, with
//     no shared memory.  The 8 columns are the heads of one query token, or of several where a
//     group has fewer, so the maximum over a group stays within a quad.
//   Selection: a CTA per (query, KV head) with its keys in shared memory.  Radix passes over the
//     range that still holds the k-th best, 256 equal parts of it at a time, and one ordered
//     pass over the blocks that writes those above it and the first of its equals.
#include <algorithm>
#include <cmath>

#include "block_mma.cuh"

namespace echo {

// the row of block entry e of (b, h), -1 when it is not held or lies outside the rows
struct BlockTable {
  const int32_t *table;
  int32_t heads, max_blocks, n_kv;
  __device__ __forceinline__ int64_t row(int b, int h, int e) const {
    const int32_t id = table[(static_cast<int64_t>(b) * heads + (heads > 1 ? h : 0)) * max_blocks + e];
    return id < 0 ? -1 : heads > 1 ? id : static_cast<int64_t>(id) * n_kv + h;
  }
};

// a context length within what the table can hold
__device__ __forceinline__ int held_len(int len, int64_t most, int32_t *status, bool report) {
  if (len > most) {
    if (report) set_status(status, ECHO_DEV_BAD_INDEX);
    len = static_cast<int>(most);
  }
  return max(len, 0);
}

// ---------------------------------------------------------------------------
// summaries
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 128;

struct SummaryParams {
  const uint8_t *rows;
  int64_t row_bytes;
  int32_t n_rows, bs;
  BlockTable tab;
  const int32_t *old_len, *new_len;
  int32_t B;
  uint32_t *summary;
  float k_scale;  // 2^-k_shift
  int32_t *status;
};

// blocks [first, end) of request b that are summed up anew
__device__ __forceinline__ int2 redone(const SummaryParams &P, int b, bool report) {
  const int64_t most = static_cast<int64_t>(P.tab.max_blocks) * P.bs;
  const int n = held_len(P.new_len[b], most, P.status, report);
  const int o = P.old_len ? held_len(P.old_len[b], most, P.status, report) : 0;
  if (n == o) return make_int2(0, 0);
  return make_int2(min(o, n) / P.bs, (n + P.bs - 1) / P.bs);
}

template <int FMT>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (FMT == ECHO_BLOCK_FP4) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (FMT == ECHO_BLOCK_FP4) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kSumThreads) block_summary_kernel(const SummaryParams P) {
  constexpr bool kFp4 = FMT == ECHO_BLOCK_FP4;
  constexpr int kWords = kFp4 ? 16 : 4;               // pairs of dims that a thread holds
  constexpr int kLanes = D / (2 * kWords);            // threads of a token
  constexpr int kTokens = kSumThreads / kLanes;       // tokens a round
  constexpr int kRounds = kFp4 ? 2 : 8;               // rounds of loads in flight
  extern __shared__ int32_t sum_cu[];                 // [B + 1] exclusive sums of the redone blocks
  __shared__ uint32_t part[4][2][D / 2];
  __shared__ int32_t wsum[4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();

  // ----- the line of redone blocks -----
  const int per = (P.B + kSumThreads - 1) / kSumThreads;
  int mine = 0;
  for (int b = tid * per; b < min(P.B, (tid + 1) * per); ++b) {
    const int2 r = redone(P, b, blockIdx.x == 0);
    mine += r.y - r.x;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < warp; ++w) at += wsum[w];
  for (int b = tid * per; b < min(P.B, (tid + 1) * per); ++b) {
    sum_cu[b] = at;
    const int2 r = redone(P, b, false);
    at += r.y - r.x;
  }
  if (tid == kSumThreads - 1) sum_cu[P.B] = at;
  __syncthreads();
  const int64_t units = static_cast<int64_t>(sum_cu[P.B]) * P.tab.n_kv;

  const int t0 = tid / kLanes, c = tid % kLanes;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int line = static_cast<int>(u / P.tab.n_kv), h = static_cast<int>(u - static_cast<int64_t>(line) * P.tab.n_kv);
    int b = 0, end = P.B;
    while (end - b > 1) {
      const int mid = (b + end) >> 1;
      if (sum_cu[mid] <= line) b = mid;
      else end = mid;
    }
    const int e = redone(P, b, false).x + line - sum_cu[b];
    const int64_t row = P.tab.row(b, h, e);
    if (row >= P.n_rows && tid == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
    if (row < 0 || row >= P.n_rows) continue;  // (the same for the whole CTA)
    // tokens of the block (rounds past the last one read it again: a minimum does not mind)
    const int n = min(P.bs, held_len(P.new_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, nullptr, false) - e * P.bs);
    const uint8_t *src = P.rows + row * P.row_bytes;
    uint32_t lo[kWords], hi[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) lo[i] = kFp4 ? 0x7c007c00u : 0x7f807f80u, hi[i] = lo[i] | 0x80008000u;
    for (int t = 0; t < n; t += kTokens * kRounds) {
      uint4 x[kRounds];
      uint32_t sc[kRounds];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int tk = min(t + r * kTokens + t0, n - 1);
        if constexpr (kFp4) {
          const uint8_t *sub = src + (tk / kSubTokens) * Fp4Sub<D>::kBytes;
          x[r] = *reinterpret_cast<const uint4 *>(sub + (tk % kSubTokens) * (D / 2) + c * 16);
          sc[r] = *reinterpret_cast<const uint16_t *>(sub + Fp4Sub<D>::kKeyScales + (tk % kSubTokens) * (D / 16) + c * 2);
        } else {
          x[r] = *reinterpret_cast<const uint4 *>(src + tk * (2 * D) + c * 16);
        }
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        if constexpr (kFp4) {
          const uint32_t s2 = e4m3x2_to_half2(sc[r]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            e2m1x8_to_half2(w[i], f);
            const uint32_t s = __byte_perm(s2, 0, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t v = hmul2(f[k], s);
              lo[4 * i + k] = min2<FMT>(lo[4 * i + k], v);
              hi[4 * i + k] = max2<FMT>(hi[4 * i + k], v);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) lo[i] = min2<FMT>(lo[i], w[i]), hi[i] = max2<FMT>(hi[i], w[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int d = kLanes; d < 32; d <<= 1) {
        lo[i] = min2<FMT>(lo[i], __shfl_xor_sync(~0u, lo[i], d));
        hi[i] = max2<FMT>(hi[i], __shfl_xor_sync(~0u, hi[i], d));
      }
    if (lane < kLanes) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) part[warp][0][c * kWords + i] = lo[i], part[warp][1][c * kWords + i] = hi[i];
    }
    __syncthreads();
    if (tid < D) {
      const int m = tid / (D / 2), i = tid % (D / 2);
      uint32_t v = part[0][m][i];
#pragma unroll
      for (int w = 1; w < 4; ++w) v = m ? max2<FMT>(v, part[w][m][i]) : min2<FMT>(v, part[w][m][i]);
      if constexpr (kFp4) {  // (6 significant bits: exact in bf16, a power of two less too)
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        v = pack2<false>(f.x * P.k_scale, f.y * P.k_scale);
      }
      P.summary[row * D + tid] = v;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
constexpr int kScoreWarps = 4;
constexpr int kScoreCols = 64;  // query columns that a CTA lays out at a time

struct ScoreParams {
  const uint16_t *q;
  const uint8_t *summary;
  int32_t n_rows, bs;
  BlockTable tab;
  const int32_t *ctx_len;
  int32_t n_q, n_heads, group;
  int32_t pad_log2;       // columns of a query token: 2^pad_log2, of which `group` or fewer differ
  int32_t cols;           // columns of a KV head, a multiple of 8
  int32_t wide;           // columns of a query token where the group has more than 8 heads
  int32_t chunk;          // columns laid out at a time: whole query tokens if they fit
  int32_t ctas, tiles;    // CTAs of a (b, h), 16-block tiles that a warp of one takes
  float scale;            // |scale|
  uint32_t q_sign;
  float *scores;
  int32_t *status;
};

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(const ScoreParams P) {
  constexpr int kStride = 4 * D + 64;       // bytes of a column; + 64: its quads on other banks
  constexpr int kChunks = D / 16;           // 16-byte pieces of a summary row that a lane holds
  __shared__ __align__(16) uint8_t qs[kScoreCols * kStride];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  const int pair = blockIdx.x / P.ctas, part = blockIdx.x - pair * P.ctas;
  const int b = pair / P.tab.n_kv, h = pair - b * P.tab.n_kv;
  pdl_launch_dependents();
  pdl_wait();
  const int len = held_len(P.ctx_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, P.status,
                           part == 0 && h == 0 && threadIdx.x == 0);
  const int blocks = (len + P.bs - 1) / P.bs;
  const int first = part * (kScoreWarps * 16) * P.tiles;
  if (first >= blocks) return;

  for (int c0 = 0; c0 < P.cols; c0 += P.chunk) {
    const int nc = min(P.chunk, P.cols - c0);
    if (c0) __syncthreads();
    // [q-, q+] of the columns; a group's last head fills its padding (a maximum does not mind)
    for (int i = threadIdx.x; i < nc * (D / 8); i += kScoreWarps * 32) {
      const int col = i / (D / 8), d8 = i % (D / 8), cc = c0 + col;
      int j, g;
      if (P.pad_log2 <= 3) {
        j = cc >> P.pad_log2, g = cc & ((1 << P.pad_log2) - 1);
      } else {
        j = cc / P.wide, g = cc - j * P.wide;
      }
      j = min(j, P.n_q - 1), g = min(g, P.group - 1);
      uint4 x = *reinterpret_cast<const uint4 *>(P.q + ((static_cast<int64_t>(b) * P.n_q + j) * P.n_heads + h * P.group + g) * D + d8 * 8);
      uint32_t w[4] = {x.x ^ P.q_sign, x.y ^ P.q_sign, x.z ^ P.q_sign, x.w ^ P.q_sign}, n[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t neg = ((w[k] >> 15) & 0x10001u) * 0xffffu;  // all ones in the halves below zero
        n[k] = w[k] & neg, w[k] &= ~neg;
      }
      *reinterpret_cast<uint4 *>(qs + col * kStride + d8 * 16) = make_uint4(n[0], n[1], n[2], n[3]);
      *reinterpret_cast<uint4 *>(qs + col * kStride + 2 * D + d8 * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    for (int t = 0; t < P.tiles; ++t) {
      const int e0 = first + (t * kScoreWarps + warp) * 16;
      if (e0 >= blocks) break;
      uint4 a[2][kChunks];
      bool held[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = e0 + r8 + 8 * k;
        const int64_t row = e < blocks ? P.tab.row(b, h, e) : -1;
        held[k] = row >= 0 && row < P.n_rows;
        if (row >= P.n_rows) set_status(P.status, ECHO_DEV_BAD_INDEX);
        const uint8_t *src = P.summary + (held[k] ? row : 0) * (4 * D) + c4 * 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          a[k][i] = held[k] ? *reinterpret_cast<const uint4 *>(src + i * 64) : make_uint4(0u, 0u, 0u, 0u);
      }
      float best[2][2];  // of column parity and block
#pragma unroll
      for (int k = 0; k < 4; ++k) best[k >> 1][k & 1] = -INFINITY;
      for (int cg = 0; cg < nc; cg += 8) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t *qp = qs + (cg + r8) * kStride + c4 * 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint4 q = *reinterpret_cast<const uint4 *>(qp + i * 64);
          const uint32_t x[4] = {a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y}, y[4] = {a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w};
          mma16816<false>(acc, x, q.x, q.y);
          mma16816<false>(acc, y, q.z, q.w);
        }
        // acc[p + 2 k]: column 2 c4 + p of block k.  One value per (query token, block)
        const int cc = c0 + cg + 2 * c4;
        if (P.pad_log2 == 0) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < 2; ++k) best[p][k] = acc[p + 2 * k];
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = fmaxf(acc[2 * k], acc[1 + 2 * k]);
            if (P.pad_log2 >= 2) v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
            if (P.pad_log2 >= 3) v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
            best[0][k] = P.pad_log2 > 3 ? fmaxf(best[0][k], v) : v;
          }
        }
        int j = cc >> P.pad_log2, n_out = P.pad_log2 ? 1 : 2;
        bool write = (cc & ((1 << min(P.pad_log2, 3)) - 1) & ~1) == 0;
        bool more = false;  // an earlier chunk had heads of this token too
        if (P.pad_log2 > 3) {
          const int at = c0 + cg;
          j = at / P.wide;
          write = at + 8 == (j + 1) * P.wide || cg + 8 == nc;
          more = j * P.wide < c0;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (!write || p >= n_out || j + p >= P.n_q || (P.pad_log2 > 3 && c4)) continue;
          const int nb = (len - (P.n_q - 1 - j - p) + P.bs - 1) / P.bs;  // (may be negative: nothing)
          float *dst = P.scores + ((static_cast<int64_t>(b) * P.n_q + j + p) * P.tab.n_kv + h) * P.tab.max_blocks;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (e0 + r8 + 8 * k < nb) {
              float v = held[k] ? best[p][k] * P.scale : -INFINITY;
              if (more) v = fmaxf(v, dst[e0 + r8 + 8 * k]);  // (written by this thread)
              dst[e0 + r8 + 8 * k] = v;
            }
        }
        if (P.pad_log2 > 3 && write) best[0][0] = best[0][1] = -INFINITY;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
constexpr uint32_t kMustKey = 0xffffffffu;  // a block that is always taken; 0: one that may not be
constexpr int kSelBins = 256;

struct SelectParams {
  const float *scores;
  const int32_t *ctx_len;
  int32_t n_q, bs, k, first, last;
  BlockTable tab;  // (table: optional)
  int32_t *sel, *sel_rows, *len_out;
  int32_t *status;
};

template <int T>
__global__ void __launch_bounds__(T) block_select_kernel(const SelectParams P) {
  constexpr int W = T / 32;
  extern __shared__ uint32_t sel_smem[];
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint32_t red[4][W];
  __shared__ uint32_t pick[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  const int bj = static_cast<int>(row / P.tab.n_kv), h = static_cast<int>(row - static_cast<int64_t>(bj) * P.tab.n_kv);
  const int b = bj / P.n_q, j = bj - b * P.n_q;
  pdl_launch_dependents();
  pdl_wait();
  const int ctx = held_len(P.ctx_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, P.status, j == 0 && h == 0 && tid == 0);
  const int len = max(ctx - (P.n_q - 1 - j), 0), nb = (len + P.bs - 1) / P.bs;
  if (P.len_out && h == 0 && tid == 0) P.len_out[bj] = len;
  uint32_t *keys = sel_smem;                        // [max_blocks]
  uint32_t *cnt = sel_smem + P.tab.max_blocks;      // [ceil(max_blocks / T) * W]
  const float *src = P.scores + row * P.tab.max_blocks;

  uint32_t n_ok = 0, n_must = 0, lo = kMustKey, hi = 0;
  for (int i = tid; i < nb; i += T) {
    uint32_t key;
    if (P.tab.table && P.tab.row(b, h, i) < 0) key = 0;
    else if (i < P.first || i >= nb - P.last) key = kMustKey;
    else {
      const float s = src[i];
      key = s != s ? 1u : score_key(s);  // (a score that is NaN comes last)
    }
    keys[i] = key;
    n_ok += key != 0, n_must += key == kMustKey;
    if (key != 0 && key != kMustKey) lo = min(lo, key), hi = max(hi, key);
  }
  n_ok = __reduce_add_sync(~0u, n_ok), n_must = __reduce_add_sync(~0u, n_must);
  lo = __reduce_min_sync(~0u, lo), hi = __reduce_max_sync(~0u, hi);
  if (lane == 0) red[0][warp] = n_ok, red[1][warp] = n_must, red[2][warp] = lo, red[3][warp] = hi;
  __syncthreads();
  n_ok = n_must = hi = 0, lo = kMustKey;
#pragma unroll
  for (int w = 0; w < W; ++w) n_ok += red[0][w], n_must += red[1][w], lo = min(lo, red[2][w]), hi = max(hi, red[3][w]);

  // ----- the key above which all are taken, and how many of its equals -----
  uint32_t thr = 0, need = 0;
  if (n_ok > static_cast<uint32_t>(P.k)) {
    uint32_t want = P.k - n_must;  // (first + last <= k)
    thr = kMustKey - 1;
    while (want) {  // the want-th largest of the keys in [lo, hi]
      const uint32_t span = hi - lo;
      const int shift = max(0, 24 - __clz(span));
      for (int i = tid; i < kSelBins; i += T) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < nb; i += T) {
        const uint32_t key = keys[i];
        if (key >= lo && key <= hi) atomicAdd(&hist[(key - lo) >> shift], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // lane l holds bins 255 - 8 l .. 248 - 8 l
        uint32_t n[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = hist[kSelBins - 1 - 8 * lane - i], sum += n[i];
        uint32_t upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t x = __shfl_up_sync(~0u, upto, d);
          if (lane >= d) upto += x;
        }
        uint32_t above = upto - sum;
        if (above < want && upto >= want) {
          int i = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i == k && above + n[k] < want) above += n[k], i = k + 1;
          pick[0] = kSelBins - 1 - 8 * lane - i;
          pick[1] = above;
          pick[2] = pick_reg(n, i);
        }
      }
      __syncthreads();
      const uint32_t bin = pick[0], in = pick[2];
      want -= pick[1];
      lo += bin << shift;
      const uint32_t width = (1u << shift) - 1;
      hi = hi - lo > width ? lo + width : hi;
      if (in == want) {          // the whole part
        thr = lo - 1;
        break;
      }
      if (shift == 0) {          // equal keys: the first of them
        thr = lo, need = want;
        break;
      }
    }
  }

  // ----- the blocks in order -----
  const int rounds = (nb + T - 1) / T;
  for (int r = 0; r < rounds; ++r) {
    const int i = r * T + tid;
    const uint32_t key = i < nb ? keys[i] : 0u;
    const uint32_t gt = __ballot_sync(~0u, key > thr), eq = __ballot_sync(~0u, key == thr && key != 0);
    if (lane == 0) cnt[r * W + warp] = __popc(gt) | __popc(eq) << 16;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t base = 0;
    for (int r = 0; r < rounds * W; r += 32) {
      const uint32_t x = r + lane < rounds * W ? cnt[r + lane] : 0u;
      uint32_t upto = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += y;
      }
      if (r + lane < rounds * W) cnt[r + lane] = base + upto - x;
      base += __shfl_sync(~0u, upto, 31);
    }
    if (lane == 0) pick[0] = (base & 0xffffu) + min(base >> 16, need);
  }
  __syncthreads();
  int32_t *sel = P.sel + row * P.k, *rows = P.sel_rows ? P.sel_rows + row * P.k : nullptr;
  for (int r = 0; r < rounds; ++r) {
    const int i = r * T + tid;
    const uint32_t key = i < nb ? keys[i] : 0u;
    const bool gt = key > thr, eq = key == thr && key != 0;
    const uint32_t below = (1u << lane) - 1, c = cnt[r * W + warp];
    const uint32_t g = (c & 0xffffu) + __popc(__ballot_sync(~0u, gt) & below);
    const uint32_t q = (c >> 16) + __popc(__ballot_sync(~0u, eq) & below);
    if (gt || (eq && q < need)) {
      const uint32_t at = g + min(q, need);
      sel[at] = i;
      if (rows) rows[at] = static_cast<int32_t>(P.tab.row(b, h, i));
    }
  }
  for (int i = pick[0] + tid; i < P.k; i += T) {
    sel[i] = -1;
    if (rows) rows[i] = -1;
  }
}

}  // namespace echo

namespace echo_host {

static int sm_count(int *sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block selection device");
}

template <int FMT, int D>
static int go_summary(const echo::SummaryParams &P, cudaStream_t stream) {
  static std::atomic<bool> attr[kMaxDevices];
  const int smem = (P.B + 1) * 4;
  if (smem > 40960)
    if (int rr = smem_limit_once(attr, echo::block_summary_kernel<FMT, D>, (16384 + 1) * 4, "block summary smem attribute")) return rr;
  int sms = 0;
  if (int rr = sm_count(&sms)) return rr;
  const int64_t most = static_cast<int64_t>(P.B) * P.tab.max_blocks * P.tab.n_kv;
  const int64_t grid = std::min<int64_t>(most, static_cast<int64_t>(sms) * 12);
  cudaError_t e = launch_pdl(echo::block_summary_kernel<FMT, D>, dim3(static_cast<unsigned>(grid)), dim3(echo::kSumThreads), smem, stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block summary launch");
}

int launch_block_summary(const echo_block_summary_args *a, cudaStream_t stream) {
  echo::SummaryParams P{};
  P.rows = reinterpret_cast<const uint8_t *>(a->rows);
  P.row_bytes = 2 * echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.n_rows = a->n_rows, P.bs = a->block_tokens;
  P.tab = {a->table, a->table_heads, a->max_blocks, a->n_kv_heads};
  P.old_len = a->old_len, P.new_len = a->new_len, P.B = a->B;
  P.summary = reinterpret_cast<uint32_t *>(a->summary);
  P.k_scale = std::ldexp(1.f, -a->k_shift);
  P.status = a->dev_status;
  if (a->format == ECHO_BLOCK_FP4)
    return a->head_dim == 128 ? go_summary<ECHO_BLOCK_FP4, 128>(P, stream) : go_summary<ECHO_BLOCK_FP4, 64>(P, stream);
  return a->head_dim == 128 ? go_summary<ECHO_BLOCK_BF16, 128>(P, stream) : go_summary<ECHO_BLOCK_BF16, 64>(P, stream);
}

int launch_block_scores(const echo_block_scores_args *a, cudaStream_t stream) {
  echo::ScoreParams P{};
  P.q = a->q, P.summary = reinterpret_cast<const uint8_t *>(a->summary);
  P.n_rows = a->n_rows, P.bs = a->block_tokens;
  P.tab = {a->table, a->table_heads, a->max_blocks, a->n_kv_heads};
  P.ctx_len = a->ctx_len;
  P.n_q = a->n_q, P.n_heads = a->n_heads, P.group = a->n_heads / a->n_kv_heads;
  P.pad_log2 = 0;
  while ((1 << P.pad_log2) < P.group && P.pad_log2 <= 3) ++P.pad_log2;
  P.wide = (P.group + 7) & ~7;
  P.cols = P.pad_log2 > 3 ? P.n_q * P.wide : ((P.n_q << P.pad_log2) + 7) & ~7;
  P.chunk = P.pad_log2 > 3 && P.wide <= echo::kScoreCols ? echo::kScoreCols / P.wide * P.wide : echo::kScoreCols;
  P.scale = std::fabs(a->scale), P.q_sign = a->scale < 0.f ? 0x80008000u : 0u;
  P.scores = a->scores, P.status = a->dev_status;
  int sms = 0;
  if (int rr = sm_count(&sms)) return rr;
  // a tile per warp, or more where that still leaves every SM several CTAs
  const int64_t pairs = static_cast<int64_t>(a->B) * a->n_kv_heads, per_cta = echo::kScoreWarps * 16;
  const int64_t ctas = (a->max_blocks + per_cta - 1) / per_cta;
  P.tiles = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ctas, ctas * pairs / (16 * sms))));
  P.ctas = static_cast<int>((ctas + P.tiles - 1) / P.tiles);
  const dim3 grid(static_cast<unsigned>(P.ctas * pairs));
  cudaError_t e = a->head_dim == 128 ? launch_pdl(echo::block_scores_kernel<128>, grid, dim3(echo::kScoreWarps * 32), 0, stream, P)
                                     : launch_pdl(echo::block_scores_kernel<64>, grid, dim3(echo::kScoreWarps * 32), 0, stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block scores launch");
}

template <int T>
static int go_select(const echo::SelectParams &P, int64_t rows, cudaStream_t stream) {
  static std::atomic<bool> attr[kMaxDevices];
  const int64_t smem = (P.tab.max_blocks + (static_cast<int64_t>(P.tab.max_blocks) + T - 1) / T * (T / 32)) * 4;
  if (smem > 40960)
    if (int rr = smem_limit_once(attr, echo::block_select_kernel<T>, 212992, "block selection smem attribute")) return rr;
  cudaError_t e = launch_pdl(echo::block_select_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(T), static_cast<size_t>(smem), stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block selection launch");
}

int launch_block_select(const echo_block_select_args *a, cudaStream_t stream) {
  echo::SelectParams P{};
  P.scores = a->scores, P.ctx_len = a->ctx_len;
  P.n_q = a->n_q, P.bs = a->block_tokens, P.k = a->k, P.first = a->first, P.last = a->last;
  P.tab = {a->table, a->table_heads, a->max_blocks, a->n_kv_heads};
  P.sel = a->sel, P.sel_rows = a->sel_rows, P.len_out = a->len_out, P.status = a->dev_status;
  const int64_t rows = static_cast<int64_t>(a->B) * a->n_q * a->n_kv_heads;
  if (a->max_blocks <= 1024) return go_select<128>(P, rows, stream);
  if (a->max_blocks <= 8192) return go_select<256>(P, rows, stream);
  return go_select<1024>(P, rows, stream);
}

}  // namespace echo_host
