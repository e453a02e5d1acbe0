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
//   Summary: a warp per (block, KV head), or a CTA where blocks are large: 16-byte loads of its keys, eight
//     a lane under way, packed minima and maxima, joined over the lanes.  The blocks that changed are one
//     line over the requests, found by every CTA from the lengths.  8 prompts of 16384 tokens (8 KV heads of
//     128 dims, bf16, blocks of 64): 39-41 us, 4.5-4.75 TB/s; one more token for 64 requests: 5.4 us, three chained
//     loads (length, id, keys) and a launch.
//   Scores: 16 blocks x 8 columns with mma.m16n8k16.  The order of a contraction's dims is free,
//     so a lane reads 16 contiguous bytes of "its" two blocks per 8 dims of a quarter and feeds them
//     as they are: a warp has the 16 summaries (8 KB) in registers after one round of loads, with
//     no shared memory.  The 8 columns are the heads of one query token, or of several where a
//     group has fewer, so the maximum over a group stays within a quad.
//     64 requests of up to 131072 tokens, blocks of 64, 64 heads on 8 of 128 dims: 70 us, 0.89 of the copy
//     rate; 16 of them 22-23 us (0.70: start and end), 17 where L2 still has the summaries.  Many query tokens (512 of them against 1024 blocks: 97 us, 177 TFLOP/s) are bound by
//     instructions, 235 for 16 products of 8 columns; the tensor cores' own operands in shared memory would
//     serve them better.
//   Selection: one to 32 warps per (query, KV head), a thread with 4 to 32 blocks that follow one another,
//     their scores in registers.  The k-th best is found from counts over the range of the scores
//     (block_pick.cuh), then a sum over the threads gives each the place of what it writes: those above,
//     and the first of its equals.
//     8000 rows of 1024 blocks: 30 us, bound by instructions (the pipe of comparisons 63% busy); 256 rows of
//     2048: 6.5 us, of which a launch and the chain of loads, counts and barriers are nearly all.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "block_mma.cuh"
#include "block_pick.cuh"

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
  // (the sum passes 31 bits for the longest contexts in blocks of more than 1024 tokens)
  return make_int2(min(o, n) / P.bs, (static_cast<uint32_t>(n) + P.bs - 1) / static_cast<uint32_t>(P.bs));
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

// TEAM threads take a block: a warp, or the CTA
template <int FMT, int D, int TEAM>
__global__ void __launch_bounds__(kSumThreads) block_summary_kernel(const SummaryParams P) {
  constexpr bool kFp4 = FMT == ECHO_BLOCK_FP4;
  constexpr int kWords = kFp4 ? 16 : 4;               // pairs of dims that a thread holds
  constexpr int kLanes = D / (2 * kWords);            // threads of a token
  constexpr int kTeams = kSumThreads / TEAM;
  constexpr int kTokens = TEAM / kLanes;              // tokens a round
  constexpr int kRounds = 8;                          // rounds of loads in flight
  extern __shared__ int32_t sum_cu[];                 // [B + 1] exclusive sums of the redone blocks
  __shared__ uint32_t part[TEAM == 32 ? 1 : 4][2][D / 2];
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

  const int t0 = tid % TEAM / kLanes, c = tid % kLanes;
  // where a (block, KV head) lies and how many tokens it has; row -1: past the end, or not there
  int64_t row = -1, next_row = -1;
  int n = 0, next_n = 0;
  auto look_up = [&](int64_t u) {
    next_row = -1;
    if (u >= units) return;
    const int line = static_cast<int>(u / P.tab.n_kv), h = static_cast<int>(u - static_cast<int64_t>(line) * P.tab.n_kv);
    int b = 0, end = P.B;
    while (end - b > 1) {
      const int mid = (b + end) >> 1;
      if (sum_cu[mid] <= line) b = mid;
      else end = mid;
    }
    const int e = redone(P, b, false).x + line - sum_cu[b];
    next_row = P.tab.row(b, h, e);
    next_n = min(P.bs, held_len(P.new_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, nullptr, false) - e * P.bs);
  };
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kTeams + tid / TEAM, stride = static_cast<int64_t>(gridDim.x) * kTeams;
  look_up(u0);
  for (int64_t u = u0; u < units; u += stride) {
    row = next_row, n = next_n;
    if (row < 0 || row >= P.n_rows) {  // (the same for the whole team)
      if (row >= 0 && tid % TEAM == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
      look_up(u + stride);
      continue;
    }
    // (lanes past the last token read it again: a minimum does not mind)
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
        if (t + r * kTokens >= n) break;
        if constexpr (kFp4) {
          const uint8_t *sub = src + (tk / kSubTokens) * Fp4Sub<D>::kBytes;
          x[r] = load16_here(sub + (tk % kSubTokens) * (D / 2) + c * 16);
          sc[r] = load2_here(sub + Fp4Sub<D>::kKeyScales + (tk % kSubTokens) * (D / 16) + c * 2);
        } else {
          x[r] = load16_here(src + tk * (2 * D) + c * 16);
        }
      }
      if (t == 0) look_up(u + stride);  // (while the loads are under way)
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (t + r * kTokens >= n) break;
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
    if constexpr (TEAM == 32) {
      // Joined over the lanes of the same dims, each of which hands half of its words over and keeps the
      // other: minima, and maxima as minima of what is less, first (4 bits: 28 shuffles a lane, not 96).
      // What is left are D / 32 words from word `at` on: one store.
      constexpr int kLeft = 2 * kWords / kTokens;
      const uint32_t flip = lane & 16 ? 0x80008000u : 0u;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t less = hi[i] ^ 0x80008000u, give = lane & 16 ? lo[i] : less;
        lo[i] = min2<FMT>(lane & 16 ? less : lo[i], __shfl_xor_sync(~0u, give, 16));
      }
      int at = c * kWords;
#pragma unroll
      for (int d = 8, k = kWords / 2; d >= kLanes; d >>= 1, k >>= 1) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const uint32_t give = lane & d ? lo[i] : lo[i + k];
          lo[i] = min2<FMT>(lane & d ? lo[i + k] : lo[i], __shfl_xor_sync(~0u, give, d));
        }
        if (lane & d) at += k;
      }
      uint32_t v[kLeft];
#pragma unroll
      for (int i = 0; i < kLeft; ++i) {  // (4 bits: 6 significant ones, exact in bf16, a power of two less too)
        v[i] = lo[i] ^ flip;
        if constexpr (kFp4) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
          v[i] = pack2<false>(f.x * P.k_scale, f.y * P.k_scale);
        }
      }
      uint32_t *dst = P.summary + row * D + (lane & 16 ? D / 2 : 0) + at;
      if constexpr (kLeft == 4) *reinterpret_cast<uint4 *>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
      else *reinterpret_cast<uint2 *>(dst) = make_uint2(v[0], v[1]);
    } else {
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
        P.summary[row * D + tid] = v;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
constexpr int kScoreWarps = 4;
constexpr int kScoreCols = 64;  // query columns that a CTA lays out at a time
constexpr int kScoreAhead = 4;  // 16-byte pieces of them that a thread has under way

struct ScoreParams {
  const uint16_t *q;
  const uint8_t *summary;
  int32_t n_rows, bs;
  BlockTable tab;
  const int32_t *ctx_len;
  int32_t n_q, n_heads, group;
  int32_t cols;           // columns of a KV head, a multiple of 8
  int32_t wide;           // columns of a query token where the group has more than 8 heads
  int32_t chunk;          // columns laid out at a time: whole query tokens if they fit
  int32_t ctas, tiles;    // CTAs along the blocks of a (b, h), 16-block tiles that a warp of one takes
  int32_t parts, span;    // CTAs along its columns, columns that one takes (whole chunks)
  float scale;            // |scale|
  uint32_t q_sign;
  float *scores;
  int32_t *status;
};

// PAD: a query token has 2^PAD columns, of which `group` or fewer differ; 4: P.wide columns
template <int D, int PAD>
__global__ void __launch_bounds__(kScoreWarps * 32, 4) block_scores_kernel(const ScoreParams P) {
  constexpr int kStride = 4 * D + 64;       // bytes of a column; + 64: its quads on other banks
  constexpr int kChunks = D / 16;           // 16-byte pieces of a summary row that a lane holds
  __shared__ __align__(16) uint8_t qs[kScoreCols * kStride];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  // (the KV heads of the same blocks beside one another: their rows are neighbours in memory)
  const int bp = blockIdx.x / P.tab.n_kv, h = blockIdx.x - bp * P.tab.n_kv;
  const int line = bp / P.parts, c_from = (bp - line * P.parts) * P.span;
  const int b = line / P.ctas, part = line - b * P.ctas;
  pdl_launch_dependents();
  pdl_wait();
  const int len = held_len(P.ctx_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, P.status,
                           part == 0 && h == 0 && c_from == 0 && threadIdx.x == 0);
  // (a block may have any number of tokens: the sum passes 31 bits)
  const int blocks = (static_cast<uint32_t>(len) + P.bs - 1) / static_cast<uint32_t>(P.bs), c_end = min(c_from + P.span, P.cols);
  const int first = part * (kScoreWarps * 16) * P.tiles;
  if (first >= blocks) return;

  // summaries of blocks r8 and r8 + 8 of a tile; their rows are looked up a tile ahead
  uint4 a[2][kChunks];
  int64_t row[2];
  bool there[2];
  auto look_up = [&](int t) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = first + (t * kScoreWarps + warp) * 16 + r8 + 8 * k;
      row[k] = t < P.tiles && e < blocks ? P.tab.row(b, h, e) : -1;
    }
  };
  auto load = [&](int t) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (row[k] >= P.n_rows) set_status(P.status, ECHO_DEV_BAD_INDEX);
      there[k] = row[k] >= 0 && row[k] < P.n_rows;
      const uint8_t *src = P.summary + (there[k] ? row[k] : 0) * (4 * D) + c4 * 32;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        a[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (there[k]) a[k][i] = load16_here(src + i / 2 * 128 + i % 2 * 16);
      }
    }
    look_up(t + 1);
  };

  for (int c0 = c_from; c0 < c_end; c0 += P.chunk) {
    const int nc = min(P.chunk, c_end - c0);
    if (c0 == c_from || P.tiles > 1) {   // (a single tile stays in the registers)
      look_up(0);
      load(0);     // (under way while the queries are laid out)
    }
    if (c0 != c_from) __syncthreads();
    // [q-, q+] of the columns; a group's last head fills its padding (a maximum does not mind)
    for (int i0 = threadIdx.x; i0 < nc * (D / 8); i0 += kScoreAhead * kScoreWarps * 32) {
      uint4 x[kScoreAhead];
#pragma unroll
      for (int r = 0; r < kScoreAhead; ++r) {
        const int i = i0 + r * kScoreWarps * 32, cc = c0 + i / (D / 8);
        if (i >= nc * (D / 8)) break;
        int j, g;
        if constexpr (PAD <= 3) {
          j = cc >> PAD, g = cc & ((1 << PAD) - 1);
        } else {
          j = cc / P.wide, g = cc - j * P.wide;
        }
        j = min(j, P.n_q - 1), g = min(g, P.group - 1);
        x[r] = load16_here(P.q + ((static_cast<int64_t>(b) * P.n_q + j) * P.n_heads + h * P.group + g) * D + i % (D / 8) * 8);
      }
#pragma unroll
      for (int r = 0; r < kScoreAhead; ++r) {
        const int i = i0 + r * kScoreWarps * 32, col = i / (D / 8), d8 = i % (D / 8);
        if (i >= nc * (D / 8)) break;
        uint32_t w[4] = {x[r].x ^ P.q_sign, x[r].y ^ P.q_sign, x[r].z ^ P.q_sign, x[r].w ^ P.q_sign}, n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t neg = ((w[k] >> 15) & 0x10001u) * 0xffffu;  // all ones in the halves below zero
          n[k] = w[k] & neg, w[k] &= ~neg;
        }
        // piece 4 i + c is what lane c of a quad feeds with its i-th: it reads 32 bytes (a sector) of every 128
        uint8_t *dst = qs + col * kStride + (4 * (d8 / 8 * 2 + d8 % 2) + d8 % 8 / 2) * 16;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(n[0], n[1], n[2], n[3]);
        *reinterpret_cast<uint4 *>(dst + 2 * D) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();
    for (int t = 0; t < P.tiles; ++t) {
      const int e0 = first + (t * kScoreWarps + warp) * 16;
      if (e0 >= blocks) break;
      const bool held[2] = {there[0], there[1]};
      // the score of block r8 + 8 k of the tile for query token j, if the token sees the block's first one
      auto put = [&](int j, int k, float v, bool more) {
        const int e = e0 + r8 + 8 * k;
        if (j >= P.n_q || e >= blocks || e * P.bs >= len - (P.n_q - 1 - j)) return;
        float *dst = P.scores + ((static_cast<int64_t>(b) * P.n_q + j) * P.tab.n_kv + h) * P.tab.max_blocks + e;
        v = (k ? held[1] : held[0]) ? v * P.scale : -INFINITY;
        *dst = more ? fmaxf(v, *dst) : v;   // (more: heads of an earlier chunk, written by this thread)
      };
      float best[2] = {-INFINITY, -INFINITY};  // (PAD 4: of a token's columns so far)
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
        if (cg + 8 >= nc && t + 1 < P.tiles) load(t + 1);   // (the registers are free)
        // acc[p + 2 k]: column 2 c4 + p of block k.  One value per (query token, block)
        if constexpr (PAD == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k) put(c0 + cg + 2 * c4, k, acc[2 * k], false), put(c0 + cg + 2 * c4 + 1, k, acc[1 + 2 * k], false);
        } else {
          float v[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            v[k] = fmaxf(acc[2 * k], acc[1 + 2 * k]);
            if (PAD >= 2) v[k] = fmaxf(v[k], __shfl_xor_sync(~0u, v[k], 1));
            if (PAD >= 3) v[k] = fmaxf(v[k], __shfl_xor_sync(~0u, v[k], 2));
          }
          if constexpr (PAD == 1) {
            const int j = (c0 + cg + 2 * c4) >> 1;
            put(j, 0, v[0], false), put(j, 1, v[1], false);
          } else if constexpr (PAD <= 3) {   // (two lanes or four have them both: one writes each)
            const int j = (c0 + cg + 2 * c4) >> PAD;
            if (c4 % (1 << (PAD - 1)) < 2) put(j, c4 & 1, c4 & 1 ? v[1] : v[0], false);
          } else {
            best[0] = fmaxf(best[0], v[0]), best[1] = fmaxf(best[1], v[1]);
            const int at = c0 + cg, j = at / P.wide;
            if (at + 8 == (j + 1) * P.wide || cg + 8 == nc) {
              if (c4 < 2) put(j, c4, c4 ? best[1] : best[0], j * P.wide < c0);
              best[0] = best[1] = -INFINITY;
            }
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
constexpr int kSelBins = 256;               // parts of a row's range of scores
constexpr int kSelRows = 4;                 // rows of a CTA that takes one per warp

struct SelectParams {
  const float *scores;
  const int32_t *ctx_len;
  uint32_t n;         // rows: (query, KV head)
  int32_t n_q, bs, k, first, last;
  BlockTable tab;     // (table: optional)
  int32_t ids, more;  // block ids below `ids` have a row for each KV head, id `ids` for heads below `more` (a
                      // table of each head's rows: 0)
  int32_t *sel, *sel_rows, *len_out;
  int32_t vec;        // rows of `scores` and of the table lie on 16-byte boundaries
  int32_t *status;
};

// W warps a row (one: kSelRows rows a CTA), R blocks a thread, one after another: the order within a
// thread is then free, and one sum over the threads gives each its place in the list
template <int W, int R>
__global__ void __launch_bounds__(W == 1 ? kSelRows * 32 : W * 32) block_select_kernel(const SelectParams P) {
  __shared__ PickSpace<W, kSelBins> space[W == 1 ? kSelRows : 1];
  __shared__ uint32_t cnt[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = W == 1 ? lane : threadIdx.x;
  const uint32_t row = W == 1 ? blockIdx.x * kSelRows + warp : blockIdx.x;   // (rows: below 2^31)
  auto &S = space[W == 1 ? warp : 0];
  pdl_launch_dependents();
  pdl_wait();
  if (row >= P.n) return;
  const int bj = row / static_cast<uint32_t>(P.tab.n_kv), h = row - bj * P.tab.n_kv;
  const int b = static_cast<uint32_t>(bj) / static_cast<uint32_t>(P.n_q), j = bj - b * P.n_q;
  const float *src = P.scores + static_cast<int64_t>(row) * P.tab.max_blocks;
  const int ctx = held_len(P.ctx_len[b], static_cast<int64_t>(P.tab.max_blocks) * P.bs, P.status, j == 0 && h == 0 && tid == 0);
  const int len = max(ctx - (P.n_q - 1 - j), 0), nb = (static_cast<uint32_t>(len) + P.bs - 1) / static_cast<uint32_t>(P.bs);
  if (P.len_out && h == 0 && tid == 0) P.len_out[bj] = len;

  // Scores of blocks i0 and up; NaN: not to be chosen by its score (a block that is not there or not held,
  // or one of `must`, which is taken in any case); a score that is NaN becomes -inf
  const int i0 = tid * R;
  float score[R], lo = INFINITY, hi = -INFINITY;  // (range of the finite ones)
  uint32_t must = 0, n_ok = 0, n_must;
  pick_clear(S);
  const int32_t ids_end = P.tab.table ? P.ids + (h < P.more) : 1;   // of this head's entries
  const int32_t *ids = P.tab.table ? P.tab.table + (static_cast<int64_t>(b) * P.tab.heads + (P.tab.heads > 1 ? h : 0)) * P.tab.max_blocks : nullptr;
  {
    // (all loads before the first use, not one by one where the branches below want them)
    int32_t id[R];
#pragma unroll
    for (int r = 0; r < R; ++r) score[r] = 0.f, id[r] = 0;
    if (P.vec) {
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        if (i0 + r >= nb) break;
        const uint4 x = load16_here(src + i0 + r);
        score[r] = __uint_as_float(x.x), score[r + 1] = __uint_as_float(x.y);
        score[r + 2] = __uint_as_float(x.z), score[r + 3] = __uint_as_float(x.w);
        if (ids) {
          const uint4 y = load16_here(ids + i0 + r);
          id[r] = y.x, id[r + 1] = y.y, id[r + 2] = y.z, id[r + 3] = y.w;
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (i0 + r >= nb) break;
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(score[r]) : "l"(src + i0 + r));
        if (ids) asm volatile("ld.global.s32 %0, [%1];" : "=r"(id[r]) : "l"(ids + i0 + r));
      }
    }
    const uint32_t plain = max(nb - P.first - P.last, 0);   // blocks that are neither of the first nor of the last
    int32_t top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = i0 + r < nb && static_cast<uint32_t>(id[r]) < static_cast<uint32_t>(ids_end);
      const bool by_score = static_cast<uint32_t>(i0 + r - P.first) < plain;
      if (i0 + r < nb) top = max(top, id[r]);
      float s = score[r] == score[r] ? score[r] : -INFINITY;
      must |= there && !by_score ? 1u << r : 0u;
      s = there && by_score ? s : NAN;
      n_ok += s == s;
      if (fabsf(s) < INFINITY) lo = fminf(lo, s), hi = fmaxf(hi, s);
      score[r] = s;
    }
    if (ids && top >= ids_end) set_status(P.status, ECHO_DEV_BAD_INDEX);
  }
  static_assert(R <= 32, "a bit of `must` each");
  {  // (counts of 32768 at most: both in one word)
    uint32_t both = n_ok | __popc(must) << 16, k0 = score_key(lo), k1 = score_key(hi);
    pick_stats(S, both, k0, k1);
    n_ok = both & 0xffffu, n_must = both >> 16, lo = key_score(k0), hi = key_score(k1);
  }

  // ----- the score above which all are taken, and how many of its equals -----
  const uint32_t want = P.k - n_must;  // (first + last <= k)
  float thr = -INFINITY;
  uint32_t need = ~0u >> 1;            // (all of them)
  if (want == 0) {
    thr = INFINITY, need = 0;
  } else if (n_ok > want) {
    // 256 equal parts of the scores' range; an infinite score goes to an end
    const float step = hi > lo ? fminf(kSelBins / (hi - lo), 3e38f) : 0.f, from = -lo * step;
    auto each = [&](auto &&f) {
#pragma unroll
      for (int r = 0; r < R; ++r) f(score[r]);
    };
    auto bin = [&](float s) { return static_cast<int>(min(__float2uint_rz(fmaf(s, step, from)), kSelBins - 1u)); };
    uint32_t key;
    pick_kth(S, want, each, [](float s) { return s == s; }, bin, [](float s) { return score_key(s); }, key, need);
    // The search by halving may end at a key that no score has, with none of its equals needed.  All but one of
    // them are floats between two scores; 0x7fffffff, between the keys of zero and of the largest number below
    // it, would be -0.0, which equals zero: the key of that number parts them as well.
    thr = key_score(key - (key == 0x7fffffffu));
  }

  // ----- the blocks in order -----
  int32_t *sel = P.sel + static_cast<int64_t>(row) * P.k, *rows = P.sel_rows ? P.sel_rows + static_cast<int64_t>(row) * P.k : nullptr;
  uint32_t gt = must, eq = 0;   // above the threshold, and equal to it
#pragma unroll
  for (int r = 0; r < R; ++r) gt |= score[r] > thr ? 1u << r : 0u, eq |= score[r] == thr ? 1u << r : 0u;
  const uint32_t mine = __popc(gt) | __popc(eq) << 16;
  uint32_t at = mine, taken;     // of the blocks before the thread's, and of all
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(~0u, at, d);
    if (lane >= d) at += x;
  }
  if constexpr (W > 1) {
    if (lane == 31) cnt[warp] = at;
    __syncthreads();
    const uint32_t x = lane < W ? cnt[lane % W] : 0u;
    at += __reduce_add_sync(~0u, lane < warp ? x : 0u), taken = __reduce_add_sync(~0u, x);
  } else {
    taken = __shfl_sync(~0u, at, 31);
  }
  at -= mine;
  for (uint32_t m = gt | eq; m; m &= m - 1) {
    const int r = __ffs(m) - 1;
    const bool equal = eq >> r & 1;
    const uint32_t q = at >> 16, to = (at & 0xffffu) + min(q, need);
    if (!equal || q < need) {
      sel[to] = i0 + r;
      if (rows) rows[to] = P.tab.heads > 1 ? ids[i0 + r] : ids[i0 + r] * P.tab.n_kv + h;
    }
    at += equal ? 0x10000u : 1u;
  }
  const int n = (taken & 0xffffu) + min(taken >> 16, need);
  for (int i = n + tid; i < P.k; i += W * 32) {
    sel[i] = -1;
    if (rows) rows[i] = -1;
  }
}

}  // namespace echo

namespace echo_host {

template <int FMT, int D, int TEAM>
static int go_summary(const echo::SummaryParams &P, cudaStream_t stream) {
  static std::atomic<bool> attr[kMaxDevices];
  const int smem = (P.B + 1) * 4;
  if (smem > 40960)
    if (int rr = smem_limit_once(attr, echo::block_summary_kernel<FMT, D, TEAM>, (16384 + 1) * 4, "block summary smem attribute")) return rr;
  int sms = 0;
  if (int rr = sm_count(&sms, "block selection device")) return rr;
  const int64_t most = static_cast<int64_t>(P.B) * P.tab.max_blocks * P.tab.n_kv;
  constexpr int kTeams = echo::kSumThreads / TEAM;
  const int64_t ctas = (most + kTeams - 1) / kTeams;
  const int64_t grid = std::min<int64_t>(ctas, static_cast<int64_t>(sms) * 16);
  cudaError_t e = launch_pdl(echo::block_summary_kernel<FMT, D, TEAM>, dim3(static_cast<unsigned>(grid)), dim3(echo::kSumThreads), smem, stream, P);
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
  // A warp a block: no barriers, and no threads without a token (8 prompts of 16384 tokens, 8 KV heads of
  // 128 dims, bf16, blocks of 16 / 32 / 64: 86 / 52 / 41 us by CTAs, 42 / 40 / 40 by warps; in 4 bits
  // blocks of 64 took 45, take 26).  Larger blocks of bf16 by CTAs: a warp has 16 keys under way at once,
  // and a step that changes one block of each request would wait for all of it.
  if (a->format == ECHO_BLOCK_FP4)
    return a->head_dim == 128 ? go_summary<ECHO_BLOCK_FP4, 128, 32>(P, stream) : go_summary<ECHO_BLOCK_FP4, 64, 32>(P, stream);
  if (a->block_tokens * a->head_dim <= 64 * 128)
    return a->head_dim == 128 ? go_summary<ECHO_BLOCK_BF16, 128, 32>(P, stream) : go_summary<ECHO_BLOCK_BF16, 64, 32>(P, stream);
  return a->head_dim == 128 ? go_summary<ECHO_BLOCK_BF16, 128, echo::kSumThreads>(P, stream)
                            : go_summary<ECHO_BLOCK_BF16, 64, echo::kSumThreads>(P, stream);
}

int launch_block_scores(const echo_block_scores_args *a, cudaStream_t stream) {
  echo::ScoreParams P{};
  P.q = a->q, P.summary = reinterpret_cast<const uint8_t *>(a->summary);
  P.n_rows = a->n_rows, P.bs = a->block_tokens;
  P.tab = {a->table, a->table_heads, a->max_blocks, a->n_kv_heads};
  P.ctx_len = a->ctx_len;
  P.n_q = a->n_q, P.n_heads = a->n_heads, P.group = a->n_heads / a->n_kv_heads;
  int pad = 0;
  while ((1 << pad) < P.group && pad <= 3) ++pad;
  P.wide = (P.group + 7) & ~7;
  P.cols = pad > 3 ? P.n_q * P.wide : ((P.n_q << pad) + 7) & ~7;
  P.chunk = pad > 3 && P.wide <= echo::kScoreCols ? echo::kScoreCols / P.wide * P.wide : echo::kScoreCols;
  P.scale = std::fabs(a->scale), P.q_sign = a->scale < 0.f ? 0x80008000u : 0u;
  P.scores = a->scores, P.status = a->dev_status;
  int sms = 0;
  if (int rr = sm_count(&sms, "block selection device")) return rr;
  // a tile per warp, or more where that still leaves every SM the 4 CTAs that it holds at once (16 requests of
  // 131072 tokens, 8 KV heads, from L2: 17 us; with 3 or 12 CTAs an SM 21 and 19)
  const int64_t pairs = static_cast<int64_t>(a->B) * a->n_kv_heads, per_cta = echo::kScoreWarps * 16;
  const int64_t ctas = (a->max_blocks + per_cta - 1) / per_cta;
  P.tiles = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, ctas * pairs / (4 * sms))));
  P.ctas = static_cast<int>((ctas + P.tiles - 1) / P.tiles);
  // columns (a prompt's query tokens) over several CTAs where blocks and heads give the SMs too few; a
  // token whose heads do not fit one chunk stays with one thread, which joins them
  const int64_t chunks = (P.cols + P.chunk - 1) / P.chunk, want = (12ll * sms + P.ctas * pairs - 1) / (P.ctas * pairs);
  const int64_t each = P.wide > echo::kScoreCols ? chunks : (chunks + std::min(chunks, want) - 1) / std::min(chunks, want);
  P.span = static_cast<int>(each * P.chunk), P.parts = static_cast<int>((chunks + each - 1) / each);
  const dim3 grid(static_cast<unsigned>(P.ctas * pairs * P.parts));
  auto go = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    auto *kernel = pad == 0 ? echo::block_scores_kernel<D, 0> : pad == 1 ? echo::block_scores_kernel<D, 1>
                 : pad == 2 ? echo::block_scores_kernel<D, 2> : pad == 3 ? echo::block_scores_kernel<D, 3> : echo::block_scores_kernel<D, 4>;
    return launch_pdl(kernel, grid, dim3(echo::kScoreWarps * 32), 0, stream, P);
  };
  cudaError_t e = a->head_dim == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block scores launch");
}

template <int W, int R>
static int go_select(const echo::SelectParams &P, cudaStream_t stream) {
  const uint32_t ctas = W == 1 ? (P.n + echo::kSelRows - 1) / echo::kSelRows : P.n;
  cudaError_t e = launch_pdl(echo::block_select_kernel<W, R>, dim3(ctas), dim3(W == 1 ? echo::kSelRows * 32 : W * 32), 0,
                             stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block selection launch");
}

int launch_block_select(const echo_block_select_args *a, cudaStream_t stream) {
  echo::SelectParams P{};
  P.scores = a->scores, P.ctx_len = a->ctx_len;
  P.n = static_cast<uint32_t>(a->B) * a->n_q * a->n_kv_heads;   // (below 2^31)
  P.n_q = a->n_q, P.bs = a->block_tokens, P.k = a->k, P.first = a->first, P.last = a->last;
  P.tab = {a->table, a->table_heads, a->max_blocks, a->n_kv_heads};
  const int32_t rows = a->n_rows > 0 ? a->n_rows : 0x7fffffff, heads = a->table_heads > 1 ? 1 : a->n_kv_heads;
  P.ids = rows / heads, P.more = rows % heads;
  P.sel = a->sel, P.sel_rows = a->sel_rows, P.len_out = a->len_out, P.status = a->dev_status;
  P.vec = a->max_blocks % 4 == 0 && reinterpret_cast<uintptr_t>(a->scores) % 16 == 0 && reinterpret_cast<uintptr_t>(a->table) % 16 == 0;
  // the keys of a row in the registers of the threads that hold them: 8 or 16 each where rows fill the SMs
  // (8000 rows of 512 blocks: one warp 15.2 us, two 17.6, four 23.3), fewer each where they do not and a
  // thread's own keys are what a row waits for (256 rows of 4096: 16 warps 6.6 us, 8 warps 8.5).  Both of
  // 1024 blocks: 256 rows 4.6 and 4.4 us, 32 rows 3.6 and 3.9, 4000 rows 22.1 and 16.4
  int sms = 0;
  if (int rr = sm_count(&sms, "block selection device")) return rr;
  const bool few = P.n <= 4u * sms;
  if (a->max_blocks <= 256) return go_select<1, 8>(P, stream);
  if (a->max_blocks <= 512) return few ? go_select<4, 4>(P, stream) : go_select<1, 16>(P, stream);
  if (a->max_blocks <= 1024) return few ? go_select<8, 4>(P, stream) : go_select<4, 8>(P, stream);
  if (a->max_blocks <= 2048) return go_select<8, 8>(P, stream);
  if (a->max_blocks <= 4096) return few ? go_select<16, 8>(P, stream) : go_select<8, 16>(P, stream);
  if (a->max_blocks <= 8192) return go_select<32, 8>(P, stream);
  if (a->max_blocks <= 16384) return go_select<32, 16>(P, stream);
  return go_select<32, 32>(P, stream);
}

}  // namespace echo_host
