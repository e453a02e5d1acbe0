// block_evict.cu -- the softmax weight that each cached token gathers, and the eviction that
// keeps the heaviest tokens of a request.
//
// Gathered weight of token p of (b, KV head h), over the call's query tokens j and the group's
// heads g, with the log-sum-exp that the attention returned:
//   acc'_p = decay * acc_p + sum_{j: p < len_j} sum_g exp(scale * q_jg . k_p - lse_jg)
// One read of the keys (the values are not needed), 2 D bytes a token in bf16, against
// 2 D flops and one exponential per query row.
//
// Eviction to `keep` tokens: the first `sinks` slots and the tokens of the last `recent`
// positions stay, then the heaviest, ties to the lower slot.  Of n = len slots, those below
// `keep` whose token goes are holes, and as many tokens at or above `keep` stay; the i-th hole
// takes the i-th of them.  Sources lie at or above `keep`, targets below, so the moves need no
// order, and a call that is repeated on the same inputs does the same again.
//
// sm_103a design.
//   Weights: S^T = K Q^T with mma.m16n8k16, tokens as the 16 rows and query rows as the 8
//     columns.  A contraction's dims may come in any order, so a lane reads 16 contiguous bytes
//     of its token's key and feeds them as they are (4-bit rows: 16 bytes of codes, converted in
//     place); keys go from memory to registers with nothing in between, two sub-blocks of 16
//     tokens a warp at a time (4 bits: one, and the codes of four under way), the exponentials of a
//     column summed over the quad; a lane adds what its token had, read a round ahead.  16 requests of up to
//     32768 tokens, 64 heads on 8 of 128 dims: bf16 130 us (0.96 of the copy rate; 138 to 146 on new inputs
//     every call), 4 bits 74 us (0.51: conversions and products; what a token had, read where it was added, cost another 50).
//   Eviction: a CTA per (b, h) finds the weight of the last token that stays from counts over the
//     range of the weights (block_pick.cuh), and lists holes and movers in order; the
//     moves follow in the same CTA when they are few, else in a second kernel over the whole GPU.
//     8 prompts of 32768 tokens cut to 4096 (8 KV heads, bf16): 70 us, 27 for the lists (64 CTAs, each a
//     chain of passes: keys 8, the threshold 6, marks 4, lists 3, weights 3) and 43 for 240 MB of moves; 32
//     requests of 4100 cut to 4096: 12.5 us, the same chain.
#include <algorithm>
#include <cmath>

#include "block_mma.cuh"
#include "block_pick.cuh"

namespace echo {

// ---------------------------------------------------------------------------
// gathered weights
// ---------------------------------------------------------------------------
constexpr int kWtWarps = 4;
constexpr int kWtCols = 64;   // query columns that a CTA lays out at a time

struct WeightParams {
  const uint16_t *q;
  const uint8_t *rows;
  int64_t row_bytes;
  int32_t n_rows, bsub;
  const int32_t *table;
  int32_t table_heads, max_blocks;
  const int32_t *ctx_len, *old_len;
  int32_t n_q, n_heads, n_kv, group;
  float scale_log2;            // |scale| log2 e, over the keys' power of two
  uint32_t q_sign;
  const float *lse, *acc;
  float *acc_out;
  float decay;
  int32_t ctas, subs;          // CTAs of a (b, h), sub-blocks that a warp of one takes (even, at most 32)
  int32_t *status;
};

template <int FMT, int D>
__global__ void __launch_bounds__(kWtWarps * 32, 4) block_weights_kernel(const WeightParams P) {
  constexpr bool F16 = FMT == ECHO_BLOCK_FP4;
  constexpr int kStride = 2 * D + 64;               // bytes of a column; + 64: its quads on other banks
  constexpr int kPieces = D / 32;                   // 16-byte pieces of a column's dims per lane
  constexpr int kLoads = F16 ? 1 : kPieces;         // 16-byte loads of a token per lane (4 bits, D = 64: 8 bytes)
  constexpr int kU = F16 ? 1 : 2;                   // sub-blocks of a step
  constexpr int kDeep = F16 ? 4 : 1;                // steps whose loads are under way
  constexpr int kRun = kU * kDeep;                  // sub-blocks of a round of them
  constexpr int kOut = kRun / 2;                    // tokens of a round per lane: lane, lane + 32, ...
  __shared__ __align__(16) uint8_t qs[kWtCols * kStride];
  __shared__ float2 col[kWtCols];                   // scale and lse of a column, both times log2 e
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  const int pair = blockIdx.x / P.ctas, part = blockIdx.x - pair * P.ctas;
  const int b = pair / P.n_kv, h = pair - b * P.n_kv;
  pdl_launch_dependents();
  pdl_wait();
  const int most = P.max_blocks * P.bsub * kSubTokens;
  int len = P.ctx_len[b];
  if (len > most) {
    if (part == 0 && h == 0 && threadIdx.x == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
    len = most;
  }
  const int nsub = (max(len, 0) + kSubTokens - 1) / kSubTokens;
  const int first = part * kWtWarps * P.subs;
  if (first >= nsub) return;
  const int s0 = first + warp * P.subs, s1 = min(s0 + P.subs, nsub);
  const int old = P.old_len ? min(max(P.old_len[b], 0), len) : P.acc ? len : 0;
  const int rows_q = P.n_q * P.group;

  // where this lane's sub-block of the warp's run lies
  int64_t where = -1;
  if (s0 + lane < s1) {
    const int e = (s0 + lane) / P.bsub, in = s0 + lane - e * P.bsub;
    const int32_t id = P.table[(static_cast<int64_t>(b) * P.table_heads + (P.table_heads > 1 ? h : 0)) * P.max_blocks + e];
    const int64_t row = id < 0 ? -1 : P.table_heads > 1 ? id : static_cast<int64_t>(id) * P.n_kv + h;
    if (row >= P.n_rows) set_status(P.status, ECHO_DEV_BAD_INDEX);
    else if (row >= 0) where = row * P.row_bytes + static_cast<int64_t>(in) * (F16 ? Fp4Sub<D>::kBytes : kSubTokens * D * 2);
  }
  const int64_t out0 = (static_cast<int64_t>(b) * P.n_kv + h) * most;

  // tokens r8 and r8 + 8 of each sub-block
  uint4 a[kDeep][kU][2][kLoads];
  uint32_t sc[kDeep][kU][2];
  bool held[kDeep][kU];
  auto load = [&](auto &a, auto &sc, auto &held, int s) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      int64_t at = __shfl_sync(~0u, where, (s - s0 + u) & 31);
      if (s + u >= s1) at = -1;
      held[u] = at >= 0;
      const uint8_t *src = P.rows + (at < 0 ? 0 : at);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int tk = r8 + 8 * k;
        sc[u][k] = 0;
        if constexpr (F16) {
          a[u][k][0] = make_uint4(0u, 0u, 0u, 0u);
          if (at >= 0) {
            if constexpr (D == 128) {
              a[u][k][0] = load16_here(src + tk * (D / 2) + c4 * 16);
              sc[u][k] = load2_here(src + Fp4Sub<D>::kKeyScales + tk * (D / 16) + c4 * 2);
            } else {
              const uint2 y = load8_here(src + tk * (D / 2) + c4 * 8);
              a[u][k][0].x = y.x, a[u][k][0].y = y.y;
              sc[u][k] = load1_here(src + Fp4Sub<D>::kKeyScales + tk * (D / 16) + c4);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            a[u][k][i] = make_uint4(0u, 0u, 0u, 0u);
            if (at >= 0) a[u][k][i] = load16_here(src + tk * (2 * D) + (i / 2 * 8 + c4 * 2 + i % 2) * 16);
          }
        }
      }
    }
  };

  // what the tokens of a round gathered before, a round ahead
  float before[kOut], before_next[kOut];
  const int end = min(len, s1 * kSubTokens);
  auto load_before = [&](int s) {
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const int p = s * kSubTokens + 32 * i + lane;
      before_next[i] = 0.f;
      if (p < min(old, end)) asm volatile("ld.global.f32 %0, [%1];" : "=f"(before_next[i]) : "l"(P.acc + out0 + p));
    }
  };

  for (int c0 = 0; c0 < rows_q; c0 += kWtCols) {
    const int nc = min(kWtCols, rows_q - c0), nc8 = (nc + 7) & ~7;
    if (c0 == 0) load_before(s0);
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
      if (s0 + d * kU < s1) load(a[d], sc[d], held[d], s0 + d * kU);   // (under way while the queries are laid out)
    if (c0) __syncthreads();
    // the queries as columns: piece 4 i + c holds what lane c of a quad feeds with its i-th piece.
    for (int i = warp; i < nc8; i += kWtWarps) {   // a column per warp
      const int rq = c0 + i, j = rq / P.group;
      const int64_t at = (static_cast<int64_t>(b) * P.n_q + j) * P.n_heads + h * P.group + rq - j * P.group;
      const bool on = i < nc;
      uint2 x = make_uint2(0u, 0u);               // dims 4 lane and up
      if (on && lane < D / 4) x = *reinterpret_cast<const uint2 *>(P.q + at * D + 4 * lane);
      float scale = P.scale_log2;
      int piece;                                  // of this lane's dims
      if constexpr (F16) {
        // scaled by the power of two that brings the row's largest entry to [1, 2)
        const float x0 = __uint_as_float(x.x << 16), x1 = __uint_as_float(x.x & 0xffff0000u);
        const float x2 = __uint_as_float(x.y << 16), x3 = __uint_as_float(x.y & 0xffff0000u);
        float m = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        e = max(min(e, 126), -126);  // (zero rows, subnormal and infinite maxima)
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        x = make_uint2(pack2<true>(x0 * inv, x1 * inv), pack2<true>(x2 * inv, x3 * inv));
        scale *= __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        const int c = 4 * lane / (D / 4), k = (4 * lane % (D / 4)) / 8;  // lane c reads dims c D / 4 and up
        piece = 4 * k + c;
      } else {
        const int d8 = lane / 2;                  // lane c reads 32 bytes (a sector) of every 128, in two pieces
        piece = 4 * (d8 / 8 * 2 + d8 % 2) + d8 % 8 / 2;
      }
      x.x ^= P.q_sign, x.y ^= P.q_sign;
      if (lane < D / 4) *reinterpret_cast<uint2 *>(qs + i * kStride + piece * 16 + (lane & 1) * 8) = x;
      // (a row that saw nothing, lse = -inf, gives no weight)
      const float lse = on && lane == 0 ? P.lse[at] : -INFINITY;
      if (lane == 0) col[i] = make_float2(scale, lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f);
    }
    __syncthreads();
    for (int at = s0; at < s1; at += kRun) {
    float sum[kOut];
#pragma unroll
    for (int i = 0; i < kOut; ++i) sum[i] = 0.f, before[i] = before_next[i];
    if (c0 == 0) load_before(at + kRun);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int s = at + d * kU;
      if (s >= s1) break;
      bool held_now[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) held_now[u] = held[d][u];
      auto next = [&] {      // (the registers are free)
        if (s + kU * kDeep < s1) load(a[d], sc[d], held[d], s + kU * kDeep);
      };
      // 4 bits: the A fragments, piece i of a lane's dims in two steps of 16 (bf16: as they were loaded)
      uint32_t f[F16 ? kU : 1][F16 ? kPieces : 1][2][4];
      if constexpr (F16) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t word[4] = {a[d][u][k][0].x, a[d][u][k][0].y, a[d][u][k][0].z, a[d][u][k][0].w};
              uint32_t v[4];
              e2m1x8_to_half2(word[i], v);
              const uint32_t s2 = __byte_perm(e4m3x2_to_half2(sc[d][u][k]), 0, D == 128 && i >= 2 ? 0x3232 : 0x1010);
              f[u][i][0][k] = hmul2(v[0], s2), f[u][i][0][2 + k] = hmul2(v[1], s2);
              f[u][i][1][k] = hmul2(v[2], s2), f[u][i][1][2 + k] = hmul2(v[3], s2);
            }
        next();
      }
      float x[kU][4], w[kU][2] = {};
      auto products = [&](int cg) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[u][k] = 0.f;
        const uint8_t *qp = qs + (cg + r8) * kStride + c4 * 16;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint4 q = *reinterpret_cast<const uint4 *>(qp + i * 64);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            if constexpr (F16) {
              mma16816<true>(x[u], f[u][i][0], q.x, q.y);
              mma16816<true>(x[u], f[u][i][1], q.z, q.w);
            } else {
              const uint32_t y[4] = {a[d][u][0][i].x, a[d][u][1][i].x, a[d][u][0][i].y, a[d][u][1][i].y};
              const uint32_t z[4] = {a[d][u][0][i].z, a[d][u][1][i].z, a[d][u][0][i].w, a[d][u][1][i].w};
              mma16816<false>(x[u], y, q.x, q.y);
              mma16816<false>(x[u], z, q.z, q.w);
            }
          }
        }
      };
      // tokens that every query sees (the last n_q - 1 are looked at one by one)
      const bool edge = (s + kU) * kSubTokens > len - (P.n_q - 1);
      auto weights = [&](int cg) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = cg + 2 * c4 + p;
          const float2 m = col[c];
          const int seen = edge ? len - (P.n_q - 1 - min((c0 + c) / P.group, P.n_q - 1)) : 0x7fffffff;
#pragma unroll
          for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float e = ex2(fmaf(x[u][p + 2 * k], m.x, -m.y));
              w[u][k] += c < nc && (!edge || (s + u) * kSubTokens + r8 + 8 * k < seen) ? e : 0.f;
            }
        }
      };
      for (int cg = 0; cg + 8 < nc8; cg += 8) {
        products(cg);
        weights(cg);
      }
      products(nc8 - 8);
      if (!F16) next();
      weights(nc8 - 8);
      // the quad's sum of token r8 + 8 k goes to the lane of that token
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[u][k] += __shfl_xor_sync(~0u, w[u][k], 1);
          w[u][k] += __shfl_xor_sync(~0u, w[u][k], 2);
          w[u][k] = __shfl_sync(~0u, w[u][k], (lane & 7) * 4);
        }
        const int i = d * kU + u;     // (sub-block of the round: tokens 16 i and up of it)
        if (lane / 16 == i % 2 && held_now[u]) sum[i / 2] = lane & 8 ? w[u][1] : w[u][0];
      }
    }
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const int p = at * kSubTokens + 32 * i + lane;
      if (p >= end) continue;
      // (a later chunk of columns adds to what this thread wrote for the one before)
      P.acc_out[out0 + p] = (c0 ? P.acc_out[out0 + p] : before[i] * P.decay) + sum[i];
    }
    }
  }
}

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------
constexpr uint32_t kMustKey = 0xffffffffu;  // of a token that stays in any case
constexpr int kEvBins = 2048;          // parts of the weights' range
constexpr int kEvAhead = 8;           // slots a thread has under way
constexpr int kEvVecs = 4;            // 16-byte pieces of weights, and of positions, a thread has under way
constexpr int kEvStaged = 32768;      // tokens whose keys a CTA keeps in shared memory

struct EvictParams {
  uint8_t *rows;
  int64_t row_bytes;
  int32_t n_rows, bsub;
  const int32_t *table;
  int32_t table_heads, max_blocks, n_kv, B;
  const int32_t *len;
  int32_t *len_out;
  int32_t keep, sinks, recent;
  const float *acc;
  float *acc_out;
  const int32_t *pos, *pos_len, *next_pos;
  int32_t *pos_out;
  int32_t *moves;                     // [B * n_kv]
  int2 *list;                         // [B * n_kv][keep] (from, to)
  int32_t move_here;                  // moves made by the CTA that lists them
  int32_t move_ctas;
  int32_t *status;
};

__device__ __forceinline__ int64_t ev_row(const EvictParams &P, int b, int h, int slot, int &off) {
  const int bs = P.bsub * kSubTokens, e = slot / bs;
  off = slot - e * bs;
  const int32_t id = P.table[(static_cast<int64_t>(b) * P.table_heads + (P.table_heads > 1 ? h : 0)) * P.max_blocks + e];
  return id < 0 ? -1 : P.table_heads > 1 ? id : static_cast<int64_t>(id) * P.n_kv + h;
}

// The keys and values of tokens list[first] .. list[first + 7] (of `count`) from slot x to slot y, by a
// warp: a lane looks up a token's places, then all loads are under way before the first store.
constexpr int kMoveAhead = 8;

template <int FMT, int D>
__device__ __forceinline__ void move_tokens(const EvictParams &P, int b, int h, const int2 *list, int first, int count, int lane) {
  constexpr bool kFp4 = FMT == ECHO_BLOCK_FP4;
  // bytes from the start of `rows` to the token's key (bf16) or to its sub-block (4 bits; the token in
  // the lowest 4 bits, which are zeros otherwise), -1: not to be moved
  int64_t from = -1, to = -1;
  if (lane < kMoveAhead && first + lane < count) {
    const int2 m = list[first + lane];
    int o0, o1;
    const int64_t r0 = ev_row(P, b, h, m.x, o0), r1 = ev_row(P, b, h, m.y, o1);
    if (r0 < 0 || r1 < 0 || r0 >= P.n_rows || r1 >= P.n_rows) {
      set_status(P.status, ECHO_DEV_BAD_INDEX);
    } else if constexpr (kFp4) {
      from = r0 * P.row_bytes + o0 / kSubTokens * Fp4Sub<D>::kBytes + o0 % kSubTokens;
      to = r1 * P.row_bytes + o1 / kSubTokens * Fp4Sub<D>::kBytes + o1 % kSubTokens;
    } else {
      from = r0 * P.row_bytes + o0 * (2 * D);
      to = r1 * P.row_bytes + o1 * (2 * D);
    }
  }
  if constexpr (kFp4) {
    static_assert(Fp4Sub<D>::kBytes % 16 == 0, "a token's number fits under a sub-block's place");
    // lanes 0-7: a part of the value codes each, D / 16 bytes; from 8: a value scale each; from 16: key
    // codes, 16 bytes each; 31: the key scales
    auto place = [&](int64_t at) -> uint8_t * {
      const int t = static_cast<int>(at & 15);
      uint8_t *sub = P.rows + (at - t);
      if (lane < 8) return sub + Fp4Sub<D>::kValues + ((t >> 3) * 64 + lane * 8 + (t & 7)) * (D / 16);
      if (lane < 16) return sub + Fp4Sub<D>::kValueScales + (t >> 3) * (D / 2) + (lane - 8) * 8 + (t & 7);
      if (lane < 31) return sub + t * (D / 2) + (lane - 16) * 16;
      return sub + Fp4Sub<D>::kKeyScales + t * (D / 16);
    };
    const bool bytes16 = lane >= 16 && lane < 16 + D / 32, scale = lane >= 8 && lane < 8 + D / 16, part = lane < 8 || lane == 31;
    uint4 x[kMoveAhead];
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int64_t at = __shfl_sync(~0u, from, u);
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at < 0) continue;
      const uint8_t *s = place(at);
      if (bytes16) x[u] = *reinterpret_cast<const uint4 *>(s);
      else if (scale) x[u].x = *s;
      else if (part && D == 128) *reinterpret_cast<uint2 *>(&x[u]) = *reinterpret_cast<const uint2 *>(s);
      else if (part) x[u].x = *reinterpret_cast<const uint32_t *>(s);
    }
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int64_t at = __shfl_sync(~0u, to, u);
      if (at < 0) continue;
      uint8_t *d = place(at);
      if (bytes16) *reinterpret_cast<uint4 *>(d) = x[u];
      else if (scale) *d = static_cast<uint8_t>(x[u].x);
      else if (part && D == 128) *reinterpret_cast<uint2 *>(d) = make_uint2(x[u].x, x[u].y);
      else if (part) *reinterpret_cast<uint32_t *>(d) = x[u].x;
    }
  } else {
    constexpr int kHalf = D / 8;    // 16-byte pieces of a key
    const int64_t piece = lane < kHalf ? lane * 16 : static_cast<int64_t>(P.bsub) * kSubTokens * D * 2 + (lane - kHalf) * 16;
    uint4 x[kMoveAhead];
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int64_t at = __shfl_sync(~0u, from, u);
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0 && lane < 2 * kHalf) x[u] = load16_here(P.rows + at + piece);
    }
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int64_t at = __shfl_sync(~0u, to, u);
      if (at >= 0 && lane < 2 * kHalf) *reinterpret_cast<uint4 *>(P.rows + at + piece) = x[u];
    }
  }
}

// STAGED: the keys of a context in shared memory; otherwise they are made again from what they come of
template <int FMT, int D, int T, bool STAGED>
__global__ void __launch_bounds__(T, 1024 / T) block_evict_kernel(const EvictParams P) {
  constexpr int W = T / 32;
  extern __shared__ __align__(16) uint32_t ev_keys[];
  __shared__ PickSpace<W, kEvBins> S;
  __shared__ uint32_t wcnt[3][W];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / P.n_kv, h = blockIdx.x - b * P.n_kv;
  pdl_launch_dependents();
  pdl_wait();
  const int most = P.max_blocks * P.bsub * kSubTokens;
  int n = P.len[b];
  if (n > most) {
    if (h == 0 && tid == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
    n = most;
  }
  n = max(n, 0);
  const int end = min(n, P.keep);
  if (h == 0 && tid == 0) P.len_out[b] = end;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * most;
  const float *acc = P.acc + base;
  const int32_t *pos = P.pos ? P.pos + base : nullptr;
  float *acc_out = P.acc_out + base;
  int32_t *pos_out = P.pos ? P.pos_out + base : nullptr;
  const int known = P.pos ? min(max(P.pos_len[b], 0), n) : 0;
  const int nxt = P.pos ? P.next_pos[b] : 0;
  auto pos_of = [&](int i) { return i < known ? pos[i] : nxt - n + i; };

  // weights and positions of slots [0, upto) as they are, loads ahead of the stores (which may go to
  // the same memory)
  auto copy = [&](int upto) {
    for (int i0 = tid; i0 < upto; i0 += kEvAhead * T) {
      float x[kEvAhead];
      int y[kEvAhead];
#pragma unroll
      for (int r = 0; r < kEvAhead; ++r) {
        const int i = i0 + r * T;
        x[r] = i < upto ? acc[i] : 0.f;
        y[r] = pos_out && i < upto ? pos_of(i) : 0;
      }
#pragma unroll
      for (int r = 0; r < kEvAhead; ++r) {
        const int i = i0 + r * T;
        if (i < upto) {
          acc_out[i] = x[r];
          if (pos_out) pos_out[i] = y[r];
        }
      }
    }
  };
  if (n <= P.keep) {
    copy(n);
    if (tid == 0) P.moves[blockIdx.x] = 0;
    return;
  }

  auto make_key = [&](int i, float s, int at) -> uint32_t {
    if (i < P.sinks || (pos && at >= nxt - P.recent)) return kMustKey;
    return s != s ? 1u : score_key(s);  // (a weight that is NaN goes first)
  };
  auto key_of = [&](int i) { return make_key(i, acc[i], pos ? pos_of(i) : 0); };
  pick_clear(S);
  const uint32_t zero = score_key(0.f);
  uint32_t lo = kMustKey, hi = 0, n_must = 0;   // (of the weights above zero)
  for (int i0 = 4 * tid; i0 < n; i0 += kEvVecs * 4 * T) {
    uint4 x[kEvVecs], y[kEvVecs];   // (four slots each, which the table has in any case; all under way at once)
#pragma unroll
    for (int r = 0; r < kEvVecs; ++r) {
      const int i = i0 + r * 4 * T;
      x[r] = y[r] = make_uint4(0u, 0u, 0u, 0u);
      if (i < n) x[r] = load16_here(acc + i);
      if (i < known) y[r] = load16_here(pos + i);
    }
#pragma unroll
    for (int r = 0; r < kEvVecs; ++r) {
      const int i = i0 + r * 4 * T;
      if (i >= n) break;
      const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w}, at[4] = {y[r].x, y[r].y, y[r].z, y[r].w};
      uint32_t key[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        key[k] = make_key(i + k, __uint_as_float(w[k]), i + k < known ? static_cast<int>(at[k]) : nxt - n + i + k);
        if (i + k >= n) continue;
        if (key[k] == kMustKey) ++n_must;
        else if (key[k] > zero) lo = min(lo, key[k]), hi = max(hi, key[k]);
      }
      if constexpr (STAGED) *reinterpret_cast<uint4 *>(ev_keys + i) = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  pick_stats(S, n_must, lo, hi);
  auto key_at = [&](int i) -> uint32_t {
    if constexpr (STAGED) return ev_keys[i];
    else return key_of(i);
  };

  // ----- the key above which all stay, and how many of its equals (n > keep: some go) -----
  uint32_t thr = kMustKey - 1, need = 0;
  bool all_equal = false;    // all that equal thr stay
  if (n_must > static_cast<uint32_t>(P.keep)) {  // (more recent positions than their number: the first slots of them)
    thr = kMustKey, need = P.keep;
  } else if (n_must < static_cast<uint32_t>(P.keep)) {
    // equal parts of the keys' range (a weight's exponent and leading bits) above zero
    const int shift = hi > lo ? max(0, 21 - __clz(hi - lo)) : 0;
    auto bin = [&](uint32_t k) { return k <= lo ? 0 : static_cast<int>(min((k - lo) >> shift, kEvBins - 1u)); };
    auto each = [&](auto &&f) {
#pragma unroll 4
      for (int i = tid; i < n; i += T) f(key_at(i));
    };
    all_equal = pick_kth(S, P.keep - n_must, each, [](uint32_t k) { return k != kMustKey; }, bin, [](uint32_t k) { return k; }, thr, need);
  }
  __syncthreads();

  // ----- holes and movers in order -----
  // A thread takes a run of slots (an odd number: no bank conflicts); equals that stay, then holes and movers, are counted over the
  // runs.  Movers and holes are as many.
  const int per = (n + T - 1) / T | 1, i0 = static_cast<int>(min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(n))), i1 = min(i0 + per, n);
  auto scan = [&](uint32_t mine, int which) -> uint32_t {  // exclusive sum over the threads
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) wcnt[which][warp] = upto;
    __syncthreads();
    return upto - mine + __reduce_add_sync(~0u, lane < warp ? wcnt[which][lane % W] : 0u);
  };
  uint32_t eq0 = 0;
  if (!all_equal) {
    uint32_t eq = 0;
    for (int i = i0; i < i1; ++i) eq += key_at(i) == thr;
    eq0 = scan(eq, 0);
  }
  // whether slot i's token is one of those that stay; called for the slots of the run one after another
  auto stays = [&](int i) {
    const uint32_t key = key_at(i);
    const bool equal = key == thr, yes = key > thr || (equal && (all_equal || eq0 < need));
    eq0 += equal;
    return yes;
  };
  // (as bits, the first 64 slots of a run: all of it where keys are in shared memory)
  uint32_t holes = 0, movers = 0, marks[2];
  const uint32_t eq_first = eq0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int from = i0 + 32 * half, to = min(from + 32, i1);
    uint32_t m = 0;
#pragma unroll 8
    for (int i = from; i < to; ++i) m |= stays(i) == (i >= P.keep) ? 1u << (i - from) : 0u;
    const uint32_t below = P.keep >= from + 32 ? ~0u : P.keep > from ? (1u << (P.keep - from)) - 1 : 0u;
    holes += __popc(m & below), movers += __popc(m & ~below);
    marks[half] = m;
  }
  for (int i = i0 + 64; i < i1; ++i) {
    const bool mark = stays(i) == (i >= P.keep);
    holes += mark && i < P.keep, movers += mark && i >= P.keep;
  }
  uint32_t hole_at = scan(holes, 1), mover_at = scan(movers, 2);
  int2 *list = P.list + static_cast<int64_t>(blockIdx.x) * P.keep;
  auto note = [&](int i) {
    if (i < P.keep) list[hole_at++].y = i;
    else list[mover_at++].x = i;
  };
#pragma unroll
  for (int half = 0; half < 2; ++half)
    for (uint32_t m = marks[half]; m; m &= m - 1) note(i0 + 32 * half + __ffs(m) - 1);
  if (i1 - i0 > 64) {       // (longer runs: looked at once more)
    eq0 = eq_first;
    for (int i = i0; i < i1; ++i)
      if (stays(i) == (i >= P.keep) && i - i0 >= 64) note(i);
  }
  __syncthreads();
  const uint32_t count = __reduce_add_sync(~0u, lane < W ? wcnt[2][lane % W] : 0u);
  if (tid == 0) P.moves[blockIdx.x] = count;

  // ----- weights and positions: those that keep their slot, then those that move -----
  // (in place the first pass writes what is there)
  copy(end);
  __syncthreads();
  for (uint32_t i = tid; i < count; i += T) {
    const int2 m = list[i];
    acc_out[m.y] = acc[m.x];
    if (pos_out) pos_out[m.y] = pos_of(m.x);
  }
  if (P.move_here)
    for (int i = warp * kMoveAhead; i < static_cast<int>(count); i += W * kMoveAhead) move_tokens<FMT, D>(P, b, h, list, i, count, lane);
}

constexpr int kMvWarps = 8;

template <int FMT, int D>
__global__ void __launch_bounds__(kMvWarps * 32) block_move_kernel(const EvictParams P) {
  const int pair = blockIdx.x / P.move_ctas, part = blockIdx.x - pair * P.move_ctas;
  const int b = pair / P.n_kv, h = pair - b * P.n_kv;
  pdl_launch_dependents();
  pdl_wait();
  const int count = P.moves[pair];
  const int2 *list = P.list + static_cast<int64_t>(pair) * P.keep;
  for (int i = (part * kMvWarps + (threadIdx.x >> 5)) * kMoveAhead; i < count; i += P.move_ctas * kMvWarps * kMoveAhead)
    move_tokens<FMT, D>(P, b, h, list, i, count, threadIdx.x & 31);
}

}  // namespace echo

namespace echo_host {

int launch_block_weights(const echo_block_weights_args *a, cudaStream_t stream) {
  echo::WeightParams P{};
  P.q = a->q, P.rows = reinterpret_cast<const uint8_t *>(a->rows);
  P.row_bytes = 2 * echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.n_rows = a->n_rows, P.bsub = a->block_tokens / echo::kSubTokens;
  P.table = a->table, P.table_heads = a->table_heads, P.max_blocks = a->max_blocks;
  P.ctx_len = a->ctx_len, P.old_len = a->old_len;
  P.n_q = a->n_q, P.n_heads = a->n_heads, P.n_kv = a->n_kv_heads, P.group = a->n_heads / a->n_kv_heads;
  P.scale_log2 = std::ldexp(std::fabs(a->scale) * 1.4426950408889634f, -a->k_shift);
  P.q_sign = a->scale < 0.f ? 0x80008000u : 0u;
  P.lse = a->lse, P.acc = a->acc, P.acc_out = a->acc_out, P.decay = a->decay;
  P.status = a->dev_status;
  int sms = 0;
  if (int rr = sm_count(&sms, "block eviction device")) return rr;
  const int64_t pairs = static_cast<int64_t>(a->B) * a->n_kv_heads;
  const int64_t nsub = static_cast<int64_t>(a->max_blocks) * P.bsub;
  // two sub-blocks a warp, or more where every SM still has several CTAs (a CTA's first loads and queries
  // take as long as some 8 sub-blocks: 16 requests of 32768 tokens 135 us with half as many a warp, 130)
  P.subs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, nsub * pairs / (2 * echo::kWtWarps * 24ll * sms))) * 2);
  P.ctas = static_cast<int>((nsub + echo::kWtWarps * P.subs - 1) / (echo::kWtWarps * P.subs));
  const dim3 grid(static_cast<unsigned>(P.ctas * pairs)), block(echo::kWtWarps * 32);
  cudaError_t e;
  if (a->format == ECHO_BLOCK_FP4)
    e = a->head_dim == 128 ? launch_pdl(echo::block_weights_kernel<ECHO_BLOCK_FP4, 128>, grid, block, 0, stream, P)
                           : launch_pdl(echo::block_weights_kernel<ECHO_BLOCK_FP4, 64>, grid, block, 0, stream, P);
  else
    e = a->head_dim == 128 ? launch_pdl(echo::block_weights_kernel<ECHO_BLOCK_BF16, 128>, grid, block, 0, stream, P)
                           : launch_pdl(echo::block_weights_kernel<ECHO_BLOCK_BF16, 64>, grid, block, 0, stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block weights launch");
}

size_t block_evict_workspace_bytes(int32_t B, int32_t n_kv_heads, int32_t keep) {
  const size_t pairs = static_cast<size_t>(B) * n_kv_heads;
  return (pairs * 4 + 255) / 256 * 256 + pairs * keep * sizeof(int2);
}

template <int FMT, int D>
static int go_evict(echo::EvictParams P, cudaStream_t stream) {
  static std::atomic<bool> attr[kMaxDevices];
  const int64_t pairs = static_cast<int64_t>(P.B) * P.n_kv;
  const int64_t most = static_cast<int64_t>(P.max_blocks) * P.bsub * echo::kSubTokens;
  const bool staged = most <= echo::kEvStaged;
  const int smem = staged ? static_cast<int>(most) * 4 : 0;
  if (smem > 32768)   // (beside 9 KB of its own)
    if (int rr = smem_limit_once(attr, echo::block_evict_kernel<FMT, D, 1024, true>, echo::kEvStaged * 4, "block eviction smem attribute")) return rr;
  int sms = 0;
  if (int rr = sm_count(&sms, "block eviction device")) return rr;
  const int64_t moves = std::max<int64_t>(0, std::min<int64_t>(P.keep, most - P.keep));
  P.move_here = moves <= 256;
  P.move_ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((moves + 63) / 64, 8ll * sms / pairs)));
  // threads by the slots a pair may have
  const dim3 grid(static_cast<unsigned>(pairs));
  cudaError_t e = most <= 8192 ? launch_pdl(echo::block_evict_kernel<FMT, D, 512, true>, grid, dim3(512), smem, stream, P)
                : staged       ? launch_pdl(echo::block_evict_kernel<FMT, D, 1024, true>, grid, dim3(1024), smem, stream, P)
                               : launch_pdl(echo::block_evict_kernel<FMT, D, 1024, false>, grid, dim3(1024), smem, stream, P);
  if (e == cudaSuccess && !P.move_here)
    e = launch_pdl(echo::block_move_kernel<FMT, D>, dim3(static_cast<unsigned>(pairs * P.move_ctas)), dim3(echo::kMvWarps * 32), 0, stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block eviction launch");
}

int launch_block_evict(const echo_block_evict_args *a, cudaStream_t stream) {
  echo::EvictParams P{};
  P.rows = reinterpret_cast<uint8_t *>(a->rows);
  P.row_bytes = 2 * echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.n_rows = a->n_rows, P.bsub = a->block_tokens / echo::kSubTokens;
  P.table = a->table, P.table_heads = a->table_heads, P.max_blocks = a->max_blocks, P.n_kv = a->n_kv_heads, P.B = a->B;
  P.len = a->len, P.len_out = a->len_out;
  P.keep = a->keep, P.sinks = a->sinks, P.recent = a->recent;
  P.acc = a->acc, P.acc_out = a->acc_out;
  P.pos = a->pos, P.pos_len = a->pos_len, P.next_pos = a->next_pos, P.pos_out = a->pos_out;
  P.moves = static_cast<int32_t *>(a->workspace);
  P.list = reinterpret_cast<int2 *>(static_cast<uint8_t *>(a->workspace) + (static_cast<size_t>(a->B) * a->n_kv_heads * 4 + 255) / 256 * 256);
  P.status = a->dev_status;
  if (a->format == ECHO_BLOCK_FP4)
    return a->head_dim == 128 ? go_evict<ECHO_BLOCK_FP4, 128>(P, stream) : go_evict<ECHO_BLOCK_FP4, 64>(P, stream);
  return a->head_dim == 128 ? go_evict<ECHO_BLOCK_BF16, 128>(P, stream) : go_evict<ECHO_BLOCK_BF16, 64>(P, stream);
}

}  // namespace echo_host
