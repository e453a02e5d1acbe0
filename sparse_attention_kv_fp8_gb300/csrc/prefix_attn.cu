// prefix_attn.cu -- decode attention of requests that share a prefix: the prefix's keys and
// values are read once for all query rows of a group, as tensor-core tiles of 256 rows.
//
// For query row r of a request of group g (prefix tokens P_g, own tokens O_b):
//   x_p = scale * q_r . k_p,   out = sum_{P_g and O_b} 2^(x_p log2 e - m) v_p / l.
// A softmax over two sets of tokens is the merge of the two softmaxes by their maxima and sums,
// so the prefix goes through this kernel, the own tokens through the kernel of
// echo_block_attention (with its result left in fp32), and a last kernel merges the two.
// 4 D flops per query row and token against 4 D bytes per token and KV head (bf16): from
// about 280 rows a KV head on the tensor cores are the bound, below it HBM.
//
// sm_103a design.
//   A CTA holds the queries of a tile of up to 256 rows (two sub-tiles of 128) in shared memory
//     and walks over chunks of 128 prefix tokens:  S = Q K^T (tcgen05.mma, M = 128 rows, N = 128
//     tokens) into tensor memory, softmax by a warpgroup per sub-tile (a thread per row), P back
//     into the tensor memory that S took (two bf16 terms of 64 columns each, or one in fp16), O += P V
//     with P as the tensor-memory operand and V read along the tokens, once for each term.  While one sub-tile's warpgroup is at
//     its softmax, the tensor cores work for the other; one thread issues all products, which
//     run in the order of their issue, so S may overwrite the P that the product before it read.
//   Blocks come by TMA, a box per run of tokens inside a block, into a ring of key and value
//     tiles in the 128-byte swizzle.  4-bit rows come as they are (one bulk copy per sub-block of
//     16 tokens) and four warps, two sub-blocks each, convert them, exactly, to fp16 tiles.
//   Lazy maximum as in the decode kernel: O is rescaled (in tensor memory) only when a score
//     exceeds its row's maximum by 2^8.
//   All chunks of all (group, KV head, row tile) form one line, cut into equal pieces by the
//     lengths on the device, one per CTA.  Each (tile, piece) leaves its maxima, sums and O in
//     fp32: pieces that begin with a tile in a row per query row, the others in a slot per CTA.
//     The merge kernel takes them in order, so results do not depend on timing.
//   64 requests of 64 heads (8 KV heads of 128 dims), a prefix of 32768: bf16 84 us, 810 TFLOP/s of 4 D a row
//     and token (256 requests: 287 us, 955), 4 bits 72 us.  The tensor cores are busy half of the time (half as
//     many products again in bf16, for the weights' second term) and the exponentials' pipe a fifth: a
//     warpgroup's chunk is a chain (scores, maximum, weights, hand-over) that two sub-tiles cover only in part;
//     more would need registers for a third.  A prefix of 131072 for 8 requests, one sub-tile: 107 us, 0.76 of
//     the copy rate, the chain.  Short ones (1000 tokens: 11 us) are two kernels' chains of latencies.
#include <algorithm>
#include <cmath>

#include "block_mma.cuh"

namespace echo {

constexpr int kPxChunk = 128;         // prefix tokens of a step
constexpr int kPxRows = 256;          // query rows of a CTA's tile (two sub-tiles)
constexpr int kPxMaxGrid = 160;
constexpr float kPxLazy = 8.f;        // log2 of how far a score may exceed its row's maximum
constexpr float kPxLift = 7.f;        // fp16 weights are kept 2^7 up (their subnormals begin 2^-21 below the maximum)
constexpr float kPxNone = -3.4028234664e38f;
constexpr float kPxMinScale = 1e-37f; // of a row's scores: not zero, a masked score's infinity stays what it is

struct PrefixParams {
  const uint16_t *q;
  const uint8_t *rows;
  int64_t row_bytes;
  int32_t n_rows, bs, box;            // box: tokens of a TMA box, a divisor of bs
  const int32_t *table;               // [n_groups][heads][max_blocks]
  int32_t heads, max_blocks;
  const int32_t *len, *start;         // [n_groups], [n_groups + 1]
  int32_t n_groups;
  int32_t B, n_q, n_heads, n_kv, group;
  float scale_log2;                   // |scale| log2 e, over the keys' power of two
  float v_scale;                      // one over the values' power of two
  uint32_t q_sign;
  float *first_o;                     // [B n_q n_heads][D]: pieces that begin with their tile
  float2 *first_ml;
  float *rest_o;                      // [kPxMaxGrid][kPxRows][D]: of a CTA's first piece otherwise
  float2 *rest_ml;
  const float *own_o, *own_lse;       // [B n_q n_heads][D], or NULL
  uint16_t *out;
  float *lse;
  int32_t grid, room;                 // CTAs; whether some are left to the own tokens
  int32_t *status;
};

// ---------------------------------------------------------------------------
// the line of chunks
// ---------------------------------------------------------------------------
struct PxGroup {
  int b0, rows;       // first request, query rows of a KV head
  int len, tiles, chunks;
};

__device__ __forceinline__ PxGroup px_group(const PrefixParams &P, int g, bool report) {
  PxGroup x;
  const int s0 = P.start[g], s1 = P.start[g + 1];
  x.b0 = min(max(s0, 0), P.B);
  const int b1 = min(max(s1, x.b0), P.B);
  x.rows = (b1 - x.b0) * P.n_q * P.group;
  const int most = P.max_blocks * P.bs, n = P.len[g];
  x.len = min(max(n, 0), most);
  if (report && (n > most || s0 < 0 || s1 > P.B || s1 < s0)) set_status(P.status, ECHO_DEV_BAD_INDEX);
  x.tiles = (x.rows + kPxRows - 1) / kPxRows;
  x.chunks = (x.len + kPxChunk - 1) / kPxChunk;
  return x;
}
// (below 2^31 - 1024 over groups that do not overlap: the host checks the sizes)
__device__ __forceinline__ int px_units(const PrefixParams &P, const PxGroup &x) { return P.n_kv * x.tiles * x.chunks; }
// Group starts that are not ascending make groups overlap, and their line may be longer: sums stop at kPxMost,
// and a line of that length is taken for an empty one.
constexpr uint32_t kPxMost = 0x7fffffffu;
__device__ __forceinline__ uint32_t px_add(uint32_t a, uint32_t b) { return min(a + b, kPxMost); }

// Group g (the same for the whole warp): from the lane that has it, `mine`, where there is one a lane.
__device__ __forceinline__ PxGroup px_group_of(const PrefixParams &P, const PxGroup &mine, int g) {
  if (P.n_groups > 32) return px_group(P, g, false);
  PxGroup x;
  x.b0 = __shfl_sync(~0u, mine.b0, g), x.rows = __shfl_sync(~0u, mine.rows, g), x.len = __shfl_sync(~0u, mine.len, g);
  x.tiles = __shfl_sync(~0u, mine.tiles, g), x.chunks = __shfl_sync(~0u, mine.chunks, g);
  return x;
}

// exclusive sum over the lanes of a warp, and the total (0 instead of kPxMost)
__device__ __forceinline__ int px_scan(uint32_t mine, int &total) {
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, upto, d);
    if ((threadIdx.x & 31) >= d) upto = px_add(upto, y);
  }
  const uint32_t all = __shfl_sync(~0u, upto, 31);
  total = all == kPxMost ? 0 : static_cast<int>(all);
  return static_cast<int>(upto - mine);
}

// How the tiles are cut.  Whole: every tile of group g into ceil(chunks / whole) equal pieces, one
// per CTA, the row tiles of a KV head beside one another, so that they read the same blocks at the
// same time.  Otherwise (whole == 0): the line of all chunks into shares of `per`, one per CTA, which may
// begin and end inside a tile.  A CTA that changes tiles takes as long as kPxChange chunks more, so
// whole pieces are taken where they are no longer than a share by more.
constexpr int kPxChange = 5;
// Where the own tokens have work for many SMs, shares of up to kPxRoom chunks leave them half: they wait for
// those of a short prefix less than the SMs would wait for them (64 requests of 64 heads, a prefix of
// 2048 and own tokens of up to 100 / 1000: 31.0 / 52.3 -> 25.7 / 43.2 us, of 4096 and 1000 56.7 -> 49.7; 16
// requests, 2048 and 100 21.9 -> 18.7).
constexpr int kPxRoom = 6;
constexpr int kPxFewGroups = 8;       // (more groups: their tiles are not tried)

struct PxPlan {
  int whole, per, total;
};

__device__ __forceinline__ PxPlan px_plan(const PrefixParams &P, const PxGroup &mine, int total) {  // (by a whole warp)
  PxPlan x{0, 0, total};
  x.per = static_cast<int>((static_cast<uint32_t>(total) + P.grid - 1) / static_cast<uint32_t>(P.grid));
  if (P.room) {  // (half of the SMs, as far as that makes no share longer than kPxRoom)
    const uint32_t half = (static_cast<uint32_t>(total) + P.grid / 2) / (static_cast<uint32_t>(P.grid) / 2 + 1);
    x.per = max(x.per, static_cast<int>(min(half, static_cast<uint32_t>(kPxRoom))));
  }
  if (total == 0 || P.n_groups > kPxFewGroups) return x;
  const int lane = threadIdx.x & 31, len = x.per + lane;
  int64_t pieces = 0;
  for (int g = 0; g < P.n_groups; ++g) {
    const PxGroup y = px_group_of(P, mine, g);
    pieces += static_cast<int64_t>(P.n_kv) * y.tiles * ((static_cast<uint32_t>(y.chunks) + len - 1) / static_cast<uint32_t>(len));
  }
  const uint32_t fits = __ballot_sync(~0u, lane <= kPxChange && pieces <= P.grid);
  if (fits) x.whole = x.per + __ffs(fits) - 1;
  return x;
}
// pieces of a tile, and their length
__device__ __forceinline__ int px_pieces(const PxPlan &x, const PxGroup &y, int &len) {
  const int n = (y.chunks + x.whole - 1) / x.whole;
  len = n ? (y.chunks + n - 1) / n : 0;
  return n;
}

// One CTA's place: the piece of tile (g, h, t) from chunk c on, n chunks long.
struct PxLine {
  int g, h, t, c, n;
  PxGroup x;
  int left;       // chunks of this CTA's share from c on

  __device__ __forceinline__ void piece() { n = min(x.chunks - c, left); }

  // the first piece (by a whole warp)
  __device__ __forceinline__ bool begin(const PrefixParams &P, bool report) {
    const int lane = threadIdx.x & 31;
    const int run = (P.n_groups + 31) / 32, g0 = min(lane * run, P.n_groups), g1 = min(g0 + run, P.n_groups);
    uint32_t sum = 0;
    int total;
    PxGroup last{};
    for (int i = g0; i < g1; ++i) last = px_group(P, i, report), sum = px_add(sum, px_units(P, last));
    const int before = px_scan(sum, total), mine = sum;
    const PxPlan plan = px_plan(P, last, total);
    if (plan.whole) {
      int at = blockIdx.x;
      for (g = 0; g < P.n_groups; ++g) {
        x = px_group_of(P, last, g);
        int len;
        const int pieces = px_pieces(plan, x, len), all = P.n_kv * x.tiles * pieces;
        if (at >= all) {
          at -= all;
          continue;
        }
        const int row = at / x.tiles;      // (KV head, piece)
        t = at - row * x.tiles;
        h = row / pieces;
        c = (row - h * pieces) * len;
        left = n = min(len, x.chunks - c);
        return true;
      }
      return false;
    }
    if (static_cast<int64_t>(plan.per) * blockIdx.x >= total) return false;
    const int u0 = plan.per * blockIdx.x;
    left = min(plan.per, total - u0);
    int at = 0, off = 0;
    const bool own = u0 >= before && u0 < before + mine;
    if (own) {
      int u = before;
      for (at = g0;; ++at) {
        const int k = px_units(P, px_group(P, at, false));
        if (u0 < u + k) break;
        u += k;
      }
      off = u0 - u;
    }
    const int src = __ffs(__ballot_sync(~0u, own)) - 1;
    g = __shfl_sync(~0u, at, src);
    off = __shfl_sync(~0u, off, src);
    x = px_group_of(P, last, g);
    const uint32_t tile = static_cast<uint32_t>(off) / static_cast<uint32_t>(x.chunks);
    c = off - tile * x.chunks;
    h = tile / static_cast<uint32_t>(x.tiles), t = tile - h * x.tiles;
    piece();
    return true;
  }

  __device__ __forceinline__ bool next(const PrefixParams &P) {
    left -= n;
    if (left <= 0) return false;
    c = 0;            // (a piece ends with its tile or with the share)
    if (++t == x.tiles) {
      t = 0;
      if (++h == P.n_kv) {
        h = 0;
        do {
          x = px_group(P, ++g, false);
        } while (x.tiles == 0 || x.chunks == 0);  // (chunks are left: there is such a group)
      }
    }
    piece();
    return true;
  }

  // rows of sub-tile s
  __device__ __forceinline__ int sub_rows(int s) const { return min(max(x.rows - t * kPxRows - s * 128, 0), 128); }
};

// the cache row of a prefix token (a token below the prefix's length), -1: not held
__device__ __forceinline__ int64_t px_row(const PrefixParams &P, int g, int h, int token, int &off, bool report) {
  const uint32_t e = static_cast<uint32_t>(token) / static_cast<uint32_t>(P.bs);
  off = token - e * P.bs;
  const int32_t id = P.table[(static_cast<int64_t>(g) * P.heads + (P.heads > 1 ? h : 0)) * P.max_blocks + e];
  if (id < 0) return -1;
  const int64_t row = P.heads > 1 ? id : static_cast<int64_t>(id) * P.n_kv + h;
  if (row < P.n_rows) return row;
  if (report) set_status(P.status, ECHO_DEV_BAD_INDEX);
  return -1;
}

// (b, query token, head) of row r of a tile's group
__device__ __forceinline__ int64_t px_out_row(const PrefixParams &P, const PxLine &L, int r) {
  const uint32_t per = P.n_q * P.group, b = static_cast<uint32_t>(r) / per, rq = r - b * per, j = rq / static_cast<uint32_t>(P.group);
  return (static_cast<int64_t>(L.x.b0 + b) * P.n_q + j) * P.n_heads + L.h * P.group + rq - j * P.group;
}

// ---------------------------------------------------------------------------
// tensor-core helpers (beside those of echo_common.cuh)
// ---------------------------------------------------------------------------
__host__ __device__ constexpr uint32_t px_idesc(bool f16, int N, int b_mn) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (128u >> 4 << 24);
}
// MN-major operand in the 128-byte swizzle: groups of 64 elements along N `lbo` bytes apart, groups
// of 8 rows along K 1024 bytes apart
__device__ __forceinline__ uint64_t px_mn_desc(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// A descriptor's upper half is the same for all of an operand's steps: the lower one (addresses in
// units of 16 bytes) is what a step changes.
struct PxDesc {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit PxDesc(uint64_t d) : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
};
__device__ __forceinline__ void px_mma_ss(uint32_t d, const PxDesc &a, const PxDesc &b, uint32_t step, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a.lo + step), "r"(a.hi), "r"(b.lo + step), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void px_mma_ts(uint32_t d, uint32_t a, const PxDesc &b, uint32_t step, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b.lo + step), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void px_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void px_more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void px_fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void px_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void px_fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void px_tma(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void px_bulk(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void px_store8(float *p, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ float px_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// mbar_wait() without a look at the clock before the wait has become a long one: reading it takes
// longer than most waits here
__device__ __forceinline__ bool px_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, status);
}
// a wait without the abort flag, for what is in flight when a kernel gives up
__device__ __forceinline__ void px_drain(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < kWaitLimitNs) {
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int FMT, int D>
struct PxCfg {
  static constexpr bool kFp4 = FMT == ECHO_BLOCK_FP4;
  static constexpr uint32_t kBlock = 128 * 128;             // 128 rows or tokens of 64 dims
  static constexpr uint32_t kTile = kBlock * (D / 64);      // of all dims
  static constexpr int kSlots = kFp4 ? (D == 128 ? 3 : 6) : D == 128 ? 5 : 9;  // ring of key and value tiles
  static constexpr int kRaw = kFp4 ? 3 : 0;                 // stages of 4-bit chunks
  static constexpr uint32_t kRawBytes = 8 * 18 * D;
  static constexpr int kConvWarps = kFp4 ? 4 : 0;
  // Warpgroups: two of softmax, one of the producer and the issuer (and two idle warps), one that
  // converts.  A launch gives every thread the same registers (168 of 384 threads, 128 of 512); they
  // are handed over to the softmax, whose threads keep a row of 128 scores.  (Two threads a row, 64
  // scores each, meet for the maximum in every chunk: 70 us where one took 65, both with one term a
  // weight.)
  static constexpr int kLoadWarp = 8, kConvWarp = 12;
  static constexpr int kThreads = 32 * (kConvWarp + kConvWarps);
  static constexpr int kRegs = kFp4 ? 128 : 168, kRegsSoft = kFp4 ? 176 : 208, kRegsLoad = kFp4 ? 80 : 88, kRegsConv = kFp4 ? 80 : 0;
  static_assert(2 * kRegsSoft + kRegsLoad + kRegsConv <= kRegs * kThreads / 128, "registers of the launch");
  static constexpr uint32_t kOffQ = 0, kOffRing = 2 * kTile, kOffRaw = kOffRing + kSlots * kTile;
  static constexpr uint32_t kOffCtl = kOffRaw + kRaw * kRawBytes;
};

// Chunks whose `held` is kept: the producer is at most kSlots chunks ahead of the issuer, the
// softmax at most two behind it.
constexpr int kPxHeld = 16;

struct PxCtl {
  uint64_t kv_full[9], kv_empty[9], raw_full[3], raw_empty[3];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], o_free[2], drain, fix;  // (p: half the tokens each)
  uint32_t held[kPxHeld]; // which sub-blocks of 16 tokens of a chunk are held, a bit each
  uint32_t tmem;
  int abort;
  PxLine line[8];         // a softmax warp's place, which it does not need in registers meanwhile
};

// tokens 32 w .. 32 w + 31 of a chunk: held and below the length
__device__ __forceinline__ uint32_t px_seen(uint32_t held, int w, int tokens) {
  const uint32_t two = held >> (2 * w);
  const int n = tokens - 32 * w;
  return ((two & 1 ? 0xffffu : 0u) | (two & 2 ? 0xffff0000u : 0u)) & (n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1);
}

template <int FMT, int D>
__global__ void __launch_bounds__(PxCfg<FMT, D>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap map, const PrefixParams P) {
  using C = PxCfg<FMT, D>;
  constexpr bool F16 = C::kFp4;
  constexpr float kLift = F16 ? kPxLift : 0.f;
  constexpr uint32_t kIdescS = px_idesc(F16, kPxChunk, 0), kIdescO = px_idesc(F16, D, 1);
  extern __shared__ uint8_t px_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(px_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  PxCtl *ctl = reinterpret_cast<PxCtl *>(smem + C::kOffCtl);
  float *qscale = reinterpret_cast<float *>(ctl + 1);   // [kPxRows] (4-bit rows)
  const uint32_t q_at = smem_u32(smem + C::kOffQ), ring = smem_u32(smem + C::kOffRing);
  volatile int *abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&ctl->kv_full[i], F16 ? C::kConvWarps : 1);
      mbar_init(&ctl->kv_empty[i], 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&ctl->raw_full[i], 1);
      mbar_init(&ctl->raw_empty[i], C::kConvWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_full[s], 4);
      mbar_init(&ctl->s_full[s], 2);   // the products, and the issuer (for `held`)
      mbar_init(&ctl->p_full[s][0], 4);
      mbar_init(&ctl->p_full[s][1], 4);
      mbar_init(&ctl->o_full[s], 1);
      mbar_init(&ctl->o_free[s], 4);
    }
    mbar_init(&ctl->drain, 1);
    mbar_init(&ctl->fix, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kLoadWarp + 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;   // S of the sub-tiles at columns 0 and 128, O at 256 and 256 + D
  pdl_wait();
  pdl_launch_dependents();

  PxLine L;
  const bool any = L.begin(P, blockIdx.x == 0 && warp == 0);
  if (warp < C::kLoadWarp) {
    px_more_regs<C::kRegsSoft>();
    if (any) {
    // ===================== softmax: a warpgroup per sub-tile, a thread per row =====================
    const int s = warp >> 2, w4 = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t s_at = tmem + s * 128 + lanes, o_at = tmem + 256 + s * D + lanes;
    uint32_t ph_s = 0, ph_o = 0;
    int done = 0;       // chunks of the pieces before
    bool ok = true, active = L.sub_rows(s) > 0;

    // the queries of this warp's 32 rows: D / 8 lanes a row, 16 bytes each
    auto load_q = [&]() {
      constexpr int kLanes = D / 8, kPer = 32 / kLanes, kAhead = 8;
      const int n = L.sub_rows(s), d8 = lane % kLanes, mine = w4 * 32 + lane;
      const int64_t at = mine < n ? px_out_row(P, L, L.t * kPxRows + s * 128 + mine) : -1;
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += kAhead * kPer) {
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t from = __shfl_sync(~0u, at, r0 + u * kPer + lane / kLanes);
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          if (from >= 0) x[u] = *reinterpret_cast<const uint4 *>(P.q + from * D + d8 * 8);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int r = w4 * 32 + r0 + u * kPer + lane / kLanes;
          uint32_t v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          if constexpr (F16) {  // scaled by the power of two that brings the row's largest entry to [1, 2)
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v[k] << 16)), fabsf(__uint_as_float(v[k] & 0xffff0000u))));
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
            int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
            e = max(min(e, 126), -126);  // (zero rows, subnormal and infinite maxima)
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = pack2<true>(__uint_as_float(v[k] << 16) * inv, __uint_as_float(v[k] & 0xffff0000u) * inv);
            if (d8 == 0) qscale[s * 128 + r] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
          }
          uint8_t *dst = smem + C::kOffQ + s * C::kTile + (d8 >> 3) * C::kBlock + r * 128 + (((d8 & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4 *>(dst) = make_uint4(v[0] ^ P.q_sign, v[1] ^ P.q_sign, v[2] ^ P.q_sign, v[3] ^ P.q_sign);
        }
      }
      px_fence_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[s]);
    };

    if (active) load_q();
    for (bool more = true; more && ok;) {
      const int n = L.n, len0 = L.x.len - L.c * kPxChunk;  // (tokens from the piece's first on)
      const bool rows = active && w4 * 32 < L.sub_rows(s);  // of this warp
      if (lane == 0) ctl->line[warp] = L;
      __syncwarp();
      // (a row of zeros has the least scale; times a small softmax scale it would be zero, and a masked score's
      // infinity times that NaN: the host's bound on scale_log2 holds for the product)
      const float c = F16 && active ? fmaxf(P.scale_log2 * qscale[s * 128 + w4 * 32 + lane], kPxMinScale) : P.scale_log2;
      float m = kPxNone, l = 0.f;
      for (int i = 0; active && i < n; ++i) {
        if (!px_wait(&ctl->s_full[s], ph_s, abort, P.status)) {
          ok = false;
          break;
        }
        ph_s ^= 1;
        tc_fence_after();
        if (rows) {
          const uint32_t held = ctl->held[(done + i) % kPxHeld];
          const int tokens = len0 - i * kPxChunk;
          if (held != 0xffu || tokens < kPxChunk) {  // scores of tokens that are not there (rare: a loop)
#pragma unroll 1
            for (int w = 0; w < 4; ++w)
              for (uint32_t no = ~px_seen(held, w, tokens); no; no &= no - 1)
                asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(s_at + w * 32 + __ffs(no) - 1), "r"(0xff800000u)
                             : "memory");
            px_wait_st();
          }
          float v[4][32];      // S of the row
#pragma unroll
          for (int b = 0; b < 4; ++b) tmem_ld_32x32b_x32(s_at + b * 32, v[b]);
          tmem_wait_ld();
#pragma unroll
          for (int b = 0; b < 4; ++b) reg_fence_32(v[b]);
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 32; k += 8)
#pragma unroll
              for (int x = 0; x < 4; ++x) tops[x] = px_max3(tops[x], v[b][k + 2 * x], v[b][k + 2 * x + 1]);
          const float2 c2 = make_float2(c, c);
          float2 sums[2];
          uint32_t p[16], rest[F16 ? 1 : 16];
          // Weights of 32 tokens.  In bf16 two terms, the second the bf16 of what the first leaves out, as in the
          // decode kernel (one term: 2^-8 of a weight at most; the outputs' distance to 64 bits is then 2.1e-3
          // where all of two terms' 1.65e-3 is their own rounding to bf16; half as many products less, 64 us for
          // 83).  With 4-bit rows one fp16 term, as there: 2^-11 (two: 102 us for 72).
          auto weights = [&](int b) {
            const float2 m2 = make_float2(-m, -m);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 y = __ffma2_rn(make_float2(v[b][2 * k], v[b][2 * k + 1]), c2, m2);
              const float2 e = make_float2(ex2(y.x), ex2(y.y));
              sums[k & 1] = __fadd2_rn(sums[k & 1], e);
              p[k] = pack2<F16>(e.x, e.y);
              if constexpr (!F16) {
                const float2 left = __ffma2_rn(make_float2(__uint_as_float(p[k] << 16), __uint_as_float(p[k] & 0xffff0000u)),
                                               make_float2(-1.f, -1.f), e);
                rest[k] = pack2<F16>(left.x, left.y);
              }
            }
          };
          auto put = [&](int b) {
            px_st16(s_at + b * 16, p);
            if constexpr (!F16) px_st16(s_at + 64 + b * 16, rest);
          };
          // The first weights are worked out with the maximum as it was, beside the search for the new
          // one, which seldom is far above it; if it is (and with a piece's first chunk) again.
          sums[0] = sums[1] = make_float2(0.f, 0.f);
          weights(0);
          const float top = fmaxf(px_max3(tops[0], tops[1], tops[2]), tops[3]);
          const float x = top == -INFINITY ? kPxNone : fmaf(top, c, -kLift);
          if (__any_sync(~0u, i == 0 || x - m > kPxLazy)) {
            const float up = fmaxf(m, x), f = ex2(m - up);
            m = up;
            l *= f;
            if (i > 0) {
#pragma unroll 1
              for (int b = 0; b < D / 16; ++b) {
                uint32_t o[16];
                asm volatile(
                    "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                    : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]), "=r"(o[8]),
                      "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                    : "r"(o_at + b * 16)
                    : "memory");
                asm volatile("tcgen05.wait::ld.sync.aligned;"
                             : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]), "+r"(o[6]), "+r"(o[7]),
                               "+r"(o[8]), "+r"(o[9]), "+r"(o[10]), "+r"(o[11]), "+r"(o[12]), "+r"(o[13]), "+r"(o[14]), "+r"(o[15])
                             :
                             : "memory");
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                px_st16(o_at + b * 16, o);
              }
            }
            tmem_ld_32x32b_x32(s_at, v[0]);  // (read once more: registers are short)
            tmem_wait_ld();
            reg_fence_32(v[0]);
            sums[0] = sums[1] = make_float2(0.f, 0.f);
            weights(0);
          }
          put(0);
          weights(1);
          put(1);
          px_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[s][0]);
          weights(2);
          put(2);
          weights(3);
          put(3);
          l += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
          px_wait_st();
        } else if (lane == 0) {
          mbar_arrive(&ctl->p_full[s][0]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[s][1]);
      }
      if (!ok) break;
      done += n;
      L = ctl->line[warp];
      // where this row's part goes
      const bool valid = w4 * 32 + lane < L.sub_rows(s), head = L.c == 0;
      const int64_t to = head ? (valid ? px_out_row(P, L, L.t * kPxRows + s * 128 + w4 * 32 + lane) : 0)
                              : static_cast<int64_t>(blockIdx.x) * kPxRows + s * 128 + w4 * 32 + lane;
      __syncwarp();
      // every product with the queries is done: the next piece's go in
      more = L.next(P);
      const bool was = active;
      active = more && L.sub_rows(s) > 0;
      if (active) load_q();
      if (!was) continue;
      if (!px_wait(&ctl->o_full[s], ph_o, abort, P.status)) {
        ok = false;
        break;
      }
      ph_o ^= 1;
      tc_fence_after();
      if (rows) {
        float *dst = (head ? P.first_o : P.rest_o) + to * D;
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
          float v[32];
          tmem_ld_32x32b_x32(o_at + b * 32, v);
          tmem_wait_ld();
          reg_fence_32(v);
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) px_store8(dst + b * 32 + k, v + k);
          }
        }
        if (valid) (head ? P.first_ml : P.rest_ml)[to] = make_float2(m == kPxNone && l == 0.f ? -INFINITY : m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free[s]);
    }
    }
  } else if (warp < C::kConvWarp) {
    px_fewer_regs<C::kRegsLoad>();
    if (any && warp == C::kLoadWarp) {
    // ===================== producer =====================
    const int boxes = F16 ? kPxChunk / kSubTokens : kPxChunk / P.box, box = F16 ? kSubTokens : P.box;
    int k = 0, asked = 0;  // chunks, and (bf16) tiles, asked for
    bool ok = true;
    // the row and offset of this lane's box of a chunk, looked up a chunk ahead
    int off = 0;
    int64_t row = -1;
    uint32_t ph_fix = 0;
    auto look_up = [&](int chunk) {
      const int token = chunk * kPxChunk + lane * box;
      row = lane < boxes && token < L.x.len ? px_row(P, L.g, L.h, token, off, true) : -1;
    };
    look_up(L.c);
    for (bool more = true; more && ok;) {
      const int n = L.n, c0 = L.c, len = L.x.len;
      for (int i = 0; i < n && ok; ++i) {
        const int64_t row_now = row;
        const int off_now = off;
        if (i + 1 < n) {
          look_up(c0 + i + 1);
        } else {
          more = L.next(P);
          if (more) look_up(L.c);
        }
        const uint32_t held = __ballot_sync(~0u, row_now >= 0);
        if constexpr (F16) {
          const int st = k % C::kRaw;
          if (k >= C::kRaw && !px_wait(&ctl->raw_empty[st], (k / C::kRaw - 1) & 1, abort, P.status)) {
            ok = false;
            break;
          }
          __syncwarp();
          if (lane == 0) {
            ctl->held[k % kPxHeld] = held;
            mbar_arrive_expect_tx(&ctl->raw_full[st], __popc(held) * 18 * D);
          }
          __syncwarp();
          if (row_now >= 0)
            px_bulk(smem_u32(smem + C::kOffRaw) + st * C::kRawBytes + lane * 18 * D,
                    P.rows + row_now * P.row_bytes + (off_now / kSubTokens) * Fp4Sub<D>::kBytes, 18 * D, &ctl->raw_full[st]);
        } else {
          uint32_t subs = held;   // the same by 16 tokens
          if (box != kSubTokens) {
            subs = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) subs |= (held >> (x * kSubTokens / box) & 1) << x;
          }
          if (lane == 0) ctl->held[k % kPxHeld] = subs;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int tile = 2 * k + v, st = tile % C::kSlots;
            if (tile >= C::kSlots && !px_wait(&ctl->kv_empty[st], (tile / C::kSlots - 1) & 1, abort, P.status)) {
              ok = false;
              break;
            }
            __syncwarp();
            // values that no query sees have to be zeros (a weight of zero times NaN is NaN): the tile
            // is waited for here, mended, and handed on
            const int tokens = len - (c0 + i) * kPxChunk;
            const bool mend = v == 1 && (subs != 0xffu || tokens < kPxChunk);
            uint64_t *bar = mend ? &ctl->fix : &ctl->kv_full[st];
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(held) * box * 2 * D);
            __syncwarp();
            if (row_now >= 0) {
#pragma unroll
              for (int hb = 0; hb < D / 64; ++hb)
                px_tma(ring + st * C::kTile + hb * C::kBlock + lane * box * 128, &map, bar, hb * 64, off_now,
                       static_cast<int>(2 * row_now + v));
            }
            if (mend) {
              if (!px_wait(&ctl->fix, ph_fix, abort, P.status)) {
                px_drain(&ctl->fix, ph_fix);
                ok = false;
                break;
              }
              ph_fix ^= 1;
              uint8_t *tile_at = smem + C::kOffRing + st * C::kTile;
#pragma unroll
              for (int w = 0; w < 4; ++w)
                if (!(px_seen(subs, w, tokens) >> lane & 1))
                  for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<uint4 *>(tile_at + (x >> 3) * C::kBlock + (w * 32 + lane) * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              px_fence_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl->kv_full[st]);
            }
            asked = tile + 1;
          }
        }
        if (ok) ++k;
      }
    }
    if (*abort) {  // let every copy this warp started land before the CTA exits
      constexpr int kDepth = F16 ? (C::kRaw ? C::kRaw : 1) : C::kSlots;
      const int n = F16 ? k : asked;
      for (int j = max(n - kDepth, 0); j < n; ++j) px_drain(F16 ? &ctl->raw_full[j % kDepth] : &ctl->kv_full[j % kDepth], (j / kDepth) & 1);
    }
    } else if (any && warp == C::kLoadWarp + 1) {
    // ===================== tensor-core issuer: one thread =====================
    if (elect_one()) {
      uint32_t ph_q[2] = {0, 0}, ph_p[2] = {0, 0}, ph_free[2] = {1, 1};  // (O is free at first)
      int k = 0;        // tiles taken from the ring
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && px_wait(bar, parity, abort, P.status); };
      auto full = [&](int tile) { return wait(&ctl->kv_full[tile % C::kSlots], (tile / C::kSlots) & 1); };
      auto scores = [&](int s, int tile) {     // S of sub-tile s
        tc_fence_after();
        const PxDesc a(kmajor_sw128_desc(q_at + s * C::kTile)), b(kmajor_sw128_desc(ring + (tile % C::kSlots) * C::kTile));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          px_mma_ss(tmem + s * 128, a, b, ((kk >> 2) * C::kBlock + (kk & 3) * 32) >> 4, kIdescS, kk > 0);
        mma_commit(&ctl->s_full[s]);
        mbar_arrive(&ctl->s_full[s]);
      };
      auto values = [&](int s, int tile, int half, bool more) {  // O of sub-tile s, half the tokens, the terms of P
        tc_fence_after();
        const PxDesc b(px_mn_desc(ring + (tile % C::kSlots) * C::kTile, C::kBlock));
#pragma unroll
        for (int kk = 0; kk < kPxChunk / 32; ++kk)
#pragma unroll
          for (int term = 0; term < (F16 ? 1 : 2); ++term)
            px_mma_ts(tmem + 256 + s * D, tmem + s * 128 + term * 64 + half * 32 + kk * 8, b, (half * 64 + kk * 16) * 128 >> 4, kIdescO,
                      more || kk > 0 || term > 0);
      };
      auto release = [&](int tile) { mma_commit(&ctl->kv_empty[tile % C::kSlots]); };
      for (bool more = true; more && ok; more = ok && L.next(P)) {
        const int subs = L.sub_rows(1) > 0 ? 2 : 1;
        if (!full(k)) break;
        for (int s = 0; s < subs; ++s) {
          if (!wait(&ctl->q_full[s], ph_q[s])) break;
          ph_q[s] ^= 1;
          scores(s, k);
        }
        if (!ok) break;
        release(k);
        for (int i = 0; i < L.n && ok; ++i, k += 2) {
          const bool last = i + 1 == L.n;
          if (!full(k + 1) || (!last && !full(k + 2))) break;
          for (int s = 0; s < subs; ++s) {
            if (!wait(&ctl->p_full[s][0], ph_p[s])) break;
            if (i == 0) {
              if (!wait(&ctl->o_free[s], ph_free[s])) break;
              ph_free[s] ^= 1;
            }
            values(s, k + 1, 0, i > 0);
            if (!wait(&ctl->p_full[s][1], ph_p[s])) break;
            ph_p[s] ^= 1;
            values(s, k + 1, 1, true);
            if (s == subs - 1) release(k + 1);
            if (last) {
              mma_commit(&ctl->o_full[s]);
            } else {
              scores(s, k + 2);
              if (s == subs - 1) release(k + 2);
            }
          }
        }
      }
      if (!ok) {  // no product may run on when the tensor memory goes
        mma_commit(&ctl->drain);
        px_drain(&ctl->drain, 0);
      }
    }
    }
  } else if constexpr (F16) {
    px_fewer_regs<C::kRegsConv>();
    if (any) {
    // ===================== 4-bit rows to fp16 tiles: two sub-blocks a warp, a lane per (token, half of the dims) ====
    constexpr int kWords = D / 16;      // 8-code words of a lane
    const int tk = lane & 15, hf = lane >> 4;
    int k = 0;
    bool ok = true;
    // one sub-block's keys or values as rows of a tile
    auto convert = [&](uint8_t *tile, int sub, const uint32_t (&w)[kWords], const uint32_t (&sc)[kWords / 2], bool on) {
      const int r = sub * kSubTokens + tk;
      uint8_t *dst = tile + (D == 128 ? hf * C::kBlock : 0u) + r * 128;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t s2 = __byte_perm(e4m3x2_to_half2(sc[i / 2]), 0, 0x1010);
        uint32_t h[4];
        e2m1x8_to_half2(w[i], h);
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] = on ? hmul2(h[v], s2) : 0u;
        const int piece = D == 128 ? i : hf * kWords + i;
        *reinterpret_cast<uint4 *>(dst + ((piece ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    };
    for (bool more = true; more && ok; more = ok && L.next(P)) {
      for (int i = 0; i < L.n && ok; ++i, ++k) {
        const int st = k % C::kRaw, tokens = L.x.len - (L.c + i) * kPxChunk;
        if (!px_wait(&ctl->raw_full[st], (k / C::kRaw) & 1, abort, P.status)) {
          ok = false;
          break;
        }
        const uint32_t held = ctl->held[k % kPxHeld];
        const uint8_t *src = smem + C::kOffRaw + st * C::kRawBytes;
#pragma unroll
        for (int v = 0; v < 2; ++v) {    // keys, then values
          uint32_t w[2][kWords], sc[2][kWords / 2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint8_t *from = src + ((warp - C::kConvWarp) * 2 + u) * 18 * D;
            if (v == 0) {                // codes [16][D / 2], scales [16][D / 16]
#pragma unroll
              for (int x = 0; x < kWords / 4; ++x) {
                const uint4 y = *reinterpret_cast<const uint4 *>(from + tk * (D / 2) + hf * (D / 4) + x * 16);
                w[u][4 * x] = y.x, w[u][4 * x + 1] = y.y, w[u][4 * x + 2] = y.z, w[u][4 * x + 3] = y.w;
              }
#pragma unroll
              for (int x = 0; x < kWords / 2; ++x) sc[u][x] = from[Fp4Sub<D>::kKeyScales + tk * (D / 16) + hf * (D / 32) + x];
            } else {                     // codes [2][8][8 tokens][D / 16], scales [2][D / 16][8 tokens]
              const uint8_t *vc = from + Fp4Sub<D>::kValues + (tk >> 3) * (4 * D) + (hf * 4 * 8 + (tk & 7)) * (D / 16);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if constexpr (D == 128) {
                  const uint2 y = *reinterpret_cast<const uint2 *>(vc + x * 8 * (D / 16));
                  w[u][2 * x] = y.x, w[u][2 * x + 1] = y.y;
                } else {
                  w[u][x] = *reinterpret_cast<const uint32_t *>(vc + x * 8 * (D / 16));
                }
              }
#pragma unroll
              for (int x = 0; x < kWords / 2; ++x)
                sc[u][x] = from[Fp4Sub<D>::kValueScales + (tk >> 3) * (D / 2) + (hf * (D / 32) + x) * 8 + (tk & 7)];
            }
          }
          if (v == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->raw_empty[st]);
          }
          const int tile = 2 * k + v, sl = tile % C::kSlots;
          if (tile >= C::kSlots && !px_wait(&ctl->kv_empty[sl], (tile / C::kSlots - 1) & 1, abort, P.status)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int sub = (warp - C::kConvWarp) * 2 + u;
            convert(smem + C::kOffRing + sl * C::kTile, sub, w[u], sc[u], (held >> sub & 1) && sub * kSubTokens + tk < tokens);
          }
          px_fence_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->kv_full[sl]);
        }
      }
    }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kLoadWarp + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// merge: RW warps per query row, each with every RW-th piece
// ---------------------------------------------------------------------------
constexpr int kPxMergeWarps = 8;

template <int D, int RW>
__global__ void __launch_bounds__(kPxMergeWarps * 32) prefix_merge_kernel(const PrefixParams P) {
  constexpr int kPer = D / 32;      // dims of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine_of = warp % RW;      // which of the row's warps
  __shared__ float4 joined[RW > 1 ? kPxMergeWarps : 1][32];
  __shared__ float2 joined_ml[RW > 1 ? kPxMergeWarps : 1];
  const int64_t all = static_cast<int64_t>(P.B) * P.n_q * P.n_heads;
  const int64_t at_row = static_cast<int64_t>(blockIdx.x) * (kPxMergeWarps / RW) + warp / RW, row = at_row < all ? at_row : all - 1;
  pdl_launch_dependents();
  // (Where the row's tile lies is found before the wait: it comes of the call's inputs alone, and the
  // prefix's kernel, which lets this one and the own tokens' start, has waited for whatever wrote them.
  // That it is seen here without a wait goes, as in the own tokens' kernel, beyond what the documents promise.)
  const uint32_t bj = static_cast<uint32_t>(row) / static_cast<uint32_t>(P.n_heads), head = static_cast<uint32_t>(row) - bj * P.n_heads;
  const int b = bj / static_cast<uint32_t>(P.n_q), j = bj - b * P.n_q, h = head / static_cast<uint32_t>(P.group);

  // where the row's tile lies on the line
  const int run = (P.n_groups + 31) / 32, g0 = min(lane * run, P.n_groups), g1 = min(g0 + run, P.n_groups);
  uint32_t mine = 0;
  int u = 0, total, at = -1, r = 0;
  PxGroup last{};
  for (int g = g0; g < g1; ++g) {
    const PxGroup x = last = px_group(P, g, false);
    const int in = (b - x.b0) * P.n_q * P.group;   // (rows of a request outside the group are not below x.rows)
    if (at < 0 && x.chunks > 0 && b >= x.b0 && in < x.rows) at = g, u = mine, r = in + j * P.group + head - h * P.group;
    mine = px_add(mine, px_units(P, x));
  }
  u += px_scan(mine, total);
  const PxPlan plan = px_plan(P, last, total);
  const uint32_t who = __ballot_sync(~0u, at >= 0 && total > 0);
  int first = 0, pieces = 0, step = 1;   // the tile's first CTA, how many pieces it has, their CTAs' distance
  if (who) {
    const int src = __ffs(who) - 1;
    at = __shfl_sync(~0u, at, src);
    u = __shfl_sync(~0u, u, src);
    r = __shfl_sync(~0u, r, src);
    const PxGroup x = px_group_of(P, last, at);
    const int tile = r / kPxRows;
    if (plan.whole) {
      int len;
      for (int g = 0; g < at; ++g) {
        const PxGroup y = px_group_of(P, last, g);
        first += P.n_kv * y.tiles * px_pieces(plan, y, len);
      }
      pieces = px_pieces(plan, x, len);
      first += h * pieces * x.tiles + tile;
      step = x.tiles;
    } else {
      u += (h * x.tiles + tile) * x.chunks;
      first = u / plan.per;
      pieces = (u + x.chunks - 1) / plan.per - first + 1;
    }
    r %= kPxRows;
  }

  pdl_wait();
  auto load = [&](const float *o, float (&x)[kPer]) {   // (under way from here on)
    if constexpr (kPer == 4) {
      const uint4 y = load16_here(o);
      x[0] = __uint_as_float(y.x), x[1] = __uint_as_float(y.y), x[2] = __uint_as_float(y.z), x[3] = __uint_as_float(y.w);
    } else {
      const uint2 y = load8_here(o);
      x[0] = __uint_as_float(y.x), x[1] = __uint_as_float(y.y);
    }
  };
  float own_x[kPer], own_lse = -INFINITY;
#pragma unroll
  for (int k = 0; k < kPer; ++k) own_x[k] = 0.f;
  if (mine_of == 0 && P.own_o) {
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(own_lse) : "l"(P.own_lse + row));
    load(P.own_o + row * D + lane * kPer, own_x);
  }
  float top = -INFINITY, sum = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  constexpr int kAhead = RW > 1 ? 6 : 4;
  for (int p0 = mine_of; p0 < pieces; p0 += kAhead * RW) {   // pieces p0, p0 + RW, ...
    float2 ml[kAhead];
    float x[kAhead][kPer];
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      ml[p] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[p][k] = 0.f;
      const int i = p0 + p * RW;
      if (i < pieces) {   // (the first in a row per query row, the others in their CTAs' slots)
        const int64_t from = i ? static_cast<int64_t>(first + i * step) * kPxRows + r : row;
        const uint2 y = load8_here((i ? P.rest_ml : P.first_ml) + from);
        ml[p] = make_float2(__uint_as_float(y.x), __uint_as_float(y.y));
        load((i ? P.rest_o : P.first_o) + from * D + lane * kPer, x[p]);
      }
    }
    float up = top;
#pragma unroll
    for (int p = 0; p < kAhead; ++p) up = fmaxf(up, ml[p].x);
    const float f = top == -INFINITY ? 0.f : ex2(top - up);
    sum *= f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] *= f;
    top = up;
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      if (ml[p].x == -INFINITY) continue;  // (nothing seen; a sum that is NaN has a maximum all the same)
      const float e = ex2(ml[p].x - top);
      sum = fmaf(ml[p].y, e, sum);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(x[p][k], e, acc[k]);
    }
  }
  if constexpr (RW > 1) {   // the row's warps, in order
    if (lane == 0) joined_ml[warp] = make_float2(top, sum);
    float *mine_at = reinterpret_cast<float *>(&joined[warp][lane]);
#pragma unroll
    for (int k = 0; k < kPer; ++k) mine_at[k] = acc[k];
    __syncthreads();
    if (mine_of != 0 || at_row >= all) return;
#pragma unroll
    for (int w = 1; w < RW; ++w) {
      const float2 ml = joined_ml[warp + w];
      if (ml.x == -INFINITY) continue;
      const float up = fmaxf(top, ml.x), f = top == -INFINITY ? 0.f : ex2(top - up), e = ex2(ml.x - up);
      const float *o = reinterpret_cast<const float *>(&joined[warp + w][lane]);
      top = up;
      sum = fmaf(ml.y, e, sum * f);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(o[k], e, acc[k] * f);
    }
  } else if (at_row >= all) {
    return;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] *= P.v_scale;
  if (P.own_o) {                    // divided by its sum already: weight 2^lse, sum 1
    const float lse = own_lse * 1.4426950408889634f;
    if (lse != -INFINITY) {
      const float up = fmaxf(top, lse), f = top == -INFINITY ? 0.f : ex2(top - up), e = ex2(lse - up);
      top = up;
      sum = fmaf(sum, f, e);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(own_x[k], e, acc[k] * f);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : sum;  // (a NaN sum stays one)
  uint32_t *dst = reinterpret_cast<uint32_t *>(P.out + row * D + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) dst[k] = pack2<false>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  if (P.lse && lane == 0) P.lse[row] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

}  // namespace echo

namespace echo_host {

size_t block_attention_workspace_bytes(int32_t rows, int32_t head_dim);
int launch_block_attention_f32(const echo_block_attention_args *a, float *out, cudaStream_t stream);

// workspace: pieces that begin with a tile | pieces that do not | the own tokens' results | the
// decode kernel's own workspace
struct PxSpace {
  size_t first_ml, rest_o, rest_ml, own_o, own_lse, own_ws, end;
};
static PxSpace px_space(int64_t rows, int32_t rows_per_kv_head, int32_t head_dim) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  PxSpace s;
  s.first_ml = up(static_cast<size_t>(rows) * head_dim * 4);
  s.rest_o = s.first_ml + up(static_cast<size_t>(rows) * 8);
  s.rest_ml = s.rest_o + up(static_cast<size_t>(echo::kPxMaxGrid) * echo::kPxRows * head_dim * 4);
  s.own_o = s.rest_ml + up(static_cast<size_t>(echo::kPxMaxGrid) * echo::kPxRows * 8);
  s.own_lse = s.own_o + up(static_cast<size_t>(rows) * head_dim * 4);
  s.own_ws = s.own_lse + up(static_cast<size_t>(rows) * 4);
  s.end = s.own_ws + up(block_attention_workspace_bytes(rows_per_kv_head, head_dim));
  return s;
}

size_t prefix_attention_workspace_bytes(int32_t B, int32_t n_q, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  return px_space(static_cast<int64_t>(B) * n_q * n_heads, n_q * (n_heads / n_kv_heads), head_dim).end;
}

typedef CUresult (*PFN_encodeTiledX)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                     const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// keys and values of bf16 rows as [2 n_rows][block_tokens][head_dim], boxes of `box` tokens and 64 dims
static int px_map(const echo::PrefixParams &P, int D, CUtensorMap *map) {
  static std::atomic<PFN_encodeTiledX> known{nullptr};
  PFN_encodeTiledX enc = known.load(std::memory_order_acquire);
  if (!enc) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      set_error("cuTensorMapEncodeTiled unavailable from the driver");
      return ECHO_ECUDA;
    }
    enc = reinterpret_cast<PFN_encodeTiledX>(p);
    known.store(enc, std::memory_order_release);
  }
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(P.bs), 2 * static_cast<cuuint64_t>(P.n_rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(P.bs) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(P.box), 1}, es[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t *>(P.rows), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("tensor map for rows failed (CUresult %d)", static_cast<int>(r));
    return ECHO_ECUDA;
  }
  return ECHO_OK;
}

template <int FMT, int D>
static int go_prefix(const echo::PrefixParams &P, cudaStream_t stream) {
  using C = echo::PxCfg<FMT, D>;
  constexpr int kSmem = C::kOffCtl + sizeof(echo::PxCtl) + (C::kFp4 ? echo::kPxRows * 4 : 0) + 1024;
  static_assert(kSmem <= 232448, "prefix attention: shared memory of one CTA");
  static std::atomic<bool> attr[kMaxDevices];
  if (int rr = smem_limit_once(attr, echo::prefix_attn_kernel<FMT, D>, kSmem, "prefix attention smem attribute")) return rr;
  // (the warpgroups' shares have to fit what the launch gets: a build that needs fewer registers is refused)
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, echo::prefix_attn_kernel<FMT, D>);
    if (e != cudaSuccess) return cuda_fail(e, "prefix attention attributes");
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < C::kRegs) {
    set_error("prefix attention was built with %d registers, its warpgroups need %d", regs.load(), C::kRegs);
    return ECHO_ENOTSUP;
  }
  CUtensorMap map{};
  if (!C::kFp4)
    if (int rr = px_map(P, D, &map)) return rr;
  cudaError_t e = launch_pdl(echo::prefix_attn_kernel<FMT, D>, dim3(P.grid), dim3(C::kThreads), kSmem, stream, map, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "prefix attention launch");
}

template <int D, int RW>
static cudaError_t go_merge(const echo::PrefixParams &P, int64_t rows, cudaStream_t stream) {
  constexpr int64_t per = echo::kPxMergeWarps / RW;
  return launch_pdl(echo::prefix_merge_kernel<D, RW>, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(echo::kPxMergeWarps * 32), 0,
                    stream, P);
}

int launch_prefix_attention(const echo_prefix_attention_args *a, cudaStream_t stream) {
  int sms = 0;
  if (int rr = sm_count(&sms, "prefix attention device")) return rr;
  const int64_t rows = static_cast<int64_t>(a->B) * a->n_q * a->n_heads;
  const PxSpace s = px_space(rows, a->n_q * (a->n_heads / a->n_kv_heads), a->head_dim);
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  echo::PrefixParams P{};
  P.q = a->q, P.rows = reinterpret_cast<const uint8_t *>(a->rows);
  P.row_bytes = 2 * echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.n_rows = a->n_rows, P.bs = a->block_tokens;
  for (P.box = 128; a->block_tokens % P.box; P.box /= 2) {
  }
  P.table = a->prefix_table, P.heads = a->prefix_heads, P.max_blocks = a->max_prefix_blocks;
  P.len = a->prefix_len, P.start = a->group_start, P.n_groups = a->n_groups;
  P.B = a->B, P.n_q = a->n_q, P.n_heads = a->n_heads, P.n_kv = a->n_kv_heads, P.group = a->n_heads / a->n_kv_heads;
  // (not zero: it has to leave a masked score's infinity what it is)
  P.scale_log2 = std::max(std::ldexp(std::fabs(a->scale) * 1.4426950408889634f, -a->k_shift), echo::kPxMinScale);
  P.v_scale = std::ldexp(1.f, -a->v_shift);
  P.q_sign = a->scale < 0.f ? 0x80008000u : 0u;
  P.first_o = reinterpret_cast<float *>(ws), P.first_ml = reinterpret_cast<float2 *>(ws + s.first_ml);
  P.rest_o = reinterpret_cast<float *>(ws + s.rest_o), P.rest_ml = reinterpret_cast<float2 *>(ws + s.rest_ml);
  P.out = a->out, P.lse = a->lse, P.status = a->dev_status;
  P.grid = std::min(sms, echo::kPxMaxGrid);
  P.room = a->table && static_cast<int64_t>(a->B) * a->n_kv_heads * 4 >= sms;
  if (a->table) P.own_o = reinterpret_cast<float *>(ws + s.own_o), P.own_lse = reinterpret_cast<float *>(ws + s.own_lse);

  int r;
  if (a->format == ECHO_BLOCK_FP4) r = a->head_dim == 128 ? go_prefix<ECHO_BLOCK_FP4, 128>(P, stream) : go_prefix<ECHO_BLOCK_FP4, 64>(P, stream);
  else r = a->head_dim == 128 ? go_prefix<ECHO_BLOCK_BF16, 128>(P, stream) : go_prefix<ECHO_BLOCK_BF16, 64>(P, stream);
  if (r) return r;
  if (a->table) {
    echo_block_attention_args o{};
    o.q = a->q, o.rows = a->rows, o.n_rows = a->n_rows, o.format = a->format, o.block_tokens = a->block_tokens, o.head_dim = a->head_dim;
    o.table = a->table, o.table_heads = a->table_heads, o.max_blocks = a->max_blocks, o.ctx_len = a->ctx_len;
    o.B = a->B, o.n_q = a->n_q, o.n_heads = a->n_heads, o.n_kv_heads = a->n_kv_heads, o.scale = a->scale;
    o.lse = reinterpret_cast<float *>(ws + s.own_lse), o.workspace = ws + s.own_ws, o.dev_status = a->dev_status;
    o.k_shift = a->k_shift, o.v_shift = a->v_shift;
    if (int rr = launch_block_attention_f32(&o, reinterpret_cast<float *>(ws + s.own_o), stream)) return rr;
  }
  // four warps a row where there are few rows (1024 of a prefix of 2048: 14.8 us in all, with one 16.4), one
  // where four would make several waves of CTAs (4096 of a prefix of 32768: 83.4 us, with four 90.2)
  const cudaError_t e = a->head_dim == 128 ? (rows <= 2048 ? go_merge<128, 4>(P, rows, stream) : go_merge<128, 1>(P, rows, stream))
                         : (rows <= 2048 ? go_merge<64, 4>(P, rows, stream) : go_merge<64, 1>(P, rows, stream));
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "prefix attention merge launch");
}

}  // namespace echo_host
