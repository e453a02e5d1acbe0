// block_pick.cuh -- the want-th largest of a set of keys that a warp or a block holds, for the
// selections over block scores and over gathered weights.
//
// One pass counts the keys in equal parts of their range, and the part that holds the want-th largest is
// found from the counts.  Its keys, a few as a rule, are gathered and ranked against one another, a
// thread each; more of them (equal ones above all: 410 zeros ranked take 15 us) are settled by halving
// their range, which sees at once how many equal its lowest.  (Halving the whole range takes up to 31
// passes: a row of 1024 block scores 19 us, 8 prompts of 32768 weights 102 us in all.)
#pragma once

#include "block_rows.cuh"

namespace echo {

// Scratch of a group of W warps that counts in BINS parts.
template <int W, int BINS>
struct PickSpace {
  static constexpr int kBins = BINS, kFew = W * 32 < 96 ? W * 32 : 96;
  alignas(16) uint32_t hist[BINS];
  uint32_t red[3][W];
  uint32_t pick[3];
  uint32_t few[kFew], n_few;
};

template <int W>
__device__ __forceinline__ void pick_sync() {
  if constexpr (W > 1) __syncthreads();
  else __syncwarp();
}

// sum over the group (turn: 0 and 1 by turns, so that one barrier does)
template <int W, int BINS>
__device__ __forceinline__ uint32_t pick_sum(PickSpace<W, BINS> &S, uint32_t x, int turn) {
  x = __reduce_add_sync(~0u, x);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) S.red[turn][threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) x += S.red[turn][w];
  }
  return x;
}
template <int W, int BINS>
__device__ __forceinline__ uint32_t pick_min(PickSpace<W, BINS> &S, uint32_t x, int turn) {
  x = __reduce_min_sync(~0u, x);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) S.red[turn][threadIdx.x >> 5] = x;
    __syncthreads();
    x = S.red[turn][0];
#pragma unroll
    for (int w = 1; w < W; ++w) x = min(x, S.red[turn][w]);
  }
  return x;
}

// sum of n, minimum of lo and maximum of hi over the group, with one barrier
template <int W, int BINS>
__device__ __forceinline__ void pick_stats(PickSpace<W, BINS> &S, uint32_t &n, uint32_t &lo, uint32_t &hi) {
  n = __reduce_add_sync(~0u, n), lo = __reduce_min_sync(~0u, lo), hi = __reduce_max_sync(~0u, hi);
  if constexpr (W > 1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) S.red[0][warp] = n, S.red[1][warp] = lo, S.red[2][warp] = hi;
    __syncthreads();
    n = __reduce_add_sync(~0u, lane < W ? S.red[0][lane % W] : 0u);
    lo = __reduce_min_sync(~0u, S.red[1][lane % W]), hi = __reduce_max_sync(~0u, S.red[2][lane % W]);
  } else {
    __syncwarp();
  }
}

// Empties the counts: before a barrier that comes before pick_kth.
template <int W, int BINS>
__device__ __forceinline__ void pick_clear(PickSpace<W, BINS> &S) {
  const int tid = W > 1 ? threadIdx.x : threadIdx.x & 31;
  for (int i = tid; i < BINS; i += W * 32) S.hist[i] = 0;
  if (tid == 0) S.n_few = 0;
}

// thr and need such that the keys whose ord() lies above thr, and the first `need` whose ord() is thr,
// are the `want` largest (0 < want < their number) of the keys that count.  each(f) calls f on each key of
// the thread; counts(key): whether it is one of them; ord(key) orders them as whole numbers above 0;
// bin(key) in [0, BINS) does not fall as ord(key) grows.  Returns whether all that equal thr are
// taken.
template <int W, int BINS, class Each, class Counts, class Bin, class Ord>
__device__ __forceinline__ bool pick_kth(PickSpace<W, BINS> &S, uint32_t want, Each &&each, Counts &&counts, Bin &&bin, Ord &&ord,
                                         uint32_t &thr, uint32_t &need) {
  const int lane = threadIdx.x & 31, tid = W > 1 ? threadIdx.x : lane;
  each([&](auto key) {
    if (counts(key)) atomicAdd(&S.hist[bin(key)], 1u);
  });
  pick_sync<W>();
  int part;
  uint32_t above, in;
  if constexpr (BINS <= 256) {   // every warp by itself: 8 parts a lane, the first lane the highest ones
    static_assert(BINS == 256, "two 16-byte pieces a lane");
    const uint4 hi4 = *reinterpret_cast<const uint4 *>(&S.hist[252 - 8 * lane]), lo4 = *reinterpret_cast<const uint4 *>(&S.hist[248 - 8 * lane]);
    const uint32_t n[8] = {hi4.w, hi4.z, hi4.y, hi4.x, lo4.w, lo4.z, lo4.y, lo4.x};
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += n[i];
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    above = upto - sum;
    const int src = __ffs(__ballot_sync(~0u, upto >= want)) - 1;
    int i = 0;
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (i == k && above + n[k] < want) above += n[k], i = k + 1;
    part = __shfl_sync(~0u, 255 - 8 * lane - i, src), above = __shfl_sync(~0u, above, src), in = __shfl_sync(~0u, pick_reg(n, i), src);
  } else {       // a thread holds kPer bins, the first thread the highest ones
    constexpr int kPer = BINS / (W * 32) > 0 ? BINS / (W * 32) : 1;
    static_assert(BINS % kPer == 0 && (BINS / kPer) % 32 == 0, "whole warps of bins");
    const bool on = tid < BINS / kPer;
    uint32_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n[i] = on ? S.hist[BINS - 1 - kPer * tid - i] : 0u, sum += n[i];
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    if constexpr (W > 1) {
      if (lane == 31) S.red[0][threadIdx.x >> 5] = upto;
      __syncthreads();
      for (int w = 0; w < (threadIdx.x >> 5); ++w) upto += S.red[0][w];
    }
    above = upto - sum;
    if (on && above < want && upto >= want) {
      int i = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (i == k && above + n[k] < want) above += n[k], i = k + 1;
      S.pick[0] = BINS - 1 - kPer * tid - i, S.pick[1] = above, S.pick[2] = pick_reg(n, i);
    }
    pick_sync<W>();
    part = S.pick[0], above = S.pick[1], in = S.pick[2];
  }
  want -= above;
  if (in <= S.kFew) {
    each([&](auto key) {
      if (bin(key) == part && counts(key)) S.few[atomicAdd(&S.n_few, 1u)] = ord(key);
    });
    pick_sync<W>();
    if (tid < in) {           // (in any order: only counts come of it)
      const uint32_t mine = S.few[tid];
      uint32_t above = 0, equal = 0;
#pragma unroll 4
      for (int i = 0; i < in; ++i) above += S.few[i] > mine, equal += S.few[i] == mine;
      if (above < want && above + equal >= want) S.pick[0] = mine, S.pick[1] = want - above, S.pick[2] = equal;  // (its equals: the same)
    }
    pick_sync<W>();
    thr = S.pick[0], need = S.pick[1];
    return need == S.pick[2];
  }
  uint32_t lo = ~0u, hi = 0;   // the part's keys
  each([&](auto key) {
    if (bin(key) == part && counts(key)) lo = min(lo, ord(key)), hi = max(hi, ord(key));
  });
  lo = pick_min(S, lo, 0);
  hi = ~pick_min(S, ~hi, 1);
  // of the keys in [lo, hi], more than `want` (or all) lie above `below`, above_hi < want above `top`
  uint32_t below = lo - 1, top = hi, above_hi = 0, mid = lo;   // (many equal to the lowest: seen at once)
  need = 0;
  for (int turn = 0;; turn ^= 1) {
    if (top - below == 1) {    // equal keys: the first of them
      thr = top, need = want - above_hi;
      return false;
    }
    uint32_t c = 0;
    each([&](auto key) { c += counts(key) && ord(key) > mid && ord(key) <= hi; });
    c = pick_sum(S, c, turn);
    if (c == want) {
      thr = mid;      // (a key in between, or one of which none is needed)
      return false;
    }
    if (c > want) below = mid;
    else top = mid, above_hi = c;
    mid = below + (top - below) / 2;
  }
}

}  // namespace echo
