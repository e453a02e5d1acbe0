// block_tables.cu -- block tables and slot maps of a serving step, from request lengths.
//
// Request b goes from old_len[b] to new_len[b] tokens.  With nb(n) = ceil(n / bs):
//   f_b = max(0, nb(old) - nb(new)) blocks return to the free stack,
//   a_b = max(0, nb(new) - nb(old)) blocks are taken from it,
//   n_b = max(0, new - old) tokens are listed with their slots.
// Everything follows from the exclusive sums F, A, N of the three: freed block i of b is
// entry count + F_b + i of the stack, grown block i of b is entry top - 1 - (A_b + i) with
// top = count + sum f, and token i of the list belongs to the b with N_b <= i < N_{b+1}.
//
// One launch: every CTA forms the three sums itself (B <= 16384 lengths, read from L2; the
// sums stay in shared memory) and then takes its share of the blocks and of the list, so
// no CTA waits for another.  A stack entry at or above `count` is read where it comes from
// (the shrinking request's table), never from the stack the same launch is writing.
// Bound by latency: 64 decoding requests 2.7 us (lengths, sums, search, id, store, an entry
// per thread; four in a row per thread took 3.3 us more), 256 requests in a mixed step with a
// list of 2^20 entries 7.6 us, of which the launch and the sums take 3.2, the list's stores (8
// MB) and the moved blocks 2.2 to 2.9, and the searches and the table's look-ups the rest.
#include <algorithm>

#include "block_rows.cuh"

namespace echo {

constexpr int kTabThreads = 256;

struct TablesParams {
  const int32_t *old_len, *new_len;
  int32_t B, bs, shift;  // shift: log2 of bs, or -1
  int32_t *table;
  int32_t *free_blocks;
  int32_t max_blocks, n_blocks;
  const int32_t *free_count;
  int32_t *free_count_out;
  int32_t *slot_map, *positions, *cu_new, *len_out;
  int32_t max_new;
  int32_t *status;
};

// block of position p, blocks of n tokens (a shift for a power of two: the divisions were a
// quarter of the kernel's instructions)
__device__ __forceinline__ int block_of(const TablesParams &P, uint32_t p) {
  return static_cast<int>(P.shift >= 0 ? p >> P.shift : p / static_cast<uint32_t>(P.bs));
}
__device__ __forceinline__ int blocks_of(const TablesParams &P, int n) {
  return block_of(P, static_cast<uint32_t>(n) + static_cast<uint32_t>(P.bs) - 1);
}

// the largest i in [0, n) with cu[i] <= x (cu ascending, cu[0] <= x): the owner of entry x
// of a list whose exclusive sums are cu
__device__ __forceinline__ int owner_of(const int32_t *cu, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TablesParams P) {
  extern __shared__ int32_t tab_smem[];
  int32_t *cuN = tab_smem, *cuA = cuN + P.B + 1, *cuF = cuA + P.B + 1;
  __shared__ int32_t warp_sum[3][kTabThreads / 32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int cap = P.max_blocks * P.bs;
  const int count0 = *P.free_count;
  const int count = min(max(count0, 0), P.n_blocks);
  int bad = count != count0;

  // ===== exclusive sums over the requests: a run of consecutive requests per thread =====
  const int per = (P.B + kTabThreads - 1) / kTabThreads;
  const int b0 = min(t * per, P.B), b1 = min(b0 + per, P.B);
  int32_t n = 0, a = 0, f = 0;
  for (int b = b0; b < b1; ++b) {
    const int o0 = P.old_len[b], w0 = P.new_len[b];
    const int o = min(max(o0, 0), cap), w = min(max(w0, 0), cap);
    bad |= (o != o0) | (w != w0);
    const int no = blocks_of(P, o), nw = blocks_of(P, w);
    cuN[b] = n, cuA[b] = a, cuF[b] = f;  // sums within the thread's run for now
    n += max(w - o, 0), a += max(nw - no, 0), f += max(no - nw, 0);
  }
  int32_t sn = n, sa = a, sf = f;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int xn = __shfl_up_sync(~0u, sn, d), xa = __shfl_up_sync(~0u, sa, d), xf = __shfl_up_sync(~0u, sf, d);
    if (lane >= d) sn += xn, sa += xa, sf += xf;
  }
  if (lane == 31) warp_sum[0][warp] = sn, warp_sum[1][warp] = sa, warp_sum[2][warp] = sf;
  __syncthreads();
  int32_t en = sn - n, ea = sa - a, ef = sf - f, tn = 0, ta = 0, tf = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    const int xn = warp_sum[0][w], xa = warp_sum[1][w], xf = warp_sum[2][w];
    if (w < warp) en += xn, ea += xa, ef += xf;
    tn += xn, ta += xa, tf += xf;
  }
  for (int b = b0; b < b1; ++b) cuN[b] += en, cuA[b] += ea, cuF[b] += ef;
  if (t == 0) cuN[P.B] = tn, cuA[P.B] = ta, cuF[P.B] = tf;
  __syncthreads();
  const int top = min(count + tf, P.n_blocks);
  bad |= count + tf > P.n_blocks;
  // growth is granted in request order while it fits: b gets its blocks iff A_{b+1} <= top
  const bool exhausted = ta > top;

  // entry s of the stack after the pushes
  auto stack_at = [&](int s) -> int32_t {
    if (s < count) return P.free_blocks[s];
    const int j = s - count, b = owner_of(cuF, P.B, j);
    const int w = min(max(P.new_len[b], 0), cap);
    return P.table[static_cast<size_t>(b) * P.max_blocks + blocks_of(P, w) + (j - cuF[b])];
  };
  auto grown = [&](int j) -> int32_t {  // the j-th block handed out
    const int32_t id = stack_at(top - 1 - j);
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(P.n_blocks) ? id : -1;
  };

  const int gthreads = gridDim.x * kTabThreads, gt = blockIdx.x * kTabThreads + t;
  const int rt = gthreads - 1 - gt;  // the blocks go to the other end's threads: both at once
  // ===== the list of new tokens =====
  const int listed = min(tn, P.max_new);
  bad |= tn > P.max_new;
  // the slot and position of the token at entry i < listed of the list, request b its owner
  auto entry = [&](int i, int b, int32_t &slot, int32_t &pos) {
    slot = pos = -1;
    if (cuA[b + 1] != cuA[b] && cuA[b + 1] > top) return;  // left without its blocks
    const int o = min(max(P.old_len[b], 0), cap), nbo = blocks_of(P, o);
    const int p = o + (i - cuN[b]), k = block_of(P, p);
    const int32_t id = k < nbo ? P.table[static_cast<size_t>(b) * P.max_blocks + k] : stack_at(top - 1 - (cuA[b] + k - nbo));
    if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(P.n_blocks)) bad = 1;
    else slot = id * P.bs + (p - k * P.bs), pos = p;
  };
  const bool wide = ((reinterpret_cast<uintptr_t>(P.slot_map) | reinterpret_cast<uintptr_t>(P.positions)) & 15) == 0;
  if (P.max_new <= gthreads || !wide) {  // an entry per thread: the shortest chain of loads
    for (int i = gt; i < P.max_new; i += gthreads) {
      int32_t slot = -1, pos = -1;
      if (i < listed) entry(i, owner_of(cuN, P.B, i), slot, pos);
      P.slot_map[i] = slot;
      if (P.positions) P.positions[i] = pos;
    }
  } else {                               // four neighbours: one search and mostly one id
    for (int i = 4 * gt; i < P.max_new; i += 4 * gthreads) {
      int32_t slot[4] = {-1, -1, -1, -1}, pos[4] = {-1, -1, -1, -1};
      // one look-up per block that they touch (mostly one, two where a block or a request ends)
      int b = i < listed ? owner_of(cuN, P.B, i) : 0;
      for (int u = 0; u < 4 && i + u < listed;) {
        while (cuN[b + 1] <= i + u) ++b;
        int32_t s0, p0;
        entry(i + u, b, s0, p0);
        const int run = s0 >= 0 ? min(P.bs - (p0 - block_of(P, p0) * P.bs), cuN[b + 1] - i - u) : 1;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (v >= u && v - u < run && s0 >= 0) slot[v] = s0 + (v - u), pos[v] = p0 + (v - u);
        u += run;
      }
      if (i + 4 <= P.max_new) {
        *reinterpret_cast<int4 *>(P.slot_map + i) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        if (P.positions) *reinterpret_cast<int4 *>(P.positions + i) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u < P.max_new) {
            P.slot_map[i + u] = slot[u];
            if (P.positions) P.positions[i + u] = pos[u];
          }
      }
    }
  }
  // ===== the blocks that moved =====
  for (int j = rt; j < ta; j += gthreads) {
    const int b = owner_of(cuA, P.B, j);
    if (cuA[b + 1] > top) break;  // this request and every later one with a need get nothing
    const int o = min(max(P.old_len[b], 0), cap);
    const int32_t id = grown(j);
    bad |= id < 0;
    P.table[static_cast<size_t>(b) * P.max_blocks + blocks_of(P, o) + (j - cuA[b])] = id;
  }
  for (int j = rt; j < tf; j += gthreads) {
    const int32_t id = stack_at(count + j);
    bad |= static_cast<uint32_t>(id) >= static_cast<uint32_t>(P.n_blocks);
    if (count + j < P.n_blocks) P.free_blocks[count + j] = id;
  }
  // ===== per-request outputs =====
  for (int b = rt; b <= P.B; b += gthreads) {
    if (P.cu_new) P.cu_new[b] = cuN[b];
    if (P.len_out && b < P.B) {
      const bool have = cuA[b + 1] == cuA[b] || cuA[b + 1] <= top;
      P.len_out[b] = min(max(have ? P.new_len[b] : P.old_len[b], 0), cap);
    }
  }
  if (blockIdx.x == 0 && t == 0) {
    int taken = ta;
    if (exhausted) taken = cuA[owner_of(cuA, P.B + 1, top)];  // the largest sum that fits
    *P.free_count_out = top - taken;
    if (exhausted) set_status(P.status, ECHO_DEV_POOL_EXHAUSTED);
  }
  if (bad) set_status(P.status, ECHO_DEV_BAD_INDEX);
}

}  // namespace echo

namespace echo_host {

int launch_block_tables(const echo_block_tables_args *a, cudaStream_t stream) {
  echo::TablesParams P{};
  P.old_len = a->old_len;
  P.new_len = a->new_len;
  P.B = a->B;
  P.bs = a->block_tokens;
  P.shift = -1;
  for (int k = 0; k < 31; ++k)
    if (a->block_tokens == 1 << k) P.shift = k;
  P.table = a->table;
  P.free_blocks = a->free_blocks;
  P.max_blocks = a->max_blocks;
  P.n_blocks = a->n_blocks;
  P.free_count = a->free_count;
  P.free_count_out = a->free_count_out;
  P.slot_map = a->slot_map;
  P.positions = a->positions;
  P.cu_new = a->cu_new;
  P.len_out = a->len_out;
  P.max_new = a->max_new;
  P.status = a->dev_status;
  const size_t smem = 3 * (static_cast<size_t>(a->B) + 1) * sizeof(int32_t);
  static std::atomic<bool> attr[kMaxDevices];
  if (int rr = smem_limit_once(attr, echo::block_tables_kernel, 3 * (16384 + 1) * sizeof(int32_t),
                               "block tables smem attribute"))
    return rr;
  // an entry per thread while that fits the GPU (four CTAs per SM), then four and more each; and
  // the tables' blocks, which may all be on their way back, four to a thread on up to 152 CTAs
  // (finished requests on one CTA against 152: 125 requests of 26011 tokens in blocks of 32, 18
  // of them finished, 20.3 / 3.9 us; 256 of 131072 in blocks of 16, 40 finished, 407 / 6.5; with
  // nothing to return 64 requests take 2.8 / 2.9)
  const auto ctas = [](int64_t n, int64_t each) { return (n + each - 1) / each; };
  const int64_t by_list = ctas(a->max_new, echo::kTabThreads);
  const int64_t by_blocks = std::min<int64_t>(152, ctas(static_cast<int64_t>(a->B) * a->max_blocks, 4 * echo::kTabThreads));
  const int64_t grid = std::min<int64_t>(608, std::max<int64_t>({1, by_list, by_blocks}));
  const cudaError_t e = launch_pdl(echo::block_tables_kernel, dim3(static_cast<unsigned>(grid)), dim3(echo::kTabThreads), smem, stream, P);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "block tables launch");
}

}  // namespace echo_host
