// qk_norm_rope.cu -- per-head RMS norm and rotation of queries and keys, with the keys and
// values written to their cache rows (bf16 or 4-bit) in the same pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A head is held by head_dim / 8 lanes, 16 bytes each, and never leaves registers until its
// results are stored; the mean is a shuffle sum over those lanes.  A warp takes `span` heads
// of one kind (q, k or v) of its tokens, kBatch at a time with the next batch's loads in
// flight; cosines, sines and weights are read and multiplied once for them.  Bound by HBM:
// 16384 tokens x (64 + 8 + 8) heads of 128 in 117 us, 5.8 TB/s of the 6.67 TB/s that a copy
// reaches here (0.87; 8-byte accesses and 32 warps an SM: with one 16-byte load per lane, the
// partners shuffled between lanes and 16 warps it was 180 us); 8191 tokens x 40 heads of 64
// into a 4-bit cache 19.7 us (0.69; first loads and tail), a decode step's tokens 3 us (latency).
#include <cmath>

#include "block_rows.cuh"

namespace echo {

constexpr int kRopeThreads = 128;

struct RopeParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int32_t T, n_heads, n_kv_heads;
  const float *q_weight, *k_weight;
  float eps;
  int32_t interleaved;
  const float *cos_sin;
  int32_t max_pos, rope_dim;
  const int32_t *positions;
  uint16_t *q_out, *k_out, *v_out;
  const int32_t *slot_map;
  uint16_t *rows;
  int32_t n_rows, format, bs;
  float k_up, v_up, k_down, v_down;    // 4-bit rows: 2^shift of keys and values, and the inverse
  int64_t row_elems;
  int32_t span, kv_span;               // heads of a warp: q, and k or v
  int32_t q_chunks, k_chunks, chunks;  // warps per token group: of q, of k (and of v), in all
  int32_t *status;
};

__device__ __forceinline__ void unpack_bf16x8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One lane's 8 entries as 4-bit codes, with the scale of the 16 dimensions it shares with its
// neighbour (lane ^ 1): s = e4m3(amax / 6) and the nearest codes to x / s, ties to even.
// No exact division is needed.  x has 8 significant bits and s at most 4, so x / s lies on a
// border between codes (3 bits) exactly or at least 2^-8 away from it; amax / 6 and the
// borders between scales (5 bits) likewise.  A product with the reciprocal, off by 2^-22,
// rounded to fp16 (11 bits), is the border itself in the first case and stays on its side in
// the second, and the hardware's round-half-to-even then decides as the definition does.
// Taken times a power of two `up`, which moves the scale alone.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float up, uint32_t &scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
  scale = e4m3_from_half(__float2half_rn(amax * (up * (1.f / 6.f))));
  const uint32_t sh = e4m3x2_to_half2(scale);
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffff)));
  const float r = s > 0.f ? __fdividef(up, s) : 0.f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(__floats2half2_rn(x[2 * i] * r, x[2 * i + 1] * r));
    y[2 * i] = f.x, y[2 * i + 1] = f.y;
  }
  return e2m1x8_from_float(y);
}

// the values 8 codes stand for, times a power of two, as bf16 (exact: a code has 2 significant
// bits, a scale 4)
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t scale, float down) {
  uint32_t h[4];
  e2m1x8_to_half2(codes, h);
  const uint32_t s2 = e4m3x2_to_half2(scale | (scale << 8));
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = hmul2(h[i], s2);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
  const uint4 u = pack_bf16x8(x);
  const __nv_bfloat162 d = __floats2bfloat162_rn(down, down);
  auto mul = [&](uint32_t w) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), d);
    return *reinterpret_cast<const uint32_t *>(&y);
  };
  return make_uint4(mul(u.x), mul(u.y), mul(u.z), mul(u.w));
}

// Kinds of heads, in the order of a token's chunks; a warp works on one kind.
enum RopeKind { kRopeQ, kRopeK, kRopeV };

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t float2_to_bf16x2(float2 x) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}
// the factor 1 / sqrt(mean x^2 + eps) of a head, from each lane's part of the sum
template <int D>
__device__ __forceinline__ float norm_factor(float ss, float eps) {
#pragma unroll
  for (int d = D / 16; d > 0; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

// Where the keys and values of one token go.
struct RopeDst {
  const RopeParams &P;
  int64_t t, blk;
  int off;
  bool in;
  // the row of KV head h, null when it is not written
  __device__ __forceinline__ uint16_t *row(int h, bool report) const {
    if (blk < 0) return nullptr;
    const int64_t r = blk * P.n_kv_heads + h;
    if (r >= P.n_rows) {
      if (report) set_status(P.status, ECHO_DEV_BAD_INDEX);
      return nullptr;
    }
    return P.rows + r * P.row_elems;
  }
};

// Rotated heads that stay bf16 (queries, and keys of bf16 rows).  A lane holds both ends of
// its pairs: two units of four dims, half a rotation apart (half-split), or side by side
// (interleaved, and the dims past the rotation), so nothing but the norm's sum crosses lanes.
template <int D, int kBatch, bool kInter>
__device__ __forceinline__ void rope_pairs(const RopeParams &P, const RopeDst &W, const uint16_t *src, const float *wt,
                                           int pos, bool is_q, int h0, int h1, int l) {
  const int half = P.rope_dim >> 1, rl = P.rope_dim >> 3;  // lanes that rotate
  const bool rot = l < rl;
  const int ua = kInter ? 8 * l : rot ? 4 * l : P.rope_dim + 8 * (l - rl), ub = kInter || !rot ? ua + 4 : ua + half;
  uint2 ra[kBatch], rb[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      ra[u] = rb[u] = make_uint2(0u, 0u);
      if (h + u < h1) {  // (whatever the position: the loads need not wait for it)
        ra[u] = *reinterpret_cast<const uint2 *>(src + static_cast<int64_t>(h + u) * D + ua);
        rb[u] = *reinterpret_cast<const uint2 *>(src + static_cast<int64_t>(h + u) * D + ub);
      }
    }
  };
  load(h0);
  // u' = r (a ca - b sb),  v' = r (b cb + a sa): cosine or sine times the operand's weight
  // (half-split: unit a against unit b; interleaved: within each unit, see below)
  float ca[4], cb[4], sa[4], sb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ca[i] = cb[i] = 1.f, sa[i] = sb[i] = 0.f;
  if (W.in && rot) {
    const float *row = P.cos_sin + static_cast<int64_t>(pos) * P.rope_dim + 4 * l;
    const float4 c = *reinterpret_cast<const float4 *>(row), s = *reinterpret_cast<const float4 *>(row + half);
    if constexpr (kInter) {  // pairs 4l .. 4l + 3: two in unit a, two in unit b
      ca[0] = ca[1] = c.x, ca[2] = ca[3] = c.y, cb[0] = cb[1] = c.z, cb[2] = cb[3] = c.w;
      sa[0] = sa[1] = s.x, sa[2] = sa[3] = s.y, sb[0] = sb[1] = s.z, sb[2] = sb[3] = s.w;
    } else {
      ca[0] = cb[0] = c.x, ca[1] = cb[1] = c.y, ca[2] = cb[2] = c.z, ca[3] = cb[3] = c.w;
      sa[0] = sb[0] = s.x, sa[1] = sb[1] = s.y, sa[2] = sb[2] = s.z, sa[3] = sb[3] = s.w;
    }
  }
  if (wt) {
    const float4 wa = *reinterpret_cast<const float4 *>(wt + ua), wb = *reinterpret_cast<const float4 *>(wt + ub);
    const float a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) ca[i] *= a[i], cb[i] *= b[i], sa[i] *= a[i], sb[i] *= b[i];
  }
  for (int h = h0; h < h1; h += kBatch) {
    uint2 oa[kBatch], ob[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float2 a0 = bf16x2_to_float2(ra[u].x), a1 = bf16x2_to_float2(ra[u].y);
      const float2 b0 = bf16x2_to_float2(rb[u].x), b1 = bf16x2_to_float2(rb[u].y);
      float2 r = make_float2(1.f, 1.f);
      if (wt) {
        const float2 q = __ffma2_rn(a0, a0, __ffma2_rn(a1, a1, __ffma2_rn(b0, b0, __fmul2_rn(b1, b1))));
        r.x = r.y = norm_factor<D>(q.x + q.y, P.eps);
      }
      float2 u0, u1, v0, v1;
      if constexpr (kInter) {
        // the pair (x, y) of a unit: (x c - y s, y c + x s), weights folded into each operand
        u0 = make_float2(fmaf(-a0.y, sa[1], a0.x * ca[0]), fmaf(a0.x, sa[0], a0.y * ca[1]));
        u1 = make_float2(fmaf(-a1.y, sa[3], a1.x * ca[2]), fmaf(a1.x, sa[2], a1.y * ca[3]));
        v0 = make_float2(fmaf(-b0.y, sb[1], b0.x * cb[0]), fmaf(b0.x, sb[0], b0.y * cb[1]));
        v1 = make_float2(fmaf(-b1.y, sb[3], b1.x * cb[2]), fmaf(b1.x, sb[2], b1.y * cb[3]));
      } else if (rot) {
        const float2 nb0 = make_float2(-sb[0], -sb[1]), nb1 = make_float2(-sb[2], -sb[3]);
        u0 = __ffma2_rn(b0, nb0, __fmul2_rn(a0, make_float2(ca[0], ca[1])));
        u1 = __ffma2_rn(b1, nb1, __fmul2_rn(a1, make_float2(ca[2], ca[3])));
        v0 = __ffma2_rn(a0, make_float2(sa[0], sa[1]), __fmul2_rn(b0, make_float2(cb[0], cb[1])));
        v1 = __ffma2_rn(a1, make_float2(sa[2], sa[3]), __fmul2_rn(b1, make_float2(cb[2], cb[3])));
      } else {               // (0 * inf would reach the entries that stay)
        u0 = __fmul2_rn(a0, make_float2(ca[0], ca[1])), u1 = __fmul2_rn(a1, make_float2(ca[2], ca[3]));
        v0 = __fmul2_rn(b0, make_float2(cb[0], cb[1])), v1 = __fmul2_rn(b1, make_float2(cb[2], cb[3]));
      }
      if constexpr (kInter) {
        if (!rot) {
          u0 = make_float2(a0.x * ca[0], a0.y * ca[1]), u1 = make_float2(a1.x * ca[2], a1.y * ca[3]);
          v0 = make_float2(b0.x * cb[0], b0.y * cb[1]), v1 = make_float2(b1.x * cb[2], b1.y * cb[3]);
        }
      }
      oa[u] = make_uint2(float2_to_bf16x2(__fmul2_rn(u0, r)), float2_to_bf16x2(__fmul2_rn(u1, r)));
      ob[u] = make_uint2(float2_to_bf16x2(__fmul2_rn(v0, r)), float2_to_bf16x2(__fmul2_rn(v1, r)));
    }
    if (h + kBatch < h1) load(h + kBatch);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!W.in || h + u >= h1) continue;
      auto store = [&](uint16_t *dst) {
        __stcs(reinterpret_cast<uint2 *>(dst + ua), oa[u]);
        __stcs(reinterpret_cast<uint2 *>(dst + ub), ob[u]);
      };
      if (is_q) {
        store(P.q_out + (W.t * P.n_heads + h + u) * D);
      } else {
        if (P.k_out) store(P.k_out + (W.t * P.n_kv_heads + h + u) * D);
        if (uint16_t *row = W.row(h + u, l == 0)) store(row + static_cast<int64_t>(W.off) * D);
      }
    }
  }
}

// Values, and keys of 4-bit rows: a lane holds 8 neighbouring dims, as the rows do; the
// partners of half-split pairs come from another lane.
template <int D, int kBatch, bool kInter>
__device__ __forceinline__ void rope_rows(const RopeParams &P, const RopeDst &W, const uint16_t *src, const float *wt,
                                          int pos, bool is_v, int h0, int h1, int l, int lane) {
  constexpr int kLanes = D / 8;
  const int half = P.rope_dim >> 1, d0 = 8 * l;
  const bool rot = d0 < P.rope_dim, low = d0 < half, fp4 = P.format == ECHO_BLOCK_FP4;
  const int pd = kInter || !rot ? d0 : low ? d0 + half : d0 - half;   // the partners' dims
  const int partner = (lane & ~(kLanes - 1)) + pd / 8;
  uint4 raw[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h + u < h1) raw[u] = *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(h + u) * D + d0);
    }
  };
  load(h0);
  // y = r (x c + partner s): the cosine times the own weight, the signed sine times the partner's
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (!is_v) {
    auto four = [](const float *p, float *to) {
      const float4 v = *reinterpret_cast<const float4 *>(p);
      to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
    };
    if (W.in && rot) {
      const float *row = P.cos_sin + static_cast<int64_t>(pos) * P.rope_dim;
      float cv[8], sv[8];
      if constexpr (kInter) {
        four(row + d0 / 2, cv), four(row + half + d0 / 2, sv);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = cv[i / 2], s[i] = i % 2 == 0 ? -sv[i / 2] : sv[i / 2];
      } else {
        const float *at = row + (low ? d0 : d0 - half);
        four(at, cv), four(at + 4, cv + 4), four(at + half, sv), four(at + half + 4, sv + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = cv[i], s[i] = low ? -sv[i] : sv[i];
      }
    }
    if (wt) {
      float wo[8], wp[8];
      four(wt + d0, wo), four(wt + d0 + 4, wo + 4), four(wt + pd, wp), four(wt + pd + 4, wp + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] *= wo[i], s[i] *= wp[kInter ? i ^ 1 : i];
    }
  }
  for (int h = h0; h < h1; h += kBatch) {
    uint4 cur[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) cur[u] = raw[u];
    if (h + kBatch < h1) load(h + kBatch);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint4 o = cur[u];
      if (!is_v) {
        uint32_t w[4] = {cur[u].x, cur[u].y, cur[u].z, cur[u].w};
        float2 x[4], q = make_float2(0.f, 0.f), r = make_float2(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = bf16x2_to_float2(w[i]);
          q = __ffma2_rn(x[i], x[i], q);
        }
        if (wt) r.x = r.y = norm_factor<D>(q.x + q.y, P.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t pw = kInter ? __byte_perm(w[i], 0, 0x1032) : __shfl_sync(~0u, w[i], partner);
          if (!rot) pw = 0;
          const float2 y = __ffma2_rn(bf16x2_to_float2(pw), make_float2(s[2 * i], s[2 * i + 1]),
                                      __fmul2_rn(x[i], make_float2(c[2 * i], c[2 * i + 1])));
          w[i] = float2_to_bf16x2(__fmul2_rn(y, r));
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
      }
      uint32_t codes = 0, scale = 0;
      if (fp4) {             // (every lane: the scale is a shuffle)
        float x[8];
        unpack_bf16x8(o, x);
        codes = quantise8(x, is_v ? P.v_up : P.k_up, scale);
      }
      if (!W.in || h + u >= h1) continue;
      uint16_t *out = is_v ? P.v_out : P.k_out;
      if (out) {
        *reinterpret_cast<uint4 *>(out + (W.t * P.n_kv_heads + h + u) * D + d0) =
            fp4 ? dequantise8(codes, scale, is_v ? P.v_down : P.k_down) : o;
      }
      uint16_t *row = W.row(h + u, l == 0);
      if (!row) continue;
      if (fp4) {
        using Sub = Fp4Sub<D>;
        uint8_t *sub = reinterpret_cast<uint8_t *>(row) + W.off / kSubTokens * Sub::kBytes;
        const int tk = W.off % kSubTokens;
        if (!is_v) {
          *reinterpret_cast<uint32_t *>(sub + tk * (D / 2) + l * 4) = codes;
          if (!(l & 1)) sub[Sub::kKeyScales + tk * (D / 16) + l / 2] = static_cast<uint8_t>(scale);
        } else {
          constexpr int kPart = D / 8;     // dims of a part: 16 (two lanes) or 8 (one lane)
          *reinterpret_cast<uint32_t *>(sub + Sub::kValues + (tk / 8) * (4 * D) + ((d0 / kPart) * 8 + tk % 8) * (D / 16) +
                                        (d0 % kPart) / 2) = codes;
          if (!(l & 1)) sub[Sub::kValueScales + (tk / 8) * (D / 2) + (l / 2) * 8 + tk % 8] = static_cast<uint8_t>(scale);
        }
      } else {
        *reinterpret_cast<uint4 *>(row + (is_v ? static_cast<int64_t>(P.bs) * D : 0) + static_cast<int64_t>(W.off) * D + d0) = o;
      }
    }
  }
}

template <int D, int kBatch, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 8) qk_norm_rope_kernel(const RopeParams P) {
  constexpr int kLanes = D / 8;          // lanes of a head
  constexpr int kTokens = 32 / kLanes;   // tokens of a warp
  pdl_launch_dependents();
  pdl_wait();
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int64_t tb = wid / P.chunks;
  const int chunk = static_cast<int>(wid - tb * P.chunks);
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int64_t tok = tb * kTokens + lane / kLanes;
  if (tb * kTokens >= P.T) return;       // (the whole warp)
  const int64_t t = min(tok, static_cast<int64_t>(P.T) - 1);
  const int pos = P.positions[t];
  const bool in = tok < P.T && pos >= 0 && pos < P.max_pos;
  if (tok < P.T && pos >= P.max_pos && l == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);

  const int kind = chunk < P.q_chunks ? kRopeQ : chunk < P.q_chunks + P.k_chunks ? kRopeK : kRopeV;
  const int h0 = kind == kRopeQ ? chunk * P.span : (chunk - P.q_chunks) % P.k_chunks * P.kv_span;
  const int h1 = kind == kRopeQ ? min(h0 + P.span, P.n_heads) : min(h0 + P.kv_span, P.n_kv_heads);
  const int slot = P.slot_map && kind != kRopeQ ? P.slot_map[t] : -1;
  const int blk = slot >= 0 ? slot / P.bs : -1;
  const RopeDst W{P, t, blk, slot - blk * P.bs, in};
  if (kind == kRopeQ || (kind == kRopeK && P.format == ECHO_BLOCK_BF16))
    rope_pairs<D, kBatch, kInter>(P, W, kind == kRopeQ ? P.q + t * P.q_stride : P.k + t * P.k_stride,
                                  kind == kRopeQ ? P.q_weight : P.k_weight, pos, kind == kRopeQ, h0, h1, l);
  else
    rope_rows<D, kBatch, kInter>(P, W, kind == kRopeK ? P.k + t * P.k_stride : P.v + t * P.v_stride, P.k_weight, pos,
                                 kind == kRopeV, h0, h1, l, lane);
}

}  // namespace echo

namespace echo_host {

template <int D, int kBatch, bool kInter>
static cudaError_t launch_rope(echo::RopeParams P, bool values, int span, int kv_span, cudaStream_t stream) {
  // equal runs of whole batches, none longer than the span (24 heads: 12 + 12, not 16 + 8)
  const auto even = [](int heads, int most) {
    const int runs = (heads + most - 1) / most, run = (heads + runs - 1) / runs;
    return (run + kBatch - 1) / kBatch * kBatch;
  };
  P.span = even(P.n_heads, span);
  P.kv_span = even(P.n_kv_heads, kv_span);
  P.q_chunks = (P.n_heads + P.span - 1) / P.span;
  P.k_chunks = (P.n_kv_heads + P.kv_span - 1) / P.kv_span;
  P.chunks = P.q_chunks + (values ? 2 : 1) * P.k_chunks;
  constexpr int kTokens = 256 / D;
  const int64_t warps = (static_cast<int64_t>(P.T) + kTokens - 1) / kTokens * P.chunks;
  const int64_t grid = (warps * 32 + echo::kRopeThreads - 1) / echo::kRopeThreads;
  return launch_pdl(echo::qk_norm_rope_kernel<D, kBatch, kInter>, dim3(static_cast<unsigned>(grid)), dim3(echo::kRopeThreads),
                    0, stream, P);
}

// How many heads a warp takes (q, then k or v), and how many of them at a time.  Few heads in
// all: one each, the shortest chain; many: long runs, cosines and weights read once for them.
// In warps at one head each (T / (256 / D) times the heads), us for 1, 2 of 8 and 4, 4 of 16
// and 8 heads: 2560 warps 4.2 / 6.2 / 8.3, 10240 8.2 / 6.2 / 9.0, 81920 42.6 / 22.6 / 24.8
// (heads of 64), 163840 67.7 / 36.8 / 36.2, 655360 256 / 127 / 119 (heads of 128).
template <int D, bool kInter>
static cudaError_t launch_rope_dim(const echo::RopeParams &P, bool values, cudaStream_t stream) {
  const int64_t warps = (static_cast<int64_t>(P.T) + 256 / D - 1) / (256 / D) * (P.n_heads + (values ? 2 : 1) * static_cast<int64_t>(P.n_kv_heads));
  if (warps <= 4096) return launch_rope<D, 1, kInter>(P, values, 1, 1, stream);
  // Long runs want 8 and more KV heads: beside a warp's 16 query heads others would have 2 (16 + 4
  // heads of 128, 8 and 4 against 16 and 8: 7311 tokens into 4-bit rows 24.2 / 31.0, 16000 into
  // bf16 rows 42.3 / 44.5).  The kernels with batches of 4 spill 148 to 176 bytes a thread (the
  // format is a run-time branch: those of bf16 rows hold the quantisation too, and win all the
  // same, as above), those with batches of 2 up to 24, and 4-bit rows win with long runs of
  // batches of 2 sooner (2 of 8 and 4, 2 of 16 and 8, 4 of 16 and 8: 64000 warps
  // 18.9 / 18.6 / 18.0, 81920 20.7 / 19.8 / 23.2, 201340 50.5 / 47.4 / 53.4).
  const bool fp4 = P.format == ECHO_BLOCK_FP4;
  if (P.n_kv_heads < 8 || warps <= (fp4 ? 65536 : 163840)) return launch_rope<D, 2, kInter>(P, values, 8, 4, stream);
  if (fp4) return launch_rope<D, 2, kInter>(P, values, 16, 8, stream);
  return launch_rope<D, 4, kInter>(P, values, 16, 8, stream);
}

int launch_qk_norm_rope(const echo_qk_norm_rope_args *a, cudaStream_t stream) {
  echo::RopeParams P{};
  P.q = a->q, P.k = a->k, P.v = a->v;
  P.q_stride = a->q_stride, P.k_stride = a->k_stride, P.v_stride = a->v_stride;
  P.T = a->T, P.n_heads = a->n_heads, P.n_kv_heads = a->n_kv_heads;
  P.q_weight = a->q_weight, P.k_weight = a->k_weight, P.eps = a->eps;
  P.interleaved = a->interleaved;
  P.cos_sin = a->cos_sin, P.max_pos = a->max_pos, P.rope_dim = a->rope_dim;
  P.positions = a->positions;
  P.q_out = a->q_out, P.k_out = a->k_out, P.v_out = a->v_out;
  P.slot_map = a->slot_map, P.rows = a->rows, P.n_rows = a->n_rows;
  P.format = a->format, P.bs = a->block_tokens;
  P.row_elems = echo::block_row_elems(a->format, a->block_tokens, a->head_dim);
  P.k_up = std::ldexp(1.f, a->k_shift), P.v_up = std::ldexp(1.f, a->v_shift);
  P.k_down = std::ldexp(1.f, -a->k_shift), P.v_down = std::ldexp(1.f, -a->v_shift);
  P.status = a->dev_status;
  // value heads have work only when something takes them
  const bool values = a->v && (a->slot_map || a->v_out);
  const cudaError_t e = a->head_dim == 128
                            ? (a->interleaved ? launch_rope_dim<128, true>(P, values, stream) : launch_rope_dim<128, false>(P, values, stream))
                            : (a->interleaved ? launch_rope_dim<64, true>(P, values, stream) : launch_rope_dim<64, false>(P, values, stream));
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "qk norm + rope launch");
}

}  // namespace echo_host
