// qk_norm_rope.cu -- per-head RMS norm and rotation of queries and keys, with the keys and
// values written to their cache rows (bf16 or 4-bit) in the same pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A head is read by head_dim / 8 lanes, one 16-byte load each, and never leaves registers
// until its results are stored: the mean is a shuffle sum over those lanes, the partner of
// a half-split pair sits in the lane rope_dim / 16 away (a shuffle of the bf16 pairs as
// loaded), of an interleaved pair in the same lane; a 4-bit scale covers 16 dimensions, so
// two neighbouring lanes.  A warp takes kHeads heads of one kind (q, k or v) of its tokens:
// their loads are issued together (bytes in flight), and cosines, sines and weights are read
// and multiplied once for them.  Bound by HBM.
#include "block_rows.cuh"

namespace echo {

constexpr int kRopeThreads = 256;

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
  int64_t row_elems;
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

// One lane's 8 entries as 4-bit codes: the scale of the 16 dimensions it shares with its
// neighbour (lane ^ 1), s = e4m3(amax / 6) by IEEE division, and the nearest codes to x / s.
// x has 8 significant bits and s at most 4, so x / s is a rounding border of the code grid
// exactly or at least 2^-8 away from it: rounding x * (1 / s) to fp16 (11 bits) gives the
// border back in the first case and stays off it in the second, and the hardware's
// round-half-to-even then decides as the definition does.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t &scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
  scale = e4m3_from_float(__fdiv_rn(amax, 6.f));
  const uint32_t sh = e4m3x2_to_half2(scale);
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffff)));
  const float r = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __half2float(__float2half_rn(fminf(fmaxf(x[i] * r, -8.f), 8.f)));
  return e2m1x8_from_float(y);
}

// the values 8 codes stand for, as bf16 (exact: a code has 2 significant bits, a scale 4)
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t scale) {
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
  return pack_bf16x8(x);
}

// Kinds of heads, in the order of a token's chunks; a warp works on one kind.
enum RopeKind { kRopeQ, kRopeK, kRopeV };

template <int D, int kHeads, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams P) {
  constexpr int kLanes = D / 8;          // lanes of a head
  constexpr int kTokens = 32 / kLanes;   // tokens of a warp
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int64_t tb = wid / P.chunks;
  int chunk = static_cast<int>(wid - tb * P.chunks);
  const int lane = threadIdx.x & 31, l = lane % kLanes, d0 = 8 * l;
  const int64_t tok = tb * kTokens + lane / kLanes;
  if (tb * kTokens >= P.T) return;       // (the whole warp)
  const int64_t t = min(tok, static_cast<int64_t>(P.T) - 1);
  const int pos = __ldg(P.positions + t);
  const bool in = tok < P.T && pos >= 0 && pos < P.max_pos;
  if (tok < P.T && pos >= P.max_pos && l == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);

  const int kind = chunk < P.q_chunks ? kRopeQ : chunk < P.q_chunks + P.k_chunks ? kRopeK : kRopeV;
  const int h0 = (kind == kRopeQ ? chunk : (chunk - P.q_chunks) % P.k_chunks) * kHeads;
  const int heads = kind == kRopeQ ? P.n_heads : P.n_kv_heads;
  const uint16_t *src = (kind == kRopeQ   ? P.q + t * P.q_stride
                         : kind == kRopeK ? P.k + t * P.k_stride
                                          : P.v + t * P.v_stride) + static_cast<int64_t>(h0) * D + d0;
  uint4 raw[kHeads];
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (in && h0 + u < heads) raw[u] = *reinterpret_cast<const uint4 *>(src + u * D);
  }

  // y = r * (x * c + partner * s): the cosine times the own weight, the signed sine times
  // the partner's
  const int half = P.rope_dim >> 1;
  const bool rot = d0 < P.rope_dim, low = d0 < half;
  const float *wt = kind == kRopeQ ? P.q_weight : P.k_weight;
  const int pd = kInter || !rot ? d0 : low ? d0 + half : d0 - half;   // the partners' dims
  float2 c[4], s[4];
  if (kind != kRopeV) {
    float cw[8], sw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cw[i] = 1.f, sw[i] = 0.f;
    if (in && rot) {
      const float *row = P.cos_sin + static_cast<int64_t>(pos) * P.rope_dim;
      if constexpr (kInter) {
        const float4 cc = *reinterpret_cast<const float4 *>(row + d0 / 2);
        const float4 ss = *reinterpret_cast<const float4 *>(row + half + d0 / 2);
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) cw[2 * i] = cw[2 * i + 1] = cv[i], sw[2 * i] = -sv[i], sw[2 * i + 1] = sv[i];
      } else {
        const float *cr = row + (low ? d0 : d0 - half);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 cc = reinterpret_cast<const float4 *>(cr)[i];
          const float4 ss = reinterpret_cast<const float4 *>(cr + half)[i];
          cw[4 * i] = cc.x, cw[4 * i + 1] = cc.y, cw[4 * i + 2] = cc.z, cw[4 * i + 3] = cc.w;
          sw[4 * i] = ss.x, sw[4 * i + 1] = ss.y, sw[4 * i + 2] = ss.z, sw[4 * i + 3] = ss.w;
        }
        if (low) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sw[i] = -sw[i];
        }
      }
    }
    if (wt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(wt + d0) + i);
        const float4 b = __ldg(reinterpret_cast<const float4 *>(wt + pd) + i);
        cw[4 * i] *= a.x, cw[4 * i + 1] *= a.y, cw[4 * i + 2] *= a.z, cw[4 * i + 3] *= a.w;
        if constexpr (kInter) sw[4 * i] *= b.y, sw[4 * i + 1] *= b.x, sw[4 * i + 2] *= b.w, sw[4 * i + 3] *= b.z;
        else sw[4 * i] *= b.x, sw[4 * i + 1] *= b.y, sw[4 * i + 2] *= b.z, sw[4 * i + 3] *= b.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = make_float2(cw[2 * i], cw[2 * i + 1]), s[i] = make_float2(sw[2 * i], sw[2 * i + 1]);
  }
  // the lane that holds the other half of this lane's pairs (half-split)
  const int partner = (lane & ~(kLanes - 1)) + pd / 8;
  const int slot = P.slot_map && kind != kRopeQ ? __ldg(P.slot_map + t) : -1;
  const int64_t blk = slot >= 0 ? slot / P.bs : 0;
  const int off = slot >= 0 ? slot - static_cast<int>(blk) * P.bs : 0;

#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    if (h0 + u >= heads) break;          // (warp-uniform)
    uint4 o = raw[u];                    // a value head passes through
    if (kind != kRopeV) {
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      uint32_t pw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pw[i] = kInter ? __byte_perm(w[i], 0, 0x1032) : __shfl_sync(~0u, w[i], partner);
        if (!rot) pw[i] = 0;             // (0 * inf would reach the entries that stay)
      }
      float2 x[4], r2 = make_float2(1.f, 1.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      if (wt) {
        float2 q2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) q2 = __ffma2_rn(x[i], x[i], q2);
        float ss = q2.x + q2.y;
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
        r2.x = r2.y = rsqrtf(fmaf(ss, 1.f / D, P.eps));
      }
      uint32_t ow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = make_float2(__uint_as_float(pw[i] << 16), __uint_as_float(pw[i] & 0xffff0000u));
        const float2 y = __fmul2_rn(__ffma2_rn(p, s[i], __fmul2_rn(x[i], c[i])), r2);
        const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
        ow[i] = *reinterpret_cast<const uint32_t *>(&b);
      }
      o = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
    if (kind == kRopeQ) {
      if (in) *reinterpret_cast<uint4 *>(P.q_out + (t * P.n_heads + h0 + u) * D + d0) = o;
      continue;
    }
    uint32_t codes = 0, scale = 0;
    if (P.format == ECHO_BLOCK_FP4) {    // (every lane: the scale is a shuffle)
      float x[8];
      unpack_bf16x8(o, x);
      codes = quantise8(x, scale);
    }
    if (!in) continue;
    uint16_t *out = kind == kRopeV ? P.v_out : P.k_out;
    if (out) {
      *reinterpret_cast<uint4 *>(out + (t * P.n_kv_heads + h0 + u) * D + d0) =
          P.format == ECHO_BLOCK_FP4 ? dequantise8(codes, scale) : o;
    }
    if (slot < 0) continue;
    const int64_t row = blk * P.n_kv_heads + h0 + u;
    if (row >= P.n_rows) {
      if (l == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
      continue;
    }
    uint16_t *base = P.rows + row * P.row_elems;
    if (P.format == ECHO_BLOCK_FP4) {
      using Sub = Fp4Sub<D>;
      uint8_t *sub = reinterpret_cast<uint8_t *>(base) + off / kSubTokens * Sub::kBytes;
      const int tk = off % kSubTokens;
      if (kind == kRopeK) {
        *reinterpret_cast<uint32_t *>(sub + tk * (D / 2) + l * 4) = codes;
        if (!(l & 1)) sub[Sub::kKeyScales + tk * (D / 16) + l / 2] = static_cast<uint8_t>(scale);
      } else {
        constexpr int kPart = D / 8;     // dims of a part: 16 (two lanes) or 8 (one lane)
        *reinterpret_cast<uint32_t *>(sub + Sub::kValues + (tk / 8) * (4 * D) + ((d0 / kPart) * 8 + tk % 8) * (D / 16) +
                                      (d0 % kPart) / 2) = codes;
        if (!(l & 1)) sub[Sub::kValueScales + (tk / 8) * (D / 2) + (l / 2) * 8 + tk % 8] = static_cast<uint8_t>(scale);
      }
    } else {
      *reinterpret_cast<uint4 *>(base + (kind == kRopeV ? static_cast<int64_t>(P.bs) * D : 0) + static_cast<int64_t>(off) * D + d0) = o;
    }
  }
}

}  // namespace echo

namespace echo_host {

template <int D, int kHeads, bool kInter>
static cudaError_t launch_rope(echo::RopeParams P, bool values, cudaStream_t stream) {
  P.q_chunks = (P.n_heads + kHeads - 1) / kHeads;
  P.k_chunks = (P.n_kv_heads + kHeads - 1) / kHeads;
  P.chunks = P.q_chunks + (values ? 2 : 1) * P.k_chunks;
  constexpr int kTokens = 256 / D;
  const int64_t warps = (static_cast<int64_t>(P.T) + kTokens - 1) / kTokens * P.chunks;
  const int64_t grid = (warps * 32 + echo::kRopeThreads - 1) / echo::kRopeThreads;
  echo::qk_norm_rope_kernel<D, kHeads, kInter><<<static_cast<unsigned>(grid), echo::kRopeThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_rope_dim(const echo::RopeParams &P, bool values, bool many, cudaStream_t stream) {
  if (many) return P.interleaved ? launch_rope<D, 8, true>(P, values, stream) : launch_rope<D, 8, false>(P, values, stream);
  return P.interleaved ? launch_rope<D, 1, true>(P, values, stream) : launch_rope<D, 1, false>(P, values, stream);
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
  P.status = a->dev_status;
  // value heads have work only when something takes them
  const bool values = a->v && (a->slot_map || a->v_out);
  const bool many = static_cast<int64_t>(a->T) * (a->n_heads + 2 * a->n_kv_heads) >= 16384;
  const cudaError_t e = a->head_dim == 128 ? launch_rope_dim<128>(P, values, many, stream) : launch_rope_dim<64>(P, values, many, stream);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "qk norm + rope launch");
}

}  // namespace echo_host
