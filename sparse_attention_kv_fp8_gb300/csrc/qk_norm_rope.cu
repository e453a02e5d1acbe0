// qk_norm_rope.cu -- per-head RMS norm and rotation of queries and keys, with the keys and
// values written to their cache rows (bf16 or 4-bit) in the same pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A head is read by head_dim / 8 lanes, one 16-byte load each, and never leaves registers
// until its results are stored: the mean is a shuffle sum over those lanes, the partner of
// a half-split pair sits in the lane rope_dim / 16 away (a shuffle), of an interleaved pair
// in the same lane; a 4-bit scale covers 16 dimensions, so two neighbouring lanes.  A lane
// group takes kHeads heads of one token: their loads are issued together (bytes in flight)
// and the token's cosines and sines are read once for them.  Bound by HBM.
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
  int32_t heads;      // q + k + v heads that have work
  int32_t chunks;     // lane groups per token
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

template <int D, int kHeads>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams P) {
  constexpr int kLanes = D / 8;  // lanes of a head
  const int64_t group = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes, d0 = 8 * l;
  // groups of one warp may belong to different tokens: shuffles run over the whole warp,
  // so no lane leaves early
  const int64_t tok = group / P.chunks;
  const int chunk = static_cast<int>(group - tok * P.chunks);
  const int64_t t = min(tok, static_cast<int64_t>(P.T) - 1);
  const int pos = __ldg(P.positions + t);
  const bool in = tok < P.T && pos >= 0 && pos < P.max_pos;
  if (tok < P.T && pos >= P.max_pos && l == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
  const int slot = P.slot_map ? __ldg(P.slot_map + t) : -1;
  const int nk = P.n_heads + P.n_kv_heads;

  uint4 raw[kHeads];
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const int h = chunk * kHeads + u;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (in && h < P.heads) {
      const uint16_t *src = h < P.n_heads ? P.q + t * P.q_stride + static_cast<int64_t>(h) * D
                            : h < nk      ? P.k + t * P.k_stride + static_cast<int64_t>(h - P.n_heads) * D
                                          : P.v + t * P.v_stride + static_cast<int64_t>(h - nk) * D;
      raw[u] = *reinterpret_cast<const uint4 *>(src + d0);
    }
  }
  // the rotation as y' = y * c + partner * s, with the sign of the sine folded in
  const int half = P.rope_dim >> 1;
  const bool rot = d0 < P.rope_dim;
  const bool low = d0 < half;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (in && rot && chunk * kHeads < nk) {
    const float *row = P.cos_sin + static_cast<int64_t>(pos) * P.rope_dim;
    if (P.interleaved) {
      const float4 cc = *reinterpret_cast<const float4 *>(row + d0 / 2);
      const float4 ss = *reinterpret_cast<const float4 *>(row + half + d0 / 2);
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) c[2 * i] = c[2 * i + 1] = cv[i], s[2 * i] = -sv[i], s[2 * i + 1] = sv[i];
    } else {
      const float *cr = row + (low ? d0 : d0 - half);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cc = reinterpret_cast<const float4 *>(cr)[i];
        const float4 ss = reinterpret_cast<const float4 *>(cr + half)[i];
        c[4 * i] = cc.x, c[4 * i + 1] = cc.y, c[4 * i + 2] = cc.z, c[4 * i + 3] = cc.w;
        s[4 * i] = ss.x, s[4 * i + 1] = ss.y, s[4 * i + 2] = ss.z, s[4 * i + 3] = ss.w;
      }
      if (low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    }
  }
  // the lane that holds the other half of this lane's pairs (half-split)
  const int partner = (threadIdx.x & 31 & ~(kLanes - 1)) + (rot ? (low ? l + half / 8 : l - half / 8) : l);
  const int64_t blk = slot >= 0 ? slot / P.bs : 0;
  const int off = slot >= 0 ? slot - static_cast<int>(blk) * P.bs : 0;

#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const int h = chunk * kHeads + u;
    const bool is_q = h < P.n_heads, is_v = h >= nk;
    float x[8];
    unpack_bf16x8(raw[u], x);
    const float *wt = is_q ? P.q_weight : P.k_weight;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
    if (!is_v && wt) {
      const float r = 1.f / sqrtf(ss * (1.f / D) + P.eps);
      const float4 w0 = __ldg(reinterpret_cast<const float4 *>(wt + d0)), w1 = __ldg(reinterpret_cast<const float4 *>(wt + d0) + 1);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    }
    float y[8];
    if (P.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(~0u, x[i], partner);
    }
    uint4 o = raw[u];  // a value head passes through
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(y[i], s[i], x[i] * c[i]);
      o = pack_bf16x8(x);
    }
    const bool live = in && h < P.heads;
    if (is_q) {
      if (live) *reinterpret_cast<uint4 *>(P.q_out + (t * P.n_heads + h) * D + d0) = o;
    }
    uint32_t codes = 0, scale = 0;
    if (P.format == ECHO_BLOCK_FP4) {  // (every lane: the scale is a shuffle)
      unpack_bf16x8(o, x);
      codes = quantise8(x, scale);
    }
    if (is_q || !live) continue;
    const int hk = is_v ? h - nk : h - P.n_heads;
    uint16_t *out = is_v ? P.v_out : P.k_out;
    if (out) {
      *reinterpret_cast<uint4 *>(out + (t * P.n_kv_heads + hk) * D + d0) =
          P.format == ECHO_BLOCK_FP4 ? dequantise8(codes, scale) : o;
    }
    if (slot < 0 || !P.rows) continue;
    const int64_t row = blk * P.n_kv_heads + hk;
    if (row >= P.n_rows) {
      if (l == 0) set_status(P.status, ECHO_DEV_BAD_INDEX);
      continue;
    }
    uint16_t *base = P.rows + row * P.row_elems;
    if (P.format == ECHO_BLOCK_FP4) {
      using Sub = Fp4Sub<D>;
      uint8_t *sub = reinterpret_cast<uint8_t *>(base) + off / kSubTokens * Sub::kBytes;
      const int tk = off % kSubTokens;
      if (!is_v) {
        *reinterpret_cast<uint32_t *>(sub + tk * (D / 2) + l * 4) = codes;
        if (!(l & 1)) sub[Sub::kKeyScales + tk * (D / 16) + l / 2] = static_cast<uint8_t>(scale);
      } else {
        constexpr int kPart = D / 8;  // dims of a part: 16 (two lanes) or 8 (one lane)
        *reinterpret_cast<uint32_t *>(sub + Sub::kValues + (tk / 8) * (4 * D) + ((d0 / kPart) * 8 + tk % 8) * (D / 16) +
                                      (d0 % kPart) / 2) = codes;
        if (!(l & 1)) sub[Sub::kValueScales + (tk / 8) * (D / 2) + (l / 2) * 8 + tk % 8] = static_cast<uint8_t>(scale);
      }
    } else {
      *reinterpret_cast<uint4 *>(base + (is_v ? static_cast<int64_t>(P.bs) * D : 0) + static_cast<int64_t>(off) * D + d0) = o;
    }
  }
}

}  // namespace echo

namespace echo_host {

template <int D, int kHeads>
static cudaError_t launch_rope(echo::RopeParams P, cudaStream_t stream) {
  P.chunks = (P.heads + kHeads - 1) / kHeads;
  const int64_t threads = static_cast<int64_t>(P.T) * P.chunks * (D / 8);
  const int64_t grid = (threads + echo::kRopeThreads - 1) / echo::kRopeThreads;
  echo::qk_norm_rope_kernel<D, kHeads><<<static_cast<unsigned>(grid), echo::kRopeThreads, 0, stream>>>(P);
  return cudaGetLastError();
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
  P.heads = a->n_heads + a->n_kv_heads + (a->v && (a->slot_map || a->v_out) ? a->n_kv_heads : 0);
  const bool many = static_cast<int64_t>(a->T) * P.heads >= 16384;
  cudaError_t e;
  if (a->head_dim == 128) e = many ? launch_rope<128, 4>(P, stream) : launch_rope<128, 1>(P, stream);
  else e = many ? launch_rope<64, 4>(P, stream) : launch_rope<64, 1>(P, stream);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, "qk norm + rope launch");
}

}  // namespace echo_host
