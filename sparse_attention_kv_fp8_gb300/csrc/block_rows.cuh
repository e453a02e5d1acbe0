// block_rows.cuh -- the block-row layouts of include/echo.h (one block of tokens of one
// KV head per row), the conversions of their 4-bit entries, and the launch that the block calls share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "echo_common.cuh"

namespace echo {

constexpr int kSubTokens = 16;  // tokens of a sub-block, the unit of the 4-bit layout

// byte offsets of a 4-bit sub-block's parts (head_dim D): key codes at 0
template <int D>
struct Fp4Sub {
  static constexpr int kValues = 8 * D;
  static constexpr int kKeyScales = 16 * D;
  static constexpr int kValueScales = 17 * D;
  static constexpr int kBytes = 18 * D;
};

// 16-bit elements of a row (the arguments are already checked)
__host__ __device__ inline int64_t block_row_elems(int format, int block_tokens, int head_dim) {
  return format == ECHO_BLOCK_FP4 ? static_cast<int64_t>(block_tokens) / kSubTokens * 9 * head_dim
                                  : static_cast<int64_t>(2) * block_tokens * head_dim;
}

// two e2m1 codes (byte i of w, low nibble first) as fp16; exact.  The conversion takes the
// low byte of a register half: one shift serves the two odd bytes (four separate byte
// extractions cost 1.5x the whole conversion on the integer pipe: 17.3 cycles a word against
// 11.6 with the halves).
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b16 l, u;\n .reg .b8 p, q, r, s;\n mov.b32 {l, u}, %2;\n mov.b16 {p, q}, l;\n mov.b16 {r, s}, u;\n"
      " cvt.rn.f16x2.e2m1x2 %0, p;\n cvt.rn.f16x2.e2m1x2 %1, r;\n}\n"
      : "=r"(h[0]), "=r"(h[2])
      : "r"(w));
  asm("{\n .reg .b16 l, u;\n .reg .b8 p, q, r, s;\n mov.b32 {l, u}, %2;\n mov.b16 {p, q}, l;\n mov.b16 {r, s}, u;\n"
      " cvt.rn.f16x2.e2m1x2 %0, p;\n cvt.rn.f16x2.e2m1x2 %1, r;\n}\n"
      : "=r"(h[1]), "=r"(h[3])
      : "r"(w >> 8));
}

// eight values to e2m1 codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t e2m1x8_from_float(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// two e4m3 scales (low byte first) as fp16; exact
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(two));
  return h;
}

__device__ __forceinline__ uint32_t e4m3_from_half(__half x) {
  uint16_t r;
  const uint32_t two = __half_as_ushort(x);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(two));
  return r & 0xffu;
}

// 16 bytes, loaded where this stands: a plain load may be moved down to its first use, where one of
// several that should be under way at once then waits for the one before
__device__ __forceinline__ uint4 load16_here(const void *p) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 load8_here(const void *p) {
  uint2 x;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t load2_here(const void *p) {
  uint16_t x;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t load1_here(const void *p) {
  uint32_t x;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace echo

namespace echo_host {

// SMs of the current device; `what` names the call in the error
inline int sm_count(int *sms, const char *what) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? ECHO_OK : cuda_fail(e, what);
}

// Launch that may be made ready while the kernel before it on the stream still runs (programmatic
// stream serialization): for kernels that call pdl_wait() before they touch any memory (prefix attention's
// own tokens and merge read the call's inputs before: they say why).
// Their loads are plain ones: the non-coherent path (__ldg) is for data that nothing writes while
// the kernel is there, and the kernel before it, still running then, may write any input.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              Args &&...args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace echo_host
