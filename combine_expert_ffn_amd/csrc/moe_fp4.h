// Internal declarations of the experts on 4-bit weights.
#pragma once

#include "moe_fp8.h"

namespace moe {

// Scale byte of a block of 4-bit values from the bits of its largest magnitude: the
// biased exponent of the smallest power of two with amax <= 7 * 2^(byte - 127).  7 =
// 1.75 * 2^2, so as fp8_scale_byte (448 = 1.75 * 2^8) with another exponent.  255
// (NaN) for an infinity or NaN, whose bits are the largest.
__device__ __forceinline__ int fp4_scale_byte(uint32_t amax) {
  const int b = (int)((amax + 0x1fffffu) >> 23) - 2;
  return amax >= 0x7f800000u ? 255 : (amax == 0 ? 127 : (b < 0 ? 0 : b));
}
// Eight codes (a register) times a power of two, exact in bf16 (from its smallest
// normal value on); NaN with scale byte 255, whose factor is an infinity.
__device__ __forceinline__ bf16x8_t widen4(uint32_t v, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

int launch_quant_weights_fp4(const moe_shape* s, const void* W_gu, const void* W_down,
                             const moe_fp4_weights* w, hipStream_t st);
int launch_dequant_weights_fp4(const moe_shape* s, const moe_fp4_weights* w, void* W_gu,
                               void* W_down, hipStream_t st);
size_t fp4_workspace_bytes(const moe_shape* s);
int launch_ffn_fwd_fp4(const moe_shape* s, const void* xq, const uint8_t* xs,
                       const int32_t* xrows, const int32_t* offsets,
                       const int32_t* tile_offsets, const moe_fp4_weights* w, void* h, void* a,
                       void* yp, void* ws, hipStream_t st);
// The same for few rows per expert (gemm_fp4_small.hip), and the rule that takes it.
bool fp4_small(const moe_shape* s);
size_t fp4_small_workspace_bytes(const moe_shape* s);
int launch_ffn_fwd_fp4_small(const moe_shape* s, const void* xq, const uint8_t* xs,
                             const int32_t* xrows, const int32_t* offsets,
                             const moe_fp4_weights* w, void* h, void* a, void* yp, void* ws,
                             hipStream_t st);

}  // namespace moe
