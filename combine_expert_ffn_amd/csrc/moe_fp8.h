// Internal declarations of the 8-bit expert path and the weight update.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

int validate_shape(const moe_shape* s);  // abi.cpp

// Bytes per row of scales for k values: a multiple of 4, so that four blocks'
// scales are one aligned 32-bit load.
inline int64_t fp8_scale_ld(int64_t k) { return (cdiv(k, MOE_FP8_BLOCK) + 3) / 4 * 4; }

// ---------------------------------------------------------------------------
// the block format
// ---------------------------------------------------------------------------
// Scale byte of a block with largest finite magnitude amax (>= 0): the biased
// exponent of the smallest power of two with amax <= 448 * 2^(byte - 127).
// 448 = 1.75 * 2^8, so the exponent is amax's own less 8, one more if its
// mantissa is above 1.75 (adding 0x1fffff carries exactly then).
__device__ __forceinline__ int fp8_scale_byte(float amax) {
  const int b = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
  return amax == 0.f ? 127 : (b < 0 ? 0 : b);
}
// 2^(127 - byte), the factor into the block's units; byte <= 247 for a finite
// amax, so it is a normal float.
__device__ __forceinline__ float fp8_inv_scale(int byte) {
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^(byte - 127); subnormal for byte 0.
__device__ __forceinline__ float fp8_scale_value(int byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)byte << 23);
}
// |x| for finite x, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.f;
}
// Four floats in the block's units -> four e4m3 bytes, to nearest even
// (v_cvt_pk_fp8_f32; magnitudes are at most 448, and an infinity is made a NaN
// by the caller's finite_or_nan).
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}
__device__ __forceinline__ float finite_or_nan(float x) {
  return fabsf(x) < __builtin_inff() ? x : __builtin_nanf("");
}

// Largest value over each row of 8 or 16 lanes, in every lane of it: lanes swapped
// within pairs and quads, then the halves of 8 and of 16 mirrored.
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
  auto step = [](float x, int moved) { return fmaxf(x, __int_as_float(moved)); };
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, true));
  if constexpr (N == 16)
    v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, true));
  return v;
}
// Eight e4m3 values (two registers) times a power of two, exact in bf16
// (from its smallest normal value on).
__device__ __forceinline__ bf16x8_t widen(int lo, int hi, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Loads and stores of N words, with PAST past the caches (non-temporal): for data of
// which no cache holds the beginning when the end is reached.
template <int N, bool PAST>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N)));
  static __device__ __forceinline__ type load(const void* p) {
    return PAST ? __builtin_nontemporal_load((const type*)p) : *(const type*)p;
  }
  static __device__ __forceinline__ void store(void* p, type v) {
    if constexpr (PAST) __builtin_nontemporal_store(v, (type*)p);
    else *(type*)p = v;
  }
};
// The size from which on that is so: half of the last-level cache, 256 MB.
constexpr int64_t kPastCaches = 128 << 20;

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
int launch_quant_rows(const moe_shape* s, const void* src, int64_t rows, const int32_t* n_rows,
                      void* q, uint8_t* qs, hipStream_t st);
int launch_quant_weights(const moe_shape* s, const void* W_gu, const void* W_down,
                         const moe_fp8_weights* w, hipStream_t st);
// The 8-bit experts.  ws: q of a (or dh) [T*K][F] ([T*K][2F]), then its scales.
size_t fp8_workspace_bytes(const moe_shape* s);
int launch_ffn_fwd_fp8(const moe_shape* s, const void* xq, const uint8_t* xs,
                       const int32_t* xrows, const int32_t* offsets,
                       const int32_t* tile_offsets, const moe_fp8_weights* w, void* h, void* a,
                       void* yp, void* ws, hipStream_t st);
int launch_ffn_dgrad_fp8(const moe_shape* s, const void* dq, const uint8_t* ds,
                         const int32_t* xrows, const float* gates, const void* h,
                         const int32_t* offsets, const int32_t* tile_offsets,
                         const moe_fp8_weights* w, void* dh, void* dxp, void* ag, void* ws,
                         hipStream_t st);
// The same for few rows per expert (gemm_fp8_small.hip), and the rule that takes it.
bool fp8_small(const moe_shape* s, bool dgrad);
size_t fp8_small_workspace_bytes(const moe_shape* s);
int launch_ffn_fwd_fp8_small(const moe_shape* s, const void* xq, const uint8_t* xs,
                             const int32_t* xrows, const int32_t* offsets,
                             const moe_fp8_weights* w, void* h, void* a, void* yp, void* ws,
                             hipStream_t st);
int launch_ffn_dgrad_fp8_small(const moe_shape* s, const void* dq, const uint8_t* ds,
                               const int32_t* xrows, const float* gates, const void* h,
                               const int32_t* offsets, const moe_fp8_weights* w, void* dh,
                               void* dxp, void* ag, void* ws, hipStream_t st);
int launch_adamw(const moe_adamw_tensor* t, int n, const moe_adamw_hyper* hp, hipStream_t st);

}  // namespace moe
