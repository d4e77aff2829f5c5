// Internal declarations of the layer's norm.
#pragma once

#include "moe_internal.h"

namespace moe {

// Rows that a block of 256 threads works on at once, by the width: 16, 64 or 256
// lanes to a row.
inline int norm_lanes(int64_t d) { return d <= 512 ? 16 : (d <= 2048 ? 64 : 256); }
// Blocks of the backward pass, each of which leaves one row of partial sums of
// dgamma in the workspace: four per CU at most, and, past one per CU, so many that each
// walks over 64 rows of up to 512, 16 of up to 2048 or 8 of more, since a row of sums in
// float32 is twice a row of the input.  In us, dx and dgamma together, bf16, with a block for every row or four of
// up to 2048 / with these: 1500 x 4096 26 / 16, 4096 x 4096 32 / 27, 2048 x 16384 99 / 52, 4096 x
// 2048 19 / 16; 16 rows where it is 8: 1500 x 4096 17.  8192 x 640: 11.3 / 11.0, with 32 rows 13.6.
constexpr int64_t kNormParts = 1024;
inline int64_t norm_parts(int64_t T, int64_t d) {
  const int64_t at_once = 256 / norm_lanes(d), n = cdiv(T, at_once);
  const int64_t m = T / (at_once == 1 ? 8 : 4 * at_once);
  return n <= 256 ? n : (m < 256 ? 256 : (m < kNormParts ? m : kNormParts));
}
inline size_t norm_workspace_bytes(const moe_shape* s) {
  const size_t b = align_up((size_t)(norm_parts(s->T, s->d) * s->d) * sizeof(float), 256);
  return b < 256 ? 256 : b;
}

int launch_rmsnorm(const moe_shape* s, const void* x, const void* res, const void* gamma,
                   float eps, void* r, void* y, void* q, uint8_t* qs, float* rstd,
                   hipStream_t st);
int launch_rmsnorm_bwd(const moe_shape* s, const void* dy, const void* r, const void* gamma,
                       const float* rstd, const void* dres, void* dx, float* dgamma,
                       bool accumulate, float* parts, hipStream_t st);

}  // namespace moe
