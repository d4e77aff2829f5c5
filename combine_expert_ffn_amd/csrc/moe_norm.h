// Internal declarations of the layer's norm.
#pragma once

#include "moe_internal.h"

namespace moe {

// Blocks of the backward pass, each of which leaves one row of partial sums of
// dgamma in the workspace: four per CU at most.
constexpr int64_t kNormParts = 1024;
// Rows that a block of 256 threads works on at once, by the width: 16, 64 or 256
// lanes to a row.
inline int norm_lanes(int64_t d) { return d <= 512 ? 16 : (d <= 2048 ? 64 : 256); }
inline int64_t norm_parts(int64_t T, int64_t d) {
  const int64_t n = cdiv(T, 256 / norm_lanes(d));
  return n < kNormParts ? n : kNormParts;
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
