// libmoe C ABI: host-side validation of the norm and of the calls on 4-bit
// weights.  As in abi.cpp, everything is checked before the first launch.
#include "moe_fp4.h"
#include "moe_norm.h"

#include <math.h>

using namespace moe;

#define REQUIRE(p)                                                            \
  do {                                                                        \
    if (!(p)) return set_error(MOE_ERR_NULL, "%s: %s is NULL", __func__, #p); \
  } while (0)
#define ALIGNED(p, n)                                                                        \
  do {                                                                                       \
    if ((uintptr_t)(p) % (n))                                                                \
      return set_error(MOE_ERR_ARG, "%s: %s is not %d-byte aligned", __func__, #p, (int)(n)); \
  } while (0)

static int start(const moe_shape* s) {
  set_error(MOE_OK, "");
  return validate_shape(s);
}

static int blocks_of_128(const moe_shape* s, const char* fn) {
  if (s->d % 128 || s->F % 128)
    return set_error(MOE_ERR_SHAPE, "%s: d = %lld and F = %lld must be multiples of 128", fn,
                     (long long)s->d, (long long)s->F);
  return MOE_OK;
}

static int need(const char* fn, size_t have, size_t bytes) {
  if (have < bytes)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu required", fn, have, bytes);
  return MOE_OK;
}

static int weights_fp4(const moe_fp4_weights* w, const char* fn) {
  if (!w || !w->gu || !w->gu_s || !w->down || !w->down_s)
    return set_error(MOE_ERR_NULL, "%s: w or a pointer of it is NULL", fn);
  if ((uintptr_t)w->gu % 16 || (uintptr_t)w->down % 16 || (uintptr_t)w->gu_s % 4 ||
      (uintptr_t)w->down_s % 4)
    return set_error(MOE_ERR_ARG, "%s: the codes must be 16-byte aligned, the scales 4-byte", fn);
  return MOE_OK;
}

extern "C" {

int moe_rmsnorm(const moe_shape* s, const void* x, const void* res, const void* gamma, float eps,
                void* r, void* y, void* q, uint8_t* qs, float* rstd, hipStream_t stream) {
  if (int rc = start(s)) return rc;
  if (!(eps >= 1e-30f) || !isfinite(eps))
    return set_error(MOE_ERR_ARG, "%s: eps = %g must be finite and at least 1e-30", __func__,
                     (double)eps);
  REQUIRE(gamma);
  ALIGNED(gamma, 16);
  if (q && s->d % MOE_FP8_BLOCK)
    return set_error(MOE_ERR_SHAPE, "%s: d = %lld, 8-bit rows need a multiple of %d", __func__,
                     (long long)s->d, MOE_FP8_BLOCK);
  if (s->T == 0) return MOE_OK;
  REQUIRE(x);
  if (!y && !q) return set_error(MOE_ERR_NULL, "%s: y and q are both NULL", __func__);
  if (!q != !qs) return set_error(MOE_ERR_NULL, "%s: q and qs go together", __func__);
  if (r && !res)
    return set_error(MOE_ERR_ARG, "%s: r goes with res (without it r is x)", __func__);
  ALIGNED(x, 16);
  ALIGNED(res, 16);
  ALIGNED(r, 16);
  ALIGNED(y, 16);
  ALIGNED(q, 16);
  ALIGNED(qs, 4);
  ALIGNED(rstd, 4);
  return launch_rmsnorm(s, x, res, gamma, eps, r, y, q, qs, rstd, stream);
}

size_t moe_rmsnorm_workspace_bytes(const moe_shape* s) {
  if (start(s)) return 0;
  return norm_workspace_bytes(s);
}

int moe_rmsnorm_bwd(const moe_shape* s, const void* dy, const void* r, const void* gamma,
                    const float* rstd, const void* dres, void* dx, float* dgamma, int accumulate,
                    void* ws, size_t ws_bytes, hipStream_t stream) {
  if (int rc = start(s)) return rc;
  REQUIRE(gamma);
  if (s->T > 0) {
    REQUIRE(dy);
    REQUIRE(r);
    REQUIRE(rstd);
    REQUIRE(dx);
  }
  if (accumulate & ~MOE_ACCUM_DW)
    return set_error(MOE_ERR_ARG, "%s: unknown accumulate bits 0x%x", __func__, accumulate);
  ALIGNED(dy, 16);
  ALIGNED(r, 16);
  ALIGNED(gamma, 16);
  ALIGNED(rstd, 4);
  ALIGNED(dres, 16);
  ALIGNED(dx, 16);
  ALIGNED(dgamma, 16);
  if (dgamma) {
    REQUIRE(ws);
    ALIGNED(ws, 16);
    if (int rc = need(__func__, ws_bytes, norm_workspace_bytes(s))) return rc;
  }
  return launch_rmsnorm_bwd(s, dy, r, gamma, rstd, dres, dx, dgamma, accumulate != 0, (float*)ws,
                            stream);
}

int moe_quant_weights_fp4(const moe_shape* s, const void* W_gu, const void* W_down,
                          const moe_fp4_weights* w, hipStream_t stream) {
  if (int rc = start(s)) return rc;
  if (int rc = blocks_of_128(s, __func__)) return rc;
  REQUIRE(W_gu);
  REQUIRE(W_down);
  if (int rc = weights_fp4(w, __func__)) return rc;
  ALIGNED(W_gu, 16);
  ALIGNED(W_down, 16);
  return launch_quant_weights_fp4(s, W_gu, W_down, w, stream);
}

int moe_dequant_weights_fp4(const moe_shape* s, const moe_fp4_weights* w, void* W_gu,
                            void* W_down, hipStream_t stream) {
  if (int rc = start(s)) return rc;
  if (int rc = blocks_of_128(s, __func__)) return rc;
  if (int rc = weights_fp4(w, __func__)) return rc;
  REQUIRE(W_gu);
  REQUIRE(W_down);
  ALIGNED(W_gu, 16);
  ALIGNED(W_down, 16);
  return launch_dequant_weights_fp4(s, w, W_gu, W_down, stream);
}

size_t moe_fp4_workspace_bytes(const moe_shape* s) {
  if (start(s) || blocks_of_128(s, __func__)) return 0;
  return fp4_workspace_bytes(s);
}

int moe_expert_ffn_fwd_fp4(const moe_shape* s, const void* xq, const uint8_t* xs,
                           const int32_t* pair_of_row, const int32_t* offsets,
                           const int32_t* tile_offsets, const moe_fp4_weights* w, void* h,
                           void* a, void* yp, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (int rc = start(s)) return rc;
  if (int rc = blocks_of_128(s, __func__)) return rc;
  if (int rc = weights_fp4(w, __func__)) return rc;
  if (!is16(s))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: the products need 16-bit data", __func__);
  if (s->T == 0) return MOE_OK;
  REQUIRE(xq);
  REQUIRE(xs);
  REQUIRE(offsets);
  REQUIRE(tile_offsets);
  REQUIRE(yp);
  REQUIRE(ws);
  if (pair_of_row && s->T * s->d >= (1LL << 31))
    return set_error(MOE_ERR_SHAPE, "%s: T*d = %lld, gathered rows need it below 2^31", __func__,
                     (long long)(s->T * s->d));
  ALIGNED(xq, 16);
  ALIGNED(xs, 4);
  ALIGNED(h, 16);
  ALIGNED(a, 16);
  ALIGNED(yp, 16);
  ALIGNED(ws, 16);
  if (int rc = need(__func__, ws_bytes, fp4_workspace_bytes(s))) return rc;
  return launch_ffn_fwd_fp4(s, xq, xs, pair_of_row, offsets, tile_offsets, w, h, a, yp, ws,
                            stream);
}

}  // extern "C"
