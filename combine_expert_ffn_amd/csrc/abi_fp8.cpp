// libmoe C ABI: host-side validation of the 8-bit expert calls and of the
// weight update.  As in abi.cpp, everything is checked before the first launch.
#include "moe_fp8.h"

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

namespace moe {

static int validate_fp8_shape(const moe_shape* s, const char* fn) {
  set_error(MOE_OK, "");
  if (int rc = validate_shape(s)) return rc;
  if (s->d % MOE_FP8_BLOCK || s->F % MOE_FP8_BLOCK)
    return set_error(MOE_ERR_SHAPE, "%s: d = %lld and F = %lld must be multiples of %d", fn,
                     (long long)s->d, (long long)s->F, MOE_FP8_BLOCK);
  return MOE_OK;
}

// The checks the two product calls share.
static int validate_fp8_product(const moe_shape* s, const char* fn, const void* q, const void* qs,
                                const int32_t* pair_of_row, const void* ws, size_t ws_bytes) {
  if (!is16(s))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: the 8-bit products need 16-bit data", fn);
  if (pair_of_row && s->T * s->d >= (1LL << 31))
    return set_error(MOE_ERR_SHAPE, "%s: T*d = %lld, gathered rows need it below 2^31", fn,
                     (long long)(s->T * s->d));
  if ((uintptr_t)q % 16 || (uintptr_t)qs % 4 || (uintptr_t)ws % 16)
    return set_error(MOE_ERR_ARG, "%s: the quantised rows and ws must be 16-byte aligned, their "
                     "scales 4-byte", fn);
  const size_t need = fp8_workspace_bytes(s);
  if (ws_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu required", fn, ws_bytes,
                     need);
  return MOE_OK;
}

}  // namespace moe

extern "C" {

int64_t moe_fp8_scale_ld(int64_t k) { return k < 0 ? 0 : fp8_scale_ld(k); }

size_t moe_fp8_workspace_bytes(const moe_shape* s) {
  if (validate_fp8_shape(s, __func__)) return 0;
  return fp8_workspace_bytes(s);
}

int moe_quant_rows_fp8(const moe_shape* s, const void* src, int64_t rows, const int32_t* n_rows,
                       void* q, uint8_t* qs, hipStream_t stream) {
  if (int rc = validate_fp8_shape(s, __func__)) return rc;
  if (rows < 0 || rows >= (1LL << 31))
    return set_error(MOE_ERR_SHAPE, "%s: rows = %lld outside [0, 2^31)", __func__,
                     (long long)rows);
  REQUIRE(src);
  REQUIRE(q);
  REQUIRE(qs);
  ALIGNED(src, 16);
  ALIGNED(q, 16);
  ALIGNED(qs, 4);
  if (rows == 0) return MOE_OK;
  return launch_quant_rows(s, src, rows, n_rows, q, qs, stream);
}

int moe_quant_weights_fp8(const moe_shape* s, const void* W_gu, const void* W_down,
                          const moe_fp8_weights* w, hipStream_t stream) {
  if (int rc = validate_fp8_shape(s, __func__)) return rc;
  REQUIRE(W_gu);
  REQUIRE(W_down);
  REQUIRE(w);
  REQUIRE(w->gu);
  REQUIRE(w->gu_s);
  REQUIRE(w->down);
  REQUIRE(w->down_s);
  if (w->guT || w->guT_s || w->downT || w->downT_s) {
    REQUIRE(w->guT);
    REQUIRE(w->guT_s);
    REQUIRE(w->downT);
    REQUIRE(w->downT_s);
  }
  ALIGNED(W_gu, 16);
  ALIGNED(W_down, 16);
  ALIGNED(w->gu, 16);
  ALIGNED(w->down, 16);
  ALIGNED(w->guT, 16);
  ALIGNED(w->downT, 16);
  ALIGNED(w->gu_s, 4);
  ALIGNED(w->down_s, 4);
  ALIGNED(w->guT_s, 4);
  ALIGNED(w->downT_s, 4);
  return launch_quant_weights(s, W_gu, W_down, w, stream);
}

int moe_expert_ffn_fwd_fp8(const moe_shape* s, const void* xq, const uint8_t* xs,
                           const int32_t* pair_of_row, const int32_t* offsets,
                           const int32_t* tile_offsets, const moe_fp8_weights* w, void* h,
                           void* a, void* yp, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (int rc = validate_fp8_shape(s, __func__)) return rc;
  REQUIRE(xq);
  REQUIRE(xs);
  REQUIRE(offsets);
  REQUIRE(tile_offsets);
  REQUIRE(w);
  REQUIRE(w->gu);
  REQUIRE(w->gu_s);
  REQUIRE(w->down);
  REQUIRE(w->down_s);
  REQUIRE(yp);
  REQUIRE(ws);
  ALIGNED(w->gu, 16);
  ALIGNED(w->down, 16);
  ALIGNED(w->gu_s, 4);
  ALIGNED(w->down_s, 4);
  ALIGNED(h, 16);
  ALIGNED(a, 16);
  ALIGNED(yp, 16);
  if (int rc = validate_fp8_product(s, __func__, xq, xs, pair_of_row, ws, ws_bytes)) return rc;
  if (s->T == 0) return MOE_OK;
  return launch_ffn_fwd_fp8(s, xq, xs, pair_of_row, offsets, tile_offsets, w, h, a, yp, ws,
                            stream);
}

int moe_ffn_dgrad_fp8(const moe_shape* s, const void* dq, const uint8_t* ds,
                      const int32_t* pair_of_row, const float* gates, const void* h,
                      const int32_t* offsets, const int32_t* tile_offsets,
                      const moe_fp8_weights* w, void* dh, void* dxp, void* ag, void* ws,
                      size_t ws_bytes, hipStream_t stream) {
  if (int rc = validate_fp8_shape(s, __func__)) return rc;
  REQUIRE(dq);
  REQUIRE(ds);
  REQUIRE(h);
  REQUIRE(offsets);
  REQUIRE(tile_offsets);
  REQUIRE(w);
  REQUIRE(w->guT);
  REQUIRE(w->guT_s);
  REQUIRE(w->downT);
  REQUIRE(w->downT_s);
  REQUIRE(dh);
  REQUIRE(dxp);
  REQUIRE(ws);
  if (pair_of_row) {
    REQUIRE(gates);
  } else if (gates || ag) {
    return set_error(MOE_ERR_ARG, "%s: gates and ag go with pair_of_row (rows gathered by token)",
                     __func__);
  }
  ALIGNED(w->guT, 16);
  ALIGNED(w->downT, 16);
  ALIGNED(w->guT_s, 4);
  ALIGNED(w->downT_s, 4);
  ALIGNED(h, 16);
  ALIGNED(dh, 16);
  ALIGNED(dxp, 16);
  ALIGNED(ag, 16);
  if (int rc = validate_fp8_product(s, __func__, dq, ds, pair_of_row, ws, ws_bytes)) return rc;
  if (s->T == 0) return MOE_OK;
  return launch_ffn_dgrad_fp8(s, dq, ds, pair_of_row, gates, h, offsets, tile_offsets, w, dh, dxp,
                              ag, ws, stream);
}

int moe_adamw(const moe_adamw_tensor* t, int n, const moe_adamw_hyper* hp, hipStream_t stream) {
  set_error(MOE_OK, "");
  REQUIRE(hp);
  if (n < 0) return set_error(MOE_ERR_SHAPE, "%s: n = %d < 0", __func__, n);
  if (n > 0) REQUIRE(t);
  if (!(hp->beta1 >= 0 && hp->beta1 < 1 && hp->beta2 >= 0 && hp->beta2 < 1))
    return set_error(MOE_ERR_ARG, "%s: beta1 = %g, beta2 = %g outside [0, 1)", __func__,
                     hp->beta1, hp->beta2);
  if (!((float)hp->eps > 0) || !isfinite(hp->eps) || !isfinite(hp->lr) || !isfinite(hp->grad_scale))
    return set_error(MOE_ERR_ARG, "%s: eps = %g must be positive, lr = %g and grad_scale = %g "
                     "finite", __func__, hp->eps, hp->lr, (double)hp->grad_scale);
  if (hp->step < 1)
    return set_error(MOE_ERR_ARG, "%s: step = %lld < 1", __func__, (long long)hp->step);
  if (hp->reserved != 0) return set_error(MOE_ERR_ARG, "%s: reserved must be 0", __func__);
  ALIGNED(hp->grad_scale_dev, 4);
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor& x = t[i];
    if (x.n < 0 || x.n > (1LL << 34))
      return set_error(MOE_ERR_SHAPE, "%s: tensor %d has %lld elements", __func__, i,
                       (long long)x.n);
    if (x.dtype != MOE_F32 && x.dtype != MOE_BF16 && x.dtype != MOE_F16)
      return set_error(MOE_ERR_DTYPE, "%s: tensor %d: dtype %d", __func__, i, x.dtype);
    if ((x.state8 != 0 && x.state8 != 1) || x.reserved != 0 || !isfinite(x.weight_decay))
      return set_error(MOE_ERR_ARG, "%s: tensor %d: state8 = %d, reserved = %d, weight_decay = %g",
                       __func__, i, x.state8, x.reserved, (double)x.weight_decay);
    if (x.n == 0) continue;
    if (!x.param || !x.grad || !x.m || !x.v || (x.state8 && (!x.m_s || !x.v_s)))
      return set_error(MOE_ERR_NULL, "%s: tensor %d: a required pointer is NULL", __func__, i);
    if (!x.state8 && (x.m_s || x.v_s))
      return set_error(MOE_ERR_ARG, "%s: tensor %d: scales without state8", __func__, i);
    const uintptr_t es = x.dtype == MOE_F32 ? 4 : 2;
    if ((uintptr_t)x.param % es || (uintptr_t)x.master % 4 || (uintptr_t)x.grad % 4 ||
        (!x.state8 && ((uintptr_t)x.m % 4 || (uintptr_t)x.v % 4)))
      return set_error(MOE_ERR_ARG, "%s: tensor %d: a pointer is not aligned to its type",
                       __func__, i);
  }
  return launch_adamw(t, n, hp, stream);
}

}  // extern "C"
