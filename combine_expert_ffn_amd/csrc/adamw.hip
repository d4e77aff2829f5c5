// AdamW over a list of tensors in one launch per 40 of them (formulas and the
// 8-bit state format in moe.h).  The step is bound by memory: an element of a
// bf16 weight with a float32 master moves 30 bytes with float32 states, 18.03
// with 8-bit ones, and every byte is touched once: 38 million elements with
// float32 states 170 us (6.7 TB/s).
#include "moe_fp8.h"

#include <math.h>

namespace moe {
namespace {

constexpr int kMax = 40;       // tensors per launch (the kernel's arguments hold them)
constexpr int kChunk = 2048;   // elements per workgroup: 16 lanes hold a block of 128
constexpr int64_t kBlocks = 1 << 23;  // workgroups per launch (2^31 threads): 2^34 elements

struct Tensor {
  void* param;
  float* master;
  const float* grad;
  void *m, *v;
  uint8_t *m_s, *v_s;
  int64_t n;
  float keep;     // 1 - lr * weight_decay
  uint32_t key;   // of the random rounding
  int32_t dtype;
  int32_t flags;  // kState8, kVec
};
enum { kState8 = 1, kVec = 2 };

struct Args {
  Tensor t[kMax];
  int32_t start[kMax + 1];  // first workgroup of each tensor
  int32_t n;
  float b1, a1, b2, a2;  // beta, 1 - beta
  float rate;            // lr / (1 - beta1^step)
  float root;            // 1 / sqrt(1 - beta2^step)
  float eps, scale;
  const float* scale_dev;
};

// 32 well mixed bits of an element's number (xor-shift and multiply by odd
// constants, twice; the constants are primes of a published 32-bit hash); the top
// 20 of them, and the top 20 of one more product, are the two roundings' random
// numbers.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0xC2B2AE3Du;
  return x ^ (x >> 16);
}

// e4m3 code of y (in the block's units, |y| <= 448), rounded up or down at
// random: rnd (20 bits) is added below the last kept bit.  Values under 2^-6
// have the fixed spacing 2^-9.  With LEAST a value that is not zero stays so: the
// second moment's root divides, and a stored 0 beside a first moment that was rounded
// up gave steps of 600 to 1000 times the learning rate (elements whose gradients are
// 1e-5 of their block's largest; at most 2.3 times with the least value kept).
template <bool LEAST>
__device__ __forceinline__ uint32_t round_fp8(float y, uint32_t rnd) {
  const uint32_t bits = __float_as_uint(y), mag = bits & 0x7fffffffu;
  const uint32_t normal = ((mag + rnd) >> 20) - 960u;
  const float small = floorf(__fadd_rn(fabsf(y) * 512.f, (float)rnd * 0x1p-20f));
  uint32_t code = mag >= 0x3c800000u ? normal : (uint32_t)small;
  if (LEAST && mag != 0) code = code > 1u ? code : 1u;
  code = mag < 0x7f800000u ? code : 127u;
  return code | ((bits >> 24) & 0x80u);
}

// Eight consecutive elements; a partial or unaligned block goes one at a time.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float* f) {
  if (vec) {
    Chunk<T>::unpack(*(const uint4*)p, f);
    if constexpr (Chunk<T>::N == 4) Chunk<T>::unpack(*(const uint4*)(p + 4), f + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? Elt<T>::ld(p + i) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float* f) {
  if (vec) {
    *(uint4*)p = Chunk<T>::pack(f);
    if constexpr (Chunk<T>::N == 4) *(uint4*)(p + 4) = Chunk<T>::pack(f + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) Elt<T>::st(p + i, f[i]);
  }
}

__device__ __forceinline__ void load_q(const uint8_t* q, const uint8_t* s, int64_t blk, int n,
                                       bool vec, float* f) {
  uint32_t w[2] = {0, 0};
  if (vec) {
    const uint2 v = *(const uint2*)q;
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 2] |= (uint32_t)q[i] << (8 * (i & 3));
  }
  const float scale = fp8_scale_value(n > 0 ? s[blk] : 127);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f[4 * h + 0] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 0) * scale;
    f[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 1) * scale;
    f[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 2) * scale;
    f[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 3) * scale;
  }
}
// f: zero past the block's end
template <bool LEAST>
__device__ __forceinline__ void store_q(uint8_t* q, uint8_t* s, int64_t blk, int n, bool vec,
                                        bool first, const float* f, const uint32_t* rnd) {
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, finite_abs(f[i]));
  const int byte = fp8_scale_byte(lanes_max<16>(mx));
  const float inv = fp8_inv_scale(byte);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= round_fp8<LEAST>(f[i] * inv, rnd[i]) << (8 * (i & 3));
  if (vec) {
    *(uint2*)q = uint2{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if (first && n > 0) s[blk] = (uint8_t)byte;
}

template <typename P>
__device__ __forceinline__ void update(const Args& a, const Tensor& t, int64_t e0, int lane16) {
  // every product and sum is rounded by itself (no fused multiply-add), so a
  // result depends on the formula alone
#pragma clang fp contract(off)
  const int64_t left = t.n - e0;
  const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  const bool vec = (t.flags & kVec) && n == 8;
  const bool q8 = t.flags & kState8;  // block-uniform
  const int64_t blk = e0 >> 7;
  P* param = (P*)t.param + e0;
  float g[8], m[8], v[8], p[8];
  load8(t.grad + e0, n, vec, g);
  if (t.master) load8(t.master + e0, n, vec, p);
  else load8(param, n, vec, p);
  if (q8) {
    load_q((uint8_t*)t.m + e0, t.m_s, blk, n, vec, m);
    load_q((uint8_t*)t.v + e0, t.v_s, blk, n, vec, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
  } else {
    load8((float*)t.m + e0, n, vec, m);
    load8((float*)t.v + e0, n, vec, v);
  }
  const float dev = a.scale_dev ? *a.scale_dev : 1.f;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float gi = g[i] * a.scale;
    gi = gi * dev;
    const float m0 = m[i] * a.b1, m1 = gi * a.a1;
    m[i] = m0 + m1;
    const float gg = gi * gi;
    const float v0 = v[i] * a.b2, v1 = gg * a.a2;
    v[i] = v0 + v1;
    r[i] = sqrtf(v[i]);
    const float den = r[i] * a.root;
    const float stp = m[i] * a.rate / (den + a.eps);
    const float kept = p[i] * t.keep;
    p[i] = kept - stp;
  }
  if (t.master) store8(t.master + e0, n, vec, p);
  store8(param, n, vec, p);
  if (q8) {
    uint32_t rm[8], rv[8];
    const uint32_t key = t.key ^ ((uint32_t)(e0 >> 32) * 0x85EBCA77u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = mix(((uint32_t)e0 + i) ^ key);
      rm[i] = x >> 12;
      rv[i] = (x * 0x9E3779B1u) >> 12;
      if (i >= n) m[i] = r[i] = 0.f;
    }
    store_q<false>((uint8_t*)t.m + e0, t.m_s, blk, n, vec, lane16 == 0, m, rm);
    store_q<true>((uint8_t*)t.v + e0, t.v_s, blk, n, vec, lane16 == 0, r, rv);
  } else {
    store8((float*)t.m + e0, n, vec, m);
    store8((float*)t.v + e0, n, vec, v);
  }
}

__global__ __launch_bounds__(256) void adamw_kernel(Args a) {
  const int b = blockIdx.x;
  int lo = 0, hi = a.n;  // start[lo] <= b < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.start[mid] <= b) lo = mid;
    else hi = mid;
  }
  const Tensor& t = a.t[lo];
  const int64_t e0 = (int64_t)(b - a.start[lo]) * kChunk + threadIdx.x * 8;
  const int l = threadIdx.x & 15;
  if (t.dtype == MOE_BF16) update<uint16_t>(a, t, e0, l);
  else if (t.dtype == MOE_F16) update<_Float16>(a, t, e0, l);
  else update<float>(a, t, e0, l);
}

}  // namespace

int launch_adamw(const moe_adamw_tensor* t, int n, const moe_adamw_hyper* hp, hipStream_t st) {
  Args a;
  const double c1 = 1.0 - pow(hp->beta1, (double)hp->step);
  const double c2 = 1.0 - pow(hp->beta2, (double)hp->step);
  a.b1 = (float)hp->beta1;
  a.a1 = (float)(1.0 - hp->beta1);
  a.b2 = (float)hp->beta2;
  a.a2 = (float)(1.0 - hp->beta2);
  a.rate = (float)(hp->lr / c1);
  a.root = (float)(1.0 / sqrt(c2));
  a.eps = (float)hp->eps;
  a.scale = hp->grad_scale;
  a.scale_dev = hp->grad_scale_dev;
  const uint32_t key = (uint32_t)hp->seed ^ ((uint32_t)(hp->seed >> 32) * 0x85EBCA77u) ^
                       ((uint32_t)hp->step * 0x9E3779B1u);
  for (int i = 0; i < n;) {
    a.n = 0;
    a.start[0] = 0;
    for (; i < n && a.n < kMax; ++i) {
      const moe_adamw_tensor& x = t[i];
      if (x.n == 0) continue;
      const int64_t blocks = cdiv(x.n, kChunk);
      if (a.n > 0 && a.start[a.n] + blocks > kBlocks) break;
      uintptr_t bits = (uintptr_t)x.param | (uintptr_t)x.master | (uintptr_t)x.grad;
      bits |= x.state8 ? ((uintptr_t)x.m | (uintptr_t)x.v) << 1 : (uintptr_t)x.m | (uintptr_t)x.v;
      a.t[a.n] = {x.param, x.master, x.grad, x.m, x.v, x.m_s, x.v_s, x.n,
                  (float)(1.0 - hp->lr * x.weight_decay), key ^ ((uint32_t)i * 0xC2B2AE3Du),
                  x.dtype, (x.state8 ? kState8 : 0) | (bits % 16 ? 0 : kVec)};
      a.start[a.n + 1] = a.start[a.n] + (int32_t)blocks;
      ++a.n;
    }
    if (a.n == 0) break;
    MOE_LAUNCH("adamw", st, adamw_kernel<<<a.start[a.n], 256, 0, st>>>(a));
    if (int rc = check_launch("adamw")) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
