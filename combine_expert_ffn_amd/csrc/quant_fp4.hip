// The experts' weights to 4 bits and back (the format is in moe.h).  Rows are whole
// blocks and neither codes nor scales are padded, so a matrix is one flat list of
// blocks of 32: a thread holds eight consecutive values (16 bytes in 16 bits, a
// register of codes), four threads a block.  Bound by memory: 128 experts of 2048 x 768
// bf16 (1.53 GB) quantised in 239 us (6.4 TB/s), read back in 252 (6.1); 267 and 272 with four
// groups to a thread and through the caches.
#include "moe_fp4.h"

namespace moe {
namespace {

constexpr int NT = 256;
constexpr int U = 2;                // groups of eight values per thread
constexpr int CHUNK = NT * 8 * U;   // values per step of a block; divides 128 x 128

// Both matrices as one list of chunks: the first `first` chunks are W_gu's.
template <typename T>
struct Mats {
  T* w[2];
  uint8_t *q[2], *s[2];
  int64_t first, total;
};

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
}

template <typename T, bool PAST>
__global__ __launch_bounds__(NT) void quant_weights_fp4_kernel(Mats<T> m) {
  for (int64_t c = blockIdx.x; c < m.total; c += gridDim.x) {  // block-uniform
    const int i = c >= m.first;
    const int64_t g0 = (c - (i ? m.first : 0)) * (CHUNK / 8) + threadIdx.x;  // group of eight
    uint4 raw[U][sizeof(T) / 2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < (int)sizeof(T) / 2; ++p)
        raw[u][p] = __builtin_bit_cast(
            uint4, Words<4, PAST>::load((const uint4*)(m.w[i] + (g0 + u * NT) * 8) + p));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
#pragma unroll
      for (int p = 0; p < (int)sizeof(T) / 2; ++p)
        Chunk<T>::unpack(raw[u][p], f + p * Chunk<T>::N);
      uint32_t mx = 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) mx = max(mx, __float_as_uint(f[t]) & 0x7fffffffu);
      const int byte = fp4_scale_byte(quad_max(mx));
      const float scale = fp8_scale_value(byte);
      uint32_t v = 0;
      v = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[0], f[1], scale, 0);
      v = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[2], f[3], scale, 1);
      v = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[4], f[5], scale, 2);
      v = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[6], f[7], scale, 3);
      const int64_t g = g0 + u * NT;
      Words<1, PAST>::store(m.q[i] + g * 4, byte == 255 ? 0u : v);
      if ((threadIdx.x & 3) == 0) m.s[i][g >> 2] = (uint8_t)byte;
    }
  }
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

template <typename T, bool PAST>
__global__ __launch_bounds__(NT) void dequant_weights_fp4_kernel(Mats<T> m) {
  for (int64_t c = blockIdx.x; c < m.total; c += gridDim.x) {  // block-uniform
    const int i = c >= m.first;
    const int64_t g0 = (c - (i ? m.first : 0)) * (CHUNK / 8) + threadIdx.x;
    uint32_t v[U];
    int byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = *(const uint32_t*)(m.q[i] + (g0 + u * NT) * 4);
      byte[u] = m.s[i][(g0 + u * NT) >> 2];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float scale = fp8_scale_value(byte[u]);
      float f[8];
      const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], scale, 0);
      const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], scale, 1);
      const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], scale, 2);
      const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], scale, 3);
      f[0] = a[0]; f[1] = a[1]; f[2] = b[0]; f[3] = b[1];
      f[4] = d[0]; f[5] = d[1]; f[6] = e[0]; f[7] = e[1];
#pragma unroll
      for (int p = 0; p < (int)sizeof(T) / 2; ++p)
        Words<4, PAST>::store((uint4*)(m.w[i] + (g0 + u * NT) * 8) + p,
                              __builtin_bit_cast(typename Words<4, PAST>::type,
                                                 Chunk<T>::pack(f + p * Chunk<T>::N)));
    }
  }
}

template <typename T>
Mats<T> mats(const moe_shape* s, const void* W_gu, const void* W_down, const moe_fp4_weights* w) {
  const int64_t n = s->E_l * s->F * s->d;  // a multiple of 128 x 128
  return {{(T*)W_gu, (T*)W_down}, {w->gu, w->down}, {w->gu_s, w->down_s}, 2 * n / CHUNK,
          3 * n / CHUNK};
}
template <typename T>
int grid_of(const Mats<T>& m) {
  return (int)(m.total < (1 << 20) ? m.total : (1 << 20));
}
template <typename T>
bool past_caches(const Mats<T>& m) {
  return m.total * CHUNK * (int64_t)sizeof(T) >= kPastCaches;
}
template <typename T>
int quant_t(const Mats<T>& m, hipStream_t st) {
  auto go = [&](auto kernel) {
    MOE_LAUNCH("quant_weights_fp4", st, kernel<<<grid_of(m), NT, 0, st>>>(m));
    return check_launch("quant_weights_fp4");
  };
  return past_caches(m) ? go(quant_weights_fp4_kernel<T, true>)
                        : go(quant_weights_fp4_kernel<T, false>);
}
template <typename T>
int dequant_t(const Mats<T>& m, hipStream_t st) {
  auto go = [&](auto kernel) {
    MOE_LAUNCH("dequant_weights_fp4", st, kernel<<<grid_of(m), NT, 0, st>>>(m));
    return check_launch("dequant_weights_fp4");
  };
  return past_caches(m) ? go(dequant_weights_fp4_kernel<T, true>)
                        : go(dequant_weights_fp4_kernel<T, false>);
}

}  // namespace

int launch_quant_weights_fp4(const moe_shape* s, const void* W_gu, const void* W_down,
                             const moe_fp4_weights* w, hipStream_t st) {
  if (s->dtype == MOE_BF16) return quant_t(mats<uint16_t>(s, W_gu, W_down, w), st);
  if (s->dtype == MOE_F16) return quant_t(mats<_Float16>(s, W_gu, W_down, w), st);
  return quant_t(mats<float>(s, W_gu, W_down, w), st);
}

int launch_dequant_weights_fp4(const moe_shape* s, const moe_fp4_weights* w, void* W_gu,
                               void* W_down, hipStream_t st) {
  if (s->dtype == MOE_BF16) return dequant_t(mats<uint16_t>(s, W_gu, W_down, w), st);
  if (s->dtype == MOE_F16) return dequant_t(mats<_Float16>(s, W_gu, W_down, w), st);
  return dequant_t(mats<float>(s, W_gu, W_down, w), st);
}

}  // namespace moe
