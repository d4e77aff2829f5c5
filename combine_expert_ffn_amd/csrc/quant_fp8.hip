// Block quantisation to e4m3 with power-of-two scales (the format is in moe.h):
// activation rows in blocks of 1 x 128, expert weights in blocks of 128 x 128.
// Both are one pass over memory: every value is read once into registers, the
// block's largest magnitude is formed there, and the bytes are written.  Bound by
// memory: 65536 x 2048 bf16 rows 71 us (405 MB, 5.7 TB/s); 128 experts of 2048 x 768 with
// their transposed copies 463 us (2.4 GB, 5.2 TB/s).  33 rows take one launch, 2.5 us
// (6.1 with the call).
#include "moe_fp8.h"

namespace moe {
namespace {

// Eight consecutive elements as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  Chunk<T>::unpack(*(const uint4*)p, f);
  if constexpr (Chunk<T>::N == 4) Chunk<T>::unpack(*(const uint4*)(p + 4), f + 4);
}

__device__ __forceinline__ float amax8(const float* f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(f[i]));
  return m;
}

__device__ __forceinline__ uint2 quant8(const float* f, float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = finite_or_nan(f[i]) * inv;
  return uint2{pack_fp8(y[0], y[1], y[2], y[3]), pack_fp8(y[4], y[5], y[6], y[7])};
}

// Rows: 16 lanes hold one block of 128, eight values each, so a wave reads and
// writes whole 128-byte lines.
template <typename T>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ src, int64_t rows,
                                                         const int32_t* __restrict__ n_rows,
                                                         int kb, int ld, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ qs) {
  int64_t n = rows;
  if (n_rows) n = min(n, (int64_t)max(*n_rows, 0));
  const int64_t blocks = n * kb;
  const int grp = threadIdx.x >> 4, l = threadIdx.x & 15;
  for (int64_t b = (int64_t)blockIdx.x * 16 + grp; b < blocks; b += (int64_t)gridDim.x * 16) {
    float f[8];
    load8(src + b * 128 + l * 8, f);
    const int byte = fp8_scale_byte(lanes_max<16>(amax8(f)));
    *(uint2*)(q + b * 128 + l * 8) = quant8(f, fp8_inv_scale(byte));
    const int64_t row = b / kb;
    const int k = (int)(b - row * kb);
    // lane 0 writes the scale; behind a row's last block the padding follows
    const int last = k == kb - 1 ? ld - kb : 0;
    if (l <= last) qs[row * ld + k + l] = l == 0 ? (uint8_t)byte : (uint8_t)0;
  }
}

// Four rows of four bytes -> four columns.
__device__ __forceinline__ void transpose4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3,
                                           uint32_t* c) {
  const uint32_t x0 = __builtin_amdgcn_perm(r1, r0, 0x05010400u);
  const uint32_t x1 = __builtin_amdgcn_perm(r1, r0, 0x07030602u);
  const uint32_t y0 = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
  const uint32_t y1 = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
  c[0] = __builtin_amdgcn_perm(y0, x0, 0x05040100u);
  c[1] = __builtin_amdgcn_perm(y0, x0, 0x07060302u);
  c[2] = __builtin_amdgcn_perm(y1, x1, 0x05040100u);
  c[3] = __builtin_amdgcn_perm(y1, x1, 0x07060302u);
}

// One matrix of the weights: [E_l][n][k] in blocks of 128 x 128.
struct WMat {
  const void* src;
  uint8_t *q, *s, *qT, *sT;  // qT and sT NULL: no transposed copy
  int nb, kb, ld, ldT;       // blocks along n and k; scale row bytes
};

// A workgroup takes one 128 x 128 block, a thread 8 rows x 8 columns of it in
// registers.  The transposed block goes through LDS: thread (row group g, column
// group c) writes the eight bytes of column 8c + i at 8-byte slot g ^ c of LDS
// row 8c + i (so the 16 column groups of a wave instruction fall on different
// banks), and 16 lanes read a whole row back.
template <typename T>
__global__ __launch_bounds__(256) void quant_weights_kernel(WMat m0, WMat m1, int first) {
  __shared__ uint2 tile[128][16];
  __shared__ float wave_max[4];
  const bool second = (int)blockIdx.x >= first;  // block-uniform
  const WMat m = second ? m1 : m0;
  int b = (int)blockIdx.x - (second ? first : 0);
  const int kb = b % m.kb;
  b /= m.kb;
  const int nb = b % m.nb, e = b / m.nb;
  const int K = m.kb * 128, N = m.nb * 128;
  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4;
  const size_t mat = (size_t)e * N * K;
  const T* src = (const T*)m.src + mat + (size_t)(nb * 128 + g * 8) * K + kb * 128 + c * 8;
  float f[8][8];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) load8(src + (size_t)i * K, f[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, amax8(f[i]));
  mx = lanes_max<16>(mx);
  mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  if ((tid & 63) == 0) wave_max[tid >> 6] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
  const int byte = fp8_scale_byte(mx);
  const float inv = fp8_inv_scale(byte);
  uint8_t* q = m.q + mat + (size_t)(nb * 128 + g * 8) * K + kb * 128 + c * 8;
  uint2 r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = quant8(f[i], inv);
    *(uint2*)(q + (size_t)i * K) = r[i];
  }
  const int pad = kb == m.kb - 1 ? m.ld - m.kb : 0;
  if (tid <= pad) m.s[((size_t)e * m.nb + nb) * m.ld + kb + tid] = tid == 0 ? (uint8_t)byte : 0;
  if (!m.qT) return;  // block-uniform
  uint32_t lo[8], hi[8];  // columns 0..7: rows 0..3, rows 4..7
  transpose4(r[0].x, r[1].x, r[2].x, r[3].x, lo);
  transpose4(r[0].y, r[1].y, r[2].y, r[3].y, lo + 4);
  transpose4(r[4].x, r[5].x, r[6].x, r[7].x, hi);
  transpose4(r[4].y, r[5].y, r[6].y, r[7].y, hi + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) tile[c * 8 + i][g ^ c] = uint2{lo[i], hi[i]};
  __syncthreads();
  uint8_t* qT = m.qT + mat + (size_t)(kb * 128) * N + nb * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = i * 16 + g;  // LDS row = column of the block
    *(uint2*)(qT + (size_t)col * N + c * 8) = tile[col][c ^ (col >> 3)];
  }
  const int padT = nb == m.nb - 1 ? m.ldT - m.nb : 0;
  if (tid <= padT)
    m.sT[((size_t)e * m.kb + kb) * m.ldT + nb + tid] = tid == 0 ? (uint8_t)byte : 0;
}

template <typename T>
int quant_rows_t(const moe_shape* s, const void* src, int64_t rows, const int32_t* n_rows,
                 void* q, uint8_t* qs, hipStream_t st) {
  const int kb = (int)(s->d / 128);
  const int64_t want = cdiv(rows * kb, 16);
  const int grid = (int)(want < 16384 ? want : 16384);
  MOE_LAUNCH("quant_rows", st,
             quant_rows_kernel<T><<<grid, 256, 0, st>>>((const T*)src, rows, n_rows, kb,
                                                        (int)fp8_scale_ld(s->d), (uint8_t*)q, qs));
  return check_launch("quant_rows");
}

template <typename T>
int quant_weights_t(const moe_shape* s, const void* W_gu, const void* W_down,
                    const moe_fp8_weights* w, hipStream_t st) {
  const int db = (int)(s->d / 128), fb = (int)(s->F / 128);
  const int ld_d = (int)fp8_scale_ld(s->d), ld_f = (int)fp8_scale_ld(s->F),
            ld_2f = (int)fp8_scale_ld(2 * s->F);
  const WMat gu{W_gu, (uint8_t*)w->gu, w->gu_s, (uint8_t*)w->guT, w->guT_s, 2 * fb, db, ld_d,
                ld_2f};
  const WMat dn{W_down, (uint8_t*)w->down, w->down_s, (uint8_t*)w->downT, w->downT_s, db, fb,
                ld_f, ld_d};
  const int first = (int)s->E_l * 2 * fb * db, total = first + (int)s->E_l * fb * db;
  MOE_LAUNCH("quant_weights", st,
             quant_weights_kernel<T><<<total, 256, 0, st>>>(gu, dn, first));
  return check_launch("quant_weights");
}

}  // namespace

int launch_quant_rows(const moe_shape* s, const void* src, int64_t rows, const int32_t* n_rows,
                      void* q, uint8_t* qs, hipStream_t st) {
  if (s->dtype == MOE_BF16) return quant_rows_t<uint16_t>(s, src, rows, n_rows, q, qs, st);
  if (s->dtype == MOE_F16) return quant_rows_t<_Float16>(s, src, rows, n_rows, q, qs, st);
  return quant_rows_t<float>(s, src, rows, n_rows, q, qs, st);
}

int launch_quant_weights(const moe_shape* s, const void* W_gu, const void* W_down,
                         const moe_fp8_weights* w, hipStream_t st) {
  if (s->dtype == MOE_BF16) return quant_weights_t<uint16_t>(s, W_gu, W_down, w, st);
  if (s->dtype == MOE_F16) return quant_weights_t<_Float16>(s, W_gu, W_down, w, st);
  return quant_weights_t<float>(s, W_gu, W_down, w, st);
}

}  // namespace moe
