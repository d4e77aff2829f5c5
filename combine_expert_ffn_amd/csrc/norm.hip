// Root-mean-square norm of token rows, with the residual's addition before it and
// the 8-bit rows behind it, and its backward pass (formulas in moe.h).
// Both are one pass over memory, which bounds them: 65536 x 2048 bf16 forward with
// residual, y and 8-bit rows 203 us (1.21 GB, 6.0 TB/s; 222 through the caches and with
// 2048 blocks), backward with the residual's gradient 183 us (1.07 GB, 5.9 TB/s; 202).  Not
// the backward of rows of more than 8192: a lane's eight chunks of dy, r, dres, gamma and
// dgamma leave one wave to a SIMD, so a row's loads, sum and stores follow each other: 8192 x
// 16384 bf16 235 us (3.4 TB/s), where as many values in rows of 2048 take 141.  A
// row is held in the registers of 16, 64 or 256 lanes (d up to 512, 2048, 16384), eight
// consecutive elements of a lane to a 16-byte load, so the sum of squares needs no
// second read, and 16 lanes hold a scale block of 128.  Sums are float32: a lane's own,
// then over the lanes in a fixed order.  Which products are fused into a sum is written out, so
// that a row's bits are the same in every kernel (the compiler chose otherwise in some).
// dgamma is a sum over all rows: a block keeps its columns' sums in registers while
// it walks its rows, writes one row of them, and a second launch adds those rows in
// a fixed order.  For few rows dgamma's columns are summed by further blocks of the same
// launch, which read dy and r again.
#include "moe_fp8.h"
#include "moe_norm.h"

namespace moe {
namespace {

constexpr int NT = 256;
// Rows up to which dgamma is summed from a second reading of dy and r: in us, dx and
// dgamma together in a graph, bf16, this way against partial sums: 333 x 640 3.8 / 5.4 (called one
// by one 6.6 / 9.1), 700 x 2048 4.9 / 7.4, 1024 x 640 5.5 / 5.8, 1024 x 4096 11.7 / 14.4, 1024 x
// 16384 43 / 38; 1500 x 640 6.7 / 6.3, 1500 x 2048 10.6 / 9.6, 2048 x 4096 25 / 19.
constexpr int64_t kFewRows = 1024;

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int N = (int)sizeof(T) * 8 / 16;
  uint4 v[N];
  template <bool PAST = false>
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = __builtin_bit_cast(uint4, Words<4, PAST>::load((const uint4*)p + i));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = uint4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
    for (int i = 0; i < N; ++i) Chunk<T>::unpack(v[i], f + i * Chunk<T>::N);
  }
  __device__ __forceinline__ void pack(const float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Chunk<T>::pack(f + i * Chunk<T>::N);
  }
  template <bool PAST>
  __device__ __forceinline__ void store(T* p) const {
    typedef Words<4, PAST> W;
#pragma unroll
    for (int i = 0; i < N; ++i)
      W::store((uint4*)p + i, __builtin_bit_cast(typename W::type, v[i]));
  }
};

// Sum over the L lanes of a row, in each of them.  With 256 lanes through LDS: s
// has two halves used in turn, so one barrier per row is enough.
template <int L>
__device__ __forceinline__ float row_sum(float v, float (&s)[2][NT / 64], int turn) {
#pragma unroll
  for (int o = 1; o < (L < 64 ? L : 64); o <<= 1) v += __shfl_xor(v, o, 64);
  if constexpr (L == 256) {
    float* p = s[turn & 1];
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (p[0] + p[1]) + (p[2] + p[3]);
  }
  return v;
}

template <typename T>
struct Fwd {
  const T *x, *res, *gamma;
  T *r, *y;
  uint8_t *q, *qs;
  float* rstd;
  float eps;
  int64_t rows;
  int d, ld;  // ld: scale bytes per row
};

// L lanes to a row, C chunks of eight elements to a lane (chunk c L + lane).
template <typename T, int L, int C, bool PAST>
__global__ __launch_bounds__(NT) void rmsnorm_kernel(Fwd<T> a) {
  __shared__ float s_sum[2][NT / 64];
  const int lane = threadIdx.x & (L - 1), chunks = a.d >> 3;
  const int64_t step = (int64_t)gridDim.x * (NT / L);
  const int64_t first = (int64_t)blockIdx.x * (NT / L);
  Raw8<T> gamma[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    gamma[c].zero();
    if (c * L + lane < chunks) gamma[c].load(a.gamma + (c * L + lane) * 8);
  }
  int turn = 0;
  for (int64_t row0 = first; row0 < a.rows; row0 += step, ++turn) {  // block-uniform
    const int64_t row = row0 + threadIdx.x / L;
    const bool on = row < a.rows;
    const int64_t at = row * a.d;
    Raw8<T> xr[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      xr[c].zero();
      if (on && c * L + lane < chunks) xr[c].template load<PAST>(a.x + at + (c * L + lane) * 8);
    }
    if (a.res) {  // the sum is rounded as it is stored; the norm is of the stored sum
#pragma unroll
      for (int c = 0; c < C; ++c) {
        rr[c].zero();
        if (on && c * L + lane < chunks) rr[c].template load<PAST>(a.res + at + (c * L + lane) * 8);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[8], g[8];
        xr[c].unpack(f);
        rr[c].unpack(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        xr[c].pack(f);
        if (a.r && on && c * L + lane < chunks)
          xr[c].template store<PAST>(a.r + at + (c * L + lane) * 8);
      }
    }
    auto squares = [&](float unit) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[8];
        xr[c].unpack(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[i] * unit, f[i] * unit, sum);
      }
      return sum;
    };
    // Where the sum, or the mean with eps, passes float32's range (values of 1e17 and more)
    // the row is taken in units of 2^80, eps with it (in two steps: 2^-160 is no float32).
    float unit = 1.f, mean = row_sum<L>(squares(1.f), s_sum, turn) / (float)a.d + a.eps;
    if (mean == __builtin_inff()) {  // the same for all lanes of the row
      unit = 0x1p-80f;
      if constexpr (L == 256) ++turn;
      mean = row_sum<L>(squares(unit), s_sum, turn) / (float)a.d + a.eps * unit * unit;
    }
    const float root = 1.0f / sqrtf(mean);
    const float rstd = root * unit;
    if (a.rstd && on && lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = c * L + lane;
      const bool ok = on && k < chunks;
      float f[8], g[8];
      xr[c].unpack(f);
      gamma[c].unpack(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = (f[i] * unit) * root * g[i];
      Raw8<T> y;
      y.pack(f);
      if (a.y && ok) y.template store<PAST>(a.y + at + k * 8);
      if (a.q) {  // of the rounded y, as moe_quant_rows_fp8 gives it
        y.unpack(f);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(f[i]));
        const int byte = fp8_scale_byte(lanes_max<16>(m));
        const float inv = fp8_inv_scale(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = finite_or_nan(f[i]) * inv;
        if (ok) {
          Words<2, PAST>::store(a.q + at + k * 8, {pack_fp8(f[0], f[1], f[2], f[3]),
                                                   pack_fp8(f[4], f[5], f[6], f[7])});
          // the first lane of a block writes its scale; behind the last the padding follows
          const int b = k >> 4, kb = chunks >> 4, l = k & 15;
          if (l <= (b == kb - 1 ? a.ld - kb : 0))
            a.qs[row * a.ld + b + l] = l == 0 ? (uint8_t)byte : (uint8_t)0;
        }
      }
    }
  }
}

template <typename T>
struct Bwd {
  const T *dy, *r, *gamma;
  const float* rstd;
  const T* dres;
  T* dx;
  float* parts;  // [gridDim.x][d], or dgamma itself with one block; NULL: not formed
  bool accumulate;  // with one block
  int64_t rows;
  int d;
  float* dgamma;  // FEW: the blocks behind the first row_blocks sum its columns
  int row_blocks;
};

// 32 columns of dgamma over all rows: four lanes to a row, 64 rows at a time, four in
// flight; then the lanes of a wave and the waves.
template <typename T>
__device__ __forceinline__ void sum_columns(const Bwd<T>& a, int block) {
  __shared__ float s[NT / 64][32];
  const int part = threadIdx.x & 3, col = block * 32 + part * 8;
  float acc[8] = {};
  for (int64_t t0 = threadIdx.x >> 2; t0 < a.rows; t0 += 4 * (NT / 4)) {
    Raw8<T> dy[4], r[4];
    float rstd[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t t = t0 + u * (NT / 4);
      dy[u].zero();
      r[u].zero();
      rstd[u] = 0.f;
      if (t < a.rows) {
        dy[u].load(a.dy + t * a.d + col);
        r[u].load(a.r + t * a.d + col);
        rstd[u] = a.rstd[t];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[8], x[8];
      dy[u].unpack(f);
      r[u].unpack(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f[i], x[i] * rstd[u], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = acc[i];
#pragma unroll
    for (int o = 4; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) < 4) s[threadIdx.x >> 6][part * 8 + i] = v;
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (j < 32) {
    const float v = (s[0][j] + s[1][j]) + (s[2][j] + s[3][j]);
    float* p = a.dgamma + block * 32 + j;
    *p = a.accumulate ? *p + v : v;
  }
}

template <typename T, int L, int C, bool PAST, bool FEW>
__global__ __launch_bounds__(NT) void rmsnorm_bwd_kernel(Bwd<T> a) {
  if constexpr (FEW)
    if ((int)blockIdx.x >= a.row_blocks) return sum_columns(a, (int)blockIdx.x - a.row_blocks);
  __shared__ float s_sum[2][NT / 64];
  __shared__ float s_part[L == 256 || FEW ? 1 : NT / 64][L == 256 || FEW ? 1 : C * L * 8];
  const int lane = threadIdx.x & (L - 1), chunks = a.d >> 3;
  const int64_t step = (int64_t)(FEW ? a.row_blocks : gridDim.x) * (NT / L);
  const int64_t first = (int64_t)blockIdx.x * (NT / L);
  Raw8<T> gamma[C];
  float acc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    gamma[c].zero();
    if (c * L + lane < chunks) gamma[c].load(a.gamma + (c * L + lane) * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.f;
  }
  int turn = 0;
  for (int64_t row0 = first; row0 < a.rows; row0 += step, ++turn) {  // block-uniform
    const int64_t row = row0 + threadIdx.x / L;
    const bool on = row < a.rows;
    const int64_t at = row * a.d;
    const float rstd = on ? a.rstd[row] : 0.f;
    Raw8<T> dy[C], r[C], dres[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      dy[c].zero();
      r[c].zero();
      dres[c].zero();
      if (on && c * L + lane < chunks) {
        dy[c].template load<PAST>(a.dy + at + (c * L + lane) * 8);
        r[c].template load<PAST>(a.r + at + (c * L + lane) * 8);
        if (a.dres) dres[c].template load<PAST>(a.dres + at + (c * L + lane) * 8);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], x[8], g[8];
      dy[c].unpack(f);
      r[c].unpack(x);
      gamma[c].unpack(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = x[i] * rstd;
        sum = fmaf(f[i] * g[i], xhat, sum);
        acc[c][i] = fmaf(f[i], xhat, acc[c][i]);
      }
    }
    const float mean = row_sum<L>(sum, s_sum, turn) / (float)a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], x[8], g[8], e[8];
      dy[c].unpack(f);
      r[c].unpack(x);
      gamma[c].unpack(g);
      dres[c].unpack(e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[i] = fmaf(rstd, fmaf(-(x[i] * rstd), mean, f[i] * g[i]), e[i]);
      Raw8<T> o;
      o.pack(f);
      if (on && c * L + lane < chunks) o.template store<PAST>(a.dx + at + (c * L + lane) * 8);
    }
  }
  if (FEW || !a.parts) return;  // block-uniform
  float* out = a.parts + (size_t)blockIdx.x * a.d;
  auto put = [&](float* p, float v) { *p = a.accumulate ? *p + v : v; };
  if constexpr (L == 256) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * L + lane < chunks)
#pragma unroll
        for (int i = 0; i < 8; ++i) put(out + (c * L + lane) * 8 + i, acc[c][i]);
  } else {
    // a wave's rows, then the waves
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = acc[c][i];
#pragma unroll
        for (int o = L; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
        if ((threadIdx.x & 63) < L) s_part[wave][(c * L + lane) * 8 + i] = v;
      }
    __syncthreads();
    for (int j = threadIdx.x; j < a.d; j += NT)
      put(out + j, (s_part[0][j] + s_part[1][j]) + (s_part[2][j] + s_part[3][j]));
  }
}

// dgamma from n rows of partial sums: 16 columns to a block, 64 threads to a column, each
// with eight rows in flight.
__global__ __launch_bounds__(1024) void rmsnorm_dgamma_kernel(const float* __restrict__ parts,
                                                              int n, int d, bool accumulate,
                                                              float* __restrict__ dgamma) {
  __shared__ float s[16][16];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, j = blockIdx.x * 16 + col;
  float v = 0.f;
  for (int i = grp; i < n; i += 512) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k * 64 < n ? parts[(size_t)(i + k * 64) * d + j] : 0.f;
    v += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
  }
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if ((threadIdx.x & 63) < 16) s[threadIdx.x >> 6][col] = v;
  __syncthreads();
  if (threadIdx.x < 16) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][col];
    dgamma[j] = accumulate ? dgamma[j] + t : t;
  }
}

// Calls go.template operator()<L, C>() with the row layout for width d.
template <class Go>
int with_layout(int64_t d, Go go) {
  const int L = norm_lanes(d);
  const int64_t c = cdiv(d, 8 * L);
  if (L == 16) return c <= 1 ? go.template operator()<16, 1>()
                             : (c <= 2 ? go.template operator()<16, 2>()
                                       : go.template operator()<16, 4>());
  if (L == 64) return c <= 2 ? go.template operator()<64, 2>() : go.template operator()<64, 4>();
  return c <= 2 ? go.template operator()<256, 2>()
                : (c <= 4 ? go.template operator()<256, 4>() : go.template operator()<256, 8>());
}

template <typename T>
struct GoFwd {
  Fwd<T> a;
  bool past;
  hipStream_t st;
  template <int L, int C>
  int operator()() const {
    const int64_t want = cdiv(a.rows, NT / L);
    const int grid = (int)(want < 16384 ? want : 16384);
    if (past)
      MOE_LAUNCH("rmsnorm", st, rmsnorm_kernel<T, L, C, true><<<grid, NT, 0, st>>>(a));
    else
      MOE_LAUNCH("rmsnorm", st, rmsnorm_kernel<T, L, C, false><<<grid, NT, 0, st>>>(a));
    return check_launch("rmsnorm");
  }
};
template <typename T>
struct GoBwd {
  Bwd<T> a;
  int grid;
  bool past, few;
  hipStream_t st;
  template <int L, int C>
  int operator()() const {
    auto go = [&](auto kernel) {
      MOE_LAUNCH("rmsnorm_bwd", st, kernel<<<grid, NT, 0, st>>>(a));
      return check_launch("rmsnorm_bwd");
    };
    if (few) return go(rmsnorm_bwd_kernel<T, L, C, false, true>);
    return past ? go(rmsnorm_bwd_kernel<T, L, C, true, false>)
                : go(rmsnorm_bwd_kernel<T, L, C, false, false>);
  }
};

template <typename T>
bool past_caches(const moe_shape* s) {
  return s->T * s->d * (int64_t)sizeof(T) >= kPastCaches;
}

template <typename T>
int rmsnorm_t(const moe_shape* s, const void* x, const void* res, const void* gamma, float eps,
              void* r, void* y, void* q, uint8_t* qs, float* rstd, hipStream_t st) {
  return with_layout(s->d, GoFwd<T>{{(const T*)x, (const T*)res, (const T*)gamma, (T*)r, (T*)y,
                                     (uint8_t*)q, qs, rstd, eps, s->T, (int)s->d,
                                     (int)fp8_scale_ld(s->d)}, past_caches<T>(s), st});
}

template <typename T>
int rmsnorm_bwd_t(const moe_shape* s, const void* dy, const void* r, const void* gamma,
                  const float* rstd, const void* dres, void* dx, float* dgamma, bool accumulate,
                  float* parts, hipStream_t st) {
  const int n = (int)norm_parts(s->T, s->d);
  const Bwd<T> a{(const T*)dy, (const T*)r, (const T*)gamma, rstd, (const T*)dres, (T*)dx, nullptr,
                 accumulate, s->T, (int)s->d, dgamma, (int)cdiv(s->T, NT / norm_lanes(s->d))};
  // the columns' blocks read dy and r beside blocks that write dx
  if (dgamma && n > 1 && s->T <= kFewRows && dx != dy && dx != r)
    return with_layout(s->d, GoBwd<T>{a, a.row_blocks + (int)(s->d / 32), false, true, st});
  if (n > 0) {
    const bool direct = n == 1;  // one block adds to dgamma itself
    float* p = !dgamma ? nullptr : (direct ? dgamma : parts);
    Bwd<T> b = a;
    b.parts = p;
    b.accumulate = direct && accumulate;
    if (int rc = with_layout(s->d, GoBwd<T>{b, n, past_caches<T>(s), false, st})) return rc;
    if (!dgamma || direct) return MOE_OK;
  }
  if (!dgamma) return MOE_OK;
  MOE_LAUNCH("rmsnorm_dgamma", st,
             rmsnorm_dgamma_kernel<<<(int)(s->d / 16), 1024, 0, st>>>(parts, n, (int)s->d,
                                                                      accumulate, dgamma));
  return check_launch("rmsnorm_dgamma");
}

}  // namespace

int launch_rmsnorm(const moe_shape* s, const void* x, const void* res, const void* gamma,
                   float eps, void* r, void* y, void* q, uint8_t* qs, float* rstd,
                   hipStream_t st) {
  if (s->dtype == MOE_BF16)
    return rmsnorm_t<uint16_t>(s, x, res, gamma, eps, r, y, q, qs, rstd, st);
  if (s->dtype == MOE_F16)
    return rmsnorm_t<_Float16>(s, x, res, gamma, eps, r, y, q, qs, rstd, st);
  return rmsnorm_t<float>(s, x, res, gamma, eps, r, y, q, qs, rstd, st);
}

int launch_rmsnorm_bwd(const moe_shape* s, const void* dy, const void* r, const void* gamma,
                       const float* rstd, const void* dres, void* dx, float* dgamma,
                       bool accumulate, float* parts, hipStream_t st) {
  if (s->dtype == MOE_BF16)
    return rmsnorm_bwd_t<uint16_t>(s, dy, r, gamma, rstd, dres, dx, dgamma, accumulate, parts, st);
  if (s->dtype == MOE_F16)
    return rmsnorm_bwd_t<_Float16>(s, dy, r, gamma, rstd, dres, dx, dgamma, accumulate, parts, st);
  return rmsnorm_bwd_t<float>(s, dy, r, gamma, rstd, dres, dx, dgamma, accumulate, parts, st);
}

}  // namespace moe
