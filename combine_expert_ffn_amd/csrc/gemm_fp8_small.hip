// The 8-bit expert products for few rows per expert (decoding, short prompts):
// each is one pass over the active experts' weights, so what bounds them is how
// fast those stream from memory.  A block takes 16 S weight rows (of both halves for
// gate and up) of one expert; its four waves share the reduction by blocks of 128,
// whose weights go straight to registers.  As compiled, a wave asks for one block's
// weights and rows at a time, behind the MFMAs of the one before (the loads that stand
// ahead of them in reduce_blocks are moved past the loop's exit), and the second product for its
// weights behind the quantisation: up to four memory latencies in a row, which other
// waves cover where there are many and nothing does for a single token.  The weight
// rows are the M side of 16 x 16 x 32 bf16 MFMAs, up to 16 G token rows the N side:
// e4m3 values and their power-of-two scales are exact in bf16, so the products are
// exact and only their float32 sums round, and the conversions (one instruction per
// two values) hide behind the loads.
// The first product leaves its result in float32; the second quantises the rows
// as it reads them (each wave its own blocks of 128, in registers), so no block
// needs another's column maximum.
// bf16 on an MI355X, forward: one token, 8 of 128 experts of 2048 x 768, 13.9 us (38 MB of
// weights; two launches and their chains of latencies); 64 tokens, up to 9 rows for each of
// the 128, 131 us (604 MB, 4.6 TB/s, near the 5.0 of a large copy).
#include "moe_fp8.h"

#include <math.h>

#include <algorithm>

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int WAVES = 4;
// Blocks of 128 per round of a wave, for `sets` of 16 weight rows each.
constexpr int depth(int sets) { return sets <= 2 ? 4 : 2; }

// Expert number `slot` among those with rows, and its rows; false if there are
// fewer.  Every wave finds it by itself.
__device__ __forceinline__ bool nth_expert(const int32_t* offsets, int E_l, int slot, int& e,
                                           int& m0, int& m_end) {
  const int lane = (int)(threadIdx.x & 63);
  int lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = min(k * 64 + lane, E_l - 1);
    lo[k] = offsets[j];
    hi[k] = offsets[j + 1];
  }
  bool found = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool has = k * 64 + lane < E_l && hi[k] > lo[k];
    const uint64_t b = __ballot(has);
    const int rank = (int)__builtin_amdgcn_mbcnt_hi(
        (uint32_t)(b >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b, 0u));
    const uint64_t mine = __ballot(has && rank == slot);
    if (!found && mine) {  // wave-uniform
      const int l = __builtin_ctzll(mine);
      e = k * 64 + l;
      m0 = __builtin_amdgcn_readlane(lo[k], l);
      m_end = __builtin_amdgcn_readlane(hi[k], l);
      found = true;
    }
    slot -= (int)__popcll(b);
  }
  return found;
}

// A lane's 32 values of a block of 128: row lane % 16, values 32 (lane / 16) ..+31,
// the same for both operands (the order within a block does not change its sum).
struct Raw {
  i32x4_t v[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    v[0] = *(const i32x4_t*)p;
    v[1] = *(const i32x4_t*)(p + 16);
  }
  __device__ __forceinline__ bf16x8_t part(int q, float scale) const {
    return widen(v[q >> 1][(q & 1) * 2], v[q >> 1][(q & 1) * 2 + 1], scale);
  }
};
struct Block {
  bf16x8_t v[4];
};

// Sums of the four waves' accumulators: weight set w's token group g is summed by
// wave owner(w, g).
template <int NW, int G>
struct Reduce {
  f32x4_t v[WAVES][NW][G][64];
  __device__ __forceinline__ void put(const f32x4_t (&acc)[NW][G], int wave, int lane) {
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int g = 0; g < G; ++g) v[wave][w][g][lane] = acc[w][g];
  }
  __device__ __forceinline__ f32x4_t sum(int w, int g, int lane) const {
    return (v[0][w][g][lane] + v[1][w][g][lane]) + (v[2][w][g][lane] + v[3][w][g][lane]);
  }
  static __device__ __forceinline__ int owner(int w, int g) { return (w * G + g) % WAVES; }
};

// The weights of a product: H halves `apart` rows from each other (gate and up),
// of each S consecutive groups of 16 rows; set w is group w % S of half w / S.
struct WRows {
  const uint8_t* q;   // [E_l][n][k]
  const uint8_t* s;   // [E_l][n / 128][ld]
  int n, k, ld, apart;
};

// acc[w][g] += weights . tokens over this wave's blocks of 128.  tokens(kb, g)
// gives a token group's block.
template <int S, int NW, int G, class Tokens>
__device__ __forceinline__ void reduce_blocks(const WRows& W, int e, int r0, int wave, int lane,
                                              f32x4_t (&acc)[NW][G], Tokens tokens) {
  constexpr int D = depth(NW);
  const int kbs = W.k / 128;
  const uint8_t* base = W.q + ((size_t)e * W.n + r0 + (lane & 15)) * W.k + (lane >> 4) * 32;
  // 16 S consecutive rows lie in one block of 128
  const uint8_t* sc = W.s + ((size_t)e * (W.n / 128) + r0 / 128) * W.ld;
  for (int k0 = wave; k0 < kbs; k0 += WAVES * D) {
    Raw raw[D][NW];
    int byte[D][NW / S];
#pragma unroll
    for (int t = 0; t < D; ++t) {
      const int kb = min(k0 + t * WAVES, kbs - 1);
#pragma unroll
      for (int w = 0; w < NW; ++w)
        raw[t][w].load(base + (size_t)(w / S * W.apart + w % S * 16) * W.k + kb * 128);
#pragma unroll
      for (int w = 0; w < NW / S; ++w) byte[t][w] = sc[(size_t)w * (W.apart / 128) * W.ld + kb];
    }
#pragma unroll
    for (int t = 0; t < D; ++t) {
      const int kb = k0 + t * WAVES;
      if (kb >= kbs) break;  // wave-uniform
      Block x[G];
#pragma unroll
      for (int g = 0; g < G; ++g) x[g] = tokens(kb, g);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float scale = fp8_scale_value(byte[t][w / S]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t a = raw[t][w].part(q, scale);
#pragma unroll
          for (int g = 0; g < G; ++g)
            acc[w][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x[g].v[q], acc[w][g], 0, 0, 0);
        }
      }
    }
  }
}

// Four consecutive 16-bit values.
template <typename elt>
__device__ __forceinline__ void store4(elt* p, const float* f) {
  const float t[8] = {f[0], f[1], f[2], f[3], 0, 0, 0, 0};
  const uint4 v = Chunk<elt>::pack(t);
  *(uint2*)p = uint2{v.x, v.y};
}
template <typename elt>
__device__ __forceinline__ void load4(const elt* p, float* f) {
  const uint2 v = *(const uint2*)p;
  float t[8];
  Chunk<elt>::unpack(uint4{v.x, v.y, 0, 0}, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = t[i];
}

// The quantised row operand: dispatched rows, or token rows through the plan.
struct QRows {
  const uint8_t* q;
  const uint8_t* s;
  int k, ld;
  const int32_t* xrows;  // NULL: dispatched rows
  int K;
};

template <typename elt>
struct GateUp {
  static constexpr int H = 2;
  elt *h, *a;
  float* af;  // [rows][F]
  int F;
  __device__ __forceinline__ void finish(size_t row, int j, const f32x4_t (&v)[2]) const {
    float g[4], u[4], t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = v[0][i];
      u[i] = v[1][i];
      t[i] = silu_fast(g[i]) * u[i];
    }
    *(float4*)(af + row * F + j) = float4{t[0], t[1], t[2], t[3]};
    if (h) {
      store4(h + row * 2 * F + j, g);
      store4(h + row * 2 * F + F + j, u);
    }
    if (a) store4(a + row * F + j, t);
  }
};

template <typename elt>
struct DgradAct {
  static constexpr int H = 1;
  const elt* h;
  const float* gates;    // with xrows
  const int32_t* xrows;
  elt *dh, *ag;
  float* df;  // [rows][2F]
  int F;
  __device__ __forceinline__ void finish(size_t row, int j, const f32x4_t (&v)[1]) const {
    float g[4], u[4], dg[4], du[4], av[4];
    load4(h + row * 2 * F + j, g);
    load4(h + row * 2 * F + F + j, u);
    const float gate = xrows ? gates[xrows[row]] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sg = sigmoid_fast(g[i]), d = v[0][i] * gate;
      dg[i] = d * u[i] * sg * (1.0f + g[i] * (1.0f - sg));
      du[i] = d * g[i] * sg;
      av[i] = gate * (g[i] * sg) * u[i];
    }
    *(float4*)(df + row * 2 * F + j) = float4{dg[0], dg[1], dg[2], dg[3]};
    *(float4*)(df + row * 2 * F + F + j) = float4{du[0], du[1], du[2], du[3]};
    store4(dh + row * 2 * F + j, dg);
    store4(dh + row * 2 * F + F + j, du);
    if (ag) store4(ag + row * F + j, av);
  }
};

// First product: quantised rows x W, 16 S output columns per block.
template <int S, int G, class Op>
__global__ __launch_bounds__(64 * WAVES) void small_first_kernel(
    Op op, QRows x, WRows W, const int32_t* __restrict__ offsets, int E_l) {
  constexpr int NW = Op::H * S;
  __shared__ Reduce<NW, G> red;
  int e, m0, m_end;
  if (!nth_expert(offsets, E_l, blockIdx.y, e, m0, m_end)) return;  // block-uniform
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int j0 = blockIdx.x * 16 * S;
  for (int r0 = m0 + blockIdx.z * 16 * G; r0 < m_end; r0 += gridDim.z * 16 * G) {
    const uint8_t *xp[G], *sp[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int row = min(r0 + g * 16 + (lane & 15), m_end - 1);
      const size_t src = x.xrows ? x.xrows[row] / x.K : row;
      xp[g] = x.q + src * x.k + (lane >> 4) * 32;
      sp[g] = x.s + src * x.ld;
    }
    f32x4_t acc[NW][G] = {};
    reduce_blocks<S, NW, G>(W, e, j0, wave, lane, acc, [&](int kb, int g) {
      Raw r;
      r.load(xp[g] + kb * 128);
      const float scale = fp8_scale_value(sp[g][kb]);
      Block b;
#pragma unroll
      for (int q = 0; q < 4; ++q) b.v[q] = r.part(q, scale);
      return b;
    });
    red.put(acc, wave, lane);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int row = r0 + g * 16 + (lane & 15);
        if (red.owner(t, g) == wave && row < m_end) {
          f32x4_t v[Op::H];
#pragma unroll
          for (int w = 0; w < Op::H; ++w) v[w] = red.sum(w * S + t, g, lane);
          op.finish((size_t)row, j0 + t * 16 + (lane >> 4) * 4, v);
        }
      }
    __syncthreads();
  }
}

// Second product: float32 rows, quantised here, x W; 16 S output columns per block.
template <int S, int G, typename elt>
__global__ __launch_bounds__(64 * WAVES) void small_second_kernel(
    const float* __restrict__ x, WRows W, elt* __restrict__ out,
    const int32_t* __restrict__ offsets, int E_l) {
  __shared__ Reduce<S, G> red;
  int e, m0, m_end;
  if (!nth_expert(offsets, E_l, blockIdx.y, e, m0, m_end)) return;  // block-uniform
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = blockIdx.x * 16 * S;
  for (int r0 = m0 + blockIdx.z * 16 * G; r0 < m_end; r0 += gridDim.z * 16 * G) {
    const float* xp[G];
#pragma unroll
    for (int g = 0; g < G; ++g)
      xp[g] = x + (size_t)min(r0 + g * 16 + (lane & 15), m_end - 1) * W.k + (lane >> 4) * 32;
    f32x4_t acc[S][G] = {};
    reduce_blocks<S, S, G>(W, e, c0, wave, lane, acc, [&](int kb, int g) {
      float f[32];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float4 v = *(const float4*)(xp[g] + kb * 128 + t * 4);
        f[4 * t] = v.x; f[4 * t + 1] = v.y; f[4 * t + 2] = v.z; f[4 * t + 3] = v.w;
      }
      float m = 0.f;
#pragma unroll
      for (int t = 0; t < 32; ++t) m = fmaxf(m, finite_abs(f[t]));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const int byte = fp8_scale_byte(m);
      const float inv = fp8_inv_scale(byte), scale = fp8_scale_value(byte);
      Block b;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float* y = f + q * 8 + p * 4;
          w[p] = pack_fp8(finite_or_nan(y[0]) * inv, finite_or_nan(y[1]) * inv,
                          finite_or_nan(y[2]) * inv, finite_or_nan(y[3]) * inv);
        }
        b.v[q] = widen((int)w[0], (int)w[1], scale);
      }
      return b;
    });
    red.put(acc, wave, lane);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < S; ++w)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int row = r0 + g * 16 + (lane & 15);
        if (red.owner(w, g) == wave && row < m_end) {
          const f32x4_t v = red.sum(w, g, lane);
          const float t[4] = {v[0], v[1], v[2], v[3]};
          store4(out + (size_t)row * W.n + c0 + w * 16 + (lane >> 4) * 4, t);
        }
      }
    __syncthreads();
  }
}

// Launch shape.  rows: what most experts have at most (the mean of an even routing and two
// standard deviations of a Poisson count).  S: four groups of 16 columns per block
// where that and 16 rows per block leave one block per CU or more (every block reads, and
// for the second product quantises, all of its rows: at 128 rows, 2 experts of 2048 x 2048,
// 29 us against 71 for the activation gradient's second product).  G: as many token groups
// per pass as the rows fill, fewer where blocks are few, down to one.  An expert may hold
// every token: all passes that this takes are spread over the grid's z, as far as four
// blocks per CU (surplus blocks leave at once: nothing measurable on even loads).  8 of
// 64 experts of 2048 x 768, 256 tokens, K = 1, z for the rows of an even load and for every
// token: even 21 and 20 us, Zipf 1.1 74 and 49, all on one expert 126 and 76.
struct Shape {
  int G, S;
  int64_t passes;  // of a block whose expert holds every token
  dim3 grid;
  Shape(const moe_shape* s, int cols, bool may_widen) {
    const int64_t pairs = s->T * s->K;
    const double mean = (double)pairs / (double)s->E;
    const int64_t rows = (int64_t)(mean + 2 * sqrt(mean)) + 1;
    const int64_t slots = std::max<int64_t>(1, std::min(pairs, s->E_l));
    S = may_widen && slots * cols / 64 * cdiv(rows, 16) >= 256 ? 4 : 1;
    const int64_t blocks = slots * cols / (16 * S);
    G = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    while (G > 1 && blocks * cdiv(rows, 16 * G) < (S == 1 ? 512 : 256)) G /= 2;
    const int64_t z = std::max<int64_t>(1, std::min(cdiv(s->T, 16 * G), cdiv(1024, blocks)));
    passes = cdiv(s->T, 16 * G * z);
    grid = dim3((unsigned)(cols / (16 * S)), (unsigned)slots, (unsigned)z);
  }
};

template <class Op>
int first(const char* name, const moe_shape* s, const Op& op, const QRows& x, const WRows& W,
          const int32_t* offsets, int cols, hipStream_t st) {
  const Shape sh(s, cols, Op::H == 1);
  auto go = [&](auto kernel) {
    MOE_LAUNCH(name, st, kernel<<<sh.grid, 64 * WAVES, 0, st>>>(op, x, W, offsets, (int)s->E_l));
    return check_launch(name);
  };
  if constexpr (Op::H == 1)
    if (sh.S == 4)
      return sh.G == 1 ? go(small_first_kernel<4, 1, Op>)
                       : (sh.G == 2 ? go(small_first_kernel<4, 2, Op>)
                                    : go(small_first_kernel<4, 4, Op>));
  return sh.G == 1 ? go(small_first_kernel<1, 1, Op>)
                   : (sh.G == 2 ? go(small_first_kernel<1, 2, Op>)
                                : go(small_first_kernel<1, 4, Op>));
}
template <typename elt>
int second(const char* name, const moe_shape* s, const float* x, const WRows& W, elt* out,
           const int32_t* offsets, hipStream_t st) {
  const Shape sh(s, W.n, true);
  auto go = [&](auto kernel) {
    MOE_LAUNCH(name, st, kernel<<<sh.grid, 64 * WAVES, 0, st>>>(x, W, out, offsets, (int)s->E_l));
    return check_launch(name);
  };
  if (sh.S == 4)
    return sh.G == 1 ? go(small_second_kernel<4, 1, elt>)
                     : (sh.G == 2 ? go(small_second_kernel<4, 2, elt>)
                                  : go(small_second_kernel<4, 4, elt>));
  return sh.G == 1 ? go(small_second_kernel<1, 1, elt>)
                   : (sh.G == 2 ? go(small_second_kernel<1, 2, elt>)
                                : go(small_second_kernel<1, 4, elt>));
}

template <typename elt>
int ffn_fwd_t(const moe_shape* s, const void* xq, const uint8_t* xs, const int32_t* xrows,
              const int32_t* offsets, const moe_fp8_weights* w, void* h, void* a, void* yp,
              void* ws, hipStream_t st) {
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const int ld_d = (int)fp8_scale_ld(d), ld_f = (int)fp8_scale_ld(F);
  const GateUp<elt> op{(elt*)h, (elt*)a, (float*)ws, F};
  if (int rc = first("ffn_gate_up_fp8_small", s, op,
                     QRows{(const uint8_t*)xq, xs, d, ld_d, xrows, K},
                     WRows{(const uint8_t*)w->gu, w->gu_s, 2 * F, d, ld_d, F}, offsets, F, st))
    return rc;
  return second("ffn_down_fp8_small", s, (const float*)ws,
                WRows{(const uint8_t*)w->down, w->down_s, d, F, ld_f, 0}, (elt*)yp, offsets, st);
}

template <typename elt>
int ffn_dgrad_t(const moe_shape* s, const void* dq, const uint8_t* ds, const int32_t* xrows,
                const float* gates, const void* h, const int32_t* offsets,
                const moe_fp8_weights* w, void* dh, void* dxp, void* ag, void* ws,
                hipStream_t st) {
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const int ld_d = (int)fp8_scale_ld(d), ld_2f = (int)fp8_scale_ld(2 * F);
  const DgradAct<elt> op{(const elt*)h, gates, xrows, (elt*)dh, (elt*)ag, (float*)ws, F};
  if (int rc = first("dgrad_act_fp8_small", s, op,
                     QRows{(const uint8_t*)dq, ds, d, ld_d, xrows, K},
                     WRows{(const uint8_t*)w->downT, w->downT_s, F, d, ld_d, 0}, offsets, F, st))
    return rc;
  return second("dgrad_in_fp8_small", s, (const float*)ws,
                WRows{(const uint8_t*)w->guT, w->guT_s, d, 2 * F, ld_2f, 0}, (elt*)dxp, offsets,
                st);
}

}  // namespace

// Few rows: up to 256 per expert on average, and E_l F d (mean - 11) up to 0.8e9 for the
// forward and 1.3e9 for the gradient in bf16, 1.4e9 and 1.9e9 in fp16 (where the tiles multiply
// at half the rate).  Below it these kernels are faster than the 256 x 256 tiles, whose time
// hardly falls with the rows; above, the tiles reuse each weight more.  Both sides in us on
// an MI355X, small against tiles, forward and gradient: bf16, 128 experts of 2048 x 768 at 16
// rows 174 / 171 and 187 / 202, at 32 297 / 171 and 347 / 203; 8 experts of 2048 x 1408 at 32
// 47 / 44 and 55 / 67, at 64 59 / 44 and 69 / 68; 8 of 2048 x 768 at 64 36 / 38 and 39 / 56, at
// 128 50 / 40 and 59 / 58; 4 of 640 x 384 at 256 24 / 32 and 28 / 49.  fp16: 8 of 2048 x 1408 at
// 64 59 / 59 and 69 / 86, at 128 104 / 60 and 121 / 89.
// These are even loads, and the time here follows the fullest expert, whose passes a block
// makes one after another.  So no block may need more than 8 with every token on one expert:
// over the 362 calls tried that this and the limits above let through (four shapes from
// 640 x 384 to 4096 x 1024, 4 to 128 experts, K = 1 to 8, 16 to 2048 tokens), small over tiles is
// 0.62 on even loads, 0.84 with Zipf 1.1 and 0.98 with all tokens on the same K experts
// (geometric means; worst 7.8), without it 0.65, 1.13 and 1.45 (worst 20.5, and 26 at 16384
// tokens, 64 experts of 512 x 384, all on one: 859 / 33).
static int64_t most_mean(const moe_shape* s, bool dgrad) {
  const int64_t most = (s->dtype == MOE_BF16 ? 800000000 : 1400000000) + (dgrad ? 500000000 : 0);
  return std::min<int64_t>(256, 11 + most / (s->E_l * s->F * s->d));
}
bool fp8_small(const moe_shape* s, bool dgrad) {
  return cdiv(s->T * s->K, s->E) <= most_mean(s, dgrad) &&
         std::max(Shape(s, (int)s->F, dgrad).passes, Shape(s, (int)s->d, true).passes) <= 8;
}
// For the longest batch of at most T tokens that these kernels take.
size_t fp8_small_workspace_bytes(const moe_shape* s) {
  const int64_t rows = std::min(s->T * s->K, s->E * most_mean(s, true));
  return (size_t)(rows * 2 * s->F) * sizeof(float);
}

int launch_ffn_fwd_fp8_small(const moe_shape* s, const void* xq, const uint8_t* xs,
                             const int32_t* xrows, const int32_t* offsets,
                             const moe_fp8_weights* w, void* h, void* a, void* yp, void* ws,
                             hipStream_t st) {
  return s->dtype == MOE_BF16
             ? ffn_fwd_t<uint16_t>(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st)
             : ffn_fwd_t<_Float16>(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st);
}

int launch_ffn_dgrad_fp8_small(const moe_shape* s, const void* dq, const uint8_t* ds,
                               const int32_t* xrows, const float* gates, const void* h,
                               const int32_t* offsets, const moe_fp8_weights* w, void* dh,
                               void* dxp, void* ag, void* ws, hipStream_t st) {
  return s->dtype == MOE_BF16 ? ffn_dgrad_t<uint16_t>(s, dq, ds, xrows, gates, h, offsets, w, dh,
                                                      dxp, ag, ws, st)
                              : ffn_dgrad_t<_Float16>(s, dq, ds, xrows, gates, h, offsets, w, dh,
                                                      dxp, ag, ws, st);
}

}  // namespace moe
