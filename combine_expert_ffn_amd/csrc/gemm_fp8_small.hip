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
#include "moe_small8.h"

namespace moe {
namespace {

// Blocks of 128 per round of a wave, for `sets` of 16 weight rows each.
constexpr int depth(int sets) { return sets <= 2 ? 4 : 2; }

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
      return quantised(f);
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
