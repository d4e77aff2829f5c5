// The products of 8-bit rows with 4-bit expert weights for few rows per expert
// (decoding, short prompts): one pass over the active experts' weights, so what bounds
// them is how fast those stream from memory.  As the 8-bit kernels for few rows: a
// block takes 16 S weight rows (of both halves for gate and up) of one expert, its four
// waves share the reduction by blocks of 128, the weights go straight to registers and
// are the M side of 16 x 16 x 32 bf16 MFMAs, up to 16 G token rows the N side.  e2m1
// and e4m3 values with their powers of two are exact in bf16, so the products are exact
// and only their float32 sums round.
// A lane's 32 values of a block of 128 are one 16-byte load and one scale byte.
#include "moe_fp4.h"
#include "moe_small8.h"

namespace moe {
namespace {

// Blocks of 128 per round of a wave, for `sets` of 16 weight rows each.
constexpr int depth(int sets) { return sets <= 2 ? 4 : 2; }

// The weights of a product: H halves `apart` rows from each other (gate and up),
// of each S consecutive groups of 16 rows; set w is group w % S of half w / S.
struct WRows4 {
  const uint8_t* q;   // [E_l][n][k / 2]
  const uint8_t* s;   // [E_l][n][k / 32]
  int n, k, apart;
};

// acc[w][g] += weights . tokens over this wave's blocks of 128.  tokens(kb, g)
// gives a token group's block.
template <int S, int NW, int G, class Tokens>
__device__ __forceinline__ void reduce_blocks(const WRows4& W, int e, int r0, int wave, int lane,
                                              f32x4_t (&acc)[NW][G], Tokens tokens) {
  constexpr int D = depth(NW);
  const int kbs = W.k / 128;
  const size_t row = (size_t)e * W.n + r0 + (lane & 15);
  const uint8_t* base = W.q + row * (W.k / 2) + (lane >> 4) * 16;
  const uint8_t* sc = W.s + row * (W.k / 32) + (lane >> 4);
  for (int k0 = wave; k0 < kbs; k0 += WAVES * D) {
    i32x4_t raw[D][NW];
    int byte[D][NW];
#pragma unroll
    for (int t = 0; t < D; ++t) {
      const int kb = min(k0 + t * WAVES, kbs - 1);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const size_t to = (size_t)(w / S * W.apart + w % S * 16);
        raw[t][w] = *(const i32x4_t*)(base + to * (W.k / 2) + kb * 64);
        byte[t][w] = sc[to * (W.k / 32) + kb * 4];
      }
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
        const float scale = fp8_scale_value(byte[t][w]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t a = widen4((uint32_t)raw[t][w][q], scale);
#pragma unroll
          for (int g = 0; g < G; ++g)
            acc[w][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x[g].v[q], acc[w][g], 0, 0, 0);
        }
      }
    }
  }
}

// First product: quantised rows x W_gu, 16 outputs (gate and up) per block.
template <int G, typename elt>
__global__ __launch_bounds__(64 * WAVES) void fp4_first_kernel(
    GateUp<elt> op, QRows x, WRows4 W, const int32_t* __restrict__ offsets, int E_l) {
  __shared__ Reduce<2, G> red;
  int e, m0, m_end;
  if (!nth_expert(offsets, E_l, blockIdx.y, e, m0, m_end)) return;  // block-uniform
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int j0 = blockIdx.x * 16;
  for (int r0 = m0 + blockIdx.z * 16 * G; r0 < m_end; r0 += gridDim.z * 16 * G) {
    const uint8_t *xp[G], *sp[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int row = min(r0 + g * 16 + (lane & 15), m_end - 1);
      const size_t src = x.xrows ? x.xrows[row] / x.K : row;
      xp[g] = x.q + src * x.k + (lane >> 4) * 32;
      sp[g] = x.s + src * x.ld;
    }
    f32x4_t acc[2][G] = {};
    reduce_blocks<1, 2, G>(W, e, j0, wave, lane, acc, [&](int kb, int g) {
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
    for (int g = 0; g < G; ++g) {
      const int row = r0 + g * 16 + (lane & 15);
      if (red.owner(0, g) == wave && row < m_end) {
        const f32x4_t v[2] = {red.sum(0, g, lane), red.sum(1, g, lane)};
        op.finish((size_t)row, j0 + (lane >> 4) * 4, v);
      }
    }
    __syncthreads();
  }
}

// Second product: float32 rows, quantised here, x W_down; 16 S output columns per block.
template <int S, int G, typename elt>
__global__ __launch_bounds__(64 * WAVES) void fp4_second_kernel(
    const float* __restrict__ x, WRows4 W, elt* __restrict__ out,
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

template <typename elt>
int first(const moe_shape* s, const GateUp<elt>& op, const QRows& x, const WRows4& W,
          const int32_t* offsets, hipStream_t st) {
  const Shape sh(s, (int)s->F, false);
  auto go = [&](auto kernel) {
    MOE_LAUNCH("ffn_gate_up_fp4_small", st,
               kernel<<<sh.grid, 64 * WAVES, 0, st>>>(op, x, W, offsets, (int)s->E_l));
    return check_launch("ffn_gate_up_fp4_small");
  };
  return sh.G == 1 ? go(fp4_first_kernel<1, elt>)
                   : (sh.G == 2 ? go(fp4_first_kernel<2, elt>) : go(fp4_first_kernel<4, elt>));
}
template <typename elt>
int second(const moe_shape* s, const float* x, const WRows4& W, elt* out, const int32_t* offsets,
           hipStream_t st) {
  const Shape sh(s, W.n, true);
  auto go = [&](auto kernel) {
    MOE_LAUNCH("ffn_down_fp4_small", st,
               kernel<<<sh.grid, 64 * WAVES, 0, st>>>(x, W, out, offsets, (int)s->E_l));
    return check_launch("ffn_down_fp4_small");
  };
  if (sh.S == 4)
    return sh.G == 1 ? go(fp4_second_kernel<4, 1, elt>)
                     : (sh.G == 2 ? go(fp4_second_kernel<4, 2, elt>)
                                  : go(fp4_second_kernel<4, 4, elt>));
  return sh.G == 1 ? go(fp4_second_kernel<1, 1, elt>)
                   : (sh.G == 2 ? go(fp4_second_kernel<1, 2, elt>)
                                : go(fp4_second_kernel<1, 4, elt>));
}

template <typename elt>
int ffn_fwd_t(const moe_shape* s, const void* xq, const uint8_t* xs, const int32_t* xrows,
              const int32_t* offsets, const moe_fp4_weights* w, void* h, void* a, void* yp,
              void* ws, hipStream_t st) {
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  if (int rc = first(s, GateUp<elt>{(elt*)h, (elt*)a, (float*)ws, F},
                     QRows{(const uint8_t*)xq, xs, d, (int)fp8_scale_ld(d), xrows, K},
                     WRows4{w->gu, w->gu_s, 2 * F, d, F}, offsets, st))
    return rc;
  return second(s, (const float*)ws, WRows4{w->down, w->down_s, d, F, 0}, (elt*)yp, offsets, st);
}

}  // namespace

// Few rows: see fp8_small; the same form.
static int64_t most_mean(const moe_shape* s) {
  const int64_t most = s->dtype == MOE_BF16 ? 800000000 : 1400000000;
  return std::min<int64_t>(256, 11 + most / (s->E_l * s->F * s->d));
}
bool fp4_small(const moe_shape* s) {
  return cdiv(s->T * s->K, s->E) <= most_mean(s) &&
         std::max(Shape(s, (int)s->F, false).passes, Shape(s, (int)s->d, true).passes) <= 8;
}
// For the longest batch of at most T tokens that these kernels take.
size_t fp4_small_workspace_bytes(const moe_shape* s) {
  const int64_t rows = std::min(s->T * s->K, s->E * most_mean(s));
  return (size_t)(rows * s->F) * sizeof(float);
}

int launch_ffn_fwd_fp4_small(const moe_shape* s, const void* xq, const uint8_t* xs,
                             const int32_t* xrows, const int32_t* offsets,
                             const moe_fp4_weights* w, void* h, void* a, void* yp, void* ws,
                             hipStream_t st) {
  return s->dtype == MOE_BF16
             ? ffn_fwd_t<uint16_t>(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st)
             : ffn_fwd_t<_Float16>(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st);
}

}  // namespace moe
