// The products of 8-bit rows with 4-bit expert weights for few rows per expert
// (decoding, short prompts): one pass over the active experts' weights, so what bounds
// them is how fast those stream from memory.  A block takes groups of 16 S weight rows (of
// both halves for gate and up) of one expert; its four waves share the reduction by 256
// values (128 bytes of a weight row), the weights go straight to registers and are the
// M side of the MFMAs, up to 16 G token rows the N side.
// bf16 data: v_mfma_scale_f32_16x16x128_f8f6f4 on the codes as they are, with the scales
// as bytes of the lanes.  fp16 data: codes and rows widened to bf16 with their scales
// (exact) for 16 x 16 x 32 bf16 MFMAs.
#include "moe_fp4.h"
#include "moe_small8.h"

#include <type_traits>

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2), aligned(4)));

// The weights of a product: H halves `apart` rows from each other (gate and up),
// of each S consecutive groups of 16 rows; set w is group w % S of half w / S.
struct WRows4 {
  const uint8_t* q;   // [E_l][n][k / 2]
  const uint8_t* s;   // [E_l][n][k / 32]
  int n, k, apart;
};

// A lane's part of 128 values of 16 token rows: row lane % 16, and of its values the 32
// that are paired with the lane's 32 consecutive ones of a weight row: the same 32 where
// both are widened; where the instruction takes 8-bit rows, 16 from 16 (lane / 16) on and
// 16 from 64 further on.
template <bool WIDE>
struct Tokens {
  Block b;
};
template <>
struct Tokens<false> {
  i32x8_t v;
  int scale;
};

// 8-bit rows as the token side.
template <bool WIDE, int G>
struct X8 {
  const uint8_t *q[G], *s[G];
  __device__ __forceinline__ Tokens<WIDE> get(int kb, int g, int part) const {
    Tokens<WIDE> t;
    const uint8_t* p = q[g] + kb * 128;
    const int byte = s[g][kb];
    if constexpr (WIDE) {
      Raw r;
      r.load(p + part * 32);
      const float scale = fp8_scale_value(byte);
#pragma unroll
      for (int i = 0; i < 4; ++i) t.b.v[i] = r.part(i, scale);
    } else {
      const i32x4_t lo = *(const i32x4_t*)(p + part * 16);
      const i32x4_t hi = *(const i32x4_t*)(p + part * 16 + 64);
      t.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      t.scale = byte;
    }
    return t;
  }
};
// Float32 rows, quantised here.
template <bool WIDE, int G>
struct X32 {
  const float* p[G];
  __device__ __forceinline__ Tokens<WIDE> get(int kb, int g, int part) const {
    float f[32];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int at = WIDE ? part * 32 + t * 4 : part * 16 + (t >> 2) * 64 + (t & 3) * 4;
      const float4 v = *(const float4*)(p[g] + kb * 128 + at);
      f[4 * t] = v.x; f[4 * t + 1] = v.y; f[4 * t + 2] = v.z; f[4 * t + 3] = v.w;
    }
    Tokens<WIDE> t;
    if constexpr (WIDE) {
      t.b = quantised(f);
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = fmaxf(m, finite_abs(f[i]));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      t.scale = fp8_scale_byte(m);
      const float inv = fp8_inv_scale(t.scale);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        t.v[i] = (int)pack_fp8(finite_or_nan(f[4 * i]) * inv, finite_or_nan(f[4 * i + 1]) * inv,
                               finite_or_nan(f[4 * i + 2]) * inv,
                               finite_or_nan(f[4 * i + 3]) * inv);
    }
    return t;
  }
};

// A lane's codes of NW sets of 16 weight rows, values 32 (lane / 16) ..+31 of two blocks of
// 128, and the scales of all four lanes of the row (byte lane / 16 of a word is its own): a
// byte of each lane's own would be a request of its own, 20 % of the time.
template <int S, int NW, bool PAIR>
struct Weights {
  i32x4_t v[NW][2];
  uint32_t scale[NW][2];
  // q: the lane's codes, s: the row's scales, in block 0 of set 0.  Where the second block
  // does not exist the first's codes are read again, and nothing past the row's scales
  // (PAIR: one load for both blocks, where a row has two at least).
  __device__ __forceinline__ void load(const WRows4& W, const uint8_t* q, const uint8_t* s,
                                       int kb) {
    const bool two = kb * 128 + 128 < W.k;  // wave-uniform
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const size_t to = (size_t)(w / S * W.apart + w % S * 16);
      const uint8_t* p = q + to * (W.k / 2) + kb * 64;
      v[w][0] = *(const i32x4_t*)p;
      v[w][1] = *(const i32x4_t*)(p + (two ? 64 : 0));
      const uint8_t* b = s + to * (W.k / 32) + kb * 4;
      if constexpr (PAIR) {
        const u32x2_t x = *(const u32x2_t*)(b - (two ? 0 : 4));
        scale[w][0] = two ? x[0] : x[1];
        scale[w][1] = x[1];
      } else {
        scale[w][0] = *(const uint32_t*)b;
        scale[w][1] = *(const uint32_t*)(b + (two ? 4 : 0));
      }
    }
  }
};

// acc += the lane's 32 values of a weight row set x tokens.
template <bool WIDE>
__device__ __forceinline__ f32x4_t multiply(const i32x4_t& v, uint32_t byte,
                                            const Tokens<WIDE>& x, f32x4_t acc) {
  if constexpr (WIDE) {
    const float scale = fp8_scale_value((int)(byte & 255u));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen4((uint32_t)v[i], scale), x.b.v[i], acc,
                                                    0, 0, 0);
    return acc;
  } else {
    const i32x8_t a = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
    // 4: e2m1, 0: e4m3
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x.v, acc, 4, 0, 0, (int)byte,
                                                            0, x.scale);
  }
}

// First product: quantised rows x W_gu, SwiGLU.
template <typename elt>
struct First {
  static constexpr int H = 2;
  static constexpr bool WIDE = std::is_same<elt, _Float16>::value;
  template <int G> using X = X8<WIDE, G>;
  GateUp<elt> out;
  QRows x;
  __device__ __forceinline__ int index(int r) const { return x.xrows ? x.xrows[r] : r; }
  template <int G>
  __device__ __forceinline__ void rows(X<G>& v, int g, int i) const {
    const size_t src = x.xrows ? i / x.K : i;
    v.q[g] = x.q + src * x.k;
    v.s[g] = x.s + src * x.ld;
  }
  __device__ __forceinline__ void finish(size_t r, int j, const f32x4_t (&v)[2]) const {
    out.finish(r, j, v);
  }
};
// Second product: float32 rows, quantised here, x W_down.
template <typename elt>
struct Second {
  static constexpr int H = 1;
  static constexpr bool WIDE = std::is_same<elt, _Float16>::value;
  template <int G> using X = X32<WIDE, G>;
  const float* x;
  elt* out;
  int k, n;
  __device__ __forceinline__ int index(int r) const { return r; }
  template <int G>
  __device__ __forceinline__ void rows(X<G>& v, int g, int i) const {
    v.p[g] = x + (size_t)i * k;
  }
  __device__ __forceinline__ void finish(size_t r, int j, const f32x4_t (&v)[1]) const {
    const float t[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
    store4(out + r * n + j, t);
  }
};

// A block takes `span` groups of 16 S output columns of one expert, 16 G of its rows at a
// time.  Its four waves take the units of the reduction (two blocks of 128) in turn, and
// their sums meet in LDS for each group.  With UW units to a wave at most (0: any number) it
// keeps its part of the rows in registers over the groups: read, and for the second product
// quantised, once.  Each of BUF buffers is filled with the weights of the unit that will use it
// next as soon as its last ones are used: no weights are moved between registers, which
// would wait for them.
template <int S, int G, int UW, class Op>
__global__ __launch_bounds__(64 * WAVES) void fp4_small_kernel(
    Op op, WRows4 W, const int32_t* __restrict__ offsets, int E_l, int groups, int span) {
  constexpr int NW = Op::H * S, HELD = UW > 0 ? UW : 1, BUF = 2;
  constexpr bool WIDE = Op::WIDE;
  __shared__ Reduce<NW, G> red;
  int e, m0, m_end;
  if (!nth_expert(offsets, E_l, blockIdx.y, e, m0, m_end)) return;  // block-uniform
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, part = lane >> 4;
  const int c_first = blockIdx.x * span, c_end = min(c_first + span, groups);
  const int kbs = W.k / 128, units = (kbs + 1) / 2;
  const int n = (units - wave + WAVES - 1) / WAVES;  // of this wave
  const size_t row0 = (size_t)e * W.n + (lane & 15);
  const uint8_t* q = W.q + row0 * (W.k / 2) + part * 16;
  const uint8_t* s = W.s + row0 * (W.k / 32);
  auto block = [&](int i) { return (wave + i * WAVES) * 2; };  // the first of unit i
  Weights<S, NW, (UW > 0)> buf[BUF];
  // unit i of group c, if there is such a group
  auto fetch = [&](auto& w, int c, int i) {
    if (c < c_end)  // block-uniform
      w.load(W, q + (size_t)(c * 16 * S) * (W.k / 2), s + (size_t)(c * 16 * S) * (W.k / 32),
             block(i));
  };
  for (int r0 = m0 + blockIdx.z * 16 * G; r0 < m_end; r0 += gridDim.z * 16 * G) {
    // the rows' places are asked for ahead of the weights, behind which their loads, in
    // order, would wait
    int at[G];
#pragma unroll
    for (int g = 0; g < G; ++g) at[g] = op.index(min(r0 + g * 16 + (lane & 15), m_end - 1));
    __builtin_amdgcn_sched_barrier(0);
    if (n > 0) {  // wave-uniform
#pragma unroll
      for (int b = 0; b < BUF; ++b)  // the first BUF units in order
        fetch(buf[b], c_first + b / n, b % n);
    }
    __builtin_amdgcn_sched_barrier(0);
    typename Op::template X<G> x;
#pragma unroll
    for (int g = 0; g < G; ++g) op.rows(x, g, at[g]);
    Tokens<WIDE> held[HELD][2][G];
    auto hold = [&](Tokens<WIDE> (&to)[2][G], int kb) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < G; ++g) to[h][g] = x.get(min(kb + h, kbs - 1), g, part);
    };
    if constexpr (UW > 0) {
#pragma unroll
      for (int i = 0; i < UW; ++i)
        if (i < n) hold(held[i], block(i));  // wave-uniform
    }
    auto finish_group = [&](int c, const f32x4_t (&acc)[NW][G]) {
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
            op.finish((size_t)row, (c * S + t) * 16 + (lane >> 4) * 4, v);
          }
        }
      __syncthreads();
    };
    f32x4_t acc[NW][G];
    auto unit = [&](auto& w, int i, const Tokens<WIDE> (&b)[2][G]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && block(i) + 1 >= kbs) break;  // wave-uniform
#pragma unroll
        for (int v = 0; v < NW; ++v)
#pragma unroll
          for (int g = 0; g < G; ++g)
            acc[v][g] = multiply<WIDE>(w.v[v][h], w.scale[v][h] >> (part * 8), b[h][g],
                                       acc[v][g]);
      }
    };
    auto clear = [&]() {
#pragma unroll
      for (int v = 0; v < NW; ++v)
#pragma unroll
        for (int g = 0; g < G; ++g) acc[v][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    if constexpr (UW == 2) {
      for (int c = c_first; c < c_end; ++c) {
        clear();
        if (n == 2) {  // wave-uniform
          unit(buf[0], 0, held[0]);
          fetch(buf[0], c + 1, 0);
          unit(buf[1], 1, held[1]);
          fetch(buf[1], c + 1, 1);
        } else if (n == 1) {  // both buffers hold unit 0, of this group and the next
          unit(buf[0], 0, held[0]);
          buf[0] = buf[1];
          fetch(buf[1], c + 2, 0);
        }
        finish_group(c, acc);
      }
    } else if constexpr (UW == 1) {
      for (int c = c_first; c < c_end; c += 2) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (c + b < c_end) {  // block-uniform
            clear();
            if (n > 0) {
              unit(buf[b], 0, held[0]);
              fetch(buf[b], c + b + 2, 0);
            }
            finish_group(c + b, acc);
          }
      }
    } else {
      for (int c = c_first; c < c_end; ++c) {
        clear();
        for (int i = 0; i < n; ++i) {
          hold(held[0], block(i));
          unit(buf[0], i, held[0]);
          const int to = i + 2;
          buf[0] = buf[1];
          fetch(buf[1], c + to / n, to % n);
        }
        finish_group(c, acc);
      }
    }
  }
}

// Blocks that share the groups where the routing is even: two per CU.
constexpr int kBlocks = 512;

template <class Op>
int launch(const char* name, const moe_shape* s, const Op& op, const WRows4& W, int cols,
           const int32_t* offsets, hipStream_t st) {
  const Shape sh(s, cols, Op::H == 1);
  const int groups = (int)sh.grid.x;
  // experts that have rows
  const double with_rows =
      std::max(1.0, (double)s->E_l * -expm1(-(double)(s->T * s->K) / (double)s->E));
  const int parts = (int)std::max(1.0, kBlocks / (with_rows * sh.grid.z) + 0.5);
  const int span = (int)cdiv(groups, std::min(parts, groups));
  const dim3 grid((unsigned)cdiv(groups, span), sh.grid.y, sh.grid.z);
  const int units = (W.k + 255) / 256, per_wave = (units + WAVES - 1) / WAVES;
  auto go = [&](auto kernel) {
    MOE_LAUNCH(name, st, kernel<<<grid, 64 * WAVES, 0, st>>>(op, W, offsets, (int)s->E_l, groups,
                                                             span));
    return check_launch(name);
  };
  auto by_rows = [&](auto S_) {
    constexpr int S = decltype(S_)::value;
    // as many units' rows in registers as leave two waves to a SIMD
    auto by_units = [&](auto G_, auto most) {
      constexpr int G = decltype(G_)::value, MOST = decltype(most)::value;
      if (per_wave > MOST || W.k == 128) return go(fp4_small_kernel<S, G, 0, Op>);
      if constexpr (MOST == 2)
        if (per_wave == 2) return go(fp4_small_kernel<S, G, 2, Op>);
      return go(fp4_small_kernel<S, G, 1, Op>);
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    if (sh.G == 4)
      return by_units(std::integral_constant<int, 4>{},
                      std::integral_constant<int, Op::WIDE || S == 4 ? 1 : 2>{});
    if (sh.G == 2) return by_units(Two{}, std::integral_constant<int, Op::WIDE ? 1 : 2>{});
    return by_units(One{}, Two{});
  };
  if constexpr (Op::H == 1)
    if (sh.S == 4) return by_rows(std::integral_constant<int, 4>{});
  return by_rows(std::integral_constant<int, 1>{});
}

template <typename elt>
int ffn_fwd_t(const moe_shape* s, const void* xq, const uint8_t* xs, const int32_t* xrows,
              const int32_t* offsets, const moe_fp4_weights* w, void* h, void* a, void* yp,
              void* ws, hipStream_t st) {
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const First<elt> gu{{(elt*)h, (elt*)a, (float*)ws, F},
                      {(const uint8_t*)xq, xs, d, (int)fp8_scale_ld(d), xrows, K}};
  if (int rc = launch("ffn_gate_up_fp4_small", s, gu, WRows4{w->gu, w->gu_s, 2 * F, d, F}, F,
                      offsets, st))
    return rc;
  return launch("ffn_down_fp4_small", s, Second<elt>{(const float*)ws, (elt*)yp, F, d},
                WRows4{w->down, w->down_s, d, F, 0}, d, offsets, st);
}

}  // namespace

// Few rows: up to 20 per expert on average (17 in fp16), and (x / E_l F d)^2 more with x =
// 5e7 in bf16 and 7e7 in fp16, 256 at most.  Below it these kernels are faster than the tiles,
// whose time hardly falls with the rows; above, more than 32 rows of an expert take a pass
// over its weights each, or more registers than leave two waves to a SIMD.  Both sides in us
// on an MI355X, forward, small against tiles: bf16, 128 experts of 2048 x 768 at 8 rows 88 / 121,
// at 16 96 / 121, at 20 124 / 122, at 24 146 / 123; 64 of them at 20 62 / 76, at 24 84 / 75; 16 of
// 4096 x 1024 at 20 53 / 60, at 25 68 / 60; 8 of 2048 x 1408 at 21 25 / 37, at 26 50 / 37; 8 of
// 2048 x 768 at 32 23 / 32, at 64 29 / 33; 4 of 640 x 384 at 256 15 / 26, at 400 29 / 23.  fp16: 128
// of 2048 x 768 at 16 136 / 151, at 20 183 / 152; 8 of 2048 x 1408 at 21 39 / 54, at 26 58 / 55; 8 of
// 2048 x 768 at 64 40 / 49, at 128 67 / 50.
// As for the 8-bit kernels, no block may need more than 8 passes with every token on one
// expert.
static int64_t most_mean(const moe_shape* s) {
  const bool bf16 = s->dtype == MOE_BF16;
  const double more = (bf16 ? 5e7 : 7e7) / ((double)s->E_l * (double)s->F * (double)s->d);
  return std::min<int64_t>(256, (bf16 ? 20 : 17) + (int64_t)std::min(256.0, more * more));
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
