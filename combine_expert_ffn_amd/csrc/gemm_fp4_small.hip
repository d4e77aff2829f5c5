// The products of 8-bit rows with 4-bit expert weights for few rows per expert
// (decoding, short prompts): one pass over the active experts' weights, so what bounds
// them is how fast those stream from memory.  A block takes groups of 16 S weight rows (of
// both halves for gate and up) of one expert; its four waves share the reduction by 256
// values (128 bytes of a weight row; by 128 where there are 512 at most), the weights go
// straight to registers and are the M side of the MFMAs, up to 16 G token rows the N side.
// bf16 data: v_mfma_scale_f32_16x16x128_f8f6f4 on the codes as they are, with the scales
// as bytes of the lanes.  It cuts each of eight consecutive products 13 bits below the
// largest of them, as the tiles do, which is chosen for time: with the products exact, as
// below for fp16, one token takes 13.0 us for 11.7, 64 tokens 83 for 79, 256 tokens 126 for 85
// (128 experts of 2048 x 768).  h and a keep the error of their rounding to bf16 (1.66e-3).
// Of a's values next to the border between two e4m3 values, 0.05 % of all, some fall on the
// other side, no further from a (quantised, a is 2.65e-2 off either way); y_p, 1.66e-3 from
// the definition with none of them, is 1.74e-3 at 256 tokens, up to 1.98e-3 at 16.
// fp16 data: codes and rows widened to bf16 with their scales (exact) for 16 x 16 x 32 bf16
// MFMAs.
// 128 experts of 2048 x 768, bf16, both products: one token (8 experts, 20 MB) 11.8 us, two
// launches of 6.5 and 5.0 whose chains of latencies (plan, weights, sum over waves) bound
// them; 64 tokens (316 MB) 75 us, 4.2 TB/s of weights; 256 tokens 85.
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

// A lane's codes of NW sets of 16 weight rows, values 32 (lane / 16) ..+31 of UB blocks of
// 128, and the scales of all four lanes of the row (byte lane / 16 of a word is its own): a
// byte of each lane's own would be a request of its own, 20 % of the time.
template <int S, int NW, int UB, bool PAIR>
struct Weights {
  i32x4_t v[NW][UB];
  uint32_t scale[NW][UB];
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
      const uint8_t* b = s + to * (W.k / 32) + kb * 4;
      v[w][0] = *(const i32x4_t*)p;
      if constexpr (UB == 1) {
        scale[w][0] = *(const uint32_t*)b;
        continue;
      }
      v[w][UB - 1] = *(const i32x4_t*)(p + (two ? 64 : 0));
      if constexpr (PAIR) {
        const u32x2_t x = *(const u32x2_t*)(b - (two ? 0 : 4));
        scale[w][0] = two ? x[0] : x[1];
        scale[w][UB - 1] = x[1];
      } else {
        scale[w][0] = *(const uint32_t*)b;
        scale[w][UB - 1] = *(const uint32_t*)(b + (two ? 4 : 0));
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

// Sum over the lanes up to this one.
__device__ __forceinline__ int sum_to_lane(int v) {
  auto add = [&](int x) { v += x; };
  add(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));   // within rows of 16: from 1,
  add(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));   // 2,
  add(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));   // 4
  add(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));   // and 8 lanes below
  add(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));  // lane 15 and 47 to the next row
  add(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));  // lane 31 to the upper half
  return v;
}

// Pass number `slot` over at most ROWS rows of one expert, the experts in order; false if
// there are fewer.  Every wave finds it by itself.
template <int ROWS>
__device__ __forceinline__ bool nth_pass(const int32_t* offsets, int E_l, int slot, int& e,
                                         int& r0, int& m_end) {
  const int lane = (int)(threadIdx.x & 63);
  int lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = min(k * 64 + lane, E_l - 1);
    lo[k] = offsets[j];
    hi[k] = offsets[j + 1];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k * 64 >= E_l) break;  // uniform
    const int n = k * 64 + lane < E_l ? (hi[k] - lo[k] + ROWS - 1) / ROWS : 0;
    const uint64_t some = __ballot(n > 0), many = __ballot(n > 1);
    int upto, total;  // passes up to this lane's expert, and of all 64
    if (many == 0) {  // wave-uniform: most often, and the shorter way
      upto = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(some >> 32),
                                            __builtin_amdgcn_mbcnt_lo((uint32_t)some, 0u)) + n;
      total = (int)__popcll(some);
    } else {
      upto = sum_to_lane(n);
      total = __builtin_amdgcn_readlane(upto, 63);
    }
    if (slot < total) {  // wave-uniform
      const int l = __builtin_ctzll(__ballot(slot < upto));
      const int before = __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l);
      e = k * 64 + l;
      r0 = __builtin_amdgcn_readlane(lo[k], l) + (slot - before) * ROWS;
      m_end = __builtin_amdgcn_readlane(hi[k], l);
      return true;
    }
    slot -= total;
  }
  return false;
}

// A block takes `span` groups of 16 S output columns for a pass, 16 G rows of one expert.  Its
// four waves take the units of the reduction (UB blocks of 128) in turn, and their sums meet
// in LDS for each group.  With UW units to a wave at most (0: any number) it keeps its part of
// the rows in registers over the groups: read, and for the second product quantised, once.
// With all of a wave's rows held, each of BUF buffers is filled with the weights of the unit that
// will use it next as soon as its last ones are used.  Where a wave has more units (UW = 0), or
// one of two, the second buffer's weights are moved to the first, which waits for them, and with
// UW = 0 a unit's rows are read, and for the second product quantised, where they are used, with no
// load of them in flight: 2.5 TB/s of weights (16 experts of 4096 x 1024 at 8 rows, 39 us) where
// held rows give 4.2.
template <int S, int G, int UW, int UB, bool LOOP, class Op>
__global__ __launch_bounds__(64 * WAVES) void fp4_small_kernel(
    Op op, WRows4 W, const int32_t* __restrict__ offsets, int E_l, int groups, int span,
    int most) {
  constexpr int NW = Op::H * S, HELD = UW > 0 ? UW : 1, BUF = 2;
  constexpr bool WIDE = Op::WIDE;
  __shared__ Reduce<NW, G> red;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, part = lane >> 4;
  const int c_first = blockIdx.x * span, c_end = min(c_first + span, groups);
  const int kbs = W.k / 128, units = (kbs + UB - 1) / UB;
  const int n = (units - wave + WAVES - 1) / WAVES;  // of this wave
  auto block = [&](int i) { return (wave + i * WAVES) * UB; };  // the first of unit i
  int e, r0, m_end;
  // no load has more than `most` passes; without LOOP the grid has them all
  for (int slot = blockIdx.y; slot < most && nth_pass<16 * G>(offsets, E_l, slot, e, r0, m_end);
       slot += gridDim.y) {  // block-uniform
    const size_t row0 = (size_t)e * W.n + (lane & 15);
    const uint8_t* q = W.q + row0 * (W.k / 2) + part * 16;
    const uint8_t* s = W.s + row0 * (W.k / 32);
    Weights<S, NW, UB, (UW > 0)> buf[BUF];
    // unit i of group c, if there is such a group
    auto fetch = [&](auto& w, int c, int i) {
      if (c < c_end)  // block-uniform
        w.load(W, q + (size_t)(c * 16 * S) * (W.k / 2), s + (size_t)(c * 16 * S) * (W.k / 32),
               block(i));
    };
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
    Tokens<WIDE> held[HELD][UB][G];
    auto hold = [&](Tokens<WIDE> (&to)[UB][G], int kb) {
#pragma unroll
      for (int h = 0; h < UB; ++h)
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
    auto unit = [&](auto& w, int i, const Tokens<WIDE> (&b)[UB][G]) {
#pragma unroll
      for (int h = 0; h < UB; ++h) {
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
    if constexpr (!LOOP) break;
  }
}

// Blocks that share the groups where the routing is even: two per CU; and in all, those that
// only a skewed load needs, which leave at once in others.
constexpr int kBlocks = 512, kMostBlocks = 4096;

// Whether the kernel's registers, as compiled, leave two waves to a SIMD.  (The second product
// never meets S = 1 with 64-row passes: in Shape, S = 1 says blocks * cdiv(rows, 16) < 1024, G = 4
// blocks * cdiv(rows, 64) >= 512 and rows > 32, so cdiv(rows, 16) < 2 cdiv(rows, 64), which no
// rows > 16 fulfil.)
template <class Op>
constexpr bool two_waves(int S, int G, int UW, int UB) {
  if (UB == 1) return Op::H == 2 || G < 4 || (S == 4 && !Op::WIDE);
  if (Op::H == 2) return G < 4 || UW == 0 || (UW == 1 && !Op::WIDE);
  return G == 1 || (G == 2 && (S == 1 || UW > 0));
}
// The units of a wave whose rows it keeps in registers, if that is all of them, else 0.
template <class Op>
int held_units(int G, int k) {
  const int per_wave = (k + 256 * WAVES - 1) / (256 * WAVES);
  return per_wave <= (Op::WIDE && G > 1 ? 1 : 2) ? per_wave : 0;
}
// Token groups of a pass over a reduction of k: Shape's, halved until two waves fit a SIMD.  In
// us, one wave / halved: 8 of 64 experts of 2048 x 1408 at 23 rows 37 / 31 (first product) and
// 37 / 29 (second), 8 of 1152 x 1280 at 32 rows 25.8 / 22.5; fp16: 16 of 1024 x 768 at 32 rows
// 25.4 / 21.7, 8 of 2048 x 384 at 50 rows 20.3 / 18.8, 8 of 4096 x 2048 at 18 rows 62 / 54.  It
// costs a little where 32-row passes of the second product become 16: 16 of 2048 x 4096 at 17
// rows 87 / 96, but 8 of 256 of 7168 x 2304 at 20 rows 170 / 152.  Halving everywhere would be
// slower where 64-row passes leave two waves: 128 of 128 x 768 at 32 rows 26 / 33.
template <class Op>
int pass_groups(const Shape& sh, int k) {
  int G = sh.G;
  while (G > 1 && !two_waves<Op>(sh.S, G, k <= 128 * WAVES ? 1 : held_units<Op>(G, k),
                                 k <= 128 * WAVES ? 1 : 2))
    G /= 2;
  return G;
}

template <class Op>
int launch(const char* name, const moe_shape* s, const Op& op, const WRows4& W, int cols,
           const int32_t* offsets, hipStream_t st) {
  const Shape sh(s, cols, Op::H == 1);
  const int groups = (int)sh.grid.x, G_run = pass_groups<Op>(sh, W.k);
  // passes of an even load: experts that have rows, times the passes over what most have at
  // most (as in Shape; with the mean alone 25 us instead of 23, 8 experts of 2048 x 768, 32 rows)
  const int64_t pairs = s->T * s->K, rows = 16 * G_run;
  const double mean = (double)pairs / (double)s->E;
  const double passes =
      std::max(1.0, s->E_l * -expm1(-mean)) * ceil((mean + 2 * sqrt(mean)) / (double)rows);
  // and of any load, tokens that name an expert more than once among them
  const int64_t slots = std::max<int64_t>(1, std::min(pairs, s->E_l));
  const int64_t most = slots + pairs / rows;
  // A grid of fewer passes, whose blocks take further ones, where the pass is of 16 rows and
  // there may be more than 24.  The loop costs 30 registers and often a wave per SIMD, in us
  // with / without: one token, 128 experts of 2048 x 768 12.0 / 11.8, 100 of 8 of 64 experts
  // of 2048 x 1408 19.5 / 18.9, 200 of them (32 rows) 27.4 / 23.6; but the weights of many
  // experts stream better with it: 64 tokens, 128 experts 75 / 79, 8 of them 40 / 42.
  const bool loop = G_run == 1 && most > 24;
  const int64_t parts = std::min<int64_t>(
      {(int64_t)(kBlocks / passes + 0.5), groups, loop ? groups : kMostBlocks / most});
  const int span = (int)cdiv(groups, std::max<int64_t>(1, parts));
  const int64_t x = cdiv(groups, span);
  const int64_t y =
      loop ? std::min(most, std::max(2 * (int64_t)ceil(passes), cdiv(1024, x))) : most;
  const dim3 grid((unsigned)x, (unsigned)y);
  const int held = held_units<Op>(G_run, W.k);
  auto go = [&](auto kernel) {
    MOE_LAUNCH(name, st, kernel<<<grid, 64 * WAVES, 0, st>>>(op, W, offsets, (int)s->E_l, groups,
                                                             span, (int)most));
    return check_launch(name);
  };
  auto by_rows = [&](auto S_) {
    constexpr int S = decltype(S_)::value;
    auto by_units = [&](auto G_, auto loop_) {
      constexpr int G = decltype(G_)::value;
      constexpr bool LOOP = decltype(loop_)::value;
      constexpr int MOST = Op::WIDE && G > 1 ? 1 : 2;
      // pass_groups took none of the kernels that are left out
      if constexpr (two_waves<Op>(S, G, 1, 1))
        // one block of 128 to a wave where that is all
        if (W.k <= 128 * WAVES) return go(fp4_small_kernel<S, G, 1, 1, LOOP, Op>);
      if constexpr (two_waves<Op>(S, G, 0, 2))
        if (held == 0) return go(fp4_small_kernel<S, G, 0, 2, LOOP, Op>);
      if constexpr (MOST == 2 && two_waves<Op>(S, G, 2, 2))
        if (held == 2) return go(fp4_small_kernel<S, G, 2, 2, LOOP, Op>);
      if constexpr (two_waves<Op>(S, G, 1, 2))
        if (held == 1) return go(fp4_small_kernel<S, G, 1, 2, LOOP, Op>);
      return set_error(MOE_ERR_UNSUPPORTED, "%s: no kernel", name);
    };
    typedef std::integral_constant<int, 1> One;
    if (G_run == 4) return by_units(std::integral_constant<int, 4>{}, std::false_type{});
    if (G_run == 2) return by_units(std::integral_constant<int, 2>{}, std::false_type{});
    if (loop) return by_units(One{}, std::true_type{});
    return by_units(One{}, std::false_type{});
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
// whose time hardly falls with the rows; above, an expert's rows take several passes, each over
// its weights again.  Both sides in us on an MI355X, forward, small against tiles: bf16, 128
// experts of 2048 x 768 at 8 rows 82 / 117, at 16 85 / 117, at 20 118 / 119, at 24 129 / 119; 64
// of them at 20 49 / 74, at 24 72 / 75; 16 of 4096 x 1024 at 20 49 / 60, at 25 59 / 60, at 32 65 /
// 60; 8 of 2048 x 1408 at 21 24 / 37, at 26 28 / 38, at 36 34 / 38; 8 of 2048 x 768 at 32 23 / 32,
// at 64 28 / 33; 8 of 1024 x 256 at 184 18 / 24; 4 of 640 x 384 at 256 14 / 25.  fp16: 128 of 2048
// x 768 at 16 124 / 150, at 20 165 / 151; 8 of 2048 x 1408 at 26 35 / 54; 8 of 2048 x 768 at 64
// 42 / 49, at 128 59 / 50.
// These are even loads, which for few experts would bear a higher border.  It stays below them
// because a fuller expert takes more passes, each over its weights again from L2, and the
// loads are not known here: 128 experts of 2048 x 768, Zipf 1.1, at 4 rows 62 / 73, at 16 83 /
// 99; 8 of 64 of 2048 x 1408 at 9 45 / 39, at 19 64 / 40, at 23 81 / 41; one of 512 of 2048 x
// 768 at 16 (the fullest, 950 rows) 85 / 34 where its even load is 10 / 30.  So that
// it stays within a few times the tiles' time, no expert may take more than 64 passes of
// Shape's rows with every token once.  (Passes that pass_groups halves count as one: with them
// counted apart, even loads would go to slower tiles, 128 experts of 128 x 384, fp16, at 38 rows
// 18 / 32, 256 of 512 of 128 x 1408 at 10 57 / 119, 32 of 256 of 1920 x 256 at 25 23 / 41; the most
// skewed to faster ones, 16 of 512 of 1152 x 2816, Zipf 1.1, 501 / 158.)
static int64_t most_mean(const moe_shape* s) {
  const bool bf16 = s->dtype == MOE_BF16;
  const double more = (bf16 ? 5e7 : 7e7) / ((double)s->E_l * (double)s->F * (double)s->d);
  return std::min<int64_t>(256, (bf16 ? 20 : 17) + (int64_t)std::min(256.0, more * more));
}
bool fp4_small(const moe_shape* s) {
  const int64_t rows = 16 * std::min(Shape(s, (int)s->F, false).G, Shape(s, (int)s->d, true).G);
  return cdiv(s->T * s->K, s->E) <= most_mean(s) && cdiv(s->T, rows) <= 64;
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
