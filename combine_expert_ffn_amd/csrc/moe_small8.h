// What the few-row kernels of the 8-bit and 4-bit experts share: the experts with
// rows, 8-bit rows as MFMA operands, the sum over a block's waves, the SwiGLU epilogue
// and the launch shape.  Included by their two sources, each with copies of its own.
#pragma once

#include "moe_fp8.h"

#include <math.h>

#include <algorithm>

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int WAVES = 4;

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

// A lane's 32 floats of a block of 128 (lanes 16 apart hold the rest), quantised to 8 bits.
__device__ __forceinline__ Block quantised(const float* f) {
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
}

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

}  // namespace
}  // namespace moe
