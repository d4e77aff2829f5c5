// What the tile kernels of the 8-bit and 4-bit experts share: block and wave tile,
// copies to LDS, the persistent schedule, the 8-bit row operand and the epilogues of
// the forward.  Included by their two sources, each with copies of its own.
#pragma once

#include "moe_fp8.h"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

struct BF16 {
  typedef uint16_t elt;
  static constexpr bool WIDE = false;
};
struct F16 {
  typedef _Float16 elt;
  static constexpr bool WIDE = true;
};

constexpr int BM = 256, BN = 256, NT = 512;
constexpr int WGN = 2;                    // waves along N; 4 along M
constexpr int WTM = 64, WTN = 128;        // wave tile
constexpr int TM = WTM / 32, TN = WTN / 32;
constexpr int STAGE = BM * 128;           // bytes of one operand's stage
static_assert(BM == kTileM, "row tiles come from the dispatch plan");
// Epilogue staging: 16 rows x 128 columns of floats per wave, rows 132 apart, in
// the second stage's buffer and a little past it (the first takes the next tile's
// first stage meanwhile).
constexpr int EP_LD = 132;
constexpr int EP_WAVE = 16 * EP_LD * 4;
constexpr int SMEM = 2 * STAGE + NT / 64 * EP_WAVE;
static_assert(SMEM >= 4 * STAGE, "two stages of both operands");

__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p) {
  // raw buffer (stride 0); every offset used is a valid byte of the operand
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, 0x7fffffff, 0x00020000);
}

// A wave's copy of 8 tile rows straight to LDS (no registers in between): 1024
// consecutive bytes there; lane l's 16 bytes land at chunk l % 8 of row l / 8, so the
// lane reads the chunk that the swizzle puts there.  Inline assembly, since the
// compiler would wait for all copies ahead of every LDS read; stage_wait() does, once
// per stage.
__device__ __forceinline__ void copy_rows(uint32_t off, u32x4_t r, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(off), "s"(r), "s"(at)
               : "memory", "m0");
}

// One operand's 256 rows: 4 copies per wave and stage, 64 rows apart.
struct Load {
  static constexpr int CH = BM * 128 / (NT * 16), ROWS = BM / CH;
  u32x4_t rsrc;
  uint32_t off[CH];
  __device__ __forceinline__ void set_base(const void* base) {
    const uint64_t p = (uint64_t)base;
    // raw buffer (stride 0); every offset used is a valid byte of the operand
    rsrc = u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p),
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)) & 0xffffu,
                   0x7fffffffu, 0x00020000u};
  }
  // row r starts at offset(get(r)); get may read memory, for all rows at once
  template <class Get, class Offset>
  __device__ __forceinline__ void init(const void* base, Get get, Offset offset, int tid) {
    set_base(base);
    const int row = tid >> 3;  // rows 64 apart have the same swizzle
    int at[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) at[c] = get(c * ROWS + row);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      off[c] = (uint32_t)offset(at[c]) + (uint32_t)((tid & 7) ^ swz(row)) * 16u;
  }
  // block kt to the LDS address of this wave's first 1024 bytes; on = false
  // reads nothing (no byte of the buffer is in range; LDS gets zeros), without a
  // branch, past which the compiler would sink the MFMAs before it; below = false
  // reads nothing for the lower half of the rows
  __device__ __forceinline__ void copy(int kt, uint32_t lds, bool on = true,
                                       bool below = true) const {
    const u32x4_t r = {rsrc[0], rsrc[1], on ? rsrc[2] : 0u, rsrc[3]};
    const u32x4_t rb = {rsrc[0], rsrc[1], on && below ? rsrc[2] : 0u, rsrc[3]};
#pragma unroll
    for (int c = 0; c < CH; ++c)
      copy_rows(off[c], c < CH / 2 ? r : rb, (uint32_t)kt * 128u, lds + c * ROWS * 128);
  }
};
// Waits for the wave's memory operations.
__device__ __forceinline__ void stage_wait() {
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

__device__ __forceinline__ i32x8_t read_frag(const uint8_t* tile, int row0, int kk, int lane) {
  const int fr = lane & 31, hf = lane >> 5;
  const uint8_t* p = tile + (row0 + fr) * 128;
  const int s = swz(fr);
  const i32x4_t lo = *(const i32x4_t*)(p + (((kk * 4 + hf) ^ s) << 4));
  const i32x4_t hi = *(const i32x4_t*)(p + (((kk * 4 + 2 + hf) ^ s) << 4));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Wave and lane index next to their use (the lane index opaque to the optimiser,
// so that addresses made from it are not held across the main loop).
struct Pos {
  int lane, wave, wm, wn;
  static __device__ __forceinline__ Pos of() {
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(l));
    return {l, w, w / WGN, w % WGN};
  }
};

// The block of the reduction after k, around its end.
__device__ __forceinline__ int after(int k, int nk) { return k + 1 < nk ? k + 1 : 0; }

// Persistent schedule: the blocks form G = min(8, grid) groups by block % G
// (with G = 8 a group is one XCD); group g owns tiles [g*total/G, (g+1)*total/G),
// handed out to its blocks round robin.  Where the tiles of the last round leave half of
// the blocks without one, they are split in two units of 128 rows (one wave per SIMD
// computes, the others only copy): such a unit takes 0.84 of a tile's time, in fp16 0.72.
// 8 experts of 2048 x 1408, 192 rows each (88 tiles for 256 CUs), gate and up: 32 -> 27 us
// (fp16 51 -> 37).
struct Sched {
  int u, units, lo, whole, step;
  __device__ __forceinline__ explicit Sched(int total) {
    const int nb = gridDim.x, G = nb < 8 ? nb : 8;
    const int g = blockIdx.x % G;
    lo = (int)((long)total * g / G);
    const int n = (int)((long)total * (g + 1) / G) - lo;
    step = (nb - g + G - 1) / G;
    u = blockIdx.x / G;
    const int rest = n % step;
    whole = 2 * rest <= step ? n - rest : n;
    units = whole + 2 * (n - whole);
  }
  // Tile of unit u, and which half of its rows (-1: all).
  __device__ __forceinline__ int tile(int& half) const {
    const int h = u - whole;
    half = h < 0 ? -1 : h & 1;
    return lo + (h < 0 ? u : whole + h / 2);
  }
};

// (expert, first row, row end) of M-tile mt from LDS copies of the plan, in
// scalar registers: the expert is the number of later experts whose first tile is
// not past mt, counted by all lanes at once.
__device__ __forceinline__ void row_tile(const int* s_to, const int* s_off, int E_l, int mt,
                                         int& e, int& m0, int& m_end) {
  const int lane = (int)(threadIdx.x & 63);
  e = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = 1 + k * 64 + lane;
    e += (int)__popcll(__ballot(j < E_l && s_to[min(j, E_l)] <= mt));
  }
  m0 = __builtin_amdgcn_readfirstlane(s_off[e] + (mt - s_to[e]) * kTileM);
  m_end = __builtin_amdgcn_readfirstlane(s_off[e + 1]);
}

// The row operand of a product: rows of the dispatched matrix, or token rows
// gathered through the plan.
struct Rows {
  const uint8_t* q;
  const uint8_t* s;
  int k, ld;              // bytes per row, scale bytes per row
  const int32_t* xrows;   // NULL: dispatched rows
  int K;
  template <class Scales>
  __device__ __forceinline__ void init(int m0, int m_end, Load& la, Scales& sc, int tid) const {
    const Pos w = Pos::of();
    const int sr = w.wm * WTM + (w.lane & 31);
    if (xrows) {  // block-uniform
      int sp[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) sp[i] = xrows[min(m0 + sr + i * 32, m_end - 1)];
      la.init(q, [&](int r) { return xrows[min(m0 + r, m_end - 1)]; },
              [&](int pair) { return pair / K * k; }, tid);
      sc.ra = rsrc_of(s);
#pragma unroll
      for (int i = 0; i < TM; ++i) sc.oa[i] = (uint32_t)(sp[i] / K) * (uint32_t)ld;
    } else {
      la.init(q + (size_t)m0 * k, [&](int r) { return (min(m0 + r, m_end - 1) - m0) * k; },
              [](int at) { return at; }, tid);
      sc.ra = rsrc_of(s + (size_t)m0 * ld);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        sc.oa[i] = (uint32_t)(min(m0 + sr + i * 32, m_end - 1) - m0) * (uint32_t)ld;
    }
  }
};

// Rows 16 hb .. 16 hb + 15 of accumulator tile i of this wave (all four column tiles)
// as rows of floats in the wave's own LDS area (operations of one wave on LDS complete in
// order).
__device__ __forceinline__ const float* stage_rows(const f32x16_t (&acc)[TM][TN], int i, int hb,
                                                   uint8_t* smem, const Pos& w) {
  float* reg = reinterpret_cast<float*>(smem + 2 * STAGE + w.wave * EP_WAVE);
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int r = 0; r < 8; ++r)
      reg[(8 * (r >> 2) + 4 * (w.lane >> 5) + (r & 3)) * EP_LD + j * 32 + (w.lane & 31)] =
          acc[i][j][hb * 8 + r];
  return reg;
}
__device__ __forceinline__ void ld8(const float* p, float* f) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// Stores past L2 (non-temporal).
__device__ __forceinline__ void put16(void* p, const uint4& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), (u32x4_t*)p);
}
__device__ __forceinline__ void put8(void* p, const uint2& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x2_t, v), (u32x2_t*)p);
}
// Largest magnitude of eight values; NaN is passed over.
__device__ __forceinline__ float amax8(const float* f) {
  float m = fmaxf(fabsf(f[0]), fabsf(f[1]));
#pragma unroll
  for (int t = 2; t < 8; t += 2) m = fmaxf(fmaxf(fabsf(f[t]), fabsf(f[t + 1])), m);
  return m;
}
// Where a lane's values hold an infinity (m, their largest magnitude, says so),
// infinities are made NaN, which is what they are quantised to, and m the largest
// of the rest.
__device__ __forceinline__ float without_inf(float* f, float m) {
  if (__any(m == __builtin_inff())) {
    m = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      f[t] = finite_or_nan(f[t]);
      m = fmaxf(m, finite_abs(f[t]));
    }
  }
  return m;
}
__device__ __forceinline__ uint2 quant8(const float* f, float inv) {
  return uint2{pack_fp8(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
               pack_fp8(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
}
// Epilogue of the first product: h, a and the quantised a.  A tile is 128 outputs: the
// 128 tile columns of wave column wn are 64 gate rows and the 64 up rows of the same
// outputs.  The tile's outputs are one scale block per row; its two halves' largest
// magnitudes meet in LDS.
template <class E>
struct GateUpOut {
  typedef typename E::elt elt;
  elt *h, *a;
  uint8_t *aq, *as;
  int F, ldF;
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int m0, int m_end,
                                           int nt, uint8_t* smem, float* s_max,
                                           Arrived arrived) const {
    const Pos p = Pos::of();
    const int c = (p.lane & 7) * 8, j0 = nt * 128 + p.wn * 64 + c;
    float av[TM][4][8];
    const float* blk = nullptr;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if ((q & 1) == 0) blk = stage_rows(acc, i, q >> 1, smem, p);
        const int r = (q & 1) * 8 + (p.lane >> 3), tr = p.wm * WTM + i * 32 + (q >> 1) * 16 + r;
        float g[8], u[8];
        ld8(blk + r * EP_LD + c, g);
        ld8(blk + r * EP_LD + 64 + c, u);
#pragma unroll
        for (int t = 0; t < 8; ++t) av[i][q][t] = silu_fast(g[t]) * u[t];
        if (i == 0 && q == 0) arrived();
        if (m0 + tr < m_end) {
          const size_t row = (size_t)(m0 + tr);
          if (h) {
            put16(h + row * 2 * F + j0, Chunk<elt>::pack(g));
            put16(h + row * 2 * F + F + j0, Chunk<elt>::pack(u));
          }
          if (a) put16(a + row * F + j0, Chunk<elt>::pack(av[i][q]));
        }
        const float mx = lanes_max<8>(without_inf(av[i][q], amax8(av[i][q])));
        if ((p.lane & 7) == 0) s_max[p.wn * BM + tr] = mx;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int tr = p.wm * WTM + i * 32 + q * 8 + (p.lane >> 3);
        const int byte = fp8_scale_byte(fmaxf(s_max[tr], s_max[BM + tr]));
        if (m0 + tr < m_end) {
          const size_t row = (size_t)(m0 + tr);
          put8(aq + row * F + j0, quant8(av[i][q], fp8_inv_scale(byte)));
          if (p.wn == 0 && (p.lane & 7) == 0) as[row * ldF + nt] = (uint8_t)byte;
        }
      }
  }
};

// Epilogue of a product whose result [rows][n] is stored as it is.
template <class E>
struct PlainOut {
  typedef typename E::elt elt;
  elt* out;
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int n, int m0,
                                           int m_end, int nt, uint8_t* smem,
                                           Arrived arrived) const {
    const Pos p = Pos::of();
    const int cb = nt * BN + p.wn * WTN, c = (p.lane & 15) * 8;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const float* blk = stage_rows(acc, i, hb, smem, p);
        if (i + hb == 0) arrived();
        if (cb >= n) continue;  // wave-uniform; n is a multiple of 128
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = q * 4 + (p.lane >> 4), row = m0 + p.wm * WTM + i * 32 + hb * 16 + r;
          float f[8];
          ld8(blk + r * EP_LD + c, f);
          if (row < m_end) put16(out + (size_t)row * n + cb + c, Chunk<elt>::pack(f));
        }
      }
  }
};

inline int max_row_tiles(const moe_shape* s) {
  return (int)((s->T * s->K + s->E_l * (int64_t)(kTileM - 1)) / kTileM);
}

// One block per CU of the current device (at most `tiles`).
inline int persistent_grid(long tiles) {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  return (int)(tiles < n ? (tiles > 0 ? tiles : 1) : n);
}

struct Ws {
  uint8_t *q, *s;
  Ws(const moe_shape* sh, void* ws, int64_t cols)
      : q((uint8_t*)ws), s(q + align_up((size_t)(sh->T * sh->K * cols), 256)) {}
};

}  // namespace
}  // namespace moe
