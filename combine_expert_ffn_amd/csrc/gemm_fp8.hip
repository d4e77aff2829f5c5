// Grouped expert products on 8-bit operands (gfx950): e4m3 values with a
// power-of-two scale per 128 along the reduction, float32 accumulation.
//
// bf16 data: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies each lane's 32 values by
// a scale byte of that lane's own, so the block scales of both operands enter
// without a vector instruction.  It aligns eight consecutive products (8 bytes of a
// lane) to the largest of them and cuts each 13 bits below it; the groups' sums
// and the accumulator add up in float32 (measured with single products; the unscaled
// e4m3 instruction does the same).  Choice: on normal operands the sums are 1.5e-5
// off, rms, where their bf16 rounding is 1.66e-3.  It shows in the second product
// only, through values of a or dh next to a rounding border of e4m3: 0.16 % and 0.09 %
// of them become the neighbouring value, which is as near to the unrounded one, and
// y_p and dx_p are 2.02e-3 and 1.89e-3 from the float64 definition instead of 1.66e-3.
// With exact products (as for fp16 below) 128 experts of 2048 x 768 take 791 + 432 us
// forward and 581 + 748 us backward instead of 521 + 287 and 458 + 463; the 16-bit experts'
// products take 790 + 468 and 492 + 795.
// fp16 data, whose results keep 11 bits: the values are widened to bf16 with their
// scale (exact, one instruction per two) and multiplied by
// v_mfma_f32_32x32x16_bf16 at half the rate: h 2.07e-4 and y_p 2.2e-4 off, their own rounding.
// A stage of the reduction is one block of 128 values = 128 bytes per row.
//  * block tile 256 x 256, 8 waves (2 per SIMD) of 64 x 128 = 2 x 4 MFMA tiles;
//    a wave's 128 columns are whole scale blocks of the output, so the fused
//    quantisation needs at most one exchange with another wave;
//  * two LDS stages of [rows][128 bytes], the 16-byte chunk index XOR-swizzled
//    by the row; a lane's 32 bytes are the chunks 2t + lane / 32 of two
//    consecutive pairs t, the same for both operands (the order of the values
//    within a block does not change its sum);
//  * stages are copied from memory straight to LDS, one ahead; 128-byte rows, since
//    64-byte pieces halve the rate of L2 (17 against 34 TB/s);
//  * outputs are staged through LDS to rows of 128 bytes or more and stored past
//    L2 (non-temporal), where they would push out the operands that 32 CUs share;
//  * persistent grid over the dispatch plan's row tiles, one range per XCD.
// What bounds it: moving operands to LDS and results out.  128 experts of 2048 x 768,
// 131072 rows, bf16, by the library's kernel timer: gate and up 509 us (1.62 PFLOP/s), down 289
// (1.43), activation gradient 450 (which also reads h) and input gradient 457 (1.80); the matrix
// cores are busy 43, 37, 24 and 47 % of that, and memory reads are 2.5, 1.1, 1.7 and 2.1 times
// the operands.  In variants with parts left out, gate and up / down: fragment reads and MFMAs
// alone 300 / 168 us, copies alone 319 / 160 (184 / 106 where L2 has all), everything but
// the stores 452 / 225.  A wave's memory operations complete in order, so a tile's stores (at
// the write rate of HBM) add up with the next one's copies.
// Slower: two blocks of half the size per CU, four waves of 128 x 128, rings of 64-byte
// slices, four waves that copy while the other four store.
#include "moe_fp8.h"

#include <algorithm>

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
// The same of rows k bytes apart, whose offsets are one vector register and scalars.
// half: only the first 128 of the 256 rows exist (they are read twice).
struct LoadRows {
  static constexpr int CH = BM * 128 / (NT * 16), ROWS = BM / CH;
  u32x4_t rsrc;
  uint32_t off, step, upper;
  __device__ __forceinline__ void init(const uint8_t* base, int k, bool half, int tid) {
    Load l;
    l.set_base(base);
    rsrc = l.rsrc;
    off = (uint32_t)((tid >> 3) * k) + (uint32_t)((tid & 7) ^ swz(tid >> 3)) * 16u;
    step = (uint32_t)__builtin_amdgcn_readfirstlane(ROWS * k);
    upper = (uint32_t)__builtin_amdgcn_readfirstlane(half ? 0 : 128 * k);
  }
  __device__ __forceinline__ void copy(int kt, uint32_t lds, bool on = true) const {
    const u32x4_t r = {rsrc[0], rsrc[1], on ? rsrc[2] : 0u, rsrc[3]};
#pragma unroll
    for (int c = 0; c < CH; ++c)
      copy_rows(off, r, (uint32_t)kt * 128u + (c % (CH / 2)) * step + (c / (CH / 2)) * upper,
                lds + c * ROWS * 128);
  }
};

// Waits for the wave's memory operations.
__device__ __forceinline__ void stage_wait() {
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// Scale bytes of four stages at a time: of the wave's rows (one per lane and
// 32-row tile) and of the two 64-column halves of its columns.
struct Scales {
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t oa[TM], ob[2];
  uint32_t a[TM], b[2], an[TM], bn[2];
  __device__ __forceinline__ void fetch(int k, uint32_t (&ta)[TM], uint32_t (&tb)[2]) const {
#pragma unroll
    for (int i = 0; i < TM; ++i) ta[i] = __builtin_amdgcn_raw_buffer_load_b32(ra, (int)oa[i], k, 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) tb[h] = __builtin_amdgcn_raw_buffer_load_b32(rb, (int)ob[h], k, 0);
  }
  // the group of block k now, and the one after it
  __device__ __forceinline__ void start(int k, int nk) {
    fetch(k & ~3, a, b);
    fetch((k | 3) + 1 < nk ? (k | 3) + 1 : 0, an, bn);
  }
  // both are here
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(a[i]), "+v"(an[i]));
#pragma unroll
    for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(b[h]), "+v"(bn[h]));
  }
  // A move that the compiler cannot fold: else it moves the values of the next
  // fetch instead, and waits for them.
  static __device__ __forceinline__ uint32_t moved(uint32_t v) {
    uint32_t r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
    return r;
  }
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = moved(an[i]);
    b[0] = moved(bn[0]);
    b[1] = moved(bn[1]);
  }
};

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

// One 64-deep slice: the MFMAs of the wave on a and b, and beside them the reads
// of the next slice's fragments (an into its own registers, b's four one by one
// into those the MFMAs are done with).
template <bool WIDE>
__device__ __forceinline__ void slice(const i32x8_t (&a)[TM], i32x8_t (&an)[TM], i32x8_t (&b)[TN],
                                      const uint32_t (&sa)[TM], const uint32_t (&sb)[2],
                                      f32x16_t (&acc)[TM][TN], const uint8_t* next, int kk,
                                      const Pos& w) {
  auto next_b = [&](int j) {
    return read_frag(next + STAGE, w.wn * WTN + j * 32, kk, w.lane);
  };
  auto next_a = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i) an[i] = read_frag(next, w.wm * WTM + i * 32, kk, w.lane);
  };
  if constexpr (WIDE) {
    float fa[TM], fb[2];
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[i] = fp8_scale_value((int)(sa[i] & 255u));
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[j] = fp8_scale_value((int)(sb[j] & 255u));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8_t aw[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) aw[i] = widen(a[i][2 * q], a[i][2 * q + 1], fa[i]);
      if (q == 2) next_a();
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bf16x8_t bw = widen(b[j][2 * q], b[j][2 * q + 1], fb[j >> 1]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(aw[i], bw, acc[i][j], 0, 0, 0);
        if (q == 3) b[j] = next_b(j);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    i32x8_t bn[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (j == 0) next_a();
      if (j > 0) bn[j - 1] = next_b(j - 1);
      if (j == TN - 1) bn[j] = next_b(j);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            a[i], b[j], acc[i][j], 0, 0, 0, (int)sa[i], 0, (int)sb[j >> 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = bn[j];
  }
}

// The block of the reduction after k, around its end.
__device__ __forceinline__ int after(int k, int nk) { return k + 1 < nk ? k + 1 : 0; }

// The reduction over nk blocks from block k0 around (PlainOp::ROTATE); the first stage is in the first
// buffer, the second is being copied to the other.  below: the tile has rows past
// the first 128.  idle: the wave's 64 rows lie past the tile's last, so it only copies (2 %
// of the time at 1024 rows per expert, whose last tiles are half empty).
template <bool WIDE, class LoadB>
__device__ __forceinline__ void mainloop(const Load& la, const LoadB& lb, Scales& sc, int nk,
                                         int k0, uint8_t* smem, uint32_t lds, bool below, bool idle,
                                         f32x16_t (&acc)[TM][TN]) {
  const Pos w = Pos::of();
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  int kb = k0;                        // the stage's block of the reduction
  int kc = after(after(k0, nk), nk);  // the block that is copied next
  if (idle) {  // wave-uniform: only its part of the copies, and the barriers
    for (int kt = 0; kt < nk; ++kt) {
      const int odd = kt & 1;
      stage_wait();
      __syncthreads();
      la.copy(kc, lds + odd * 2 * STAGE, kt + 2 < nk, below);
      lb.copy(kc, lds + odd * 2 * STAGE + STAGE, kt + 2 < nk);
      kc = after(kc, nk);
    }
    stage_wait();
    __syncthreads();
    return;
  }
  i32x8_t a0[TM], a1[TM], b[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) a0[i] = read_frag(smem, w.wm * WTM + i * 32, 0, w.lane);
#pragma unroll
  for (int j = 0; j < TN; ++j) b[j] = read_frag(smem + STAGE, w.wn * WTN + j * 32, 0, w.lane);
  for (int kt = 0; kt < nk;) {
    // the stages that share a register of scale bytes
    const int end = min(kt + min(4 - (kb & 3), nk - kb), nk);
    for (; kt < end; ++kt, ++kb) {
      const int odd = kt & 1;
      const uint8_t* cur = smem + odd * 2 * STAGE;
      const uint8_t* nxt = smem + (odd ^ 1) * 2 * STAGE;
      const int sh = (kb & 3) * 8;
      uint32_t sa[TM], sb[2];
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = sc.a[i] >> sh;
      sb[0] = sc.b[0] >> sh;
      sb[1] = sc.b[1] >> sh;
      __builtin_amdgcn_sched_barrier(0);
      slice<WIDE>(a0, a1, b, sa, sb, acc, cur, 1, w);
      stage_wait();
      __syncthreads();
      la.copy(kc, lds + odd * 2 * STAGE, kt + 2 < nk, below);
      lb.copy(kc, lds + odd * 2 * STAGE + STAGE, kt + 2 < nk);
      kc = after(kc, nk);
      __builtin_amdgcn_sched_barrier(0);
      slice<WIDE>(a1, a0, b, sa, sb, acc, nxt, 0, w);
    }
    if (kb == nk) kb = 0;
    sc.next();
    __builtin_amdgcn_sched_barrier(0);
    sc.fetch((kb | 3) + 1 < nk ? (kb | 3) + 1 : 0, sc.an, sc.bn);
    __builtin_amdgcn_sched_barrier(0);
  }
  stage_wait();  // the copies past the last stage write zeros to LDS
  __syncthreads();
}

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

// The weight operand [E_l][n][k] with scales [E_l][n / 128][ld].
struct Cols {
  const uint8_t* q;
  const uint8_t* s;
  int n, k, ld;
  // columns nt * 256 ..+255; n is a multiple of 128, so the last tile may be half
  __device__ __forceinline__ void init(int e, int nt, LoadRows& lb, Scales& sc, int tid) const {
    const Pos w = Pos::of();
    lb.init(q + ((size_t)e * n + (size_t)nt * BN) * k, k, nt * BN + 128 >= n, tid);
    sc.rb = rsrc_of(s + (size_t)e * (n / 128) * ld);
    sc.ob[0] = sc.ob[1] = (uint32_t)(min(nt * 2 + w.wn, n / 128 - 1) * ld);
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
// forward GEMM1: [g, u] = x^ . W_gu^[e]^T, a = silu(g) u, quantised for GEMM2.
// A tile is 128 outputs: the 128 tile columns of wave column wn are 64 gate
// rows and the 64 up rows of the same outputs.  The tile's outputs are one
// scale block per row; its two halves' largest magnitudes meet in LDS.
template <class E>
struct GateUpOp {
  typedef E type;
  typedef typename E::elt elt;
  Rows x;
  Cols w;  // n = 2F
  elt *h, *a;
  uint8_t *aq, *as;
  int F, ldF;
  static constexpr bool ROTATE = false;
  __device__ __forceinline__ int stages() const { return x.k / 128; }
  typedef Load LoadB;
  __device__ __forceinline__ void init(int e, int m0, int m_end, int nt, Load& la, LoadB& lb,
                                       Scales& sc, int tid) const {
    x.init(m0, m_end, la, sc, tid);
    lb.init(w.q + (size_t)e * w.n * w.k,
            [&](int c) {
              const int j = nt * 128 + (c >> 7) * 64 + (c & 63);
              return (((c >> 6) & 1) * F + j) * w.k;
            },
            [](int at) { return at; }, tid);
    sc.rb = rsrc_of(w.s + (size_t)e * (w.n / 128) * w.ld);
    sc.ob[0] = (uint32_t)(nt * w.ld);
    sc.ob[1] = (uint32_t)((F / 128 + nt) * w.ld);
  }
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

// Products whose result is stored as it is: forward GEMM2 (y_p = a^ . W_down^T) and
// the second of the dgrad (dx_p = dh^ . W_gu, with the transposed weights).
// ROTATE: the blocks of an XCD start at different blocks of the reduction.  Its CUs
// work on consecutive tiles; in step, all that share a panel ask for its lines at once
// and wait for memory together, started apart one fetches a line and the others find
// it in L2.  bf16, 131072 rows, us in step and rotated, down and input gradient: 64 experts of
// 2048 x 768 320 / 287 and 486 / 439, of 4096 x 1024 377 / 350 and 613 / 562, of 2048 x 1408
// 462 / 426 and 780 / 740, of 1024 x 512 126 / 116 and 183 / 171, of 1024 x 1024 185 / 179 and
// 297 / 288; fp16 within 3 % either way.  The products with SwiGLU epilogues gain nothing (gate
// and up, activation gradient: 491 / 478 and 438 / 440, 614 / 610 and 458 / 463, 870 / 868 and
// 814 / 831, 194 / 194 and 255 / 252, 395 / 396 and 469 / 463).  A row's float32 sum thus starts
// where its CU does, and its last bits with it; a start by the column tile alone would not
// depend on the row's place, and takes 312 and 478 us for 128 experts instead of 287 and 457.
template <class E>
struct PlainOp {
  typedef E type;
  typedef typename E::elt elt;
  Rows x;
  Cols w;
  elt* out;  // [rows][w.n]
  static constexpr bool ROTATE = true;
  __device__ __forceinline__ int stages() const { return x.k / 128; }
  typedef LoadRows LoadB;
  __device__ __forceinline__ void init(int e, int m0, int m_end, int nt, Load& la, LoadB& lb,
                                       Scales& sc, int tid) const {
    x.init(m0, m_end, la, sc, tid);
    w.init(e, nt, lb, sc, tid);
  }
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int m0, int m_end,
                                           int nt, uint8_t* smem, float*, Arrived arrived) const {
    const Pos p = Pos::of();
    const int cb = nt * BN + p.wn * WTN, c = (p.lane & 15) * 8;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const float* blk = stage_rows(acc, i, hb, smem, p);
        if (i + hb == 0) arrived();
        if (cb >= w.n) continue;  // wave-uniform; n is a multiple of 128
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = q * 4 + (p.lane >> 4), row = m0 + p.wm * WTM + i * 32 + hb * 16 + r;
          float f[8];
          ld8(blk + r * EP_LD + c, f);
          if (row < m_end) put16(out + (size_t)row * w.n + cb + c, Chunk<elt>::pack(f));
        }
      }
  }
};

// dgrad GEMM A: da = [gate] d^ . W_down^[e] with the SwiGLU backward; dg and du of a
// wave's 128 columns are one scale block each.
template <class E>
struct DgradActOp {
  typedef E type;
  typedef typename E::elt elt;
  Rows x;
  Cols w;  // W_down transposed, n = F
  const elt* h;
  const float* gates;  // with x.xrows
  elt *dh, *ag;
  uint8_t *dq, *ds;  // [rows][2F], [rows][ld2F]
  int F, ld2F;
  static constexpr bool ROTATE = false;
  __device__ __forceinline__ int stages() const { return x.k / 128; }
  typedef LoadRows LoadB;
  __device__ __forceinline__ void init(int e, int m0, int m_end, int nt, Load& la, LoadB& lb,
                                       Scales& sc, int tid) const {
    x.init(m0, m_end, la, sc, tid);
    w.init(e, nt, lb, sc, tid);
  }
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int m0, int m_end,
                                           int nt, uint8_t* smem, float*, Arrived arrived) const {
    const Pos p = Pos::of();
    const int cb = nt * BN + p.wn * WTN, c = (p.lane & 15) * 8;
    const int last = m_end - 1, r0 = m0 + p.wm * WTM + (p.lane >> 4);
    arrived();
    if (cb >= F) return;  // wave-uniform; F is a multiple of 128
    // h and the gates of 16 rows, loaded one half tile ahead of their use (a wave's
    // loads wait for its earlier stores)
    uint4 gv[2][4], uv[2][4];
    float gates_[2][4];
    auto fetch = [&](int s, int at) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const size_t row = (size_t)min(r0 + at + q * 4, last);
        gv[s][q] = *(const uint4*)(h + row * 2 * F + cb + c);
        uv[s][q] = *(const uint4*)(h + row * 2 * F + F + cb + c);
        gates_[s][q] = x.xrows ? gates[x.xrows[row]] : 1.f;
      }
    };
    fetch(0, 0);
#pragma unroll
    for (int b = 0; b < 2 * TM; ++b) {
      const float* blk = stage_rows(acc, b >> 1, b & 1, smem, p);
      if (b + 1 < 2 * TM) fetch((b + 1) & 1, (b + 1) * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = r0 + b * 16 + q * 4;
        float da[8], g[8], u[8], dg[8], du[8], av[8];
        ld8(blk + (q * 4 + (p.lane >> 4)) * EP_LD + c, da);
        Chunk<elt>::unpack(gv[b & 1][q], g);
        Chunk<elt>::unpack(uv[b & 1][q], u);
        const float gate = gates_[b & 1][q];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float sg = sigmoid_fast(g[t]), d = da[t] * gate;
          dg[t] = d * u[t] * sg * (1.0f + g[t] * (1.0f - sg));
          du[t] = d * g[t] * sg;
          av[t] = gate * (g[t] * sg) * u[t];
        }
        const bool ok = rr < m_end;
        const size_t row = (size_t)rr;
        if (ok) {
          put16(dh + row * 2 * F + cb + c, Chunk<elt>::pack(dg));
          put16(dh + row * 2 * F + F + cb + c, Chunk<elt>::pack(du));
          if (ag) put16(ag + row * F + cb + c, Chunk<elt>::pack(av));
        }
        const int bg = fp8_scale_byte(lanes_max<16>(without_inf(dg, amax8(dg))));
        const int bu = fp8_scale_byte(lanes_max<16>(without_inf(du, amax8(du))));
        if (ok) {
          put8(dq + row * 2 * F + cb + c, quant8(dg, fp8_inv_scale(bg)));
          put8(dq + row * 2 * F + F + cb + c, quant8(du, fp8_inv_scale(bu)));
          if ((p.lane & 15) == 0) {
            ds[row * ld2F + cb / 128] = (uint8_t)bg;
            ds[row * ld2F + (F + cb) / 128] = (uint8_t)bu;
          }
        }
      }
    }
  }
};

// Row-grouped product over the plan's tiles.  The next tile's first stage is copied
// while a tile's epilogue runs, and ahead of its stores: a wave's memory operations
// complete in order.
template <class Op>
__global__ __launch_bounds__(NT) void fp8_kernel(Op op, const int32_t* __restrict__ offsets,
                                                 const int32_t* __restrict__ tile_offsets,
                                                 int E_l, int n_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
  __shared__ float s_max[2 * BM];
  __shared__ int s_to[257], s_off[257];
  for (int j = threadIdx.x; j <= E_l; j += NT) {
    s_to[j] = tile_offsets[j];
    s_off[j] = offsets[j];
  }
  __syncthreads();
  Sched sch(s_to[E_l] * n_tiles);
  const int tid = threadIdx.x, nk = op.stages();
  // LDS address of this wave's part of buffer 0
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)((uint32_t)(uintptr_t)(lds_u8_t*)smem + (threadIdx.x >> 6) * 1024u));
  Load la;
  typename Op::LoadB lb;
  Scales sc;
  int nt, e, m0, m_end, half;
  const int k0 = Op::ROTATE ? (int)(blockIdx.x / 8) % nk : 0;
  // Finds the next unit with rows and starts its copies; false behind the last.
  auto locate = [&]() {
    for (; sch.u < sch.units; sch.u += sch.step) {  // block-uniform
      const int t = sch.tile(half);
      nt = t % n_tiles;
      row_tile(s_to, s_off, E_l, t / n_tiles, e, m0, m_end);
      if (half >= 0) {
        m0 += half * (BM / 2);
        m_end = min(m_end, m0 + BM / 2);
      }
      if (m0 >= m_end) continue;
      op.init(e, m0, m_end, nt, la, lb, sc, tid);
      la.copy(k0, lds, true, half < 0);
      lb.copy(k0, lds + STAGE);
      sc.start(k0, nk);
      return true;
    }
    return false;
  };
  // The next tile's first stage and scales are here, ahead of this one's stores.
  auto arrived = [&]() {
    stage_wait();
    sc.arrived();
  };
  if (!locate()) return;
  arrived();
  for (;;) {
    la.copy(after(k0, nk), lds + 2 * STAGE, nk > 1, half < 0);
    lb.copy(after(k0, nk), lds + 3 * STAGE, nk > 1);
    __syncthreads();  // every wave's part of stage 0 is here
    f32x16_t acc[TM][TN];
    mainloop<Op::type::WIDE>(la, lb, sc, nk, k0, smem, lds, half < 0,
                             m0 + Pos::of().wm * WTM >= m_end, acc);
    const int cm0 = m0, cm_end = m_end, cnt = nt;
    sch.u += sch.step;
    const bool more = locate();
    op.epilogue(acc, cm0, cm_end, cnt, smem, s_max, arrived);
    if (!more) break;
    __syncthreads();  // the staging is read before the next tile's stage 1 lands there
  }
}

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

template <class Op>
int launch(const char* name, const moe_shape* s, const Op& op, const int32_t* offsets,
           const int32_t* tile_offsets, int n_tiles, hipStream_t st) {
  const int grid = persistent_grid(2L * max_row_tiles(s) * n_tiles);  // two units per tile
  MOE_LAUNCH(name, st, fp8_kernel<Op><<<grid, NT, 0, st>>>(op, offsets, tile_offsets, (int)s->E_l,
                                                           n_tiles));
  return check_launch(name);
}

struct Ws {
  uint8_t *q, *s;
  Ws(const moe_shape* sh, void* ws, int64_t cols)
      : q((uint8_t*)ws), s(q + align_up((size_t)(sh->T * sh->K * cols), 256)) {}
};

template <class E>
int ffn_fwd_t(const moe_shape* s, const void* xq, const uint8_t* xs, const int32_t* xrows,
              const int32_t* offsets, const int32_t* tile_offsets, const moe_fp8_weights* w,
              void* h, void* a, void* yp, void* ws, hipStream_t st) {
  typedef typename E::elt elt;
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const int ld_d = (int)fp8_scale_ld(d), ld_f = (int)fp8_scale_ld(F);
  const Ws q(s, ws, F);
  const GateUpOp<E> gu{{(const uint8_t*)xq, xs, d, ld_d, xrows, K},
                       {(const uint8_t*)w->gu, w->gu_s, 2 * F, d, ld_d},
                       (elt*)h, (elt*)a, q.q, q.s, F, ld_f};
  if (int rc = launch("ffn_gate_up_fp8", s, gu, offsets, tile_offsets, F / 128, st)) return rc;
  const PlainOp<E> dn{{q.q, q.s, F, ld_f, nullptr, K},
                      {(const uint8_t*)w->down, w->down_s, d, F, ld_f}, (elt*)yp};
  return launch("ffn_down_fp8", s, dn, offsets, tile_offsets, (d + BN - 1) / BN, st);
}

template <class E>
int ffn_dgrad_t(const moe_shape* s, const void* dq, const uint8_t* ds, const int32_t* xrows,
                const float* gates, const void* h, const int32_t* offsets,
                const int32_t* tile_offsets, const moe_fp8_weights* w, void* dh, void* dxp,
                void* ag, void* ws, hipStream_t st) {
  typedef typename E::elt elt;
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const int ld_d = (int)fp8_scale_ld(d), ld_2f = (int)fp8_scale_ld(2 * F);
  const Ws q(s, ws, 2 * F);
  const DgradActOp<E> act{{(const uint8_t*)dq, ds, d, ld_d, xrows, K},
                          {(const uint8_t*)w->downT, w->downT_s, F, d, ld_d},
                          (const elt*)h, gates, (elt*)dh, (elt*)ag, q.q, q.s, F, ld_2f};
  if (int rc = launch("dgrad_act_fp8", s, act, offsets, tile_offsets, (F + BN - 1) / BN, st))
    return rc;
  const PlainOp<E> in{{q.q, q.s, 2 * F, ld_2f, nullptr, K},
                      {(const uint8_t*)w->guT, w->guT_s, d, 2 * F, ld_2f}, (elt*)dxp};
  return launch("dgrad_in_fp8", s, in, offsets, tile_offsets, (d + BN - 1) / BN, st);
}

}  // namespace

size_t fp8_workspace_bytes(const moe_shape* s) {
  // the gradient's share is the larger, and holds the forward's either way; the
  // larger of both kernels', so that it never falls as T grows
  const size_t rows = (size_t)(s->T * s->K);
  const size_t b = align_up(rows * 2 * s->F, 256) + align_up(rows * fp8_scale_ld(2 * s->F), 256);
  const size_t few = align_up(fp8_small_workspace_bytes(s), 256);
  return std::max({b, few, (size_t)256});
}

int launch_ffn_fwd_fp8(const moe_shape* s, const void* xq, const uint8_t* xs,
                       const int32_t* xrows, const int32_t* offsets,
                       const int32_t* tile_offsets, const moe_fp8_weights* w, void* h, void* a,
                       void* yp, void* ws, hipStream_t st) {
  if (fp8_small(s, false))
    return launch_ffn_fwd_fp8_small(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st);
  return s->dtype == MOE_BF16
             ? ffn_fwd_t<BF16>(s, xq, xs, xrows, offsets, tile_offsets, w, h, a, yp, ws, st)
             : ffn_fwd_t<F16>(s, xq, xs, xrows, offsets, tile_offsets, w, h, a, yp, ws, st);
}

int launch_ffn_dgrad_fp8(const moe_shape* s, const void* dq, const uint8_t* ds,
                         const int32_t* xrows, const float* gates, const void* h,
                         const int32_t* offsets, const int32_t* tile_offsets,
                         const moe_fp8_weights* w, void* dh, void* dxp, void* ag, void* ws,
                         hipStream_t st) {
  if (fp8_small(s, true))
    return launch_ffn_dgrad_fp8_small(s, dq, ds, xrows, gates, h, offsets, w, dh, dxp, ag, ws, st);
  return s->dtype == MOE_BF16 ? ffn_dgrad_t<BF16>(s, dq, ds, xrows, gates, h, offsets,
                                                  tile_offsets, w, dh, dxp, ag, ws, st)
                              : ffn_dgrad_t<F16>(s, dq, ds, xrows, gates, h, offsets,
                                                 tile_offsets, w, dh, dxp, ag, ws, st);
}

}  // namespace moe
