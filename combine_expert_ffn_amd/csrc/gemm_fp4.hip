// Grouped products of 8-bit rows with 4-bit expert weights (gfx950), for many rows per
// expert: e4m3 rows with a power-of-two scale per 128, e2m1 weights with one per 32,
// float32 accumulation.
// bf16 data: v_mfma_scale_f32_32x32x64_f8f6f4 takes an 8-bit and a 4-bit operand; a
// lane holds 32 consecutive values of a weight row, which are one scale block, so every
// weight scale is a byte of that lane's own and costs no vector instruction.  It runs at
// the rate of two 8-bit operands (3.96 against 4.04 PFLOP/s measured), and cuts products
// as the 8-bit kernels' comment says.  That is chosen for time (the exact products of fp16
// data take 1161 us for 128 experts of 2048 x 768 and 131072 rows, these 728); what it
// changes is that 0.05 % of a's values, next to the border between two e4m3 values, are
// quantised to the other one, for which y_p is 1.77e-3 from the definition instead of 1.66e-3.
// fp16 data: both operands widened to bf16 with their scales (exact) and multiplied by
// v_mfma_f32_32x32x16_bf16.
// Tile, waves, schedule and epilogues are the 8-bit kernels'.  What differs is the
// weights' way through LDS: a stage of the reduction is 128 values, 128 bytes of a
// row but 64 of a weight row, and 64-byte pieces halve the rate of L2.  So weights
// are copied as 256 values (128 bytes) for two stages at a time, half of the tile's
// weight rows per stage, while rows are copied each stage.
// What bounds it: 128 experts of 2048 x 768, 131072 rows, bf16, h and a kept, by the library's
// kernel timer: gate and up 455 us (1.81 PFLOP/s), down 265 (1.56); the 8-bit experts' 509 and 289.
// In variants with parts left out: fragment reads and MFMAs alone 292 / 184, with the copies
// 339 / 193, the epilogues without their stores 66 / 36 more, the stores (past the caches;
// through them 31 more in all) 50 / 35.  The matrix cores are busy 45 and 38 % of it.
// fp16: 1333 tokens, 8 of 64 experts of 2048 x 1408, K = 6, Zipf 85 and 38 us: little more than one
// round of tiles on 256 CUs.
// Slower: two blocks of 128 x 256 per CU (781 us for both products; 5 to 10 % faster at a few
// hundred rows per expert), a ring of four stages with tiles of 128 rows (534 us for 512 rows
// each instead of 372, and no faster below), the first slice without clearing (350 registers
// in memory).
#include "moe_fp4.h"
#include "moe_tile8.h"

namespace moe {
namespace {

// As stage_wait(), as a wait that the compiler sees: behind the inline assembly it would
// wait again ahead of each use of the fetched scales, for the copies of the next stage too.
__device__ __forceinline__ void all_here() {
  asm volatile("" : : : "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0) alone
  asm volatile("" : : : "memory");
}

__device__ __forceinline__ uint32_t scalar(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// The weight operand's copies: 256 rows of k / 2 bytes, in groups of 64 rows whose
// offsets from the first are scalars (group c: (c & 1) * s1 + (c >> 1) * s2).
struct Load4 {
  u32x4_t rsrc;
  uint32_t off, upper, s1, s2;
  __device__ __forceinline__ void init(const uint8_t* base, int bytes, uint32_t s1_, uint32_t s2_,
                                       int tid) {
    Load l;
    l.set_base(base);
    rsrc = l.rsrc;
    const uint32_t chunk = (uint32_t)((tid & 7) ^ swz(tid >> 3));
    off = (uint32_t)((tid >> 3) * bytes) + chunk * 16u;
    upper = (chunk & 4u) << 4;  // 64 where the chunk lies in the second 64 bytes
    s1 = scalar(s1_);
    s2 = scalar(s2_);
    // in scalar registers, whatever they were computed in
    asm volatile("" : "+s"(rsrc), "+s"(s1), "+s"(s2));
  }
  // Half h (128 of the 256 rows) of the two blocks from kb on, kb even.  Where kb is the
  // last block the second 64 bytes of a row do not exist and the first are read again.
  __device__ __forceinline__ void copy(int kb, int nk, int h, uint32_t lds, bool on) const {
    const u32x4_t r = {rsrc[0], rsrc[1], on ? rsrc[2] : 0u, rsrc[3]};
    const uint32_t o = off - (kb + 1 < nk ? 0u : upper);
    const uint32_t at = (uint32_t)kb * 64u + (h ? s2 : 0u);
    const uint32_t to = lds + (uint32_t)h * 2 * Load::ROWS * 128;
    copy_rows(o, r, scalar(at), to);
    copy_rows(o, r, scalar(at + s1), to + Load::ROWS * 128);
  }
};

// Scales of four stages at a time: bytes of the wave's rows (one register per 32-row
// tile), and the four bytes of each of the four blocks of its 128 weight rows, lane l's
// those of row l of each 64.  b[h][0] is the current block's.
struct Scales4 {
  static constexpr int H = TN / 2;
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t oa[TM], ob, s1;  // 64 rows h: ob + h * s1
  uint32_t a[TM], an[TM];
  u32x4_t b[H], bn[H];
  __device__ __forceinline__ void fetch(int k, uint32_t (&ta)[TM], u32x4_t (&tb)[H]) const {
#pragma unroll
    for (int i = 0; i < TM; ++i) ta[i] = __builtin_amdgcn_raw_buffer_load_b32(ra, (int)oa[i], k, 0);
    // past the last block's scales of the last row nothing is read (zeros)
#pragma unroll
    for (int h = 0; h < H; ++h)
      tb[h] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)(ob + (uint32_t)(k * 4) + h * s1), 0,
                                                    0);
  }
  // the group of block k now, and the one after it
  __device__ __forceinline__ void start(int k, int nk) {
    fetch(k & ~3, a, b);
    fetch((k | 3) + 1 < nk ? (k | 3) + 1 : 0, an, bn);
  }
  // both are here; k: the first block
  __device__ __forceinline__ void arrived(int k) {
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(a[i]), "+v"(an[i]));
#pragma unroll
    for (int h = 0; h < H; ++h) asm volatile("" : "+v"(b[h]), "+v"(bn[h]));
    if (k & 2) {  // block-uniform; k is even
#pragma unroll
      for (int h = 0; h < H; ++h) b[h] = u32x4_t{b[h][2], b[h][3], 0, 0};
    }
  }
  // The current block's four bytes of lane l % 32's row of every column tile, shifted by
  // the lane's half (bytes 0 and 2 are then slices 0 and 1); and on to the next block.
  // Lanes 0 .. 31 hold the rows of the even column tiles, the others those of the odd.
  __device__ __forceinline__ void step(int half, uint32_t (&sb)[TN]) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const auto p = __builtin_amdgcn_permlane32_swap(b[h][0], b[h][0], false, false);
      sb[2 * h] = p[0] >> half;
      sb[2 * h + 1] = p[1] >> half;
      b[h] = u32x4_t{b[h][1], b[h][2], b[h][3], 0};
    }
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
#pragma unroll
    for (int h = 0; h < H; ++h)
      b[h] = u32x4_t{moved(bn[h][0]), moved(bn[h][1]), moved(bn[h][2]), moved(bn[h][3])};
  }
};

// A lane's 32 values of a 64-deep slice kk of a stage: of a row, the two chunks that the
// instruction pairs with 32 consecutive 4-bit values of the other operand (found with
// single products), or, widened here, 32 consecutive ones.
template <bool WIDE>
__device__ __forceinline__ i32x8_t row_frag(const uint8_t* tile, int row0, int kk, int lane) {
  if constexpr (!WIDE) return read_frag(tile, row0, kk, lane);
  const int fr = lane & 31, hf = lane >> 5;
  const uint8_t* p = tile + (row0 + fr) * 128;
  const int s = swz(fr);
  const i32x4_t lo = *(const i32x4_t*)(p + (((kk * 4 + 2 * hf) ^ s) << 4));
  const i32x4_t hi = *(const i32x4_t*)(p + (((kk * 4 + 2 * hf + 1) ^ s) << 4));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Of a weight row, chunk 2 q + lane / 32 of its eight, q the slice of the two stages.
__device__ __forceinline__ i32x4_t weight_frag(const uint8_t* tile, int row0, int q, int lane) {
  const int fr = lane & 31;
  return *(const i32x4_t*)(tile + (row0 + fr) * 128 + (((q * 2 + (lane >> 5)) ^ swz(fr)) << 4));
}

// One 64-deep slice (CUR of its stage): the MFMAs of the wave on a and b, and beside them
// the reads of the next slice's fragments: rows from na, slice 1 - CUR of their stage,
// weights from nb, slice nq of their two stages.  sb: the weight scales, already
// shifted by the lane's half.  between(j) is what else is issued behind the MFMAs of
// column tile j: they keep the matrix core busy meanwhile, where ahead of them, behind a
// barrier, it would stand idle.
template <bool WIDE, int CUR, class Between>
__device__ __forceinline__ void slice(const i32x8_t (&a)[TM], i32x8_t (&an)[TM], i32x4_t (&b)[TN],
                                      const uint32_t (&sa)[TM], const uint32_t (&sb)[TN],
                                      f32x16_t (&acc)[TM][TN], const uint8_t* na,
                                      const uint8_t* nb, int nq, const Pos& w, Between between) {
  auto next_b = [&](int j) { return weight_frag(nb, w.wn * WTN + j * 32, nq, w.lane); };
  auto next_a = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i) an[i] = row_frag<WIDE>(na, w.wm * WTM + i * 32, 1 - CUR, w.lane);
  };
  if constexpr (WIDE) {
    float fa[TM], fb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[i] = fp8_scale_value((int)(sa[i] & 255u));
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = fp8_scale_value((int)((sb[j] >> (16 * CUR)) & 255u));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8_t aw[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) aw[i] = widen(a[i][2 * q], a[i][2 * q + 1], fa[i]);
      if (q == 2) next_a();
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bf16x8_t bw = widen4((uint32_t)b[j][q], fb[j]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(aw[i], bw, acc[i][j], 0, 0, 0);
        if (q == 3) b[j] = next_b(j);
        if (q == 0) between(j);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    i32x4_t bn[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (j == 0) next_a();
      if (j > 0) bn[j - 1] = next_b(j - 1);
      if (j == TN - 1) bn[j] = next_b(j);
      const i32x8_t bw = __builtin_shufflevector(b[j], b[j], 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
      for (int i = 0; i < TM; ++i)  // 0: e4m3, 4: e2m1
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            a[i], bw, acc[i][j], 0, 4, 0, (int)sa[i], 2 * CUR, (int)sb[j]);
      between(j);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = bn[j];
  }
}

// The reduction over nk blocks from block k0 around (k0 even; 0 if nk is odd).  Two row
// buffers take the stages in turn, two weight buffers the pairs of stages; the first
// stage and pair are in theirs, the second stage and half of the second pair are being
// copied.  A buffer is written again behind the barrier after its last read; what is
// read behind a barrier was asked for a stage ahead.  below, idle: as in the 8-bit kernels.
template <bool WIDE>
__device__ __forceinline__ void mainloop(const Load& la, const Load4& lb, Scales4& sc, int nk,
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
  int kc = after(after(k0, nk), nk);  // the block of the stage that is copied next
  int kn = kc;                        // the first block of the pair that is copied next
  auto copy_a = [&](int kt) {
    la.copy(kc, lds + (kt & 1) * 2 * STAGE, kt + 2 < nk, below);
    kc = after(kc, nk);
  };
  auto copy_b = [&](int kt) {
    const int odd = kt & 1, pair = (kt >> 1) + 1 + odd;
    lb.copy(kn, nk, odd, lds + STAGE + (pair & 1) * 2 * STAGE, 2 * pair < nk);
    if (!odd) kn = after(after(kn, nk), nk);
  };
  if (idle) {  // wave-uniform: only its part of the copies, and the barriers
    for (int kt = 0; kt < nk; ++kt) {
      all_here();
      __syncthreads();
      copy_a(kt);
      copy_b(kt);
    }
    all_here();
    __syncthreads();
    return;
  }
  const int half = (w.lane >> 5) * 8;
  i32x8_t a0[TM], a1[TM];
  i32x4_t b[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) a0[i] = row_frag<WIDE>(smem, w.wm * WTM + i * 32, 0, w.lane);
#pragma unroll
  for (int j = 0; j < TN; ++j) b[j] = weight_frag(smem + STAGE, w.wn * WTN + j * 32, 0, w.lane);
  for (int kt = 0; kt < nk;) {
    // the stages whose scales were fetched together
    const int end = min(kt + min(4 - (kb & 3), nk - kb), nk);
    do {
      const int odd = kt & 1;
      const uint8_t* cur = smem + odd * 2 * STAGE;
      const uint8_t* nxt = smem + (odd ^ 1) * 2 * STAGE;
      const uint8_t* wcur = smem + STAGE + (kt & 2) * STAGE;
      const uint8_t* wnxt = smem + STAGE + ((kt + 1) & 2) * STAGE;
      const int sh = (kb & 3) * 8;
      uint32_t sa[TM], sb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = sc.a[i] >> sh;
      sc.step(half, sb);
      __builtin_amdgcn_sched_barrier(0);
      slice<WIDE, 0>(a0, a1, b, sa, sb, acc, cur, wcur, odd * 2 + 1, w, [](int) {});
      all_here();
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      slice<WIDE, 1>(a1, a0, b, sa, sb, acc, nxt, wnxt, (odd ^ 1) * 2, w, [&](int j) {
        if (j == 0) copy_a(kt);
        if (j == 1) copy_b(kt);
      });
      ++kb;
    } while (++kt < end);
    if (kb == nk) kb = 0;
    sc.next();
    __builtin_amdgcn_sched_barrier(0);
    sc.fetch((kb | 3) + 1 < nk ? (kb | 3) + 1 : 0, sc.an, sc.bn);
    __builtin_amdgcn_sched_barrier(0);
  }
  all_here();  // the copies past the last stage write zeros to LDS
  __syncthreads();
}

// The weight operand [E_l][n][k / 2] with scales [E_l][n][k / 32].
struct Cols4 {
  const uint8_t* q;
  const uint8_t* s;
  int n, k;
  // first: the tile's first weight row; s1, s2: rows from 64-row group to group (Load4);
  // srow: the wave's first row, t1: rows to its second 64 (Scales4)
  __device__ __forceinline__ void init(int e, int first, int s1, int s2, int srow, int t1,
                                       Load4& lb, Scales4& sc, int tid) const {
    const int kq = k / 2, ks = k / 32;
    lb.init(q + ((size_t)e * n + first) * kq, kq, (uint32_t)(s1 * kq), (uint32_t)(s2 * kq), tid);
    sc.rb = __builtin_amdgcn_make_buffer_rsrc((void*)(s + (size_t)e * n * ks), (short)0, n * ks,
                                              0x00020000);
    sc.ob = (uint32_t)((srow + Pos::of().lane) * ks);
    sc.s1 = scalar((uint32_t)(t1 * ks));
  }
};

// First product: [g, u] = x^ . W_gu^[e]^T, a = silu(g) u, quantised for the second.  A
// wave column's 128 columns are 64 gate rows and the 64 up rows of the same outputs.
template <class E>
struct GateUp4 {
  typedef E type;
  Rows x;
  Cols4 w;  // n = 2F
  GateUpOut<E> out;
  static constexpr bool ROTATE = false;
  __device__ __forceinline__ void init(int e, int m0, int m_end, int nt, Load& la, Load4& lb,
                                       Scales4& sc, int tid) const {
    x.init(m0, m_end, la, sc, tid);
    const int wn = Pos::of().wn, j0 = nt * 128;
    w.init(e, j0, out.F, 64, j0 + wn * 64, out.F, lb, sc, tid);
  }
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int m0, int m_end,
                                           int nt, uint8_t* smem, float* s_max,
                                           Arrived arrived) const {
    out.epilogue(acc, m0, m_end, nt, smem, s_max, arrived);
  }
};

// Second product: y_p = a^ . W_down^T.  n is a multiple of 128, so the last tile may be
// half, whose rows are then read twice.
template <class E>
struct Down4 {
  typedef E type;
  Rows x;
  Cols4 w;  // n = d
  PlainOut<E> out;
  static constexpr bool ROTATE = true;
  __device__ __forceinline__ void init(int e, int m0, int m_end, int nt, Load& la, Load4& lb,
                                       Scales4& sc, int tid) const {
    x.init(m0, m_end, la, sc, tid);
    const bool part = nt * BN + 128 >= w.n;
    const int wn = part ? 0 : Pos::of().wn;
    w.init(e, nt * BN, 64, part ? 0 : 128, nt * BN + wn * 128, 64, lb, sc, tid);
  }
  template <class Arrived>
  __device__ __forceinline__ void epilogue(const f32x16_t (&acc)[TM][TN], int m0, int m_end,
                                           int nt, uint8_t* smem, float*, Arrived arrived) const {
    out.epilogue(acc, w.n, m0, m_end, nt, smem, arrived);
  }
};

// Row-grouped product over the plan's tiles, as the 8-bit kernel.
template <class Op>
__global__ __launch_bounds__(NT) void fp4_kernel(Op op, const int32_t* __restrict__ offsets,
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
  const int tid = threadIdx.x, nk = op.x.k / 128;
  // LDS address of this wave's part of buffer 0
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)((uint32_t)(uintptr_t)(lds_u8_t*)smem + (threadIdx.x >> 6) * 1024u));
  Load la;
  Load4 lb;
  Scales4 sc;
  int nt, e, m0, m_end, half;
  const int k0 = Op::ROTATE && nk % 2 == 0 ? (int)(blockIdx.x / 8) % (nk / 2) * 2 : 0;
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
      lb.copy(k0, nk, 0, lds + STAGE, true);
      lb.copy(k0, nk, 1, lds + STAGE, true);
      sc.start(k0, nk);
      return true;
    }
    return false;
  };
  // The next tile's first stage and scales are here, ahead of this one's stores.
  auto arrived = [&]() {
    all_here();
    sc.arrived(k0);
  };
  if (!locate()) return;
  arrived();
  for (;;) {
    la.copy(after(k0, nk), lds + 2 * STAGE, nk > 1, half < 0);
    lb.copy(after(after(k0, nk), nk), nk, 1, lds + 3 * STAGE, nk > 2);
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

template <class Op>
int launch(const char* name, const moe_shape* s, const Op& op, const int32_t* offsets,
           const int32_t* tile_offsets, int n_tiles, hipStream_t st) {
  const int grid = persistent_grid(2L * max_row_tiles(s) * n_tiles);  // two units per tile
  MOE_LAUNCH(name, st, fp4_kernel<Op><<<grid, NT, 0, st>>>(op, offsets, tile_offsets, (int)s->E_l,
                                                           n_tiles));
  return check_launch(name);
}

template <class E>
int ffn_fwd_t(const moe_shape* s, const void* xq, const uint8_t* xs, const int32_t* xrows,
              const int32_t* offsets, const int32_t* tile_offsets, const moe_fp4_weights* w,
              void* h, void* a, void* yp, void* ws, hipStream_t st) {
  typedef typename E::elt elt;
  const int d = (int)s->d, F = (int)s->F, K = (int)s->K;
  const int ld_d = (int)fp8_scale_ld(d), ld_f = (int)fp8_scale_ld(F);
  const Ws q(s, ws, F);
  const GateUp4<E> gu{{(const uint8_t*)xq, xs, d, ld_d, xrows, K},
                      {w->gu, w->gu_s, 2 * F, d},
                      {(elt*)h, (elt*)a, q.q, q.s, F, ld_f}};
  if (int rc = launch("ffn_gate_up_fp4", s, gu, offsets, tile_offsets, F / 128, st)) return rc;
  const Down4<E> dn{{q.q, q.s, F, ld_f, nullptr, K}, {w->down, w->down_s, d, F}, {(elt*)yp}};
  return launch("ffn_down_fp4", s, dn, offsets, tile_offsets, (d + BN - 1) / BN, st);
}

}  // namespace

size_t fp4_workspace_bytes(const moe_shape* s) {
  // the tiles' quantised a, or the few-row kernels' float32 a; the larger of both, so that
  // it never falls as T grows
  const size_t rows = (size_t)(s->T * s->K);
  const size_t b = align_up(rows * s->F, 256) + align_up(rows * fp8_scale_ld(s->F), 256);
  const size_t few = align_up(fp4_small_workspace_bytes(s), 256);
  return b > few ? (b > 256 ? b : 256) : (few > 256 ? few : 256);
}

int launch_ffn_fwd_fp4(const moe_shape* s, const void* xq, const uint8_t* xs,
                       const int32_t* xrows, const int32_t* offsets,
                       const int32_t* tile_offsets, const moe_fp4_weights* w, void* h, void* a,
                       void* yp, void* ws, hipStream_t st) {
  if (fp4_small(s))
    return launch_ffn_fwd_fp4_small(s, xq, xs, xrows, offsets, w, h, a, yp, ws, st);
  return s->dtype == MOE_BF16
             ? ffn_fwd_t<BF16>(s, xq, xs, xrows, offsets, tile_offsets, w, h, a, yp, ws, st)
             : ffn_fwd_t<F16>(s, xq, xs, xrows, offsets, tile_offsets, w, h, a, yp, ws, st);
}

}  // namespace moe
