// gq_tiles.h -- one block's tile of C = A B^T for operands whose rows are read in pieces of 128
// bytes: 128 codes of 8 bits (v_mfma_i32_16x16x64_i8) or 64 halves (v_mfma_f32_16x16x32_f16).  Both
// instructions take 64 bytes of 16 rows, lane l the 16 bytes of row l mod 16 at l / 16, in the same
// number of cycles, so one loop serves both; the result has column l mod 16 and rows
// 4 (l / 16) + 0..3.  B's rows are the first operand, so a lane ends with four neighbouring columns
// of one row of C.  (Products bound by the card's power gain by these over 32 x 32 ones: a loop of
// nothing else reaches 1.80 against 1.56 PFLOP/s in halves and 3.9 against 3.4 in 8 bits on random
// data.)
#pragma once

#include "gq_device.h"

namespace gq {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct F16Product {
  typedef f32x4 Four;
  static __device__ __forceinline__ Four mul(i32x4 first, i32x4 second, Four acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, first),
                                                  __builtin_bit_cast(f16x8, second), acc, 0, 0, 0);
  }
};

struct I8Product {
  typedef i32x4 Four;
  static __device__ __forceinline__ Four mul(i32x4 first, i32x4 second, Four acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(first, second, acc, 0, 0, 0);
  }
};

constexpr int kStepBytes = 128;  // of a row, one step of the loop: a whole line

// An operand's rows as one tile needs them.
struct TileRows {
  const uint8_t *first;  // the tile's first row
  int rows;              // rows there are, at most the tile's: later ones repeat the last
};

// Shape of a block's tile: WM x WN waves, a wave 16 R x 16 C results, NB buffers of a step's operands.
// After the products a wave's results leave 32 rows at a time in C passes of 64 lanes, eight columns
// each: where C is a power of two a lane has the same columns in all passes, else a pass has 16
// columns.
template <int WM_, int WN_, int R_, int C_, int NB_>
struct TileShape {
  static constexpr int WM = WM_, WN = WN_, R = R_, C = C_, NB = NB_;
  static constexpr int BM = WM * R * 16, BN = WN * C * 16, T = WM * WN * 64;
  static constexpr int kStage = (BM + BN) * kStepBytes;
  static constexpr int kOwn = 32 * C * 64, kPer = kStage / kOwn;  // a wave's part after the products
  static constexpr bool kSameCols = (C & (C - 1)) == 0;
  static_assert(R % 2 == 0 && (NB == 2 || NB == 4), "pairs of rows, buffers");
  static_assert(kPer > 0 && kPer * NB >= WM * WN, "the waves' parts fit the buffers");
  static __device__ __forceinline__ int row_of(int pass, int lane) {
    return kSameCols ? pass * (32 / C) + lane / (C * 2) : lane >> 1;
  }
  static __device__ __forceinline__ int col_of(int pass, int lane) {
    return kSameCols ? lane % (C * 2) * 8 : pass * 16 + (lane & 1) * 8;
  }
  // where four columns of a row are in a wave's part
  static __device__ __forceinline__ int place(int row, int chunk) {
    return row * (C * 64) + ((chunk ^ (kSameCols ? row & (C * 4 - 1) : row >> 2 & 3)) << 4);
  }
};

// The buffers of a block's tile (arrays of their own), and the wave's part of them once the products
// are done.
#define GQ_TILE_LDS(S)                                                              \
  __shared__ __align__(1024) uint8_t lds0[S::kStage];                               \
  __shared__ __align__(1024) uint8_t lds1[S::kStage];                               \
  __shared__ __align__(1024) uint8_t lds2[S::NB > 2 ? S::kStage : 16];              \
  __shared__ __align__(1024) uint8_t lds3[S::NB > 2 ? S::kStage : 16];              \
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);                \
  uint8_t *const own = (wave / S::kPer == 0   ? lds0                                \
                        : wave / S::kPer == 1 ? lds1                                \
                        : wave / S::kPer == 2 ? lds2                                \
                                              : lds3) +                             \
                       wave % S::kPer * S::kOwn

// Waits until at most N of the wave's loads are on their way and its LDS reads are done, then for the
// block's other waves: what was loaded before those N is in LDS for all of them, and no wave still
// reads what it read before.  (A workgroup's release would wait for all loads, as they write LDS.)
template <int N>
__device__ __forceinline__ void arrive_but() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Where row r's 16-byte chunks of a step are kept: chunk c at c XOR tile_key(r).
__device__ __forceinline__ int tile_key(int r) { return (r ^ (r >> 3 & 3)) & 7; }

// Steps step0 .. step0 + count - 1 (count at least 1) of the tile's sums.  Operands go from memory to
// LDS without registers, into NB buffers in turn, each a static array of its own: LDS reads wait for
// their own buffer's loads only.  With tile_key's order of chunks 16 rows' reads of one chunk column
// fall on 16 different places of 256 bytes.
//
// A step is four groups of products, and a group's operands are read from LDS while the group before
// is multiplied, across the barrier too: it stands before a step's last group, when the step's own
// operands are all in registers, so that its buffer is free for the step NB further on and the next
// step's has arrived.
//
// Measured in 8 bits on 4096 x 4096 (a 256 x 256 tile a CU, two buffers): a step takes 1.43 us on random
// codes and 1.14 on zeros; the matrix instructions alone 1.10 and 0.89; loading and LDS reads without them
// 0.86, whatever the data: 64 KB a step and CU, some 19 TB/s from the L2s.  On random data the card's
// power sets the clock (1.9 GHz).  Tried at 8192 x 11008 x 4096 on random codes: pieces of 64 bytes a row,
// half a line, in four buffers (422 us against 394), and with them 256 x 128 tiles, two a CU, which load
// half as much again (476 against 422); operands read after the barrier instead of across it made no
// difference (390 and 390); conflicts in LDS, see below, cost 0.11 us a step.
// Returns with every load done and every wave past its reads: the buffers are free.
template <class P, class S>
__device__ __forceinline__ void tile_product(uint8_t *lds0, uint8_t *lds1, uint8_t *lds2,
                                             uint8_t *lds3, TileRows a, TileRows b, int pitch,
                                             int step0, int count,
                                             typename P::Four (&acc)[S::R][S::C]) {
#if defined(__HIP_DEVICE_COMPILE__)  // buffer resources are a type of the device only
  constexpr int WN = S::WN, R = S::R, C = S::C, H = R / 2, NB = S::NB;
  uint8_t *const lds[4] = {lds0, lds1, lds2, lds3};
  constexpr int T = S::T, CA = S::BM * 8 / T, CB = S::BN * 8 / T;  // 16-byte chunks a thread and step
  static_assert(S::BM * 8 % T == 0 && S::BN * 8 % T == 0 && T / 8 % 32 == 0, "whole chunks");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // resources that end with the tile's last row: nothing outside the matrices is ever read
  const auto ra = __builtin_amdgcn_make_buffer_rsrc((void *)a.first, 0, a.rows * pitch, 0x00027000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc((void *)b.first, 0, b.rows * pitch, 0x00027000);
  int off_a[CA], off_b[CB];
  {
    const int row = tid >> 3, chunk = ((tid & 7) ^ tile_key(row)) << 4;  // T / 8 rows keep the key
#pragma unroll
    for (int i = 0; i < CA; ++i) off_a[i] = min(row + i * (T / 8), a.rows - 1) * pitch + chunk;
#pragma unroll
    for (int i = 0; i < CB; ++i) off_b[i] = min(row + i * (T / 8), b.rows - 1) * pitch + chunk;
  }
  const int r16 = lane & 15;
  // Lanes 16..31 take the third 16 bytes and 32..47 the second, for A and B alike: the order of a sum's
  // terms.  LDS serves lanes of both halves of a wave together: with the bytes in the lanes' order every
  // read met a conflict.
  const int quarter = (lane >> 4 & 1) << 1 | lane >> 5;
  int frag[2];  // rows 16 further on have another key: (r XOR r / 8 mod 4) mod 8 changes by 2
#pragma unroll
  for (int j = 0; j < 2; ++j) frag[j] = r16 * 128 + (((4 * j + quarter) ^ tile_key(r16)) << 4);
  const int last = step0 + count - 1;
  auto issue = [&](uint8_t *to, int k) {  // past the end: the last step again, not multiplied
    const int at = min(k, last) * kStepBytes;
#pragma unroll
    for (int i = 0; i < CA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_PTR void *)(to + (i * T + wave * 64) * 16),
                                               16, off_a[i], at, 0, 0);
#pragma unroll
    for (int i = 0; i < CB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (LDS_PTR void *)(to + S::BM * 128 + (i * T + wave * 64) * 16), 16, off_b[i], at, 0, 0);
  };
  const int odd_b = (wn * C & 1) << 5;
  i32x4 fa[2][H], fb[2][C];
  // Group s: half of the wave's rows of A (s odd: the second) times its rows of B, 64 bytes of each
  // (s / 2: which).
  auto fetch = [&](const uint8_t *from, int s) {
    const int g = s >> 1;
    if ((s & 1) == 0) {
      const uint8_t *lb = from + (S::BM + wn * C * 16) * 128;
#pragma unroll
      for (int i = 0; i < C; ++i)
        fb[g][i] = *reinterpret_cast<const i32x4 *>(lb + i * 2048 + (frag[g] ^ (i & 1) << 5 ^ odd_b));
    }
    const uint8_t *la = from + (wm * R + (s & 1) * H) * 2048;
#pragma unroll
    for (int i = 0; i < H; ++i)
      fa[s & 1][i] = *reinterpret_cast<const i32x4 *>(la + i * 2048 + (frag[g] ^ (((s & 1) * H + i) & 1) << 5));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int s) {
#pragma unroll
    for (int m = 0; m < H; ++m)
#pragma unroll
      for (int n = 0; n < C; ++n)
        acc[(s & 1) * H + m][n] = P::mul(fb[s >> 1][n], fa[s & 1][m], acc[(s & 1) * H + m][n]);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < NB; ++i) issue(lds[i], step0 + i);
  arrive_but<(NB - 1) * (CA + CB)>();
  fetch(lds[0], 0);
  auto step = [&](int i, int k) {
    fetch(lds[i], 1);
    multiply(0);
    fetch(lds[i], 2);
    multiply(1);
    fetch(lds[i], 3);
    multiply(2);
    arrive_but<(NB - 2) * (CA + CB)>();
    issue(lds[i], k + NB);
    fetch(lds[(i + 1) % NB], 0);  // of a step that is not there, after the last: not multiplied
    multiply(3);
  };
  int k = step0;
  for (; k + NB - 1 <= last; k += NB) {
#pragma unroll
    for (int i = 0; i < NB; ++i) step(i, k + i);
  }
#pragma unroll
  for (int i = 0; i < NB - 1; ++i)
    if (k + i <= last) step(i, k + i);
  arrive_but<0>();
#endif
}

// A wave's results by rows, 32 of them at a time, through its own part of LDS.  For the wave's i-th 32
// rows: pre(k, four) makes four neighbouring results of row 16 k + (lane mod 16) of the wave's what is
// exchanged, f(i, pass, row, col, lo, hi) has eight neighbouring columns from `col` of row `row`, and
// after(i) follows.  before(i) is called one turn ahead, so that what it loads arrives meanwhile: a
// load in f itself would cost its latency in every pass.
template <class P, class S, class H, class B, class F, class G>
__device__ __forceinline__ void by_rows(const typename P::Four (&acc)[S::R][S::C], uint8_t *own, H &&pre,
                                        B &&before, F &&f, G &&after) {
  constexpr int R = S::R, C = S::C;
  const int lane = threadIdx.x & 63;
  before(0);
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < C; ++n)
        *reinterpret_cast<f32x4 *>(own + S::place(m * 16 + (lane & 15), n * 4 + (lane >> 4))) =
            pre(i * 2 + m, acc[i * 2 + m][n]);
    wave_exchange();
    if (i + 1 < R / 2) before(i + 1);
#pragma unroll
    for (int p = 0; p < C; ++p) {
      const int row = S::row_of(p, lane), col = S::col_of(p, lane);
      const f32x4 lo = *reinterpret_cast<const f32x4 *>(own + S::place(row, col >> 2));
      const f32x4 hi = *reinterpret_cast<const f32x4 *>(own + S::place(row, (col >> 2) + 1));
      f(i, p, row, col, lo, hi);
    }
    wave_exchange();
    after(i);
  }
}

// What all lanes have alike, for the scalar registers: a quotient comes out of the vector ones, and a
// buffer's address from there would be asked for lane by lane at every load.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Blocks are handed to the XCDs in turn: an XCD's blocks take neighbouring tiles, which share
// operand rows in its L2.
__device__ __forceinline__ int near_tiles(int block, int total) {
  const int xcd = block & 7, each = total >> 3, more = total & 7;
  return xcd * each + min(xcd, more) + (block >> 3);
}

// Tile (m, n) of a grid of tiles, eight rows of tiles at a time.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int &m, int &n) {
  const int width = 8 * tiles_n, group = t / width, first = group * 8;
  const int high = min(tiles_m - first, 8), in = t - group * width;
  m = first + in % high;
  n = in / high;
}

}  // namespace
}  // namespace gq
