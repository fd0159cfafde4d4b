// gq_tiles.h -- one block's tile of C = A B^T for operands whose rows are read in pieces of 64
// bytes: 64 codes of 8 bits (v_mfma_i32_32x32x32_i8) or 32 halves (v_mfma_f32_32x32x16_f16).  Both
// instructions take 32 bytes of 32 rows, lane l the 16 bytes of row l mod 32 at l / 32, in the same
// number of cycles, so one loop serves both; the result has column l mod 32 and rows
// 8 i + 4 (l / 32) + 0..3.  B's rows are the first operand, so a lane ends with four neighbouring
// columns of one row of C.
#pragma once

#include "gq_device.h"

namespace gq {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct F16Product {
  typedef f32x16 Acc;
  typedef f32x4 Four;
  static __device__ __forceinline__ Acc mul(i32x4 first, i32x4 second, Acc acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, first),
                                                  __builtin_bit_cast(f16x8, second), acc, 0, 0, 0);
  }
};

struct I8Product {
  typedef i32x16 Acc;
  typedef i32x4 Four;
  static __device__ __forceinline__ Acc mul(i32x4 first, i32x4 second, Acc acc) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(first, second, acc, 0, 0, 0);
  }
};

constexpr int kStepBytes = 64;  // of a row, one step of the loop

// An operand's rows as one tile needs them.
struct TileRows {
  const uint8_t *first;  // the tile's first row
  int rows;              // rows there are, at most the tile's: later ones repeat the last
};

// Shape of a block's tile: WM x WN waves, a wave FM x FN results of 32 x 32.
template <int WM, int WN, int FM, int FN>
struct TileShape {
  static constexpr int BM = WM * FM * 32, BN = WN * FN * 32, T = WM * WN * 64;
  static constexpr int kStage = (BM + BN) * kStepBytes;  // bytes of a step's operands
};

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

// Steps step0 .. step0 + count - 1 (count even, at least 2) of the tile's sums.  Operands go from
// memory to LDS without registers, three steps ahead, in four buffers of their own names: LDS reads
// wait for their own buffer's loads only.  Row r's 16-byte chunk c is kept at chunk
// c XOR (r / 4 mod 4): 16 rows' reads of one chunk column fall on 16 different places of 256 bytes.
// Returns with every load done and every wave past its reads: the buffers are free.
template <class P, int WM, int WN, int FM, int FN>
__device__ __forceinline__ void tile_product(uint8_t *lds0, uint8_t *lds1, uint8_t *lds2,
                                             uint8_t *lds3, TileRows a, TileRows b, int pitch,
                                             int step0, int count,
                                             typename P::Acc (&acc)[FM][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)  // buffer resources are a type of the device only
  using S = TileShape<WM, WN, FM, FN>;
  constexpr int T = S::T, CA = S::BM * 4 / T, CB = S::BN * 4 / T;  // 16-byte chunks a thread and step
  static_assert(S::BM * 4 % T == 0 && S::BN * 4 % T == 0 && T / 4 % 16 == 0, "whole chunks");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // resources that end with the tile's last row: nothing outside the matrices is ever read
  const auto ra = __builtin_amdgcn_make_buffer_rsrc((void *)a.first, 0, a.rows * pitch, 0x00027000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc((void *)b.first, 0, b.rows * pitch, 0x00027000);
  int off_a[CA], off_b[CB];
  {
    const int row = tid >> 2, chunk = ((tid & 3) ^ (row >> 2 & 3)) << 4;  // T / 4 rows keep the key
#pragma unroll
    for (int i = 0; i < CA; ++i) off_a[i] = min(row + i * (T / 4), a.rows - 1) * pitch + chunk;
#pragma unroll
    for (int i = 0; i < CB; ++i) off_b[i] = min(row + i * (T / 4), b.rows - 1) * pitch + chunk;
  }
  const int r32 = lane & 31, half = lane >> 5;
  int frag[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) frag[j] = r32 * 64 + (((2 * j + half) ^ (r32 >> 2 & 3)) << 4);
  const int last = step0 + count - 1;
  auto issue = [&](uint8_t *lds, int k) {  // past the end: the last step again, not multiplied
    const int at = min(k, last) * kStepBytes;
#pragma unroll
    for (int i = 0; i < CA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_PTR void *)(lds + (i * T + wave * 64) * 16),
                                               16, off_a[i], at, 0, 0);
#pragma unroll
    for (int i = 0; i < CB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (LDS_PTR void *)(lds + S::BM * 64 + (i * T + wave * 64) * 16), 16, off_b[i], at, 0, 0);
  };
  auto step = [&](const uint8_t *now, uint8_t *free, int k) {
    arrive_but<2 * (CA + CB)>();
    issue(free, k + 3);
    const uint8_t *la = now + wm * FM * 2048, *lb = now + (S::BM + wn * FN * 32) * 64;
    i32x4 fa[2][FM], fb[2][FN];
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[j][i] = *reinterpret_cast<const i32x4 *>(la + frag[j] + i * 2048);
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[j][i] = *reinterpret_cast<const i32x4 *>(lb + frag[j] + i * 2048);
    };
    fetch(0);
    fetch(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = P::mul(fb[j][n], fa[j][m], acc[m][n]);
  };
  issue(lds0, step0);
  issue(lds1, step0 + 1);
  issue(lds2, step0 + 2);
  int k = step0;
  for (; k + 3 <= last; k += 4) {
    step(lds0, lds3, k);
    step(lds1, lds0, k + 1);
    step(lds2, lds1, k + 2);
    step(lds3, lds2, k + 3);
  }
  if (k <= last) {
    step(lds0, lds3, k);
    step(lds1, lds0, k + 1);
  }
  arrive_but<0>();
#endif
}

// A wave's results by rows, through its own part of LDS (32 rows of FN * 128 bytes): f(i, pass, row,
// col, lo, hi) with eight neighbouring columns from `col` of row `row` of the wave's i-th 32 rows; a
// lane's columns are the same in all passes.  after(i) follows each 32 rows.
template <class P, int FM, int FN, class F, class G>
__device__ __forceinline__ void by_rows(const typename P::Acc (&acc)[FM][FN], uint8_t *own, F &&f,
                                        G &&after) {
  typedef typename P::Four Four;
  constexpr int kRow = FN * 128, kChunks = FN * 8;
  const int lane = threadIdx.x & 63, r32 = lane & 31, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int chunk = (j * 8 + 2 * q + half) ^ (r32 & (kChunks - 1));
        *reinterpret_cast<Four *>(own + r32 * kRow + chunk * 16) =
            Four{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
    wave_exchange();
#pragma unroll
    for (int p = 0; p < FN * 2; ++p) {
      const int row = p * (16 / FN) + lane / (FN * 4), c = lane % (FN * 4) * 2;
      const Four lo = *reinterpret_cast<const Four *>(own + row * kRow + ((c ^ (row & (kChunks - 1))) * 16));
      const Four hi = *reinterpret_cast<const Four *>(own + row * kRow + (((c + 1) ^ (row & (kChunks - 1))) * 16));
      f(i, p, row, c * 4, lo, hi);
    }
    wave_exchange();
    after(i);
  }
}

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
