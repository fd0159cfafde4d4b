// gq_i8.hip -- gfx950 kernels of 8-bit integer matrices with a scale for each row: quantisation of
// a matrix by rows and by columns, and the product of two of them.
//
// Format.  A row of `cols` elements is `cols` codes of 8 bits in [-127, 127] and a scale, fp32:
// an element stands for code * scale.  Rows are padded with zero codes to a multiple of 128, so the
// product's K loop has no tail.  With t the row's largest magnitude, scale = fp32(t / 127) and
// inv = fp32(127 / t): the uniform grid of 127 levels of the gradient quantisers with the largest
// magnitude as its scale.  A row whose inv is not finite (t zero, or below 2^-121) has scale 0 and
// zero codes; one that holds an infinity or NaN has scale NaN and zero codes.
#include <math.h>

#include <type_traits>

#include "gq_layers.h"
#include "gq_tiles.h"

namespace gq {
namespace {

// ---------------------------------------------------------------- quantisation
struct RowScale {
  float scale, inv;  // inv 0: all codes are zero
};

__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  if (top >= 0x7F800000u) return RowScale{__uint_as_float(0x7FC00000u), 0.0f};
  const float t = __uint_as_float(top), inv = 127.0f / t;
  if (!(inv < INFINITY)) return RowScale{0.0f, 0.0f};
  return RowScale{t / 127.0f, inv};
}

// The code's byte, the other bits not cleared.  To nearest, ties to even: x * inv + 1.5 * 2^23 in one
// rounding, whose unit is 1 there, so that the exact product is rounded.  A row without codes has
// inv = 0: 0 * inf is NaN, whose byte is 0.
__device__ __forceinline__ uint32_t nearest_byte(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.0f));
}

// Up from floor(u) with probability u - floor(u), u = min(fp32(|x| inv), 127), as the gradient
// quantisers do.
__device__ __forceinline__ uint32_t drawn_byte(float x, float inv, uint32_t h) {
  const float u = fminf(fabsf(x) * inv, 127.0f);
  const int c = (int)u + ((float)h < __builtin_amdgcn_fractf(u) * 4294967296.0f);
  return (uint32_t)((__float_as_uint(x) >> 31) ? -c : c);
}

__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u),
                               __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

template <bool STOCH>
__device__ __forceinline__ u32x2 eight_codes(const float (&x)[8], float inv, const uint32_t (&h)[8]) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = STOCH ? drawn_byte(x[i], inv, h[i]) : nearest_byte(x[i], inv);
  return u32x2{four_bytes(c[0], c[1], c[2], c[3]), four_bytes(c[4], c[5], c[6], c[7])};
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}

// By rows: W waves a row, C groups of eight elements a lane held in registers, so that a row is read
// once; C = 0: a row too long for that is read twice, the second time mostly from the caches.  Bound by
// its bytes at size (8192 x 4096 bf16 17 us, 101 MB, 6.0 TB/s), by a launch below (333 x 768 5 us).
template <int DT, bool STOCH, int W, int C>
__global__ __launch_bounds__(256) void k_i8_rows(const I8QuantArgs a, int pitch) {
  constexpr int kThreads = W * 64, kRows = 256 / kThreads;
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & (kThreads - 1), wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kThreads;
  const bool there = row < a.rows;
  const int64_t at = (there ? row : 0) * a.ld;
  const int groups = pitch / 8;
  float x[C > 0 ? C : 1][8];
  uint32_t top = 0;
  if constexpr (C > 0) {
    Raw<DT, 8> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = raw_word<DT, 8>(a.x, at, (int64_t)(lane + c * kThreads) * 8, a.cols);
#pragma unroll
    for (int c = 0; c < C; ++c) open_word(raw[c], a.x, at, (int64_t)(lane + c * kThreads) * 8, a.cols, x[c]);
#pragma unroll
    for (int c = 0; c < C; ++c) top = max(top, top_of(x[c]));
  } else {
    for (int g = lane; g * 8 < a.cols; g += kThreads) {
      load_word<DT>(a.x, at, (int64_t)g * 8, a.cols, x[0]);
      top = max(top, top_of(x[0]));
    }
  }
  top = wave_max(top);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) tops[wave] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < W; ++w) top = max(top, tops[w]);
  }
  const RowScale s = row_scale(top);
  if (!there) return;
  if (lane == 0) a.scales[row] = s.scale;
  int8_t *out = a.codes + row * pitch;
  uint32_t h[8] = {};
  auto leave = [&](int g, const float (&v)[8]) {
    if constexpr (STOCH) {
      const uint32_t first = a.index_base + (uint32_t)(row * a.cols) + (uint32_t)g * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = draw(first + i, a.key_mix);
    }
    const u32x2 w = eight_codes<STOCH>(v, s.inv, h);
    *reinterpret_cast<u32x2 *>(out + (int64_t)g * 8) = s.inv == 0.0f ? u32x2{0u, 0u} : w;
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int g = lane + c * kThreads;
      if (g < groups) leave(g, x[c]);
    }
  } else {
    for (int g = lane; g < groups; g += kThreads) {
      load_word<DT>(a.x, at, (int64_t)g * 8, a.cols, x[0]);
      leave(g, x[0]);
    }
  }
}

// The columns of a matrix without rows: scales of zero, and no codes.
__global__ __launch_bounds__(256) void k_i8_no_rows(float *scales_t, int64_t cols) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < cols) scales_t[i] = 0.0f;
}

// Largest magnitudes of rows (ROWS) and columns, as bits, over a part of the matrix each: a block goes
// through 64 rows at a time of its share, 512 columns, a wave 16 rows, a lane eight columns.  This read of
// the matrix is what scales of whole columns cost: 4095 x 4096 bf16 16 us (33 MB), bound by latency.
template <int DT, bool ROWS>
__global__ __launch_bounds__(256) void k_i8_tops(const I8QuantArgs a, int rows_each) {
  __shared__ uint32_t cols_top[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * 512 + lane * 8;
  const int64_t first = (int64_t)blockIdx.y * rows_each, end = min(first + rows_each, a.rows);
  uint32_t top[8] = {};
  for (int64_t r0 = first + wave * 16; r0 < end; r0 += 64) {
    uint32_t row_top[16];
#pragma unroll
    for (int q = 0; q < 16; q += 8) {  // rows past the end: the last one again
      Raw<DT, 8> raw[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) raw[u] = raw_word<DT, 8>(a.x, min(r0 + q + u, end - 1) * a.ld, c0, a.cols);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float x[8];
        open_word(raw[u], a.x, min(r0 + q + u, end - 1) * a.ld, c0, a.cols, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = max(top[i], __float_as_uint(x[i]) & 0x7FFFFFFFu);
        row_top[q + u] = top_of(x);
      }
    }
    if constexpr (ROWS) {
      // sixteen rows' maxima over 64 lanes: at each exchange a lane keeps half of the rows
#pragma unroll
      for (int half = 8; half > 0; half >>= 1) {
        const bool upper = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const uint32_t give = upper ? row_top[i] : row_top[i + half], keep = upper ? row_top[i + half] : row_top[i];
          row_top[i] = max(keep, (uint32_t)__shfl_xor((int)give, half));
        }
      }
      row_top[0] = max(row_top[0], (uint32_t)__shfl_xor((int)row_top[0], 16));
      row_top[0] = max(row_top[0], (uint32_t)__shfl_xor((int)row_top[0], 32));
      if (lane < 16 && r0 + lane < end) a.tops[(int64_t)blockIdx.x * a.rows + r0 + lane] = row_top[0];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) cols_top[wave][lane * 8 + i] = top[i];
  __syncthreads();
  uint32_t *out = a.tops + (ROWS ? gridDim.x * a.rows : 0) + (int64_t)blockIdx.y * a.cols;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = threadIdx.x + i * 256;
    const int64_t col = (int64_t)blockIdx.x * 512 + c;
    if (col < a.cols) out[col] = max(max(cols_top[0][c], cols_top[1][c]), max(cols_top[2][c], cols_top[3][c]));
  }
}

// By columns, or both ways (ROWS), from the parts' largest magnitudes (row_parts of rows, then
// col_parts of columns).  A block takes 128 rows x 128 columns; a lane has eight columns of a row,
// whose codes by rows leave as they are and whose codes by columns cross LDS.  The draw of an element
// is shared by its two codes.  4095 x 4096 bf16 stochastic both ways 29 us: some 30 vector instructions
// an element, 7 of them the draw, beside 67 MB.  Parts of twice the length, half the maxima to read again
// here, changed nothing (29 us, and 20 for the maxima instead of 16).
template <int DT, bool STOCH, bool ROWS>
__global__ __launch_bounds__(256) void k_i8_both(const I8QuantArgs a, int pitch, int pitch_t, int row_parts,
                                                 int col_parts) {
  constexpr int kPad = 136;
  __shared__ __align__(16) uint8_t tile[128 * kPad];
  __shared__ float invs[2][128];  // of rows, of columns
  __shared__ uint32_t other[2][128];
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  const int64_t col = c0 + (tid & 15) * 8;
  Raw<DT, 8> raw[8];  // rows past the end: the last one again, not kept
#pragma unroll
  for (int p = 0; p < 8; ++p) raw[p] = raw_word<DT, 8>(a.x, min(r0 + p * 16 + (tid >> 4), a.rows - 1) * a.ld, col, a.cols);
  {
    // a thread a row or column and half of its parts
    const int i = tid & 127, half = tid >> 7;
    const uint32_t *of_cols = a.tops + (ROWS ? row_parts * a.rows : 0);
    uint32_t row_top = 0, col_top = 0;
    if (c0 + i < a.cols)
#pragma unroll 8
      for (int p = half; p < col_parts; p += 2) col_top = max(col_top, of_cols[(int64_t)p * a.cols + c0 + i]);
    if (ROWS && r0 + i < a.rows)
#pragma unroll 4
      for (int p = half; p < row_parts; p += 2) row_top = max(row_top, a.tops[(int64_t)p * a.rows + r0 + i]);
    if (half) {
      other[0][i] = row_top;
      other[1][i] = col_top;
    }
    __syncthreads();
    if (!half) {
      const RowScale r = row_scale(max(row_top, other[0][i])), c = row_scale(max(col_top, other[1][i]));
      invs[0][i] = r.inv;
      invs[1][i] = c.inv;
      if (ROWS && blockIdx.x == 0 && r0 + i < a.rows) a.scales[r0 + i] = r.scale;
      if (blockIdx.y == 0 && c0 + i < a.cols) a.scales_t[c0 + i] = c.scale;
    }
    __syncthreads();
  }
  float inv_cols[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) inv_cols[i] = invs[1][(tid & 15) * 8 + i];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = p * 16 + (tid >> 4);
    const int64_t row = r0 + r;
    float x[8];
    open_word(raw[p], a.x, min(row, a.rows - 1) * a.ld, col, a.cols, x);
    if (row >= a.rows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    }
    uint32_t h[8] = {};
    if constexpr (STOCH) {
      const uint32_t first = a.index_base + (uint32_t)(row * a.cols) + (uint32_t)col;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = draw(first + i, a.key_mix);
    }
    if constexpr (ROWS) {
      const float inv = invs[0][r];
      const u32x2 w = eight_codes<STOCH>(x, inv, h);
      if (row < a.rows)
        *reinterpret_cast<u32x2 *>(a.codes + row * pitch + col) = inv == 0.0f ? u32x2{0u, 0u} : w;
    }
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = STOCH ? drawn_byte(x[i], inv_cols[i], h[i]) : nearest_byte(x[i], inv_cols[i]);
      if (inv_cols[i] == 0.0f) c[i] = 0;
    }
    *reinterpret_cast<u32x2 *>(tile + r * kPad + (tid & 15) * 8) =
        u32x2{four_bytes(c[0], c[1], c[2], c[3]), four_bytes(c[4], c[5], c[6], c[7])};
  }
  __syncthreads();
  // four columns x sixteen rows a thread
  const int g = tid & 31, rows16 = (tid >> 5) * 16;
  u32x4 out[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t *>(tile + (rows16 + q * 4 + i) * kPad + g * 4);
    const uint32_t a01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t a23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), b23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    out[0][q] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
    out[1][q] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
    out[2][q] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
    out[3][q] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c0 + g * 4 + i < a.cols)
      *reinterpret_cast<u32x4 *>(a.codes_t + (c0 + g * 4 + i) * (int64_t)pitch_t + r0 + rows16) = out[i];
}

// ---------------------------------------------------------------- products
// out = (sum a b) sa sb (+ bias) (+ out): the sum is exact, the rest in fp32, rounded once more to
// bf16.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) { return (float)sum * sa * sb; }

__device__ __forceinline__ void put_one(const I8MatmulArgs &a, int64_t m, int64_t n, int sum) {
  float v = scaled(sum, a.a_scales[m], a.b_scales[n]);
  if (a.bias) v += a.bias[n];
  const int64_t at = m * a.ldo + n;
  if (a.out_dtype == 0) {
    float *o = static_cast<float *>(a.out) + at;
    *o = a.accumulate ? *o + v : v;
  } else {
    uint16_t *o = static_cast<uint16_t *>(a.out) + at;
    if (a.accumulate) v += __uint_as_float((uint32_t)*o << 16);
    *o = to_bf16(v);
  }
}

typedef i32x4 i32x4_e4 __attribute__((aligned(4)));

// Tiled product for more than kFewRows rows.  8192 x 11008 x 4096 takes 330-370 us by the card, 2.0-2.2
// POP/s (a loop of nothing but the instruction reaches 3.9 on random data, a library's product of this
// size took 409 us): matrix cores busy 49%, at 1.9 GHz; 1376 tiles fill 5.4 of 6 rounds, and a tile's first
// loads and stores, which nothing covers as one block fills a CU's LDS, took 11 us of its 52 when that
// was fitted.  333 x 50257 x 768 takes 32-37 us, six steps a tile: first loads and stores are most of it.
// What the epilogue needs is loaded before it: row scales read at each store cost a latency every pass
// (8192 x 11008 x 4096 391 us, 371 without).
template <class S>
__global__ __launch_bounds__(S::T) void k_i8_matmul(const I8MatmulArgs a, int pitch, int tiles_m,
                                                    int tiles_n, int steps_each) {
  constexpr int WN = S::WN, R = S::R, C = S::C;
  GQ_TILE_LDS(S);
  int bm, bn;
  tile_at(near_tiles(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, bm, bn);
  bm = uniform(bm);
  bn = uniform(bn);
  const int64_t m0 = (int64_t)bm * S::BM, n0 = (int64_t)bn * S::BN;
  const TileRows ra = {static_cast<const uint8_t *>(a.a) + m0 * pitch, (int)min((int64_t)S::BM, a.M - m0)};
  const TileRows rb = {reinterpret_cast<const uint8_t *>(a.b) + n0 * pitch, (int)min((int64_t)S::BN, a.N - n0)};
  const int step0 = blockIdx.y * steps_each;
  i32x4 acc[R][C] = {};
  tile_product<I8Product, S>(lds0, lds1, lds2, lds3, ra, rb, pitch, step0,
                             min(steps_each, pitch / kStepBytes - step0), acc);
  const int lane = threadIdx.x & 63;
  const int64_t wm0 = m0 + wave / WN * R * 16, wn0 = n0 + wave % WN * C * 16;
  static_assert(S::kSameCols, "a lane's columns");
  const int64_t n = wn0 + S::col_of(0, lane);
  auto nothing = [](int) {};
  if (gridDim.y > 1) {
    int32_t *part = a.partial + (int64_t)blockIdx.y * a.M * a.N;
    by_rows<I8Product, S>(acc, own, [](int, i32x4 v) { return __builtin_bit_cast(f32x4, v); }, nothing,
                          [&](int i, int, int row, int, f32x4 lo, f32x4 hi) {
      const int64_t m = wm0 + i * 32 + row;
      if (m >= a.M || n >= a.N) return;
      int32_t *o = part + m * a.N + n;
      const i32x4 u = __builtin_bit_cast(i32x4, lo), v = __builtin_bit_cast(i32x4, hi);
      if (n + 8 <= a.N) {
        reinterpret_cast<i32x4_e4 *>(o)[0] = u;
        reinterpret_cast<i32x4_e4 *>(o)[1] = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.N) o[e] = e < 4 ? u[e & 3] : v[e & 3];
      }
    }, nothing);
    return;
  }
  // scales of the rows that a lane has before the exchange, scales and biases of the columns that it
  // has after it; no bias is -0, which changes nothing that it is added to
  float sa[R], sb[8], bias[8];
#pragma unroll
  for (int k = 0; k < R; ++k) sa[k] = a.a_scales[min(wm0 + k * 16 + (lane & 15), a.M - 1)];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t c = min(n + e, a.N - 1);
    sb[e] = a.b_scales[c];
    bias[e] = a.bias ? a.bias[c] : -0.0f;
  }
  auto by_token = [&](int k, i32x4 v) { return f32x4{(float)v[0] * sa[k], (float)v[1] * sa[k], (float)v[2] * sa[k], (float)v[3] * sa[k]}; };
  auto finished = [&](f32x4 lo, f32x4 hi, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? lo[e & 3] : hi[e & 3]) * sb[e] + bias[e];
  };
  if (!a.accumulate && n0 + S::BN <= a.N) {
    // Nothing to add to and no row cut short: no questions at the stores but the last rows'.  Rows on
    // 128-byte lines are stored non-temporally, as every store covers whole lines.
    auto leave = [&](auto half_width, auto on_lines) {
      constexpr int kElem = decltype(half_width)::value ? 2 : 4;
      char *const out = static_cast<char *>(a.out) + (wm0 * a.ldo + n) * kElem;
      const int64_t row_bytes = a.ldo * kElem;
      const int rows = (int)min((int64_t)R * 16, a.M - wm0);
      by_rows<I8Product, S>(acc, own, by_token, nothing, [&](int i, int, int row, int, f32x4 lo, f32x4 hi) {
        float v[8];
        finished(lo, hi, v);
        if (i * 32 + row >= rows) return;
        char *o = out + (i * 32 + row) * row_bytes;
        if constexpr (kElem == 2) {
          const u32x4 w = {to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
          if constexpr (decltype(on_lines)::value)
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(o));
          else
            *reinterpret_cast<u32x4_e2 *>(o) = w;
        } else {
          f32x4_e4 *to = reinterpret_cast<f32x4_e4 *>(o);
          to[0] = f32x4{v[0], v[1], v[2], v[3]};
          to[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
      }, nothing);
    };
    if (a.out_dtype == 0)
      leave(std::false_type{}, std::false_type{});
    else if (((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.ldo * 2) & 127) == 0)
      leave(std::true_type{}, std::true_type{});
    else
      leave(std::true_type{}, std::false_type{});
    return;
  }
  by_rows<I8Product, S>(acc, own, by_token, nothing, [&](int i, int, int row, int, f32x4 lo, f32x4 hi) {
    const int64_t m = wm0 + i * 32 + row;
    if (m >= a.M || n >= a.N) return;
    float v[8];
    finished(lo, hi, v);
    const int64_t at = m * a.ldo + n;
    if (n + 8 > a.N) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (n + e < a.N) {
          if (a.out_dtype == 0) {
            float *o = static_cast<float *>(a.out) + at + e;
            *o = a.accumulate ? *o + v[e] : v[e];
          } else {
            uint16_t *o = static_cast<uint16_t *>(a.out) + at + e;
            *o = to_bf16(a.accumulate ? __uint_as_float((uint32_t)*o << 16) + v[e] : v[e]);
          }
        }
      }
    } else if (a.out_dtype == 0) {
      f32x4_e4 *o = reinterpret_cast<f32x4_e4 *>(static_cast<float *>(a.out) + at);
      f32x4 p = {v[0], v[1], v[2], v[3]}, q = {v[4], v[5], v[6], v[7]};
      if (a.accumulate) {
        p += o[0];
        q += o[1];
      }
      o[0] = p;
      o[1] = q;
    } else {
      uint16_t *o = static_cast<uint16_t *>(a.out) + at;
      if (a.accumulate) {
        float x[8];
        load_eight<1>(o, 0, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += x[e];
      }
      *reinterpret_cast<u32x4_e2 *>(o) =
          u32x4{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
    }
  }, nothing);
}

// The partial sums of the K splits; their order does not matter.
__global__ __launch_bounds__(256) void k_i8_join(const I8MatmulArgs a, int splits) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.M * a.N) return;
  int v = 0;
  for (int i = 0; i < splits; ++i) v += a.partial[(int64_t)i * a.M * a.N + t];
  put_one(a, t / a.N, t % a.N, v);
}

// Few rows of A (M <= 16, one decoded token to a small batch): the weights' bytes bound it, so each
// block streams 16 rows of B straight to registers, its waves on interleaved steps of 128, AHEAD steps
// of a wave on their way together: four, or as many as a short row has for each wave.
// v_mfma_i32_16x16x64_i8: lane l holds 16 bytes of row l mod 16 at l / 16.  fp32 / bf16 rows are
// quantised by the block into LDS while its first weights are on their way.  Packed rows are read from
// memory as they are multiplied, behind the weights, so that a step waits for all loads.  The waves' sums
// meet in LDS.  1 x 4096 by 11008 x 4096, 45 MB, takes 13.5 us, 3.3 TB/s: one wait for all weights, which are
// on their way at once, after a launch; 16 rows that a launch of their own packs 20 (15 from 9 packed
// ones, 17 from 16); 1 x 11008 by 4096 x 11008 13.6, and 16.6 from a packed row.
constexpr int kFewWaves = 8;
// LDS of M packed rows: a row is padded by a chunk, so that 16 rows lie on different banks.
inline size_t few_lds(int64_t M, int64_t pitch) { return (size_t)M * (size_t)(pitch + 16); }

// A barrier for what crosses LDS alone: loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int AT, int AHEAD>
__global__ __launch_bounds__(kFewWaves * 64) void k_i8_matmul_few(const I8MatmulArgs a, int pitch) {
  __shared__ i32x4 sums[kFewWaves][64];
  __shared__ uint32_t tops[kFewRows];
  extern __shared__ __align__(16) uint8_t packed[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quarter = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int8_t *b = a.b + min(n0 + r16, a.N - 1) * pitch + quarter * 16;
  const int steps = pitch / 128;
  i32x4 w[AHEAD][2];
  auto load = [&](int k, i32x4 (&to)[2]) {
    const i32x4 *p = reinterpret_cast<const i32x4 *>(b + (int64_t)k * 128);
    to[0] = __builtin_nontemporal_load(p);
    to[1] = __builtin_nontemporal_load(p + 4);
  };
  auto first_weights = [&]() {  // past the end: the last ones again, not multiplied
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(min(wave + i * kFewWaves, steps - 1), w[i]);
  };
  const uint8_t *rows = static_cast<const uint8_t *>(a.a);
  int row_bytes = pitch;
  const int M = (int)a.M;
  if constexpr (AT != 3) {
    row_bytes = pitch + 16;
    int shift = 0;  // a row's share of the threads: 512 >> shift, the rows rounded up to a power of two
    while ((1 << shift) < M) ++shift;
    const int threads = (kFewWaves * 64) >> shift, row = threadIdx.x / threads, t = threadIdx.x % threads;
    // A's first elements before the weights, as loads return in their order
    constexpr int kHeld = 4;
    Raw<AT, 8> raw[kHeld];
    float x[kHeld][8];
    const int64_t row_at = min(row, M - 1) * a.lda;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) raw[i] = raw_word<AT, 8>(a.a, row_at, (int64_t)(t + i * threads) * 8, a.K);
    first_weights();
    if (threadIdx.x < kFewRows) tops[threadIdx.x] = 0;
    lds_barrier();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      open_word(raw[i], a.a, row_at, (int64_t)(t + i * threads) * 8, a.K, x[i]);
      top = max(top, top_of(x[i]));
    }
    if (row < M)
      for (int g = t + kHeld * threads; g * 8 < a.K; g += threads) {
        float more[8];
        load_word<AT>(a.a, row * a.lda, (int64_t)g * 8, a.K, more);
        top = max(top, top_of(more));
      }
    for (int m = 1; m < threads && m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if (row < M && (threads < 64 ? t == 0 : (t & 63) == 0)) atomicMax(&tops[row], top);
    lds_barrier();
    if (row < M) {
      const RowScale s = row_scale(tops[row]);
      const uint32_t h[8] = {};
      auto pack = [&](int g, const float (&v)[8]) {
        const u32x2 c = eight_codes<false>(v, s.inv, h);
        *reinterpret_cast<u32x2 *>(packed + row * row_bytes + g * 8) = s.inv == 0.0f ? u32x2{0u, 0u} : c;
      };
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (t + i * threads < pitch / 8) pack(t + i * threads, x[i]);
      for (int g = t + kHeld * threads; g < pitch / 8; g += threads) {
        float more[8];
        load_word<AT>(a.a, row * a.lda, (int64_t)g * 8, a.K, more);
        pack(g, more);
      }
    }
    rows = packed;
    lds_barrier();
  } else {
    first_weights();
  }
  i32x4 acc = {0, 0, 0, 0};
  auto multiply = [&](int k, const i32x4 (&v)[2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      i32x4 u = {0, 0, 0, 0};
      if (r16 < M) u = *reinterpret_cast<const i32x4 *>(rows + (int64_t)r16 * row_bytes + k * 128 + p * 64 + quarter * 16);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[p], u, acc, 0, 0, 0);
    }
  };
  constexpr int kTurn = AHEAD * kFewWaves;
  int first = wave;
  for (; first + kTurn < steps; first += kTurn) {  // a turn, with the next one's weights on their way
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      multiply(first + i * kFewWaves, w[i]);
      load(min(first + i * kFewWaves + kTurn, steps - 1), w[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (first + i * kFewWaves < steps) multiply(first + i * kFewWaves, w[i]);
  sums[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int from = threadIdx.x >> 2, e = threadIdx.x & 3;
    int v = 0;
#pragma unroll
    for (int i = 0; i < kFewWaves; ++i) v += sums[i][from][e];
    const int64_t m = from & 15, col = n0 + 4 * (from >> 4) + e;
    if (m < a.M && col < a.N) {
      if constexpr (AT != 3) {
        float o = scaled(v, row_scale(tops[m]).scale, a.b_scales[col]);
        if (a.bias) o += a.bias[col];
        const int64_t at = m * a.ldo + col;
        if (a.out_dtype == 0) {
          float *to = static_cast<float *>(a.out) + at;
          *to = a.accumulate ? *to + o : o;
        } else {
          uint16_t *to = static_cast<uint16_t *>(a.out) + at;
          *to = to_bf16(a.accumulate ? __uint_as_float((uint32_t)*to << 16) + o : o);
        }
      } else {
        put_one(a, m, col, v);
      }
    }
  }
}

template <class S>
void tiles_of(const I8MatmulArgs &a, const I8Plan &p, hipStream_t s) {
  const int tm = (int)((a.M + S::BM - 1) / S::BM), tn = (int)((a.N + S::BN - 1) / S::BN);
  k_i8_matmul<S><<<dim3((unsigned)(tm * tn), p.splits), S::T, 0, s>>>(
      a, (int)i8_pitch(a.K), tm, tn, p.each);
}

// Parts of the largest magnitudes: 512 columns each of a row, and of a column as many as give some four
// blocks a CU, at most 256.
struct Parts {
  int rows, cols, rows_each;
};

Parts tops_parts(int64_t rows, int64_t cols) {
  Parts p;
  p.rows = (int)((cols + 511) / 512);
  int64_t n = (4 * kCus + p.rows - 1) / p.rows, most = (rows + 63) / 64;
  if (n > 256) n = 256;
  if (n > most) n = most;
  p.rows_each = (int)(((rows + n - 1) / n + 63) / 64 * 64);
  p.cols = (int)((rows + p.rows_each - 1) / p.rows_each);
  return p;
}

template <int DT, bool STOCH>
void quantize_of(const I8QuantArgs &a, hipStream_t s) {
  const int pitch = (int)i8_pitch(a.cols);
  if (!a.codes_t) {
    // a row in a wave's registers where it fits, else in a block's, else read twice
    if (a.cols <= 1024)
      k_i8_rows<DT, STOCH, 1, 2><<<(unsigned)((a.rows + 3) / 4), 256, 0, s>>>(a, pitch);
    else if (a.cols <= 4096)
      k_i8_rows<DT, STOCH, 4, 2><<<(unsigned)a.rows, 256, 0, s>>>(a, pitch);
    else if (a.cols <= 12288)
      k_i8_rows<DT, STOCH, 4, 6><<<(unsigned)a.rows, 256, 0, s>>>(a, pitch);
    else
      k_i8_rows<DT, STOCH, 4, 0><<<(unsigned)a.rows, 256, 0, s>>>(a, pitch);
    return;
  }
  const int pitch_t = (int)i8_pitch(a.rows);
  const Parts t = tops_parts(a.rows, a.cols);
  const dim3 parts((unsigned)t.rows, (unsigned)t.cols);
  const dim3 tiles((unsigned)(pitch / 128), (unsigned)(pitch_t / 128));
  if (a.codes) {
    k_i8_tops<DT, true><<<parts, 256, 0, s>>>(a, t.rows_each);
    k_i8_both<DT, STOCH, true><<<tiles, 256, 0, s>>>(a, pitch, pitch_t, t.rows, t.cols);
  } else {
    k_i8_tops<DT, false><<<parts, 256, 0, s>>>(a, t.rows_each);
    k_i8_both<DT, STOCH, false><<<tiles, 256, 0, s>>>(a, pitch, pitch_t, 0, t.cols);
  }
}

}  // namespace

size_t i8_quantize_scratch(int64_t rows, int64_t cols, bool by_cols) {
  if (!by_cols) return 0;
  const Parts p = tops_parts(rows, cols);
  return ((size_t)p.rows * (size_t)rows + (size_t)p.cols * (size_t)cols) * sizeof(uint32_t);
}

hipError_t launch_i8_quantize(const I8QuantArgs &a, int dtype, hipStream_t s) {
  if (a.rows == 0)
    k_i8_no_rows<<<(unsigned)((a.cols + 255) / 256), 256, 0, s>>>(a.scales_t, a.cols);
  else if (dtype == 0)
    a.stochastic ? quantize_of<0, true>(a, s) : quantize_of<0, false>(a, s);
  else
    a.stochastic ? quantize_of<1, true>(a, s) : quantize_of<1, false>(a, s);
  return hipGetLastError();
}

bool i8_matmul_packs_rows(int64_t M, int64_t K) { return M <= kFewRows && M * i8_pitch(K) <= 32768; }

size_t i8_matmul_scratch(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewRows) return 0;
  const I8Plan p = i8_plan(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(int32_t) : 0;
}

hipError_t launch_i8_matmul(const I8MatmulArgs &a, hipStream_t s) {
  const int pitch = (int)i8_pitch(a.K);
  if (a.M <= kFewRows) {
    const unsigned blocks = (unsigned)((a.N + 15) / 16);
    const size_t lds = few_lds(a.M, pitch);
    const int64_t steps = (pitch / 128 + kFewWaves - 1) / kFewWaves;  // of a wave
    auto few = [&](auto ahead) {
      constexpr int kAhead = decltype(ahead)::value;
      if (a.a_dtype == 0)
        k_i8_matmul_few<0, kAhead><<<blocks, kFewWaves * 64, lds, s>>>(a, pitch);
      else if (a.a_dtype == 1)
        k_i8_matmul_few<1, kAhead><<<blocks, kFewWaves * 64, lds, s>>>(a, pitch);
      else
        k_i8_matmul_few<3, kAhead><<<blocks, kFewWaves * 64, 0, s>>>(a, pitch);
    };
    if (steps == 1)
      few(std::integral_constant<int, 1>{});
    else if (steps == 2)
      few(std::integral_constant<int, 2>{});
    else
      few(std::integral_constant<int, 4>{});
    return hipGetLastError();
  }
  const I8Plan p = i8_plan(a.M, a.N, a.K);
  if (p.bm == 256)
    tiles_of<TileShape<2, 4, 8, 4, 2>>(a, p, s);
  else if (p.bm == 128)
    tiles_of<TileShape<2, 2, 4, 4, 2>>(a, p, s);
  else
    tiles_of<TileShape<1, 4, 4, 2, 2>>(a, p, s);
  if (p.splits > 1) k_i8_join<<<(unsigned)((a.M * a.N + 255) / 256), 256, 0, s>>>(a, p.splits);
  return hipGetLastError();
}

}  // namespace gq
