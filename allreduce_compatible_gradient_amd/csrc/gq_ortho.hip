// gq_ortho.hip -- gfx950 kernels that bring a matrix's singular values towards 1 by steps of
//   X <- a X + (b A + c A^2) X,   A = X X^T,   from X = G / |G|_F,
// with products alone (Newton-Schulz).  Everything is done on the shorter side: n <= m, X n x m, the
// transpose of a tall G.
//
// Numbers.  Operands of the products are halves, sums fp32, and X itself stays fp32.  Four choices
// make that enough for a result in bf16.  Halves and not bf16: 3 bits more, and all operands have
// known ranges, which powers of two bring into the halves' (X to at most 2^8 |x|, the others to
// 2^10).  The diagonals of A and of B = b A + c A^2, large where the rest is small, stay apart in fp32:
// with A = D + F,  A^2 = D^2 + D F + F D + F^2, and only F^2 is a product of rounded numbers; likewise
// X <- (a + diag B) X + (B - diag B) X.  And a X, which carries a small singular value through the
// steps that raise it up to a^steps-fold, is taken from the fp32 X.  Last, what X's halves h differ
// from X by is noise in every direction, also in those that X does not have, where it grows a-fold a
// step: (B - diag B) h + diag B X leaves -diag B (h - X) there, which for one direction in few rows came to
// 4e-2 of the result in five steps, and to all of it in eight.  Before the last two steps therefore either h carries all of X (two halves an
// element: small matrices), or diag B multiplies h as well, so that the noise is multiplied by the whole
// of B and stays in X's directions; in the last two the noise of a large diag B would count for more than
// what still grows.
// The relative error (Frobenius) before the last rounding, by a model of these roundings: 1e-4 to 1.3e-3 for random,
// heavy-tailed and nearly low-rank matrices, where halves alone have 2e-3 to 7e-3 and bf16 1e-2 to
// 1e-1; up to 3e-3 for one to eight directions, in few rows and columns too; 2e-3, at worst 1.2e-2, where
// all elements are alike, as all roundings then have one sign.  Rounding to bf16 adds 1.7e-3.
//
// Work.  A and A^2 are symmetric: tiles on and above the diagonal are computed and stored both ways.
// A step is three launches: the Gram matrix (of X's halves), its square, and the update, which
// writes X in fp32, its halves by rows for the next Gram matrix, and by columns for the next update.
// By the card 4096 x 4096 takes 1.39 to 1.41 ms (0.98 PFLOP/s of what the definition cannot do without),
// 11008 x 4096 3.43 to 3.51 (0.90), twelve of 768 x 2304 0.64 to 0.67.  A profiler, whose times add up to a
// tenth more, has 155 us for a step's Gram matrix and square and 143 for its update in the first, 278 and 401
// in the second, 50 and 78 in the third, and 53, 115 and 67 for what comes before the steps.  The
// products reach 1.0 to 1.2 PFLOP/s (a library's product of 4096 x 4096 halves took 105 us, 1.3; a loop
// of nothing but the instruction 1.8 on random data); an update's epilogue reads and writes 12 bytes
// an element of X, 31 us of its 143 at 4096 x 4096 at the card's best rate, when all tiles end
// together, and is most of it where n is small.
#include <math.h>

#include "gq_layers.h"
#include "gq_tiles.h"

namespace gq {
namespace {

constexpr float kScaleX = 256.0f, kScaleB = 1024.0f;
constexpr int kNormBlocks = 1024;

// One group of matrices; every array holds `batch` of them, one after another.
struct Work {
  float *x;             // n x mp
  _Float16 *xh;         // n x mp
  _Float16 *xt[2];      // m x np, of this step and the next
  _Float16 *f;          // n x np: A off its diagonal
  _Float16 *b;          // n x np: B off its diagonal
  float *diag_a, *diag_b;  // np
  double *norms;        // kNormBlocks
  float *partial;       // splits of the Gram matrix
  int n, m, np, mp;     // np, mp: rounded up to 64
};

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
}

__device__ __forceinline__ u32x4 eight_halves(const float (&v)[8]) {
  return u32x4{pack_half(v[0], v[1]), pack_half(v[2], v[3]), pack_half(v[4], v[5]), pack_half(v[6], v[7])};
}

// ---------------------------------------------------------------- G to X
// Sums of squares in 64 bits, one a block: four rows' eight elements a thread on their way together.
template <int DT>
__global__ __launch_bounds__(256) void k_ortho_norm(const OrthoArgs a, double *norms) {
  __shared__ double part[4];
  const int64_t base = (int64_t)blockIdx.y * a.stride_g;
  double sum = 0.0;
  const int64_t stride = (int64_t)gridDim.x * blockDim.y;
  for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += (int64_t)blockDim.x * 8)
    for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < a.rows; r += 4 * stride) {
      Raw<DT, 8> raw[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) raw[u] = raw_word<DT, 8>(a.g, base + min(r + u * stride, a.rows - 1) * a.ldg, c, a.cols);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r + u * stride >= a.rows) break;
        float x[8];
        open_word(raw[u], a.g, base + (r + u * stride) * a.ldg, c, a.cols, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)x[i] * (double)x[i];
      }
    }
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
  if ((tid & 63) == 0) part[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) norms[(int64_t)blockIdx.y * kNormBlocks + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// X in fp32 and in halves both ways, padding zero, 64 x 64 elements a block.  A matrix of zeros stays
// one; one with an infinity or NaN becomes NaN everywhere.
template <int DT, bool FLIP>
__global__ __launch_bounds__(256) void k_ortho_start(const OrthoArgs a, const Work w, int parts) {
  __shared__ float tile[64][65];
  __shared__ double sums[4];
  const int tid = threadIdx.x;
  const int64_t k = blockIdx.z;
  double sum = 0.0;
  for (int i = tid; i < parts; i += 256) sum += w.norms[k * kNormBlocks + i];
  for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
  if ((tid & 63) == 0) sums[tid >> 6] = sum;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int64_t r0 = FLIP ? j0 : i0, c0 = FLIP ? i0 : j0;  // the tile's place in G
  const int64_t base = k * a.stride_g;
  Raw<DT, 8> raw[2];  // rows past the end: the last one again, not kept
#pragma unroll
  for (int p = 0; p < 2; ++p)
    raw[p] = raw_word<DT, 8>(a.g, base + min(r0 + p * 32 + (tid >> 3), a.rows - 1) * a.ldg, c0 + (tid & 7) * 8, a.cols);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = p * 32 + (tid >> 3), c = (tid & 7) * 8;
    float x[8];
    open_word(raw[p], a.g, base + min(r0 + r, a.rows - 1) * a.ldg, c0 + c, a.cols, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (FLIP)
        tile[c + i][r] = x[i];
      else
        tile[r][c + i] = x[i];
    }
  }
  __syncthreads();
  const double total = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const double inv = total > 0.0 ? 1.0 / sqrt(total) : total == 0.0 ? 0.0 : total;
  const bool bad = !(total < INFINITY);
  auto value = [&](float g) { return bad ? NAN : (float)((double)g * inv); };
  float *x = w.x + k * w.n * w.mp;
  _Float16 *xh = w.xh + k * w.n * w.mp, *xt = w.xt[0] + k * w.m * w.np;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = p * 32 + (tid >> 3), c = (tid & 7) * 8;
    float v[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = j0 + c + i < w.m ? value(tile[r][c + i]) : 0.0f;  // (rows past n are not stored)
      h[i] = v[i] * kScaleX;
    }
    if (i0 + r < w.n) {
      const int64_t at = (int64_t)(i0 + r) * w.mp + j0 + c;
      *reinterpret_cast<f32x4 *>(x + at) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4 *>(x + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      *reinterpret_cast<u32x4 *>(xh + at) = eight_halves(h);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i0 + c + i < w.n ? value(tile[c + i][r]) * kScaleX : 0.0f;
    if (j0 + r < w.m) *reinterpret_cast<u32x4 *>(xt + (int64_t)(j0 + r) * w.np + i0 + c) = eight_halves(h);
  }
}

// ---------------------------------------------------------------- products
// A wave's 32 x 16 C halves by columns, from what by_rows' lanes hold, through the wave's part of LDS
// (columns of 72 bytes: the rows' writes fall on different banks): f(column, first row, eight rows).
template <class S, class F>
__device__ __forceinline__ void by_columns(const u32x4 (&keep)[S::C], uint8_t *own, F &&f) {
  static_assert(S::kOwn >= S::C * 16 * 72, "a wave's columns fit its part");
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int p = 0; p < S::C; ++p) {
    const int row = S::row_of(p, lane), col = S::col_of(p, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<uint16_t *>(own + (col + e) * 72 + row * 2) = (uint16_t)(keep[p][e >> 1] >> (16 * (e & 1)));
  }
  wave_exchange();
#pragma unroll
  for (int p = 0; p < S::C; ++p) {
    const int c = p * 16 + (lane >> 2), piece = lane & 3;
    const u32x2 lo = *reinterpret_cast<const u32x2 *>(own + c * 72 + piece * 16);
    const u32x2 hi = *reinterpret_cast<const u32x2 *>(own + c * 72 + piece * 16 + 8);
    f(c, piece * 8, u32x4{lo.x, lo.y, hi.x, hi.y});
  }
  wave_exchange();
}

// Tile t of the triangle of tiles on and above the diagonal, row after row.
__device__ __forceinline__ void triangle_at(int t, int tiles, int &i, int &j) {
  // row i begins at i tiles - i (i - 1) / 2
  const float b = 2.0f * tiles + 1.0f;
  i = (int)((b - sqrtf(b * b - 8.0f * t)) * 0.5f);
  while (i > 0 && i * tiles - i * (i - 1) / 2 > t) --i;
  while ((i + 1) * tiles - (i + 1) * i / 2 <= t) ++i;
  j = t - (i * tiles - i * (i - 1) / 2) + i;
}

// A symmetric product of the rows of `of` (n of them, pitch bytes each).  SQUARE false: the Gram
// matrix of X, to F and diag_a (or partial sums, where gridDim.y > 1); true: F^2, to B and diag_b.
template <bool SQUARE, class S>
__global__ __launch_bounds__(S::T) void k_ortho_symmetric(const Work w, float cb, float cc, int tiles,
                                                          int steps_each) {
  constexpr int WN = S::WN, R = S::R, C = S::C;
  GQ_TILE_LDS(S);
  const int lane = threadIdx.x & 63;
  static_assert(S::BM == S::BN, "mirrored tiles");
  // a matrix's tiles lie on one XCD or two, which read its operands once
  const int count = tiles * (tiles + 1) / 2, all = near_tiles(blockIdx.x, gridDim.x);
  const int matrix = uniform(all / count), tile = uniform(all % count);
  const int64_t k = matrix;
  int ti, tj;
  triangle_at(tile, tiles, ti, tj);
  ti = uniform(ti);
  tj = uniform(tj);
  const int pitch = (SQUARE ? w.np : w.mp) * 2, i0 = ti * S::BM, j0 = tj * S::BN;
  const uint8_t *of = reinterpret_cast<const uint8_t *>(SQUARE ? w.f : w.xh) + k * w.n * pitch;
  const TileRows ra = {of + (int64_t)i0 * pitch, min(S::BM, w.n - i0)};
  const TileRows rb = {of + (int64_t)j0 * pitch, min(S::BN, w.n - j0)};
  const int step0 = blockIdx.y * steps_each;
  f32x4 acc[R][C] = {};
  tile_product<F16Product, S>(lds0, lds1, lds2, lds3, ra, rb, pitch, step0,
                                           min(steps_each, pitch / kStepBytes - step0), acc);
  const int wi = wave / WN * R * 16, wj = wave % WN * C * 16;
  auto as_is = [](int, f32x4 v) { return v; };
  if (!SQUARE && gridDim.y > 1) {
    float *part = w.partial + ((k * gridDim.y + blockIdx.y) * count + tile) * (S::BM * S::BN);
    by_rows<F16Product, S>(acc, own, as_is, [](int) {}, [&](int i, int, int row, int col, f32x4 lo, f32x4 hi) {
      f32x4 *o = reinterpret_cast<f32x4 *>(part + (wi + i * 32 + row) * S::BN + wj + col);
      o[0] = lo;
      o[1] = hi;
    }, [](int) {});
    return;
  }
  _Float16 *const to = (SQUARE ? w.b : w.f) + k * w.n * w.np;
  const _Float16 *const f = w.f + k * w.n * w.np;
  const float *const da = w.diag_a + k * w.np;
  float *const diag = (SQUARE ? w.diag_b : w.diag_a) + k * w.np;
  constexpr int kCols = S::kSameCols ? 1 : C;  // different columns that a lane has
  float dj[kCols][8];
  if (SQUARE) {
#pragma unroll
    for (int p = 0; p < kCols; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + wj + S::col_of(p, lane) + e;
        dj[p][e] = j < w.n ? da[j] : 0.0f;
      }
  }
  u32x4 keep[C];
  f16x8 olds[2][C];
  float dis[2][C];
  by_rows<F16Product, S>(acc, own, as_is, [&](int i32) {
    if (!SQUARE) return;
#pragma unroll
    for (int p = 0; p < C; ++p) {
      const int i = min(i0 + wi + i32 * 32 + S::row_of(p, lane), w.n - 1);
      dis[i32 & 1][p] = da[i];
      olds[i32 & 1][p] = *reinterpret_cast<const f16x8 *>(f + (int64_t)i * w.np + min(j0 + wj + S::col_of(p, lane), w.np - 8));
    }
  }, [&](int i32, int p, int row, int col, f32x4 lo, f32x4 hi) {
    const int i = i0 + wi + i32 * 32 + row, j = j0 + wj + col;
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    const bool there = i < w.n && j < w.np;
    const float di = SQUARE ? dis[i32 & 1][p] : 0.0f;
    const f16x8 old = SQUARE ? olds[i32 & 1][p] : f16x8{};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool on = i == j + e, in = i < w.n && j + e < w.n;
      float r;
      if (SQUARE) {
        const float sq = v[e] * (1.0f / (kScaleB * kScaleB)), fe = (float)old[e] * (1.0f / kScaleB);
        if (on && in) diag[i] = cb * di + cc * (di * di + sq);
        r = cb * fe + cc * ((di + dj[S::kSameCols ? 0 : p][e]) * fe + sq);
      } else {
        r = v[e] * (1.0f / (kScaleX * kScaleX));
        if (on && in) diag[i] = r;
      }
      v[e] = on || !in ? 0.0f : r * kScaleB;
    }
    keep[p] = eight_halves(v);
    if (there) *reinterpret_cast<u32x4 *>(to + (int64_t)i * w.np + j) = keep[p];
  }, [&](int i32) {
    if (ti == tj) return;
    by_columns<S>(keep, own, [&](int c, int r, u32x4 h) {
      const int col = j0 + wj + c, row = i0 + wi + i32 * 32 + r;
      if (col < w.n && row < w.np) *reinterpret_cast<u32x4 *>(to + (int64_t)col * w.np + row) = h;
    });
  });
}

// The Gram matrix from the partial sums of its splits: a block 64 x 64 elements of a tile.
__global__ __launch_bounds__(256) void k_ortho_join(const Work w, int tiles, int side, int splits) {
  __shared__ float tile[64][65];
  const int subs = side / 64, tid = threadIdx.x;
  const int t = blockIdx.x / (subs * subs), sub = blockIdx.x % (subs * subs);
  const int count = tiles * (tiles + 1) / 2;
  int ti, tj;
  triangle_at(t, tiles, ti, tj);
  const int64_t k = blockIdx.z;
  const int si = sub / subs * 64, sj = sub % subs * 64;
  const int i0 = ti * side + si, j0 = tj * side + sj;
  if (i0 >= w.np || j0 >= w.np) return;
  _Float16 *f = w.f + k * w.n * w.np;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = p * 32 + (tid >> 3), c = (tid & 7) * 8;
    float v[8] = {};
    for (int s = 0; s < splits; ++s) {
      const float *part = w.partial + ((k * splits + s) * count + t) * ((int64_t)side * side) + (si + r) * side + sj + c;
      const f32x4 lo = *reinterpret_cast<const f32x4 *>(part), hi = *reinterpret_cast<const f32x4 *>(part + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += lo[e];
        v[4 + e] += hi[e];
      }
    }
    const int i = i0 + r;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + c + e;
      const bool in = i < w.n && j < w.n;
      const float x = v[e] * (1.0f / (kScaleX * kScaleX));
      if (i == j && in) w.diag_a[k * w.np + i] = x;
      v[e] = i == j || !in ? 0.0f : x * kScaleB;
      tile[r][c + e] = v[e];
    }
    if (i < w.n) *reinterpret_cast<u32x4 *>(f + (int64_t)i * w.np + j0 + c) = eight_halves(v);
  }
  if (ti == tj) return;  // (a tile on the diagonal is computed whole)
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = p * 32 + (tid >> 3), c = (tid & 7) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[c + e][r];
    if (j0 + r < w.n) *reinterpret_cast<u32x4 *>(f + (int64_t)(j0 + r) * w.np + i0 + c) = eight_halves(v);
  }
}

// X <- (a + diag B) X + (B - diag B) X; the last step's goes to `out` in bf16, by columns for a tall G.
// `early`: diag B multiplies X's halves, as the product does, and a alone X itself.
template <class S>
__global__ __launch_bounds__(S::T) void k_ortho_update(const Work w, const OrthoArgs o, float ca,
                                                       int tiles_i, int tiles_j, int early, int last) {
  constexpr int WN = S::WN, R = S::R, C = S::C;
  GQ_TILE_LDS(S);
  const int lane = threadIdx.x & 63;
  const int all = near_tiles(blockIdx.x, gridDim.x);
  const int64_t k = uniform(all / (tiles_i * tiles_j));
  int ti, tj;
  tile_at(uniform(all % (tiles_i * tiles_j)), tiles_i, tiles_j, ti, tj);
  ti = uniform(ti);
  tj = uniform(tj);
  const int pitch = w.np * 2, i0 = ti * S::BM, j0 = tj * S::BN;
  const uint8_t *b = reinterpret_cast<const uint8_t *>(w.b + k * w.n * w.np);
  const uint8_t *xt = reinterpret_cast<const uint8_t *>(w.xt[0] + k * w.m * w.np);
  const TileRows ra = {b + (int64_t)i0 * pitch, min(S::BM, w.n - i0)};
  const TileRows rb = {xt + (int64_t)j0 * pitch, min(S::BN, w.m - j0)};
  f32x4 acc[R][C] = {};
  tile_product<F16Product, S>(lds0, lds1, lds2, lds3, ra, rb, pitch, 0, pitch / kStepBytes, acc);
  const int wi = wave / WN * R * 16, wj = wave % WN * C * 16;
  float *const x = w.x + k * w.n * w.mp;
  _Float16 *const xh = w.xh + k * w.n * w.mp, *const next = w.xt[1] + k * w.m * w.np;
  const float *const diag = w.diag_b + k * w.np;
  uint16_t *const out = static_cast<uint16_t *>(o.out) + k * o.stride_o;
  const bool flip = o.rows > o.cols;
  u32x4 keep[C];
  f32x4 xs[2][C][2];
  float ds[2][C];
  by_rows<F16Product, S>(acc, own, [](int, f32x4 v) { return v; }, [&](int i32) {
#pragma unroll
    for (int p = 0; p < C; ++p) {
      const int i = min(i0 + wi + i32 * 32 + S::row_of(p, lane), w.n - 1);
      const f32x4 *at = reinterpret_cast<const f32x4 *>(x + (int64_t)i * w.mp + min(j0 + wj + S::col_of(p, lane), w.mp - 8));
      xs[i32 & 1][p][0] = at[0];
      xs[i32 & 1][p][1] = at[1];
      ds[i32 & 1][p] = diag[i];
    }
  }, [&](int i32, int p, int row, int col, f32x4 lo, f32x4 hi) {
    const int i = i0 + wi + i32 * 32 + row, j = j0 + wj + col;
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}, h[8] = {};
    const bool there = i < w.n && j < w.mp;
    if (there) {
      float *at = x + (int64_t)i * w.mp + j;
      const f32x4 x0 = xs[i32 & 1][p][0], x1 = xs[i32 & 1][p][1];
      const float d = ds[i32 & 1][p], whole = early ? ca : ca + d, rounded = early ? d * (1.0f / kScaleX) : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float was = e < 4 ? x0[e & 3] : x1[e & 3];
        v[e] = whole * was + (v[e] * (1.0f / (kScaleX * kScaleB)) + rounded * (float)(_Float16)(was * kScaleX));
        if (j + e >= w.m) v[e] = 0.0f;
        h[e] = v[e] * kScaleX;
      }
      if (!last) {
        *reinterpret_cast<f32x4 *>(at) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4 *>(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
        *reinterpret_cast<u32x4 *>(xh + (int64_t)i * w.mp + j) = eight_halves(h);
      }
    }
    if (!last) {
      keep[p] = eight_halves(h);
    } else {
      keep[p] = u32x4{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
      if (!flip && there && j < w.m) {
        uint16_t *at = out + (int64_t)i * o.ldo + j;
        if (j + 8 <= w.m) {
          *reinterpret_cast<u32x4_e2 *>(at) = keep[p];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (j + e < w.m) at[e] = (uint16_t)(keep[p][e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }, [&](int i32) {
    if (last && !flip) return;
    by_columns<S>(keep, own, [&](int c, int r, u32x4 h) {
      const int col = j0 + wj + c, row = i0 + wi + i32 * 32 + r;
      if (col >= w.m) return;
      if (!last) {
        if (row < w.np) *reinterpret_cast<u32x4 *>(next + (int64_t)col * w.np + row) = h;
      } else if (row < w.n) {
        uint16_t *at = out + (int64_t)col * o.ldo + row;
        if (row + 8 <= w.n) {
          *reinterpret_cast<u32x4_e2 *>(at) = h;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row + e < w.n) at[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
        }
      }
    });
  });
}

// ---------------------------------------------------------------- small matrices
// n <= 64, m <= MP: a block a matrix, all steps in one launch, where the tiled way takes seventeen
// launches of some 3.7 us each whatever the size.  X stays in registers, four neighbouring columns of
// a row a lane and tile (the products' own layout), its halves by rows and by columns in LDS, and so do
// F and B; rows are padded by 16 bytes, so that 16 rows' reads fall on different banks.  A wave has
// MP / 8 columns of X, and two of the sixteen tiles of A and of A^2.  64 x 147 takes 28 us, 25 of them
// without the second halves of three steps, and 67 the tiled way.
template <int DT, int MP>
__global__ __launch_bounds__(512) void k_ortho_small(const OrthoArgs a) {
  constexpr int kRow = MP * 2 + 16, kSquare = 64 * 2 + 16, kTiles = MP / 128;
  __shared__ __align__(16) uint8_t xh[64 * kRow];
  __shared__ __align__(16) uint8_t xt[MP * kSquare];
  __shared__ __align__(16) uint8_t fs[64 * kSquare];
  __shared__ __align__(16) uint8_t bs[64 * kSquare];
  __shared__ float diag_a[64], diag_b[64];
  __shared__ double sums[8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, four = (lane >> 4) * 4;
  const bool flip = a.rows > a.cols;
  const int n = (int)(flip ? a.cols : a.rows), m = (int)(flip ? a.rows : a.cols);
  const int64_t base = (int64_t)blockIdx.x * a.stride_g;
  float x[kTiles][4][4];  // tile of columns, tile of rows, columns
  double sum = 0.0;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = r * 16 + r16, j = (wave * kTiles + t) * 16 + four + e;
        x[t][r][e] = i < n && j < m ? load_one<DT>(a.g, base + (flip ? j * a.ldg + i : i * a.ldg + j)) : 0.0f;
        sum += (double)x[t][r][e] * (double)x[t][r][e];
      }
  for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += sums[w];
  const double inv = total > 0.0 ? 1.0 / sqrt(total) : 0.0;
  const bool bad = !(total < INFINITY);
  auto share = [&]() {  // X's halves
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = r * 16 + r16, j = (wave * kTiles + t) * 16 + four;
        const float *v = x[t][r];
        const u32x2 h = {pack_half(v[0] * kScaleX, v[1] * kScaleX), pack_half(v[2] * kScaleX, v[3] * kScaleX)};
        *reinterpret_cast<u32x2 *>(xh + i * kRow + j * 2) = h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint16_t *>(xt + (j + e) * kSquare + i * 2) = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
      }
  };
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][r][e] = bad ? NAN : (float)((double)x[t][r][e] * inv);
  share();
  __syncthreads();
  auto piece = [&](const uint8_t *rows, int pitch, int tile, int k) {  // 32 halves of a tile's rows
    return *reinterpret_cast<const i32x4 *>(rows + (tile * 16 + r16) * pitch + k * 64 + (lane >> 4) * 16);
  };
  const int ti = wave >> 1, tj = (wave & 1) * 2;
  for (int step = 0; step < a.steps; ++step) {
    // X's columns; where they are two halves an element, the second ones in their place (a wave reads no
    // other wave's)
    const bool early = step < a.steps - 2;
    i32x4 columns[kTiles][2];
    auto take = [&]() {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) columns[t][k] = piece(xt, kSquare, wave * kTiles + t, k);
    };
    take();
    if (early) {
      wave_exchange();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = x[t][r][e] * kScaleX;
            *reinterpret_cast<_Float16 *>(xt + ((wave * kTiles + t) * 16 + four + e) * kSquare + (r * 16 + r16) * 2) =
                (_Float16)(v - (float)(_Float16)v);
          }
      wave_exchange();
    }
    float f[2][4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int k = 0; k < MP / 32; ++k) acc = F16Product::mul(piece(xh, kRow, tj + q, k), piece(xh, kRow, ti, k), acc);
      const int i = ti * 16 + r16, j = (tj + q) * 16 + four;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[q][e] = acc[e] * (1.0f / (kScaleX * kScaleX));
        if (i == j + e) {
          diag_a[i] = f[q][e];
          f[q][e] = 0.0f;
        }
      }
      *reinterpret_cast<u32x2 *>(fs + i * kSquare + j * 2) =
          u32x2{pack_half(f[q][0] * kScaleB, f[q][1] * kScaleB), pack_half(f[q][2] * kScaleB, f[q][3] * kScaleB)};
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 2; ++k) acc = F16Product::mul(piece(fs, kSquare, tj + q, k), piece(fs, kSquare, ti, k), acc);
      const int i = ti * 16 + r16, j = (tj + q) * 16 + four;
      const float di = diag_a[i];
      float b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float sq = acc[e] * (1.0f / (kScaleB * kScaleB));
        b[e] = (a.b * f[q][e] + a.c * ((di + diag_a[j + e]) * f[q][e] + sq)) * kScaleB;
        if (i == j + e) {
          diag_b[i] = a.b * di + a.c * (di * di + sq);
          b[e] = 0.0f;
        }
      }
      *reinterpret_cast<u32x2 *>(bs + i * kSquare + j * 2) = u32x2{pack_half(b[0], b[1]), pack_half(b[2], b[3])};
    }
    __syncthreads();
    auto multiply = [&](const i32x4 (&columns)[kTiles][2], f32x4 (&acc)[kTiles][4]) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < 2; ++k) acc[t][r] = F16Product::mul(columns[t][k], piece(bs, kSquare, r, k), acc[t][r]);
    };
    f32x4 acc[kTiles][4] = {};
    multiply(columns, acc);
    if (early) {
      take();
      multiply(columns, acc);
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float s = a.a + diag_b[r * 16 + r16];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][r][e] = s * x[t][r][e] + acc[t][r][e] * (1.0f / (kScaleX * kScaleB));
      }
    if (step == a.steps - 1) break;
    __syncthreads();  // every wave is past its reads of X's halves
    share();
    __syncthreads();
  }
  uint16_t *const out = static_cast<uint16_t *>(a.out) + (int64_t)blockIdx.x * a.stride_o;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = r * 16 + r16, j = (wave * kTiles + t) * 16 + four + e;
        if (i < n && j < m) out[flip ? j * a.ldo + i : i * a.ldo + j] = to_bf16(x[t][r][e]);
      }
}

// ---------------------------------------------------------------- host
constexpr size_t kGroupBytes = (size_t)2 << 30;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Sizes {
  size_t x, xh, xt, f, diag, norms, partial;
  size_t all() const { return x + xh + 2 * xt + 2 * f + 2 * diag + norms + partial; }
};

Sizes sizes_of(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t n = rows < cols ? rows : cols, m = rows < cols ? cols : rows, np = up64(n), mp = up64(m);
  const Side g = gram_plan(batch, n, m);
  const int64_t t = (n + g.side - 1) / g.side;
  Sizes z;
  z.x = up256((size_t)(batch * n * mp) * 4);
  z.xh = up256((size_t)(batch * n * mp) * 2);
  z.xt = up256((size_t)(batch * m * np) * 2);
  z.f = up256((size_t)(batch * n * np) * 2);
  z.diag = up256((size_t)(batch * np) * 4);
  z.norms = up256((size_t)batch * kNormBlocks * 8);
  z.partial = g.splits > 1 ? up256((size_t)(batch * g.splits * (t * (t + 1) / 2)) * g.side * g.side * 4) : 0;
  return z;
}

template <bool SQUARE, class S>
void symmetric(const Work &w, const OrthoArgs &a, int64_t batch, int splits, int each, hipStream_t s) {
  const int t = (w.n + S::BM - 1) / S::BM;
  k_ortho_symmetric<SQUARE, S>
      <<<dim3((unsigned)(t * (t + 1) / 2 * batch), (unsigned)splits), S::T, 0, s>>>(w, a.b, a.c, t, each);
}

template <bool SQUARE>
void symmetric_of(const Side &p, const Work &w, const OrthoArgs &a, int64_t batch, hipStream_t s) {
  if (p.side == 256)
    symmetric<SQUARE, TileShape<2, 4, 8, 4, 2>>(w, a, batch, p.splits, p.each, s);
  else if (p.side == 192)
    symmetric<SQUARE, TileShape<2, 4, 6, 3, 2>>(w, a, batch, p.splits, p.each, s);
  else if (p.side == 128 && p.alone)
    symmetric<SQUARE, TileShape<2, 2, 4, 4, 4>>(w, a, batch, p.splits, p.each, s);
  else if (p.side == 128)
    symmetric<SQUARE, TileShape<2, 2, 4, 4, 2>>(w, a, batch, p.splits, p.each, s);
  else
    symmetric<SQUARE, TileShape<2, 2, 2, 2, 4>>(w, a, batch, p.splits, p.each, s);
}

template <class S>
void update(const Work &w, const OrthoArgs &a, int64_t batch, int early, int last, hipStream_t s) {
  const int ti = (w.n + S::BM - 1) / S::BM, tj = (w.m + S::BN - 1) / S::BN;
  k_ortho_update<S><<<(unsigned)(ti * tj * batch), S::T, 0, s>>>(w, a, a.a, ti, tj, early, last);
}

template <int DT>
void small(const OrthoArgs &a, hipStream_t s) {
  const int64_t m = a.rows < a.cols ? a.cols : a.rows;
  if (m <= 128)
    k_ortho_small<DT, 128><<<(unsigned)a.batch, 512, 0, s>>>(a);
  else if (m <= 256)
    k_ortho_small<DT, 256><<<(unsigned)a.batch, 512, 0, s>>>(a);
  else
    k_ortho_small<DT, 512><<<(unsigned)a.batch, 512, 0, s>>>(a);
}

template <int DT>
void group(const OrthoArgs &a, hipStream_t s) {
  const int64_t n = a.rows < a.cols ? a.rows : a.cols, m = a.rows < a.cols ? a.cols : a.rows;
  const Sizes z = sizes_of(a.batch, a.rows, a.cols);
  char *p = static_cast<char *>(a.scratch);
  auto take = [&](size_t bytes) {
    char *q = p;
    p += bytes;
    return q;
  };
  Work w;
  w.n = (int)n;
  w.m = (int)m;
  w.np = (int)up64(n);
  w.mp = (int)up64(m);
  w.x = reinterpret_cast<float *>(take(z.x));
  w.xh = reinterpret_cast<_Float16 *>(take(z.xh));
  w.xt[0] = reinterpret_cast<_Float16 *>(take(z.xt));
  w.xt[1] = reinterpret_cast<_Float16 *>(take(z.xt));
  w.f = reinterpret_cast<_Float16 *>(take(z.f));
  w.b = reinterpret_cast<_Float16 *>(take(z.f));
  w.diag_a = reinterpret_cast<float *>(take(z.diag));
  w.diag_b = reinterpret_cast<float *>(take(z.diag));
  w.norms = reinterpret_cast<double *>(take(z.norms));
  w.partial = reinterpret_cast<float *>(p);
  const unsigned wide = a.cols > 512 ? 256 : a.cols > 128 ? 64 : 16, high = 256 / wide;
  int64_t parts = (a.rows + 4 * high - 1) / (4 * high), most = 4096 / a.batch;
  if (most > kNormBlocks) most = kNormBlocks;
  if (most < 32) most = 32;
  if (parts > most) parts = most;
  k_ortho_norm<DT><<<dim3((unsigned)parts, (unsigned)a.batch), dim3(wide, high), 0, s>>>(a, w.norms);
  const dim3 tiles((unsigned)(w.mp / 64), (unsigned)(w.np / 64), (unsigned)a.batch);
  if (a.rows > a.cols)
    k_ortho_start<DT, true><<<tiles, 256, 0, s>>>(a, w, (int)parts);
  else
    k_ortho_start<DT, false><<<tiles, 256, 0, s>>>(a, w, (int)parts);
  const Side g = gram_plan(a.batch, n, m), square = symmetric_plan(a.batch, n, w.np / 64, false);
  const int t = (int)((n + g.side - 1) / g.side), side = update_side(a.batch, n, m);
  for (int step = 0; step < a.steps; ++step) {
    symmetric_of<false>(g, w, a, a.batch, s);
    if (g.splits > 1)
      k_ortho_join<<<dim3((unsigned)(t * (t + 1) / 2 * (g.side / 64) * (g.side / 64)), 1, (unsigned)a.batch), 256, 0, s>>>(
          w, t, g.side, g.splits);
    symmetric_of<true>(square, w, a, a.batch, s);
    const int early = step < a.steps - 2, last = step == a.steps - 1;
    if (side == 256)
      update<TileShape<2, 4, 8, 4, 2>>(w, a, a.batch, early, last, s);
    else if (side == 128)
      update<TileShape<2, 2, 4, 4, 2>>(w, a, a.batch, early, last, s);
    else
      update<TileShape<2, 2, 2, 2, 4>>(w, a, a.batch, early, last, s);
    _Float16 *was = w.xt[0];
    w.xt[0] = w.xt[1];
    w.xt[1] = was;
  }
}

}  // namespace

// Groups of at most kGroupBytes of scratch: a large batch gains nothing from more.
int64_t ortho_group(int64_t batch, int64_t rows, int64_t cols) {
  if (ortho_is_small(rows, cols)) return batch;
  const int64_t fit = (int64_t)(kGroupBytes / sizes_of(1, rows, cols).all());
  const int64_t most = fit < 1 ? 1 : fit > 4096 ? 4096 : fit;
  return batch < most ? batch : most;
}

size_t ortho_scratch(int64_t batch, int64_t rows, int64_t cols) {
  if (ortho_is_small(rows, cols)) return 0;
  const int64_t group = ortho_group(batch, rows, cols);
  const size_t whole = sizes_of(group, rows, cols).all();
  const size_t rest = batch % group ? sizes_of(batch % group, rows, cols).all() : 0;
  return whole > rest ? whole : rest;
}

hipError_t launch_orthogonalise(const OrthoArgs &a, int dtype, hipStream_t s) {
  if (ortho_is_small(a.rows, a.cols)) {
    dtype == 0 ? small<0>(a, s) : small<1>(a, s);
    return hipGetLastError();
  }
  const int64_t most = ortho_group(a.batch, a.rows, a.cols);
  for (int64_t first = 0; first < a.batch; first += most) {
    OrthoArgs part = a;
    part.g = static_cast<const char *>(a.g) + first * a.stride_g * (dtype == 0 ? 4 : 2);
    part.out = static_cast<char *>(a.out) + first * a.stride_o * 2;
    part.batch = a.batch - first < most ? a.batch - first : most;
    dtype == 0 ? group<0>(part, s) : group<1>(part, s);
  }
  return hipGetLastError();
}

}  // namespace gq
