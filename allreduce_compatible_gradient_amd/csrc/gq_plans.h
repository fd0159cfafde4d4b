// gq_plans.h -- which form of a kernel takes a size: the tiles of 8-bit products and of the orthogonalised
// update (host code, without HIP).
#pragma once

#include <math.h>
#include <stdint.h>

#include <initializer_list>

namespace gq {

constexpr int kCus = 256;

// ---------------------------------------------------------------- 8-bit products
constexpr int64_t kFewRows = 16;  // rows of A that the form without tiles takes

// Bytes of a packed row: whole steps of the product.
inline int64_t i8_pitch(int64_t cols) { return (cols + 127) / 128 * 128; }

struct I8Plan {
  int bm, bn;        // tile
  int splits, each;  // K splits and steps of each
};

// Tile and K splits of a product of more than kFewRows rows.  The tile is the one of the least expected
// time, with n blocks on the fullest CU n (step K / 128 + rest) + wait K / 128 + once, fitted to 160 sizes
// (M 17 to 8192, N 300 to 51200, K 128 to 11008), where the tile so chosen takes 1.03 times the best
// one's time in the mean: 1000 x 4096 x 4096 23.0 us with 64 x 128, 27.0 with 128 x 128, 49.9 with 256 x
// 256; 4095 x 11008 x 4096 209, 205 and 178.  Splits where tiles are few and K is long (64 x 4096 x 4096
// 11.3 us, 13.5 without).
inline I8Plan i8_plan(int64_t M, int64_t N, int64_t K) {
  struct Tile {
    int bm, bn;
    float step, rest, wait, once;  // us of a step, of the rest of a tile, and once a step and a call
  };
  constexpr Tile kTiles[3] = {{256, 256, 1.28f, 11.2f, 0.0f, 0.0f}, {128, 128, 0.46f, 3.3f, 0.11f, 4.0f}, {64, 128, 0.27f, 1.3f, 0.16f, 4.7f}};
  I8Plan p = {};
  const int64_t steps = i8_pitch(K) / 128;
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  float least = INFINITY;
  for (const Tile &t : kTiles) {
    const float each = (float)((tiles(t.bm, t.bn) + kCus - 1) / kCus);
    const float us = each * ((float)steps * t.step + t.rest) + (float)steps * t.wait + t.once;
    if (us < least) {
      least = us;
      p.bm = t.bm;
      p.bn = t.bn;
    }
  }
  int64_t splits = 1;
  if (steps >= 24) {
    splits = kCus / tiles(p.bm, p.bn);
    if (splits > steps / 8) splits = steps / 8;
    if (splits > 16) splits = 16;
    if (splits < 1) splits = 1;
  }
  p.each = (int)((steps + splits - 1) / splits);
  p.splits = (int)((steps + p.each - 1) / p.each);
  return p;
}

// ---------------------------------------------------------------- orthogonalised update
inline int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

// What one block holds: 64 x 512 takes 159 KB of LDS.
inline bool ortho_is_small(int64_t rows, int64_t cols) {
  return (rows < cols ? rows : cols) <= 64 && (rows < cols ? cols : rows) <= 512;
}

// Expected time of a launch in us: a block of a side takes `step` a step of 64 halves and `rest` besides,
// as many blocks one after another as the fullest CU has; `wait` a step and `once` come on top.  The
// symmetric products' are fitted to eleven sizes (n 256 to 6000, m 768 to 11008, batches to 48), where
// the sides so chosen are the best ones but for four launches of 22, which lose 4 to 22 us.  4096 x 4096,
// five Gram matrices and squares: 293 us less with 192 than with 256 (253 tiles against 136 on 256 CUs).
// The update's have the same loop and an epilogue of 12 bytes an element; with each side at fourteen sizes
// (n 300 to 4096, m to 11008, batches to 48) the one chosen is within 3% of the best call but twice:
// 3000 x 3000 takes 955 us with 64 (chosen), 945 with 128 and 895 with 256; 48 of 256 x 1024 305, 318
// (chosen) and 289; 12 of 768 x 2304 743, 677 (chosen) and 710; 4096 x 11008 5187, 3830 and 3511 (chosen).
struct Cost {
  int side;
  float step, rest, wait, once;
};
constexpr Cost kSymmetric[] = {{256, 0.93f, 12.8f, 0.09f, 0.8f}, {192, 0.64f, 8.3f, 0.08f, 0.3f},
                               {128, 0.31f, 4.5f, 0.29f, 3.5f}, {64, 0.28f, 0.0f, 0.0f, 3.4f}};
constexpr Cost kUpdate[] = {{256, 0.93f, 40.0f, 0.09f, 0.8f}, {128, 0.31f, 9.0f, 0.29f, 3.5f}, {64, 0.13f, 2.4f, 0.0f, 7.8f}};

inline float cost_of(const Cost &c, int64_t tiles, int64_t steps) {
  return (float)((tiles + kCus - 1) / kCus) * ((float)steps * c.step + c.rest) + (float)steps * c.wait + c.once;
}

struct Side {
  int side, splits, each;
  bool alone;  // a CU has one block at most
};

// Tiles of a symmetric product with sums of `steps`; the Gram matrix, whose sums may be long, in splits
// where its tiles leave CUs idle and a launch that joins them costs less.
inline Side symmetric_plan(int64_t batch, int64_t n, int64_t steps, bool may_split) {
  Side best = {64, 1, (int)steps, false};
  float least = INFINITY;
  for (const Cost &c : kSymmetric) {
    const int64_t t = (n + c.side - 1) / c.side, count = batch * t * (t + 1) / 2;
    int64_t most = kCus / count;
    if (most > steps / 4) most = steps / 4;
    if (most > 16) most = 16;
    if (most < 1 || !may_split) most = 1;
    for (int64_t splits : {(int64_t)1, most}) {
      const int64_t each = (steps + splits - 1) / splits;
      // partial sums are written and read, at some 4 TB/s
      const float join = splits > 1 ? 4.0f + (float)(count * splits) * (float)(c.side * c.side) * 2e-6f : 0.0f;
      const float us = cost_of(c, count * splits, each) + join;
      if (us >= least) continue;
      least = us;
      best = Side{c.side, (int)((steps + each - 1) / each), (int)each, count * splits <= kCus};
    }
  }
  return best;
}

inline Side gram_plan(int64_t batch, int64_t n, int64_t m) { return symmetric_plan(batch, n, up64(m) / 64, true); }

inline int update_side(int64_t batch, int64_t n, int64_t m) {
  int side = 64;
  float least = INFINITY;
  for (const Cost &c : kUpdate) {
    const float us = cost_of(c, batch * ((n + c.side - 1) / c.side) * ((m + c.side - 1) / c.side), up64(n) / 64);
    if (us < least) {
      least = us;
      side = c.side;
    }
  }
  return side;
}

}  // namespace gq
