// gq_embed.hip -- gfx950 kernels of a token embedding, out_t = scale * table[id_t], and of its
// gradient, dtable_v = scale * sum over the tokens t with id_t = v of dout_t.
//
// An id outside [0, vocab) stands for no token: its row is zeros, and it adds to no gradient.
#include <type_traits>

#include "gq_device.h"
#include "gq_layers.h"

namespace gq {
namespace {

template <int OT>
__device__ __forceinline__ void store_one(void *p, int64_t i, float v) {
  if constexpr (OT == 0)
    static_cast<float *>(p)[i] = v;
  else
    static_cast<uint16_t *>(p)[i] = to_bf16(v);
}

// Eight neighbouring elements at any element's alignment.
template <int OT>
__device__ __forceinline__ void store_eight(void *p, int64_t i, const float (&v)[8]) {
  if constexpr (OT == 0) {
    f32x4_e4 *o = reinterpret_cast<f32x4_e4 *>(static_cast<float *>(p) + i);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4_e2 *>(static_cast<uint16_t *>(p) + i) =
        u32x4{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
  }
}

// ---------------------------------------------------------------- lookup
// A thread eight elements of four tokens, whose rows are on their way together.  Bound by its bytes: 16383
// tokens of 4096 bf16 37 us (268 MB by algorithm; rows that come again come from the caches, 213 MB by
// the counters); eight tokens 2.5 us, a launch.
constexpr int kLookAhead = 4;

template <int DT, int OT>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
  const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (col >= a.dim) return;
  const int64_t stride = (int64_t)gridDim.y * blockDim.y * kLookAhead;
  for (int64_t t0 = ((int64_t)blockIdx.y * blockDim.y + threadIdx.y) * kLookAhead; t0 < a.tokens; t0 += stride) {
    int64_t id[kLookAhead];
    Raw<DT, 8> raw[kLookAhead];
#pragma unroll
    for (int i = 0; i < kLookAhead; ++i) id[i] = a.ids[min(t0 + i, a.tokens - 1)];
    if (a.vocab > 0) {
#pragma unroll
      for (int i = 0; i < kLookAhead; ++i)  // no token: row 0, not kept
        raw[i] = raw_word<DT, 8>(a.table, ((uint64_t)id[i] < (uint64_t)a.vocab ? id[i] : 0) * a.ld_table, col, a.dim);
    }
#pragma unroll
    for (int i = 0; i < kLookAhead; ++i) {
      if (t0 + i >= a.tokens) break;
      float x[8] = {};
      if ((uint64_t)id[i] < (uint64_t)a.vocab) open_word(raw[i], a.table, id[i] * a.ld_table, col, a.dim, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= a.scale;
      const int64_t at = (t0 + i) * a.ld_out + col;
      if (col + 8 <= a.dim) {
        store_eight<OT>(a.out, at, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < a.dim) store_one<OT>(a.out, at + e, x[e]);
      }
    }
  }
}

// ---------------------------------------------------------------- tokens in the order of their ids
// order: the tokens by id, those of one id in the order in which they stand, sorted: their ids;
// start[v]: where id v's begin, start[vocab] the number of tokens that count.  A block takes `range` ids and goes through
// all tokens twice (they come from L2: 64 KB for 8192): it counts its ids and the tokens of smaller
// ids, then puts its tokens in their places.  A wave takes a run of tokens of its own and has
// counters of its own, so places follow the tokens' order without any atomic's.  One launch whatever the
// vocabulary: 10 us for 8191 tokens, 18 for 16384, latency (tokens, counters, sums and places wait for
// each other).
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 896;  // counters of 56 KB

// HELD > 0: at most 1024 HELD tokens, which stay in registers between the two.
template <int HELD>
__global__ __launch_bounds__(kSortWaves * 64) void k_embed_sort(const int64_t *ids, int64_t tokens,
                                                                int64_t vocab, int range, int bits,
                                                                int32_t *start, int32_t *order,
                                                                int32_t *sorted) {
  extern __shared__ uint32_t counts[];  // kSortWaves x range
  __shared__ uint32_t below_of[kSortWaves], total_of[kSortWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t lo = (int64_t)blockIdx.x * range, hi = min(lo + range, vocab);
  const int64_t run = (tokens + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
  const int64_t first = wave * run, end = min(first + run, tokens);
  uint32_t *mine = counts + wave * range;
  // a token's id from the range's first on; what has no id is beyond every range
  auto load = [&](int64_t t) {
    const int64_t id = ids[max(min(t, tokens - 1), (int64_t)0)];  // (of no tokens: any place that there is)
    return t < end ? id : -1;
  };
  auto place_of = [&](int64_t id) { return (uint64_t)id < (uint64_t)vocab ? (int)id - (int)lo : 1 << 30; };
  const uint32_t here = (uint32_t)(hi - lo);
  constexpr int U = HELD > 0 ? HELD : 4;
  int64_t id[U];
  int held[U];
  if (HELD > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = load(first + lane + u * 64);
  }
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortWaves * 64) counts[i] = 0;
  __syncthreads();
  uint32_t below = 0;
  for (int64_t t = first + lane; t - lane < end; t += 64 * U) {
    if (HELD == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = load(t + u * 64);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      held[u] = place_of(id[u]);
      below += held[u] < 0;
      if ((uint32_t)held[u] < here) atomicAdd(&mine[held[u]], 1u);
    }
  }
  for (int m = 1; m < 64; m <<= 1) below += (uint32_t)__shfl_xor((int)below, m);
  if (lane == 0) below_of[wave] = below;
  __syncthreads();
  // thread r: where id lo + r begins, and in it every wave's tokens
  uint32_t total = 0;
  if ((int)threadIdx.x < range)
    for (int w = 0; w < kSortWaves; ++w) total += counts[w * range + threadIdx.x];
  uint32_t sum = total;
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t other = (uint32_t)__shfl_up((int)sum, m);
    if (lane >= m) sum += other;
  }
  if (lane == 63) total_of[wave] = sum;
  __syncthreads();
  uint32_t at = sum - total;
  for (int w = 0; w < kSortWaves; ++w) {
    at += below_of[w];
    if (w < wave) at += total_of[w];
  }
  if ((int)threadIdx.x < range) {
    if (lo + threadIdx.x < hi) start[lo + threadIdx.x] = (int32_t)at;
    if (lo + threadIdx.x == vocab - 1) start[vocab] = (int32_t)(at + total);
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = counts[w * range + threadIdx.x];
      counts[w * range + threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t t = first + lane; t - lane < end; t += 64 * U) {
    if (HELD == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = load(t + u * 64);
#pragma unroll
      for (int u = 0; u < U; ++u) held[u] = place_of(id[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = (uint32_t)held[u] < here;
      uint64_t same = __ballot(in);
      if (same == 0) continue;
      // the lanes with this lane's id, bit by bit
      const uint32_t r = in ? (uint32_t)held[u] : 0u;
      for (int b = 0; b < bits; ++b) {
        const bool set = r >> b & 1;
        const uint64_t with = __ballot(set);
        same &= set ? with : ~with;
      }
      uint32_t place = 0;
      if (in) place = mine[r];
      wave_exchange();
      const uint64_t lower = same & ((1ull << lane) - 1);
      if (in) {
        order[place + __popcll(lower)] = (int32_t)(t + u * 64);
        sorted[place + __popcll(lower)] = (int32_t)(lo + r);
        if (lower == 0) mine[r] = place + __popcll(same);
      }
      wave_exchange();
    }
  }
}

// ---------------------------------------------------------------- gradient
// Three sorts of rows.  Of at most kFew tokens, most of all: one after another with the zeros
// (k_embed_rows).  Of at most kPiece tokens: added in their order by a wave, beside the first sort, as
// a frequent id's neighbours are often frequent too and would wait for each other there.  Of more: in
// pieces, the tokens at sorted places [p kPiece, (p + 1) kPiece), which are added apart and then
// joined.  Such an id, if it has any token of a piece, has its first or its last, so a piece has at most two
// sums: of the id that its first token has, and of the one that its last has.
constexpr int kPiece = 64;
constexpr int kFew = 4;

// E elements of a row of the gradient: what was added up times the scale (plus the old values).
template <int OT, int E>
__device__ __forceinline__ void leave(const EmbedGradArgs &a, int64_t v, int64_t col, float (&acc)[E], bool lines) {
  const int64_t to = v * a.ld_out + col;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] *= a.scale;
  if (a.accumulate) {
    float old[E];
    open_word(raw_word<OT, E>(a.out, v * a.ld_out, col, a.dim), a.out, v * a.ld_out, col, a.dim, old);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] += old[i];
  }
  if (col + E > a.dim) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (col + i < a.dim) store_one<OT>(a.out, to + i, acc[i]);
    return;
  }
  if constexpr (E == 8) {
    store_eight<OT>(a.out, to, acc);
  } else {
    const u32x4 w = {__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])};
    float *o = static_cast<float *>(a.out) + to;
    if (lines)
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(o));
    else
      *reinterpret_cast<u32x4_e4 *>(o) = w;
  }
}

// Adds U tokens at most, which `of` names, to E columns a lane.
template <int DT, int E, int U, class F>
__device__ __forceinline__ void add_some(const EmbedGradArgs &a, int count, int64_t col, F &&of, float (&acc)[E]) {
  int64_t row[U];
  Raw<DT, E> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) row[u] = (int64_t)of(min(u, count - 1)) * a.ld_dout;
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = raw_word<DT, E>(a.dout, row[u], col, a.dim);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u < count) {
      float x[E];
      open_word(raw[u], a.dout, row[u], col, a.dim, x);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += x[i];
    }
  }
}

// One piece and 512 columns a block, a lane eight: the rows of the second sort whose tokens begin in
// it, a wave one, then its sums of the third, a wave a quarter of the tokens.
template <int DT, int OT>
__device__ __forceinline__ void add_piece(const EmbedGradArgs &a, const int32_t *start, const int32_t *order,
                                          const int32_t *sorted, float *sums, int piece, int64_t c0) {
  __shared__ float part[4][64][9];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t col = c0 + lane * 8;
  const int p0 = piece * kPiece, all = start[a.vocab];
  if (p0 >= all) return;
  const int p1 = min(p0 + kPiece, all);
  // of this piece's tokens, a lane one: the token, its id, where the id's tokens begin and end
  const int here = min(p0 + lane, all - 1), id = sorted[here];
  const int token0 = order[here], token1 = order[min(p0 + 64 + lane, all - 1)];
  const int s = start[id], e = start[id + 1];
  auto token = [&](int place) {  // within this piece and the next
    const int k = place - p0;
    return k < 64 ? __builtin_amdgcn_readlane(token0, k) : __builtin_amdgcn_readlane(token1, k - 64);
  };
  uint64_t some = __ballot(s == p0 + lane && p0 + lane < all && e - s > kFew && e - s <= kPiece);
  for (int k = 0; some; some &= some - 1, ++k) {
    if ((k & 3) != wave) continue;
    const int l = __builtin_ctzll(some);
    const int from = __builtin_amdgcn_readlane(s, l), to = __builtin_amdgcn_readlane(e, l);
    float acc[8] = {};
    for (int at = from; at < to; at += 16)
      add_some<DT, 8, 16>(a, to - at, col, [&](int u) { return token(at + u); }, acc);
    if (col < a.dim) leave<OT, 8>(a, __builtin_amdgcn_readlane(id, l), col, acc, false);
  }
  for (int slot = 0; slot < 2; ++slot) {
    const int l = slot == 0 ? 0 : p1 - 1 - p0;
    const int s1 = __builtin_amdgcn_readlane(s, l), e1 = __builtin_amdgcn_readlane(e, l);
    // (the same for the whole block)
    if (e1 - s1 <= kPiece || (slot == 1 && __builtin_amdgcn_readlane(id, 0) == __builtin_amdgcn_readlane(id, l))) continue;
    constexpr int kEach = kPiece / 4;
    const int from = max(s1, p0) + wave * kEach, to = min(min(e1, p1), from + kEach);
    float acc[8] = {};
    if (from < to) add_some<DT, 8, kEach>(a, to - from, col, [&](int u) { return token(from + u); }, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][lane][i] = acc[i];
    __syncthreads();
    if (wave == 0 && col < a.dim) {
      float *o = sums + ((int64_t)piece * 2 + slot) * a.dim + col;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < a.dim) o[i] = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
    }
    __syncthreads();
  }
}

// The pieces in the grid's first blocks, then the rows of at most kFew tokens, 16 a block.  The zeros of
// ids without tokens, most of the bytes, leave first, by whole lines and without a question of any
// lane's own, a wave four rows; then a wave takes a quarter of the columns of all rows of some tokens,
// the first tokens of four rows on their way together, as one token is the rule.
// 50257 x 768 fp32 from 8191 tokens 29 us (167 MB, 5.8 TB/s), 131071 x 4096 from 16384 395 us (2.28 GB, 5.8
// TB/s), bound by the stores.  With every row of up to 64 tokens added here, one after another, a call at
// the first size took 77 us, and 352 where the frequent ids are neighbours: 42 and 46 this way.
// Non-temporal stores: a call at the larger size takes 404 us against 456 with plain ones; at the first, whose
// table the last cache holds when it is written again and again, 43 against 37.
template <int DT, int OT>
__global__ __launch_bounds__(256) void k_embed_rows(const EmbedGradArgs a, const int32_t *start,
                                                    const int32_t *order, const int32_t *sorted, float *sums,
                                                    int pieces, int parts, int wide, bool lines) {
  if ((int)blockIdx.x < pieces * parts) {
    add_piece<DT, OT>(a, start, order, sorted, sums, blockIdx.x / parts, (int64_t)(blockIdx.x % parts) * 512);
    return;
  }
  constexpr int E = OT == 0 ? 4 : 8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = (int)blockIdx.x - pieces * parts;
  const int64_t v0 = (int64_t)(block / wide) * 16, col = ((int64_t)(block % wide) * 256 + wave * 64 + lane) * E;
  const int at = start[min(v0 + min(lane, 16), a.vocab)], count = __shfl_down(at, 1) - at;
  const bool row = lane < 16 && v0 + lane < a.vocab;
  if (!a.accumulate)  // a wave four rows, whole
    for (uint64_t none = __ballot(row && count == 0) & 15ull << wave * 4; none; none &= none - 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float zero[E] = {};
        const int64_t at_col = col + (c - wave) * 64 * E;
        if (at_col < a.dim) leave<OT, E>(a, v0 + __builtin_ctzll(none), at_col, zero, lines);
      }
    }
  if (col - lane * E >= a.dim) return;
  uint64_t some = __ballot(row && count > 0 && count <= kFew);
  while (some) {
    int r[4];
    int64_t from[4];
    Raw<DT, E> raw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      r[q] = some ? __builtin_ctzll(some) : -1;
      some &= some - 1;
      from[q] = (int64_t)__builtin_amdgcn_readfirstlane(order[__builtin_amdgcn_readlane(at, r[q] < 0 ? r[0] : r[q])]) * a.ld_dout;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) raw[q] = raw_word<DT, E>(a.dout, from[q], col, a.dim);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (r[q] < 0) break;
      const int s = __builtin_amdgcn_readlane(at, r[q]) + 1, e = __builtin_amdgcn_readlane(at, r[q] + 1);
      float acc[E] = {}, x[E];
      open_word(raw[q], a.dout, from[q], col, a.dim, x);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += x[i];
      if (s < e)
        add_some<DT, E, kFew - 1>(a, e - s, col, [&](int u) { return __builtin_amdgcn_readfirstlane(order[s + u]); }, acc);
      if (col < a.dim) leave<OT, E>(a, v0 + r[q], col, acc, lines);
    }
  }
}

// Rows of ids of more than kPiece tokens: a block a piece in which such an id's tokens begin (the last
// token of the piece is one of them) and 256 or 512 columns; its waves add a quarter of the
// partial sums each.
template <int OT>
__global__ __launch_bounds__(256) void k_embed_join(const EmbedGradArgs a, const int32_t *start,
                                                    const int32_t *sorted, const float *sums, bool lines) {
  constexpr int E = OT == 0 ? 4 : 8, U = 8;
  __shared__ float part[4][64][E + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p0 = blockIdx.x * kPiece, all = start[a.vocab];
  if (p0 >= all) return;
  const int id = sorted[min(p0 + kPiece, all) - 1];
  const int s = start[id], e = start[id + 1];
  if (s < p0 || e - s <= kPiece) return;
  const int64_t col = (int64_t)blockIdx.y * 64 * E + lane * E;
  const int last = (e - 1) / kPiece, count = last - (int)blockIdx.x + 1, each = (count + 3) / 4;
  const int from = (int)blockIdx.x + wave * each, to = min(from + each, last + 1);
  float acc[E] = {};
  if (col < a.dim)
    for (int p = from; p < to; p += U) {
      int64_t row[U];
      Raw<0, E> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = min(p + u, to - 1);
        row[u] = ((int64_t)q * 2 + (q == (int)blockIdx.x && s != p0)) * a.dim;
        raw[u] = raw_word<0, E>(sums, row[u], col, a.dim);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u >= to) break;
        float x[E];
        open_word(raw[u], sums, row[u], col, a.dim, x);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += x[i];
      }
    }
#pragma unroll
  for (int i = 0; i < E; ++i) part[wave][lane][i] = acc[i];
  __syncthreads();
  if (wave > 0 || col >= a.dim) return;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
  leave<OT, E>(a, id, col, acc, lines);
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

int64_t pieces_of(int64_t tokens) { return (tokens + kPiece - 1) / kPiece; }

template <int DT, int OT>
void look_up(const EmbedArgs &a, hipStream_t s) {
  const int64_t groups = (a.dim + 7) / 8;
  const unsigned bx = groups > 64 ? 256 : groups > 16 ? 64 : 16;
  const int64_t by = 256 / bx, gy = (a.tokens + by * kLookAhead - 1) / (by * kLookAhead);
  const dim3 grid((unsigned)((groups + bx - 1) / bx), (unsigned)(gy < 16384 ? gy : 16384));
  k_embed<DT, OT><<<grid, dim3(bx, (unsigned)by), 0, s>>>(a);
}

template <int DT, int OT>
void gradient(const EmbedGradArgs &a, hipStream_t s) {
  int32_t *start = static_cast<int32_t *>(a.scratch);
  int32_t *order = reinterpret_cast<int32_t *>(static_cast<char *>(a.scratch) + round_up((size_t)(a.vocab + 1) * 4));
  int32_t *sorted = order + round_up((size_t)a.tokens * 4) / 4;
  float *sums = reinterpret_cast<float *>(sorted + round_up((size_t)a.tokens * 4) / 4);
  // as many ranges as CUs, unless a range's counters would not fit LDS
  int64_t range = (a.vocab + 255) / 256;
  if (range > kMaxRange) range = kMaxRange;
  int bits = 0;
  while ((1 << bits) < range) ++bits;
  const unsigned ranges = (unsigned)((a.vocab + range - 1) / range);
  const size_t lds = (size_t)range * kSortWaves * 4;
  auto sort = [&](auto held) {
    const int64_t *ids = a.tokens > 0 ? a.ids : static_cast<const int64_t *>(a.scratch);
    k_embed_sort<decltype(held)::value><<<ranges, kSortWaves * 64, lds, s>>>(ids, a.tokens, a.vocab, (int)range, bits,
                                                                            start, order, sorted);
  };
  if (a.tokens <= kSortWaves * 64 * 2)
    sort(std::integral_constant<int, 2>{});
  else if (a.tokens <= kSortWaves * 64 * 8)
    sort(std::integral_constant<int, 8>{});
  else if (a.tokens <= kSortWaves * 64 * 16)
    sort(std::integral_constant<int, 16>{});
  else
    sort(std::integral_constant<int, 0>{});
  const bool lines = ((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.ld_out * (OT == 0 ? 4 : 2)) & 127) == 0;
  const int pieces = (int)pieces_of(a.tokens), parts = (int)((a.dim + 511) / 512);
  constexpr int kWide = 64 * (OT == 0 ? 4 : 8);
  const int wide = (int)((a.dim + 4 * kWide - 1) / (4 * kWide));
  const int64_t blocks = (int64_t)pieces * parts + (a.vocab + 15) / 16 * wide;
  k_embed_rows<DT, OT><<<(unsigned)blocks, 256, 0, s>>>(a, start, order, sorted, sums, pieces, parts, wide, lines);
  if (pieces > 1)
    k_embed_join<OT><<<dim3((unsigned)pieces, (unsigned)((a.dim + kWide - 1) / kWide)), 256, 0, s>>>(a, start, sorted, sums, lines);
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, int dtype, int out_dtype, hipStream_t s) {
  if (dtype == 0)
    out_dtype == 0 ? look_up<0, 0>(a, s) : look_up<0, 1>(a, s);
  else
    out_dtype == 0 ? look_up<1, 0>(a, s) : look_up<1, 1>(a, s);
  return hipGetLastError();
}

size_t embed_grad_scratch(int64_t tokens, int64_t vocab, int64_t dim) {
  return round_up((size_t)(vocab + 1) * 4) + 2 * round_up((size_t)tokens * 4) +
         (tokens > kPiece ? (size_t)pieces_of(tokens) * 2 * (size_t)dim * 4 : 0);
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, int dtype, int out_dtype, hipStream_t s) {
  if (dtype == 0)
    out_dtype == 0 ? gradient<0, 0>(a, s) : gradient<0, 1>(a, s);
  else
    out_dtype == 0 ? gradient<1, 0>(a, s) : gradient<1, 1>(a, s);
  return hipGetLastError();
}

}  // namespace gq
