// gq_embed.hip -- gfx950 kernels of a token embedding, out_t = scale * table[id_t], and of its
// gradient, dtable_v = scale * sum over the tokens t with id_t = v of dout_t.
//
// An id outside [0, vocab) stands for no token: its row is zeros, and it adds to no gradient.
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
// A thread eight elements of four tokens, whose rows are on their way together.
constexpr int kLookAhead = 4;

template <int DT, int OT>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
  const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (col >= a.dim) return;
  const int64_t stride = (int64_t)gridDim.y * blockDim.y * kLookAhead;
  for (int64_t t0 = ((int64_t)blockIdx.y * blockDim.y + threadIdx.y) * kLookAhead; t0 < a.tokens; t0 += stride) {
    float x[kLookAhead][8];
#pragma unroll
    for (int i = 0; i < kLookAhead; ++i) {
      const int64_t id = t0 + i < a.tokens ? a.ids[t0 + i] : -1;
      if (id >= 0 && id < a.vocab) {
        load_word<DT>(a.table, id * a.ld_table, col, a.dim, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kLookAhead; ++i) {
      if (t0 + i >= a.tokens) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= a.scale;
      const int64_t at = (t0 + i) * a.ld_out + col;
      if (col + 8 <= a.dim) {
        store_eight<OT>(a.out, at, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < a.dim) store_one<OT>(a.out, at + e, x[i][e]);
      }
    }
  }
}

// ---------------------------------------------------------------- tokens in the order of their ids
// order: the tokens by id, those of one id in the order in which they stand, sorted: their ids;
// start[v]: where id v's begin, start[vocab] the number of tokens that count.  A block takes `range` ids and goes through
// all tokens twice (they come from L2: 64 KB for 8192): it counts its ids and the tokens of smaller
// ids, then puts its tokens in their places.  A wave takes a run of tokens of its own and has
// counters of its own, so places follow the tokens' order without any atomic's.
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 896;  // counters of 56 KB
constexpr int kHeld = 16;       // tokens a lane

// HELD: at most 16384 tokens, which stay in registers between the two.
template <bool HELD>
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
  auto load = [&](int64_t t) { return t < end ? ids[t] : -1; };
  auto place_of = [&](int64_t id) { return (uint64_t)id < (uint64_t)vocab ? (int)id - (int)lo : 1 << 30; };
  const uint32_t here = (uint32_t)(hi - lo);
  constexpr int U = HELD ? kHeld : 4;
  int64_t id[U];
  int held[U];
  if (HELD) {
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = load(first + lane + u * 64);
  }
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortWaves * 64) counts[i] = 0;
  __syncthreads();
  uint32_t below = 0;
  for (int64_t t = first + lane; t - lane < end; t += 64 * U) {
    if (!HELD) {
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
    if (!HELD) {
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
// Tokens are added in their order; ids of more than kPiece tokens in pieces: those at sorted places
// [p kPiece, (p + 1) kPiece) are added apart.  An id of more than kPiece tokens that has any of a
// piece has its first or its last, so a piece has at most two sums: of the id that its first token
// has, and of the one that its last has.
constexpr int kPiece = 64;

// One piece and 512 columns a block: its waves a quarter of the tokens each, a lane eight columns.
template <int DT>
__device__ __forceinline__ void add_piece(const EmbedGradArgs &a, const int32_t *start, const int32_t *order,
                                          const int32_t *sorted, float *sums, int piece, int64_t c0) {
  __shared__ float part[4][64][9];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t col = c0 + lane * 8;
  const int p0 = piece * kPiece, all = start[a.vocab];
  if (p0 >= all) return;
  const int p1 = min(p0 + kPiece, all);
  const int ids[2] = {sorted[p0], sorted[p1 - 1]};
  for (int slot = 0; slot < (ids[0] == ids[1] ? 1 : 2); ++slot) {
    const int s = start[ids[slot]], e = start[ids[slot] + 1];
    if (e - s <= kPiece) continue;  // (the same for the whole block)
    constexpr int kEach = kPiece / 4;
    const int from = max(s, p0) + wave * kEach, to = min(min(e, p1), from + kEach);
    float acc[8] = {};
    if (col < a.dim) {
      for (int k = from; k < to; k += 8) {
        float x[8][8] = {};
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k + u < to) load_word<DT>(a.dout, (int64_t)order[k + u] * a.ld_dout, col, a.dim, x[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += x[u][i];
      }
    }
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

// E neighbouring elements from `col` of a row, zeros past its end.
template <int DT, int E>
__device__ __forceinline__ void load_some(const void *p, int64_t row_at, int64_t col, int64_t dim, float (&x)[E]) {
  if constexpr (E == 8) {
    load_word<DT>(p, row_at, col, dim, x);
  } else if (col + 4 <= dim) {
    if constexpr (DT == 0) {
      const f32x4 w = *reinterpret_cast<const f32x4_e4 *>(static_cast<const float *>(p) + row_at + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[i];
    } else {
      const u32x2 w = *reinterpret_cast<const u32x2_e2 *>(static_cast<const uint16_t *>(p) + row_at + col);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = col + i < dim ? load_one<DT>(p, row_at + col + i) : 0.0f;
  }
}

// E elements of a row of the gradient: what was added up times the scale (plus the old values).
template <int OT, int E>
__device__ __forceinline__ void leave(const EmbedGradArgs &a, int64_t v, int64_t col, float (&acc)[E], bool lines) {
  const int64_t to = v * a.ld_out + col;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] *= a.scale;
  if (a.accumulate) {
    float old[E];
    load_some<OT, E>(a.out, v * a.ld_out, col, a.dim, old);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] += old[i];
  }
  if (col + E > a.dim) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (col + i < a.dim) store_one<OT>(a.out, to + i, acc[i]);
    return;
  }
  u32x4 w;
  if constexpr (OT == 0)
    w = u32x4{__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])};
  else
    w = u32x4{to_bf16_pair(acc[0], acc[1]), to_bf16_pair(acc[2], acc[3]), to_bf16_pair(acc[4], acc[5]), to_bf16_pair(acc[6], acc[7])};
  char *o = static_cast<char *>(a.out) + to * (OT == 0 ? 4 : 2);
  if (lines)
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(o));
  else
    *reinterpret_cast<u32x4_e2 *>(o) = w;
}

// Adds the tokens of sorted places [s, e) to C groups of E columns a lane, U tokens on their way
// together.
template <int DT, int E, int C, int U>
__device__ __forceinline__ void add_tokens(const EmbedGradArgs &a, const int32_t *order, int s, int e, int64_t c0,
                                           float (&acc)[C][E]) {
  for (int k = s; k < e; k += U) {
    float x[U][C][E] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u < e) {
        const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(order[k + u]) * a.ld_dout;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c0 + c * 64 * E < a.dim) load_some<DT, E>(a.dout, row, c0 + c * 64 * E, a.dim, x[u][c]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[c][i] += x[u][c][i];
  }
}

// Rows of ids of at most kPiece tokens, and in the grid's first blocks the pieces of the others.  A
// block has 16 rows and 1024 columns.  First a wave takes four rows, a lane 16 bytes of the output at
// a time, so that the zeros of ids without tokens, most of the bytes, leave in whole lines and without
// a question of any lane's own, and adds those of at most kFew tokens; then the block's waves
// share each row of more, a part of the columns each, so that its tokens are few steps.
constexpr int kFew = 8;

template <int DT, int OT>
__global__ __launch_bounds__(256) void k_embed_rows(const EmbedGradArgs a, const int32_t *start,
                                                    const int32_t *order, const int32_t *sorted, float *sums,
                                                    int pieces, int parts, bool lines) {
  if ((int)blockIdx.x < pieces * parts) {
    add_piece<DT>(a, start, order, sorted, sums, blockIdx.x / parts, (int64_t)(blockIdx.x % parts) * 512);
    return;
  }
  constexpr int E = OT == 0 ? 4 : 8, C = 1024 / (64 * E);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wide = (int)((a.dim + 1023) / 1024), block = (int)blockIdx.x - pieces * parts;
  const int64_t v0 = (int64_t)(block / wide) * 16, from = (int64_t)(block % wide) * 1024;
  const int at = start[min(v0 + min(lane, 16), a.vocab)];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int s = __builtin_amdgcn_readlane(at, wave * 4 + r), e = __builtin_amdgcn_readlane(at, wave * 4 + r + 1);
    const int64_t v = v0 + wave * 4 + r, c0 = from + lane * E;
    if (v >= a.vocab || e - s > kFew || (a.accumulate && s == e)) continue;
    float acc[C][E] = {};
    add_tokens<DT, E, C, 4>(a, order, s, e, c0, acc);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c0 + c * 64 * E < a.dim) leave<OT, E>(a, v, c0 + c * 64 * E, acc[c], lines);
  }
  const int next = __shfl_down(at, 1);
  uint64_t more = __ballot(lane < 16 && next - at > kFew && next - at <= kPiece);
  for (; more; more &= more - 1) {
    const int r = __builtin_ctzll(more);
    const int s = __builtin_amdgcn_readlane(at, r), e = __builtin_amdgcn_readlane(at, r + 1);
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      const int64_t c0 = from + (wave + c) * 64 * E + lane * E;
      if (wave + c >= C || c0 >= a.dim) continue;
      float acc[1][E] = {};
      add_tokens<DT, E, 1, 16>(a, order, s, e, c0, acc);
      leave<OT, E>(a, v0 + r, c0, acc[0], lines);
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
      float x[U][E] = {};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t slot = p + u == (int)blockIdx.x && s != p0;
        if (p + u < to) load_some<0, E>(sums, ((int64_t)(p + u) * 2 + slot) * a.dim, col, a.dim, x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += x[u][i];
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
  const dim3 grid((unsigned)((groups + bx - 1) / bx), (unsigned)(gy < 32768 ? gy : 32768));
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
  if (a.tokens <= kSortWaves * 64 * kHeld)
    k_embed_sort<true><<<ranges, kSortWaves * 64, lds, s>>>(a.ids, a.tokens, a.vocab, (int)range, bits, start, order, sorted);
  else
    k_embed_sort<false><<<ranges, kSortWaves * 64, lds, s>>>(a.ids, a.tokens, a.vocab, (int)range, bits, start, order, sorted);
  const bool lines = ((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.ld_out * (OT == 0 ? 4 : 2)) & 127) == 0;
  const int pieces = a.tokens > kPiece ? (int)pieces_of(a.tokens) : 0, parts = (int)((a.dim + 511) / 512);
  const int64_t rows = (a.vocab + 15) / 16 * ((a.dim + 1023) / 1024);
  k_embed_rows<DT, OT><<<(unsigned)((int64_t)pieces * parts + rows), 256, 0, s>>>(a, start, order, sorted, sums, pieces,
                                                                                 parts, lines);
  constexpr int kWide = 64 * (OT == 0 ? 4 : 8);
  if (pieces)
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
