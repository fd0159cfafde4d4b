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
// order: the tokens by id, those of one id in the order in which they stand; start[v]: where id v's
// begin, start[vocab] the number of tokens that count.  A block takes `range` ids and goes through
// all tokens twice (they come from L2: 64 KB for 8192): it counts its ids and the tokens of smaller
// ids, then puts its tokens in their places.  A wave takes a run of tokens of its own and has
// counters of its own, so places follow the tokens' order without any atomic's.
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 896;  // counters of 56 KB

__global__ __launch_bounds__(kSortWaves * 64) void k_embed_sort(const int64_t *ids, int64_t tokens,
                                                                int64_t vocab, int range, int bits,
                                                                int32_t *start, int32_t *order) {
  extern __shared__ uint32_t counts[];  // kSortWaves x range
  __shared__ uint32_t below_of[kSortWaves], total_of[kSortWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t lo = (int64_t)blockIdx.x * range, hi = min(lo + range, vocab);
  uint32_t *mine = counts + wave * range;
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortWaves * 64) counts[i] = 0;
  __syncthreads();
  const int64_t run = (tokens + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
  const int64_t first = wave * run, end = min(first + run, tokens);
  uint32_t below = 0;
  constexpr int U = 4;
  for (int64_t t = first + lane; t - lane < end; t += 64 * U) {
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = t + u * 64 < end ? ids[t + u * 64] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += id[u] >= 0 && id[u] < lo;
      if (id[u] >= lo && id[u] < hi) atomicAdd(&mine[id[u] - lo], 1u);
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
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = t + u * 64 < end ? ids[t + u * 64] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = id[u] >= lo && id[u] < hi;
      uint64_t same = __ballot(in);
      if (same == 0) continue;
      // the lanes with this lane's id, bit by bit
      const uint32_t r = in ? (uint32_t)(id[u] - lo) : 0u;
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

// A block a piece and 512 columns: its waves a quarter of the tokens each, a lane eight columns.
template <int DT>
__global__ __launch_bounds__(256) void k_embed_pieces(const EmbedGradArgs a, const int32_t *start,
                                                      const int32_t *order, float *sums) {
  __shared__ float part[4][64][9];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t col = (int64_t)blockIdx.y * 512 + lane * 8;
  const int all = start[a.vocab];
  const int p0 = blockIdx.x * kPiece, p1 = min(p0 + kPiece, all);
  if (p0 >= all) return;
  int64_t last_id = -1;
  for (int slot = 0; slot < 2; ++slot) {
    const int64_t id = a.ids[order[slot == 0 ? p0 : p1 - 1]];
    const int s = start[id], e = start[id + 1];
    if (e - s <= kPiece || id == last_id) continue;  // (the same for the whole block)
    last_id = id;
    const int from = max(s, p0), to = min(e, p1);
    float acc[8] = {};
    if (col < a.dim) {
      const int b = from + wave * (kPiece / 4), end = min(b + kPiece / 4, to);
      for (int k = b; k < end; k += 8) {
        float x[8][8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (k + u < end) {
            load_word<DT>(a.dout, (int64_t)order[k + u] * a.ld_dout, col, a.dim, x[u]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
          }
        }
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
      float *o = sums + ((int64_t)blockIdx.x * 2 + slot) * a.dim + col;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < a.dim) o[i] = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
    }
    __syncthreads();
  }
}

// Rows of the table's gradient: a block some rows, a thread E neighbouring elements (16 bytes of the
// output) at a time, so that the zeros of ids without tokens, most of the bytes, leave in whole lines.
template <int DT, int OT>
__global__ __launch_bounds__(256) void k_embed_rows(const EmbedGradArgs a, const int32_t *start,
                                                    const int32_t *order, const float *sums,
                                                    int rows_each, int groups, bool lines) {
  constexpr int E = OT == 0 ? 4 : 8;
  const int64_t v0 = (int64_t)blockIdx.x * rows_each;
  const int here = (int)min((int64_t)rows_each, a.vocab - v0);
  for (int l = threadIdx.x; l < here * groups; l += 256) {
    const int r = l / groups;
    const int64_t v = v0 + r, col = (int64_t)(l - r * groups) * E;
    const int s = start[v], e = start[v + 1];
    if (a.accumulate && s == e) continue;
    const bool whole = col + E <= a.dim;
    float acc[E] = {};
    auto add = [&](const float (&x)[E]) {
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += x[i];
    };
    if (e - s <= kPiece) {
      for (int k = s; k < e; k += 4) {
        float x[4][E] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (k + u < e) {
            const int64_t at = (int64_t)order[k + u] * a.ld_dout + col;
            if (whole) {
              if constexpr (E == 8) {
                load_eight<DT>(a.dout, at, x[u]);
              } else if constexpr (DT == 0) {
                const f32x4 w = *reinterpret_cast<const f32x4_e4 *>(static_cast<const float *>(a.dout) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = w[i];
              } else {
                const u32x2 w = *reinterpret_cast<const u32x2_e2 *>(static_cast<const uint16_t *>(a.dout) + at);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  x[u][2 * i] = __uint_as_float(w[i] << 16);
                  x[u][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < E; ++i)
                if (col + i < a.dim) x[u][i] = load_one<DT>(a.dout, at + i);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) add(x[u]);
      }
    } else {
      const int p0 = s / kPiece, p1 = (e - 1) / kPiece;
      for (int p = p0; p <= p1; p += 4) {
        float x[4][E] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (p + u <= p1) {
            const int slot = p + u == p0 && s != p0 * kPiece;
            const float *from = sums + ((int64_t)(p + u) * 2 + slot) * a.dim + col;
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (col + i < a.dim) x[u][i] = from[i];
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) add(x[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] *= a.scale;
    const int64_t at = v * a.ld_out + col;
    if (a.accumulate) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (col + i < a.dim) acc[i] += load_one<OT>(a.out, at + i);
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (col + i < a.dim) store_one<OT>(a.out, at + i, acc[i]);
      continue;
    }
    u32x4 w;
    if constexpr (OT == 0) {
      w = u32x4{__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])};
    } else {
      w = u32x4{to_bf16_pair(acc[0], acc[1]), to_bf16_pair(acc[2], acc[3]), to_bf16_pair(acc[4], acc[5]), to_bf16_pair(acc[6], acc[7])};
    }
    void *o = OT == 0 ? static_cast<void *>(static_cast<float *>(a.out) + at) : static_cast<void *>(static_cast<uint16_t *>(a.out) + at);
    if (lines)
      __builtin_nontemporal_store(w, static_cast<u32x4 *>(o));
    else
      *static_cast<u32x4_e2 *>(o) = w;
  }
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
  float *sums = reinterpret_cast<float *>(reinterpret_cast<char *>(order) + round_up((size_t)a.tokens * 4));
  // as many ranges as CUs, unless a range's counters would not fit LDS
  int64_t range = (a.vocab + 255) / 256;
  if (range > kMaxRange) range = kMaxRange;
  int bits = 0;
  while ((1 << bits) < range) ++bits;
  k_embed_sort<<<(unsigned)((a.vocab + range - 1) / range), kSortWaves * 64, (size_t)range * kSortWaves * 4, s>>>(
      a.ids, a.tokens, a.vocab, (int)range, bits, start, order);
  if (a.tokens > kPiece)
    k_embed_pieces<DT><<<dim3((unsigned)pieces_of(a.tokens), (unsigned)((a.dim + 511) / 512)), 256, 0, s>>>(a, start, order, sums);
  constexpr int E = OT == 0 ? 4 : 8;
  const int64_t groups = (a.dim + E - 1) / E;
  const int64_t each = groups >= 1024 ? 1 : 1024 / groups;
  const bool lines = ((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.ld_out * (OT == 0 ? 4 : 2)) & 127) == 0;
  k_embed_rows<DT, OT><<<(unsigned)((a.vocab + each - 1) / each), 256, 0, s>>>(a, start, order, sums, (int)each,
                                                                              (int)groups, lines);
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
  return round_up((size_t)(vocab + 1) * 4) + round_up((size_t)tokens * 4) +
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
