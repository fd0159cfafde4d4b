// gq_vocab.hip -- gfx950 passes over rows of logits: the log probability of a given token with
// the row's entropy and its most likely alternatives, and the distillation loss from a teacher's
// top log probabilities with its gradient.
//
// Every pass reads a row once with the running maximum and sum of its softmax.  A block of 256
// threads streams a row, or a slice of it where there are few rows; slices are joined in their
// order by a second kernel, so results do not depend on timing.  A thread's step is a group of
// 32 elements, four 8-element chunks 2048 apart, each chunk aligned to its own size in memory: a
// row of an odd length starts inside a chunk, and the first and last chunk of a row are read
// element by element, nothing outside the row at all.
//
// With m the largest logit, c = 1 / T and d = z - m:  s = sum e^(c d), lse = c m + log s.  d is
// formed before it is scaled, so its rounding is relative to d, not to z.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "gq_lm.h"

namespace gq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef f32x4 f32x4_e4 __attribute__((aligned(4)));

constexpr int kThreads = 256;
constexpr int kPart = kThreads * 8;         // elements of one chunk of every thread
constexpr int kSweep = 4 * kPart;           // elements of one group of every thread
constexpr int kSweeps = 16;                 // groups of a thread in a slice, at most
constexpr int64_t kSlice = (int64_t)kSweep * kSweeps;
constexpr int kMaxSlices = 64;
constexpr int64_t kFill = 1024;             // blocks of a call, where its rows allow slices
constexpr int kCandidates = 1024;           // entries at or above the threshold, at most
constexpr float kLog2e = 1.44269504088896340736f;

// A slice of a row: virtual index v counts from the aligned place at or before the slice's first
// element; entry v - lead of the slice exists for lead <= v < lead + count.
struct Slice {
  const void *row;   // the row's first element
  int64_t first;     // slice's first entry in the row
  int32_t count;     // entries
  int32_t lead;      // entries from that place to the first
};

// The aligned place: a multiple of `grain` entries from the first row's beginning, 8, or a line of
// 128 bytes (log probabilities of 4095 x 50257 bf16: 92.6 us from chunks, 90.6 us from lines; the
// gradient of 1021 x 131071: 116 and 122 us).
__device__ __forceinline__ Slice slice_of(const void *logits, int elem, int64_t row, int64_t ld,
                                          int64_t vocab, int64_t part, int64_t each, int grain = 8) {
  Slice s;
  s.row = static_cast<const char *>(logits) + row * ld * elem;
  s.first = part * each;
  s.count = (int32_t)min(each, vocab - s.first);
  s.lead = (int32_t)((row * ld + s.first) & (grain - 1));
  return s;
}

__device__ __forceinline__ int sweeps_of(const Slice &s) {
  return (s.lead + s.count + kSweep - 1) / kSweep;
}

template <int DT>
__device__ __forceinline__ float entry(const Slice &s, int64_t i) {  // entry i of the slice
  if constexpr (DT == 0)
    return static_cast<const float *>(s.row)[s.first + i];
  else
    return __uint_as_float((uint32_t) static_cast<const uint16_t *>(s.row)[s.first + i] << 16);
}

// Eight entries as they lie in memory.
template <int DT>
struct Chunk {
  u32x4 w[DT == 0 ? 2 : 1];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0)
      return __uint_as_float(w[i / 4][i % 4]);
    else
      return __uint_as_float(i % 2 ? w[0][i / 2] & 0xFFFF0000u : w[0][i / 2] << 16);
  }
};

// A 16-byte load; ONCE: non-temporal, where nothing reads the row again (log probabilities of
// 4095 x 50257 bf16: 98 us with plain loads, 95 us so; loss and gradient together 195 and 190 us;
// the loss whose gradient is taken later loses the row so: 191 and 216 us for the two).
template <bool ONCE>
__device__ __forceinline__ u32x4 load_vector(const u32x4 *p) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

// The chunk at virtual index v (a multiple of 8), all of whose entries exist.
template <int DT, bool ONCE = false>
__device__ __forceinline__ Chunk<DT> load_whole(const Slice &s, int v) {
  const u32x4 *p = reinterpret_cast<const u32x4 *>(
      static_cast<const char *>(s.row) + (s.first - s.lead + v) * (DT == 0 ? 4 : 2));
  Chunk<DT> c;
  c.w[0] = load_vector<ONCE>(p);
  if constexpr (DT == 0) c.w[1] = load_vector<ONCE>(p + 1);
  return c;
}

// Any chunk of the slice; what is not there is -inf.
template <int DT>
__device__ __forceinline__ Chunk<DT> load_chunk(const Slice &s, int v) {
  const int at = v - s.lead;
  if (at >= 0 && at + 8 <= s.count) return load_whole<DT>(s, v);
  Chunk<DT> c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x =
        __float_as_uint(at + i >= 0 && at + i < s.count ? entry<DT>(s, at + i) : -INFINITY);
    if constexpr (DT == 0)
      c.w[i / 4][i % 4] = x;
    else if (i % 2 == 0)
      c.w[0][i / 2] = x >> 16;
    else
      c.w[0][i / 2] |= x;
  }
  return c;
}

// Entries of the chunk whose bit is set become -inf.
template <int DT>
__device__ __forceinline__ void strip(Chunk<DT> &x, uint32_t mask) {
  if (mask == 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!(mask >> i & 1u)) continue;
    if constexpr (DT == 0)
      x.w[i / 4][i % 4] = 0xFF800000u;
    else
      x.w[0][i / 2] = i % 2 ? (x.w[0][i / 2] & 0xFFFFu) | 0xFF800000u
                            : (x.w[0][i / 2] & 0xFFFF0000u) | 0xFF80u;
  }
}

// A thread's four chunks of sweep g; returns how many of them its wave has anything of.  Whether
// they are whole is one question a wave.
template <int DT, bool ONCE = false>
__device__ __forceinline__ int load_group(const Slice &s, int g, Chunk<DT> (&c)[4]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v = g * kSweep + wave * 512, end = s.lead + s.count;  // the wave's first chunk
  if (v >= s.lead && v + 3 * kPart + 512 <= end) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = load_whole<DT, ONCE>(s, v + j * kPart + lane * 8);
    return 4;
  }
  const int there = v >= end ? 0 : min((end - v + kPart - 1) / kPart, 4);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < there) c[j] = load_chunk<DT>(s, v + j * kPart + lane * 8);
  return there;
}

// ---------------------------------------------------------------- softmax statistics
// m: the largest entry (-inf: none above it); s = sum e^(c (x - ref)), w = sum (x - ref) e^(...),
// ref = max(m, lowest): a row masked everywhere gives s = 0.
struct Stat {
  float m, s, w;
};

__device__ __forceinline__ float ref_of(float m) { return fmaxf(m, -FLT_MAX); }

// e^(c d) with cl = c log2 e; d = -inf gives 0.
__device__ __forceinline__ float exp_of(float d, float cl) { return __builtin_amdgcn_exp2f(d * cl); }

__device__ __forceinline__ Stat moved(const Stat &a, float m, float cl) {  // to the reference of m
  if (a.s == 0.0f) return Stat{m, 0.0f, 0.0f};
  const float d = ref_of(a.m) - ref_of(m);
  const float f = exp_of(d, cl);
  return Stat{m, f * a.s, f == 0.0f ? 0.0f : f * (a.w + d * a.s)};
}

template <int DT, int N>
__device__ __forceinline__ float max_of(const Chunk<DT> (&c)[N]) {
  float m = c[0].get(0);
#pragma unroll
  for (int i = 1; i < 8 * N; ++i) m = fmaxf(m, c[i / 8].get(i % 8));
  return m;
}

// Adds chunks whose largest entry is gm.  Two partial sums: half the chain of dependent adds.
template <bool W, int DT, int N>
__device__ __forceinline__ void add_chunks(Stat &a, const Chunk<DT> (&c)[N], float gm, float cl) {
  if (gm > a.m) a = moved(a, gm, cl);
  const float ref = ref_of(a.m);
  float s[2] = {a.s, 0.0f}, w[2] = {a.w, 0.0f};
#pragma unroll
  for (int i = 0; i < 8 * N; ++i) {
    const float d = c[i / 8].get(i % 8) - ref, e = exp_of(d, cl);
    s[i & 1] += e;
    if constexpr (W) w[i & 1] = fmaf(fmaxf(d, -FLT_MAX), e, w[i & 1]);
  }
  a.s = s[0] + s[1];
  if constexpr (W) a.w = w[0] + w[1];
}

// Adds the `there` chunks of a group; returns their largest entry.
template <bool W, int DT>
__device__ __forceinline__ float add_group(Stat &a, const Chunk<DT> (&c)[4], int there, float cl) {
  if (there == 4) {
    const float gm = max_of(c);
    add_chunks<W>(a, c, gm, cl);
    return gm;
  }
  float gm = -INFINITY;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= there) break;
    const Chunk<DT> one[1] = {c[j]};
    const float m = max_of(one);
    add_chunks<W>(a, one, m, cl);
    gm = fmaxf(gm, m);
  }
  return gm;
}

// The block's statistic, the same in every thread: the maximum first, then every thread's sums at
// it, added in one order.  `room` holds one entry a wave.
template <int T>
__device__ __forceinline__ float block_max(float m, Stat *room) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6].m = m;
  __syncthreads();
  m = room[threadIdx.x % (T / 64)].m;
#pragma unroll
  for (int d = T / 128; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  return m;
}

template <bool W, int T = kThreads>
__device__ __forceinline__ Stat block_join(Stat a, float cl, Stat *room) {
  a = moved(a, block_max<T>(a.m, room), cl);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    a.s += __shfl_xor(a.s, d);
    if constexpr (W) a.w += __shfl_xor(a.w, d);
  }
  // only the sums: another wave may still be reading the maxima
  if ((threadIdx.x & 63) == 0) {
    room[threadIdx.x >> 6].s = a.s;
    room[threadIdx.x >> 6].w = a.w;
  }
  __syncthreads();
  a.s = room[threadIdx.x % (T / 64)].s;
  a.w = room[threadIdx.x % (T / 64)].w;
#pragma unroll
  for (int d = T / 128; d >= 1; d >>= 1) {
    a.s += __shfl_xor(a.s, d);
    if constexpr (W) a.w += __shfl_xor(a.w, d);
  }
  return a;
}

// A row's slices' statistics, joined: the same in every thread.
template <bool W>
__device__ __forceinline__ Stat join_slices(const Stat *in, int slices, float cl, Stat *room) {
  Stat a = {-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < slices; i += kThreads) {
    const Stat b = in[i];
    const float m = fmaxf(a.m, b.m);
    const Stat x = moved(a, m, cl), y = moved(b, m, cl);
    a = Stat{m, x.s + y.s, x.w + y.w};
  }
  return block_join<W>(a, cl, room);
}

template <int T = kThreads>
__device__ __forceinline__ double block_sum(double v, double *room) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
  __syncthreads();
  v = room[threadIdx.x % (T / 64)];
#pragma unroll
  for (int d = T / 128; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// ---------------------------------------------------------------- the largest entries
// Keys that order entries as their values, the lowest index first among equals; NaN is largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint64_t full_key(uint32_t key, uint32_t index) {
  return (uint64_t)key << 32 | (uint32_t)~index;
}

struct TopRoom {
  float group[kSweeps * kThreads];   // largest entry of each group
  uint32_t thread_max[kThreads];
  uint64_t cand[kCandidates];
  uint32_t hist[256];
  uint16_t hits[kCandidates];        // groups with an entry at or above the threshold
  uint32_t count, groups, prefix, need;
};

// Threshold t with at least k threads' maxima at or above it (0: fewer threads have an entry):
// the slice's k-th largest entry is not below it.  Bit by bit over the 256 maxima, four a lane,
// in every wave alike; stops as soon as exactly k are above.
__device__ __forceinline__ uint32_t top_threshold(const TopRoom &room, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = room.thread_max[lane + 64 * i];
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t | 1u << bit;
    int above = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) above += __popcll(__ballot(v[i] >= c));
    if (above >= k) t = c;
    if (above == k) break;
  }
  return t;
}

// The k-th largest entry of the slice by its digits, then what is above it and the lowest
// indices of what equals it.  For slices with more entries at the threshold than there is room
// for (masked or constant rows), and for NaN.
template <int DT>
__device__ void top_by_digits(const Slice &s, int k, TopRoom &room) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0, mask = 0;
  if (tid == 0) room.need = (uint32_t)k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    room.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < s.count; i += kThreads) {
      const uint32_t key = order_key(entry<DT>(s, i));
      if ((key & mask) == prefix) atomicAdd(&room.hist[key >> shift & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t need = room.need;
      int digit = 255;
      while (digit > 0 && room.hist[digit] < need) need -= room.hist[digit--];
      room.need = need;
      room.prefix = prefix | (uint32_t)digit << shift;
    }
    __syncthreads();
    prefix = room.prefix;
    mask |= 255u << shift;
  }
  const uint32_t need = room.need;
  if (tid == 0) room.count = 0;
  __syncthreads();
  for (int i = tid; i < s.count; i += kThreads) {
    const uint32_t key = order_key(entry<DT>(s, i));
    if (key > prefix) room.cand[atomicAdd(&room.count, 1u)] = full_key(key, (uint32_t)(s.first + i));
  }
  uint32_t taken = 0;
  for (int base = 0; base < s.count && taken < need; base += kThreads) {
    const int i = base + tid;
    const bool equal = i < s.count && order_key(entry<DT>(s, i)) == prefix;
    const uint64_t in_wave = __ballot(equal);
    __syncthreads();
    if ((tid & 63) == 0) room.hist[tid >> 6] = (uint32_t)__popcll(in_wave);
    __syncthreads();
    uint32_t before = taken, all = taken;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < tid >> 6) before += room.hist[w];
      all += room.hist[w];
    }
    before += (uint32_t)__popcll(in_wave & ((1ull << (tid & 63)) - 1));
    if (equal && before < need)
      room.cand[atomicAdd(&room.count, 1u)] = full_key(prefix, (uint32_t)(s.first + i));
    taken = all;
  }
  __syncthreads();
}

// Leaves the slice's min(k, count) largest entries' keys in room.cand (at least those), with
// room.count of them; room.group holds the groups' maxima, my_max this thread's.
template <int DT>
__device__ void top_candidates(const Slice &s, int k, float my_max, bool odd, TopRoom &room) {
  const int tid = threadIdx.x;
  room.thread_max[tid] = order_key(my_max);
  if (tid == 0) room.count = room.groups = 0;
  __syncthreads();
  if (!odd) {  // no NaN
    // as a value: what is not below it is taken
    const float t = key_value(max(top_threshold(room, k), order_key(-INFINITY)));
    for (int g = 0; g < sweeps_of(s); ++g)
      if (room.group[g * kThreads + tid] >= t) {
        const uint32_t n = atomicAdd(&room.groups, 1u);
        if (n < kCandidates) room.hits[n] = (uint16_t)(g * kThreads + tid);
      }
    __syncthreads();
    // a lane an entry of those groups: they are few, and a thread's own 32 would be read in turn
    const int entries = (int)min(room.groups, (uint32_t)kCandidates) * 32;
    for (int i = tid; i < entries; i += kThreads) {
      const int g = room.hits[i >> 5], e = i & 31;
      const int at =
          g / kThreads * kSweep + e / 8 * kPart + g % kThreads * 8 + (e & 7) - s.lead;
      if (at < 0 || at >= s.count) continue;
      const float x = entry<DT>(s, at);
      if (!(x >= t)) continue;
      const uint32_t n = atomicAdd(&room.count, 1u);
      if (n < kCandidates) room.cand[n] = full_key(order_key(x), (uint32_t)(s.first + at));
    }
  }
  __syncthreads();
  if (odd || room.groups > kCandidates || room.count > kCandidates) {
    __syncthreads();
    top_by_digits<DT>(s, min(k, s.count), room);
  }
}

// ---------------------------------------------------------------- log probabilities
__device__ __forceinline__ void put_top(const LogprobArgs &a, int64_t row, int place, uint64_t key,
                                        float ref, float log_s) {
  const float x = key_value((uint32_t)(key >> 32));
  const float d = (x - ref) * a.inv_t - log_s;
  a.top_ids[row * a.top + place] = (int32_t)~(uint32_t)key;
  // a masked entry; in a row whose sum is NaN it is NaN like the others
  a.top_logprobs[row * a.top + place] = x == -INFINITY && log_s == log_s ? -INFINITY : d;
}

template <int DT>
__device__ __forceinline__ void put_token(const LogprobArgs &a, int64_t row, const Stat &all) {
  const int64_t token = a.tokens[row];
  const float log_s = logf(all.s);
  float lp = 0.0f;
  if (token >= 0 && token < a.vocab) {
    const Slice s = slice_of(a.logits, DT == 0 ? 4 : 2, row, a.ld, a.vocab, 0, a.vocab);
    const float x = entry<DT>(s, token);
    lp = x == -INFINITY && all.s == all.s ? -INFINITY : (x - ref_of(all.m)) * a.inv_t - log_s;
  }
  a.logprob[row] = lp;
  a.entropy[row] = all.s == 0.0f ? 0.0f : log_s - a.inv_t * all.w / all.s;
}

// A block a slice.  One slice a row: the row's results; else the slice's statistic and its
// largest entries in order, for k_logprobs_join.  One pass: the maximum of each group is kept, so
// that the largest entries are looked for in the few groups that can hold them (a thread's maxima
// bound the k-th largest from below) and not in the row again.  4095 x 50257 bf16 with 20 entries:
// 91 us, 412 MB at 4.5 TB/s; the vector ALUs are some 70% busy with 12 instructions an entry, and
// the selection at a row's end is hidden by the other blocks of the CU; fp32 152 us, 5.4 TB/s.
// 1 x 50257 fp32 in 24 slices: 6.6 us, and 3.6 us to join them.
template <int DT, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs(const LogprobArgs a, int slices,
                                                       int64_t each) {
  __shared__ Stat stats[kThreads / 64];
  __shared__ typename std::conditional<TOP, TopRoom, int>::type room;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / slices, part = blockIdx.x % slices;
  const Slice s = slice_of(a.logits, DT == 0 ? 4 : 2, row, a.ld, a.vocab, part, each, DT == 0 ? 32 : 64);
  const float cl = a.inv_t * kLog2e;
  Stat mine = {-INFINITY, 0.0f, 0.0f};
  float my_max = -INFINITY;
  const int sweeps = sweeps_of(s);
  Chunk<DT> now[4], next[4];
  int there = load_group<DT, true>(s, 0, now), there_next = 0;
  for (int g = 0; g < sweeps; ++g) {
    if (g + 1 < sweeps) there_next = load_group<DT, true>(s, g + 1, next);
    const float gm = add_group<true>(mine, now, there, cl);
    if constexpr (TOP) room.group[g * kThreads + tid] = gm;
    my_max = fmaxf(my_max, gm);
#pragma unroll
    for (int j = 0; j < 4; ++j) now[j] = next[j];
    there = there_next;
  }
  const Stat all = block_join<true>(mine, cl, stats);
  uint64_t *keys = nullptr;
  if (slices > 1) {
    Stat *out = static_cast<Stat *>(a.scratch);
    keys = reinterpret_cast<uint64_t *>(out + (((int64_t)gridDim.x + 1) & ~1ll)) +
           (int64_t)blockIdx.x * a.top;
    if (tid == 0) out[blockIdx.x] = all;
  } else if (tid == 0) {
    put_token<DT>(a, row, all);
  }
  if constexpr (TOP) {
    top_candidates<DT>(s, a.top, my_max, all.s != all.s, room);
    const int n = (int)room.count;
    const float ref = ref_of(all.m), log_s = logf(all.s);
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = room.cand[i];
      int place = 0;
      for (int j = 0; j < n; ++j) place += room.cand[j] > key;
      if (place < a.top) {
        if (slices > 1)
          keys[place] = key;
        else
          put_top(a, row, place, key, ref, log_s);
      }
    }
    if (slices > 1)
      for (int i = n + tid; i < a.top; i += kThreads) keys[i] = 0;
  }
}

// A block a row: joins the slices; a few dozen KB, bound by latency.  With d = ceil(top / slices), the ceil(top / d)-th largest of
// the lists' d-th entries has `top` entries at or above it, so smaller ones are left out.  What is
// left is gathered in LDS, and an entry's place is the number of larger ones there; where more
// is left than fits (the largest entries all in a few slices), that number is found in every
// slice's ordered list by bisection.
constexpr int kJoinKeys = 512;
template <int DT>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(const LogprobArgs a, int slices) {
  __shared__ Stat stats[kThreads / 64];
  __shared__ uint64_t near[kJoinKeys];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, n = slices * a.top;
  const int64_t row = blockIdx.x;
  const Stat *in = static_cast<const Stat *>(a.scratch);
  const uint64_t *keys = reinterpret_cast<const uint64_t *>(in + ((a.rows * slices + 1) & ~1ll)) + row * n;
  uint32_t depth_key = 0;
  const int d = (a.top + slices - 1) / slices;
  if (a.top > 0 && slices <= 64 && lane < slices) depth_key = (uint32_t)(keys[lane * a.top + d - 1] >> 32);
  if (tid == 0) count = 0;
  const Stat all = join_slices<true>(in + row * slices, slices, a.inv_t * kLog2e, stats);
  if (tid == kThreads - 1) put_token<DT>(a, row, all);
  if (a.top == 0) return;
  uint32_t t = 0;
  const int want = (a.top + d - 1) / d;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t | 1u << bit;
    if (__popcll(__ballot(depth_key >= c)) >= want) t = c;
  }
  const uint64_t least = t != 0 ? (uint64_t)t << 32 : 1;  // 0 fills a list that is too short
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = keys[i];
    if (key < least) continue;
    const int at = atomicAdd(&count, 1);
    if (at < kJoinKeys) near[at] = key;
  }
  __syncthreads();
  const float ref = ref_of(all.m), log_s = logf(all.s);
  const int left = count;
  if (left <= kJoinKeys) {
    for (int i = tid; i < left; i += kThreads) {
      const uint64_t key = near[i];
      int place = 0;
      for (int j = 0; j < left; ++j) place += near[j] > key;
      if (place < a.top) put_top(a, row, place, key, ref, log_s);
    }
    return;
  }
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = keys[i];
    if (key < least) continue;
    int place = 0;
    for (int p = 0; p < slices && place < a.top; ++p) {
      const uint64_t *list = keys + p * a.top;
      int lo = 0, hi = a.top;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] > key)
          lo = mid + 1;
        else
          hi = mid;
      }
      place += lo;
    }
    if (place < a.top) put_top(a, row, place, key, ref, log_s);
  }
}

// ---------------------------------------------------------------- distillation
// With S the taught entries (a row's ids: inside the vocabulary, each at its first place) and R
// the rest: p_j = e^(lp_j), divided by their sum unless the rest has a bucket of its own, whose
// mass p_R = 1 - sum p_j is matched with q_R = sum of q over R.
//   loss = T^2 (sum p_j (log p_j - log q_j) + p_R (log p_R - log q_R))
//   dz_v = w T (P q_v - p_v) in S,  w T q_v (P - p_R / q_R) in R,  P = sum p_j + p_R
// P is 1 unless, with a tail, p_R counts as 0 or the entries sum to more than 1.
// q_R is summed over R itself, taught entries becoming -inf on the way, so nothing is subtracted.
// With m_R the largest logit of R and s_R = sum_R e^(c (z - m_R)) >= 1, R's terms are formed as
//   log q_R = c (m_R - m) + log s_R - log s,   dz_v = w T e^(c (z_v - m_R)) (P q_R - p_R) / s_R
// so that they stand where q_R is below fp32's range, or below fp64's.
struct Taught {
  alignas(16) int32_t id[kVocabTop];     // -1: not taught
  float p[kVocabTop];
  uint32_t in_group[kSweeps * kThreads];  // taught entries of each group of the slice
  double sums[kThreads / 64];
  Stat stats[kThreads / 64];
};

struct RowStat {   // what the gradient needs of a row
  float ref;       // largest logit
  float inv_s;     // P / sum e^(c (z - ref)); 0: the row is not taught
  float rest_ref;  // largest logit of R; without a tail `ref`
  float rest;      // (P q_R - p_R) / s_R; without a tail `inv_s`
  float scale;     // p_j = scale e^(lp_j - shift); with a tail 1
};

// As four numbers a row, for a gradient that is taken later.
__device__ __forceinline__ f32x4 pack_stat(const RowStat &r, bool tail) {
  return tail ? f32x4{r.ref, r.inv_s, r.rest_ref, r.rest} : f32x4{r.ref, r.inv_s, r.scale, 0.0f};
}

__device__ __forceinline__ RowStat unpack_stat(f32x4 q, bool tail) {
  return tail ? RowStat{q.x, q.y, q.z, q.w, 1.0f} : RowStat{q.x, q.y, q.x, q.y, q.z};
}

// Loads the row's ids: t.id[j] is -1 where entry j is not taught.  Comparisons four at a time and
// without a branch wait for LDS a few times, not once an entry (4096 x 50257 bf16, 64 taught: 190
// us with a branch each, 180 us so; 33 x 24553 fp32, 128 taught: 30 and 17 us).
template <typename Room>
__device__ __forceinline__ bool load_ids(const DistillArgs &a, int64_t row, Room &t) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid < a.top) t.id[tid] = a.top_ids[row * a.top + tid];
  __syncthreads();
  bool ok = false;
  if (tid < a.top) {
    const int32_t id = t.id[tid];
    bool again = false;
#pragma unroll 4
    for (int i = 0; i < a.top; i += 4) {  // places past the last are not before tid
      const i32x4 four = *reinterpret_cast<const i32x4 *>(&t.id[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) again |= (i + j < tid) & (four[j] == id);
    }
    ok = id >= 0 && id < a.vocab && !again;
  }
  __syncthreads();
  if (tid < a.top && !ok) t.id[tid] = -1;
  return ok;
}

struct Mass {    // of a row's taught entries
  double sum;    // sum of e^(lp - shift), in 64 bits: with a tail p_R is 1 less it
  double shift;  // with a tail 0
};

// Loads the row's ids and e^(lp - shift).  Without a tail only the entries' proportions count, so a
// sum that fp32 cannot hold well (nothing but unlikely entries, or entries that are not divided by
// their sum) is formed again relative to its largest; what is added for it is one comparison.
template <int T = kThreads, typename Room>
__device__ __forceinline__ Mass load_taught(const DistillArgs &a, int64_t row, Room &t) {
  const int tid = threadIdx.x;
  const float lp = tid < a.top ? a.top_logprobs[row * a.top + tid] : 0.0f;
  const bool ok = load_ids(a, row, t);
  double p = ok ? exp((double)lp) : 0.0;
  Mass m = {block_sum<T>(p, t.sums), 0.0};
  if (!a.tail && !(m.sum >= 0x1p-64 && m.sum <= 0x1p64)) {  // the same in every thread
    m.shift = ref_of(block_max<T>(ok ? lp : -INFINITY, t.stats));
    p = ok ? exp((double)lp - m.shift) : 0.0;
    m.sum = block_sum<T>(p, t.sums);
  }
  if (tid < a.top) t.p[tid] = (float)p;
  return m;
}

__device__ __forceinline__ int place_in(const Slice &s, int64_t id, int *bit) {
  const int v = (int)(id - s.first) + s.lead;
  const int in = v % kSweep;
  *bit = (in / kPart) * 8 + (in & 7);
  return v / kSweep * kThreads + (in % kPart) / 8;
}

// Statistic of the slice's entries in R (tail) or of all of them.
template <int DT, bool TAIL>
__device__ __forceinline__ Stat rest_stat(const DistillArgs &a, int64_t row, const Slice &s, Taught &t) {
  const int tid = threadIdx.x;
  Chunk<DT> now[4], next[4];
  int there = load_group<DT>(s, 0, now), there_next = 0;
  const float cl = a.inv_t * kLog2e;
  const int sweeps = sweeps_of(s);
  if constexpr (TAIL) {
    for (int g = 0; g < sweeps; ++g) t.in_group[g * kThreads + tid] = 0;
    load_ids(a, row, t);
    __syncthreads();
    if (tid < a.top && t.id[tid] >= s.first && t.id[tid] < s.first + s.count) {
      int bit;
      const int g = place_in(s, t.id[tid], &bit);
      atomicOr(&t.in_group[g], 1u << bit);
    }
    __syncthreads();
  }
  Stat mine = {-INFINITY, 0.0f, 0.0f};
  for (int g = 0; g < sweeps; ++g) {
    if (g + 1 < sweeps) there_next = load_group<DT>(s, g + 1, next);
    if constexpr (TAIL) {
      const uint32_t mask = t.in_group[g * kThreads + tid];
      if (mask != 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) strip(now[j], mask >> (8 * j) & 0xFFu);
    }
    add_group<false>(mine, now, there, cl);
#pragma unroll
    for (int j = 0; j < 4; ++j) now[j] = next[j];
    there = there_next;
  }
  return block_join<false>(mine, cl, t.stats);
}

// Loss and gradient constants of a row from the statistic of R (tail) or of all entries.  The
// loss is a small difference of logarithms of the same sums, so what follows the stream (128
// terms at most) is held in 64 bits: an error of R's sum then counts q_R - p_R times only.
template <int DT, bool TAIL, int T, typename Room>
__device__ __forceinline__ RowStat finish_row(const DistillArgs &a, int64_t row, Stat rest,
                                              const Mass &mass, Room &t, bool write = true) {
  const int tid = threadIdx.x;
  const float cl = a.inv_t * kLog2e;
  const bool mine = tid < a.top && t.id[tid] >= 0;
  float x = 0.0f, lp = 0.0f;
  if (mine) {
    const Slice s = slice_of(a.logits, DT == 0 ? 4 : 2, row, a.ld, a.vocab, 0, a.vocab);
    x = entry<DT>(s, t.id[tid]);
    lp = a.top_logprobs[row * a.top + tid];
  }
  float m = rest.m;
  if constexpr (TAIL) m = block_max<T>(mine ? fmaxf(x, rest.m) : rest.m, t.stats);
  const float ref = ref_of(m);
  const double inv_t = 1.0 / (double)a.temperature;
  const double shift = ((double)ref_of(rest.m) - ref) * inv_t;
  const double rest_s = rest.s == 0.0f ? 0.0 : (double)rest.s * exp(shift);
  double all_s = rest_s;
  if constexpr (TAIL) all_s += block_sum<T>(mine ? (double)exp_of(x - ref, cl) : 0.0, t.sums);
  const double log_s = log(all_s);
  double p_rest = TAIL ? fmax(1.0 - mass.sum, 0.0) : 0.0;
  const double scale = TAIL ? 1.0 : 1.0 / mass.sum;
  double term = 0.0;
  if (mine && !(lp == -INFINITY)) {
    const double log_p = TAIL ? (double)lp : (double)lp - mass.shift - log(mass.sum);
    const double log_q =
        x == -INFINITY && all_s == all_s ? -INFINITY : ((double)x - ref) * inv_t - log_s;
    term = exp(log_p) * (log_p - log_q);
  }
  double loss = block_sum<T>(term, t.sums);
  const double taught = block_sum<T>(mine ? 1.0 : 0.0, t.sums);
  // a row masked everywhere has q = 0, not 0 / 0
  const float inv_s = all_s == 0.0 ? 1.0f : (float)(1.0 / all_s);
  RowStat r = {ref, inv_s, ref, inv_s, (float)scale};
  if constexpr (TAIL) {
    // no entry is left for the rest, or q_R is 0 in 64 bits and p_R is the sum's rounding
    if (taught == (double)a.vocab || (rest_s == 0.0 && p_rest < 0x1p-16)) p_rest = 0.0;
    if (p_rest > 0.0) {
      const double log_q = rest.s == 0.0f && all_s == all_s ? -INFINITY : shift + log((double)rest.s) - log_s;
      loss += p_rest * (log(p_rest) - log_q);
    }
    const double p = mass.sum + p_rest;
    r.inv_s = all_s == 0.0 ? (float)p : (float)(p / all_s);
    r.rest_ref = ref_of(rest.m);
    r.rest = rest.s == 0.0f ? 0.0f : (float)((p * (rest_s / all_s) - p_rest) / rest.s);
  }
  const bool none = taught == 0.0 || (!TAIL && mass.sum == 0.0);
  if (none) r = RowStat{ref, 0.0f, ref, 0.0f, 0.0f};
  if (write && tid == 0) {
    a.loss[row] = none ? 0.0f : (float)(loss * a.temperature * a.temperature);
    if (a.stats) reinterpret_cast<f32x4 *>(a.stats)[row] = pack_stat(r, TAIL);
  }
  return r;
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

template <int DT>
__device__ __forceinline__ void put_grad(const DistillArgs &a, int64_t at, float v) {
  if constexpr (DT == 0)
    static_cast<float *>(a.grad)[at] = v;
  else
    static_cast<uint16_t *>(a.grad)[at] = to_bf16(v);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// What a row's entries outside S get: f e^(c (z - ref)), ref their largest.
struct RowGrad {
  float f, ref, cl;
  bool plain;  // f is finite; else an entry without probability must not become 0 times it
};

__device__ __forceinline__ float row_weight(const DistillArgs &a, int64_t row) {
  return (a.weight ? a.weight[row] : 1.0f) * a.temperature;
}

__device__ __forceinline__ RowGrad row_grad(const DistillArgs &a, const RowStat &r, float w) {
  const float f = r.inv_s == 0.0f ? 0.0f : w * r.rest;
  return RowGrad{f, r.inv_s == 0.0f ? 0.0f : r.rest_ref, a.inv_t * kLog2e, r.inv_s != 0.0f && fabsf(f) < INFINITY};
}

// Gradient of the chunk whose first entry is entry `at` of the slice; out: the row's gradient.
// Whole chunks are stored non-temporally: the gradient is not read again here, and past the
// Infinity Cache it does not push out logits (4096 x 50257 bf16: 222 us with plain stores, 209 us
// so; 1021 x 131071, loss and gradient apart: 228 and 198 us).
template <int DT, bool WHOLE>
__device__ __forceinline__ void put_chunk(const DistillArgs &a, int64_t out, const Slice &s, int at,
                                          const Chunk<DT> &c, const RowGrad &g) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float e = exp_of(c.get(i) - g.ref, g.cl);
    y[i] = g.f * e;
    if (!g.plain && (g.f == 0.0f || e == 0.0f)) y[i] = 0.0f;
  }
  if constexpr (WHOLE) {
    if constexpr (DT == 0) {
      f32x4_e4 *o = reinterpret_cast<f32x4_e4 *>(static_cast<float *>(a.grad) + out + at);
      __builtin_nontemporal_store(f32x4_e4{y[0], y[1], y[2], y[3]}, o);
      __builtin_nontemporal_store(f32x4_e4{y[4], y[5], y[6], y[7]}, o + 1);
    } else {
      __builtin_nontemporal_store(
          u32x4_e2{to_bf16_pair(y[0], y[1]), to_bf16_pair(y[2], y[3]), to_bf16_pair(y[4], y[5]),
                   to_bf16_pair(y[6], y[7])},
          reinterpret_cast<u32x4_e2 *>(static_cast<uint16_t *>(a.grad) + out + at));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i >= 0 && at + i < s.count) put_grad<DT>(a, out + at + i, y[i]);
  }
}

// The taught entry of this thread, if the slice has it: read before the row's gradient is
// written (which may replace the logits), written after it.
struct TaughtEntry {
  bool mine;
  int32_t id;
  float x, p;
};

template <int DT, typename Room>
__device__ __forceinline__ TaughtEntry taught_entry(const DistillArgs &a, const Slice &s, const Room &t) {
  TaughtEntry e = {false, -1, 0.0f, 0.0f};
  if ((int)threadIdx.x < a.top) {
    e.id = t.id[threadIdx.x];
    e.p = t.p[threadIdx.x];
    e.mine = e.id >= s.first && e.id < s.first + s.count;
    if (e.mine) e.x = entry<DT>(s, e.id - s.first);
  }
  return e;
}

template <int DT>
__device__ __forceinline__ void put_taught(const DistillArgs &a, int64_t row, const TaughtEntry &e,
                                           const RowStat &r, float w) {
  if (!e.mine) return;
  const float q = exp_of(e.x - r.ref, a.inv_t * kLog2e) * r.inv_s;
  put_grad<DT>(a, row * a.ldg + e.id, r.inv_s == 0.0f ? 0.0f : w * (q - e.p * r.scale));
}

// The gradient of a slice, from another read of it.
template <int DT>
__device__ __forceinline__ void grad_stream(const DistillArgs &a, int64_t row, const Slice &s,
                                            const RowStat &r, const Taught &t) {
  const TaughtEntry mine = taught_entry<DT>(a, s, t);
  __syncthreads();
  const float w = row_weight(a, row);
  const RowGrad g = row_grad(a, r, w);
  const int sweeps = sweeps_of(s);
  Chunk<DT> now[4], next[4];
  int there = load_group<DT>(s, 0, now), there_next = 0;
  for (int i = 0; i < sweeps; ++i) {
    if (i + 1 < sweeps) there_next = load_group<DT>(s, i + 1, next);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = i * kSweep + j * kPart + (int)threadIdx.x * 8 - s.lead;
      if (j < there) {
        if (at >= 0 && at + 8 <= s.count)
          put_chunk<DT, true>(a, row * a.ldg + s.first, s, at, now[j], g);
        else
          put_chunk<DT, false>(a, row * a.ldg + s.first, s, at, now[j], g);
      }
      now[j] = next[j];
    }
    there = there_next;
  }
  __syncthreads();
  put_taught<DT>(a, row, mine, r, w);
}

// A block a row that its registers hold (T threads, N chunks each): all of it in flight at once,
// read once, there for the largest entry, the sum and the gradient.  Chunks are counted from the
// 128-byte line that the row begins in, so that a wave's stores cover whole lines.  The chunks
// that the row's ends may cut are one more of threads 64 and 128.  4096 x 50257 bf16, loss and
// gradient: 177 us, 823 MB at 4.6 TB/s.  What is left is the time between a row's last load and its
// first store, two joins over the block, which the CU's two other blocks cover in part; an
// entry's two exponentials come on top of it.  A stream that reads the row again took
// 259 us, one block of 1024 threads a CU 346 us.
template <int T, int N>
struct RowRoom {
  alignas(16) int32_t id[kVocabTop];
  float p[kVocabTop];
  double sums[T / 64];
  Stat stats[T / 64];
  uint8_t in_chunk[N * T + 4];  // taught entries of each chunk
};

template <int DT, bool TAIL, int T, int N>
__global__ __launch_bounds__(T) void k_distill_row(const DistillArgs a) {
  __shared__ __align__(16) RowRoom<T, N> t;
  constexpr uint32_t kNone = DT == 0 ? 0xFF800000u : 0xFF80FF80u;
  constexpr int kElem = DT == 0 ? 4 : 2;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const Slice s = slice_of(a.logits, kElem, row, a.ld, a.vocab, 0, a.vocab, 128 / kElem);
  const float cl = a.inv_t * kLog2e;
  const int end = s.lead + s.count;
  const char *lines = static_cast<const char *>(s.row) - s.lead * kElem;
  Chunk<DT> c[N];
  auto load_row = [&](auto once) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (auto &w : c[j].w) w = u32x4{kNone, kNone, kNone, kNone};
      const int v = (j * T + tid) * 8;
      if (v >= s.lead && v + 8 <= end) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(lines + j * T * 8 * kElem +
                                                         (uint32_t)(tid * 8 * kElem));
        c[j].w[0] = load_vector<decltype(once)::value>(p);
        if constexpr (DT == 0) c[j].w[1] = load_vector<decltype(once)::value>(p + 1);
      }
    }
  };
  if (a.grad)
    load_row(std::true_type{});
  else
    load_row(std::false_type{});
  // the chunk of the row's end, and that of its beginning if it is another
  const bool cut = (tid == 64 && (end & 7) != 0) ||
                   (tid == 128 && (s.lead & 7) != 0 && ((s.lead ^ end) & ~7) != 0);
  const int cut_v = (tid == 64 ? end : s.lead) & ~7;
  const Mass mass = load_taught<T>(a, row, t);
  if constexpr (TAIL) {
    uint32_t *zero = reinterpret_cast<uint32_t *>(t.in_chunk);
    for (int i = tid; i < (N * T + 4) / 4; i += T) zero[i] = 0;
    __syncthreads();
    if (tid < a.top && t.id[tid] >= 0)
      atomicOr(&zero[(t.id[tid] + s.lead) >> 5], 1u << ((t.id[tid] + s.lead) & 31));
    __syncthreads();
  }
  // with a tail, taught entries leave the registers: their gradient is written apart
  auto cut_chunk = [&]() {
    Chunk<DT> x = load_chunk<DT>(s, cut_v);
    if constexpr (TAIL) strip(x, t.in_chunk[cut_v >> 3]);
    return x;
  };
  if constexpr (TAIL) {
#pragma unroll
    for (int j = 0; j < N; ++j) strip(c[j], t.in_chunk[j * T + tid]);
  }
  // Keeps the entries as they were loaded: kept widened from one use to the next, bf16 would take
  // twice the registers.
  auto repack = [&]() {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (auto &w : c[j].w) asm volatile("" : "+v"(w));
  };
  float m = max_of(c);
  repack();
  if (cut) {
    const Chunk<DT> x[1] = {cut_chunk()};
    m = fmaxf(m, max_of(x));
  }
  m = block_max<T>(m == m ? m : -INFINITY, t.stats);
  const float ref = ref_of(m);
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8 * N; ++i) sum[i & 1] += exp_of(c[i / 8].get(i % 8) - ref, cl);
  repack();
  if (cut) {
    const Chunk<DT> x = cut_chunk();
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i & 1] += exp_of(x.get(i) - ref, cl);
  }
  const Stat rest = {m, (float)block_sum<T>((double)(sum[0] + sum[1]), t.sums), 0.0f};
  const RowStat r = finish_row<DT, TAIL, T>(a, row, rest, mass, t);
  if (!a.grad) return;
  const TaughtEntry mine = taught_entry<DT>(a, s, t);
  __syncthreads();
  const float w = row_weight(a, row);
  const RowGrad g = row_grad(a, r, w);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int v = (j * T + tid) * 8;
    if (v >= s.lead && v + 8 <= end) put_chunk<DT, true>(a, row * a.ldg, s, v - s.lead, c[j], g);
  }
  if (cut) put_chunk<DT, false>(a, row * a.ldg, s, cut_v - s.lead, cut_chunk(), g);
  __syncthreads();
  put_taught<DT>(a, row, mine, r, w);
}

// A block a slice: the slice's statistic.  1021 x 131071 bf16: 58 us, 268 MB at 4.6 TB/s.
template <int DT, bool TAIL>
__global__ __launch_bounds__(kThreads) void k_distill_slices(const DistillArgs a, int slices,
                                                             int64_t each) {
  __shared__ Taught t;
  const int64_t row = blockIdx.x / slices, part = blockIdx.x % slices;
  const Slice s = slice_of(a.logits, DT == 0 ? 4 : 2, row, a.ld, a.vocab, part, each);
  const Stat rest = rest_stat<DT, TAIL>(a, row, s, t);
  if (threadIdx.x == 0) static_cast<Stat *>(a.scratch)[blockIdx.x] = rest;
}

// A block a row: the slices' statistics in their order, the loss and the gradient's constants.
// 1021 rows: 10.5 us, the latency of the taught entries' loads and of the joins in 64 bits.
template <int DT, bool TAIL>
__global__ __launch_bounds__(kThreads) void k_distill_join(const DistillArgs a, int slices) {
  __shared__ Taught t;
  const int64_t row = blockIdx.x;
  const Mass mass = load_taught(a, row, t);
  const Stat rest = join_slices<false>(static_cast<const Stat *>(a.scratch) + row * slices, slices,
                                       a.inv_t * kLog2e, t.stats);
  finish_row<DT, TAIL, kThreads>(a, row, rest, mass, t);
}

// A block a slice: the gradient from the rows' constants, or (JOIN) from the slices' statistics:
// every block joins its row's for itself, one kernel less than with the constants in between.
// 1021 x 131071 bf16: 113 us, 536 MB at 4.7 TB/s; with JOIN, 5 x 50257 fp32: 9.0 us.
template <int DT, bool JOIN, bool TAIL>
__global__ __launch_bounds__(kThreads) void k_distill_grad(const DistillArgs a, int slices,
                                                           int64_t each) {
  __shared__ Taught t;
  const int64_t row = blockIdx.x / slices, part = blockIdx.x % slices;
  const Slice s = slice_of(a.logits, DT == 0 ? 4 : 2, row, a.ld, a.vocab, part, each);
  const Mass mass = load_taught(a, row, t);
  RowStat r;
  if constexpr (JOIN) {
    const Stat rest = join_slices<false>(static_cast<const Stat *>(a.scratch) + row * slices, slices,
                                         a.inv_t * kLog2e, t.stats);
    r = finish_row<DT, TAIL, kThreads>(a, row, rest, mass, t, part == 0);
  } else {
    r = unpack_stat(reinterpret_cast<const f32x4 *>(a.stats)[row], a.tail);
  }
  grad_stream<DT>(a, row, s, r, t);
}

// Slices of a row: as many as fill the GPU a few times over, at least 2048 entries each, at most
// kSlice.
int slices_of(int64_t rows, int64_t vocab, int64_t *each, int64_t fill = kFill) {
  int64_t n = fill / rows;
  if (n > vocab / kPart) n = vocab / kPart;
  if (n > kMaxSlices) n = kMaxSlices;
  const int64_t least = (vocab + kSlice - 65) / (kSlice - 64);
  if (n < least) n = least;
  if (n < 1) n = 1;
  *each = ((vocab + n - 1) / n + 7) & ~7ll;
  return (int)((vocab + *each - 1) / *each);
}

template <int DT>
void logprobs_of(const LogprobArgs &a, int slices, int64_t each, hipStream_t s) {
  const unsigned blocks = (unsigned)(a.rows * slices);
  if (a.top > 0)
    k_logprobs<DT, true><<<blocks, kThreads, 0, s>>>(a, slices, each);
  else
    k_logprobs<DT, false><<<blocks, kThreads, 0, s>>>(a, slices, each);
  if (slices > 1) k_logprobs_join<DT><<<(unsigned)a.rows, kThreads, 0, s>>>(a, slices);
}

// The longest row that is held in registers: two blocks of 512 threads a CU with 16 chunks of bf16,
// 8 of fp32 a thread.  One block of 1024 for rows twice as long left the CU idle in its joins: 663
// x 68328 bf16 84 us, as slices 62 us; 2048 x 40000 fp32 244 and 209; 2000 x 128000 bf16 291 and
// 318, but its loss alone 203 and 119.
template <int DT>
constexpr int64_t kRowMax = 512 * (DT == 0 ? 64 : 128) - 64;

// Whether a block's registers hold a row; else its slices, one or more, leave their statistics in
// the scratch memory.  A launch has fewer than 2^32 threads, so blocks of 512 serve fewer than 2^23
// rows; kVocabRows is the limit of the others.
bool row_held(int slices, int64_t rows, int64_t vocab, int dtype) {
  return slices == 1 && vocab <= (dtype == 0 ? kRowMax<0> : kRowMax<1>) &&
         (rows < 1 << 23 || vocab <= 256 * 64 - 64);
}

template <int DT, bool TAIL>
void distill_of(const DistillArgs &a, int slices, int64_t each, hipStream_t s) {
  const unsigned rows = (unsigned)a.rows;
  // Three blocks of 256 threads and 26 chunks a CU where a row fits them (4096 x 50257 bf16: 194 us
  // when two of 512 and 16 took 212 us).
  if (row_held(slices, a.rows, a.vocab, DT)) {
    if (a.vocab <= 256 * 64 - 64)
      k_distill_row<DT, TAIL, 256, 8><<<rows, 256, 0, s>>>(a);
    else if (DT == 0 || a.vocab <= 512 * 64 - 64)
      k_distill_row<DT, TAIL, 512, 8><<<rows, 512, 0, s>>>(a);
    else if constexpr (DT == 1) {
      if (a.vocab <= 256 * 208 - 64)
        k_distill_row<DT, TAIL, 256, 26><<<rows, 256, 0, s>>>(a);
      else
        k_distill_row<DT, TAIL, 512, 16><<<rows, 512, 0, s>>>(a);
    }
    return;
  }
  const unsigned blocks = (unsigned)(a.rows * slices);
  k_distill_slices<DT, TAIL><<<blocks, kThreads, 0, s>>>(a, slices, each);
  // in place, a block's gradient would replace taught logits that another block still reads
  if (a.grad && a.grad != a.logits) {
    k_distill_grad<DT, true, TAIL><<<blocks, kThreads, 0, s>>>(a, slices, each);
    return;
  }
  DistillArgs b = a;
  if (!b.stats)
    b.stats = reinterpret_cast<float *>(static_cast<char *>(a.scratch) +
                                        (((size_t)a.rows * slices * sizeof(Stat) + 15) & ~(size_t)15));
  k_distill_join<DT, TAIL><<<(unsigned)a.rows, kThreads, 0, s>>>(b, slices);
  if (a.grad) k_distill_grad<DT, false, false><<<blocks, kThreads, 0, s>>>(b, slices, each);
}

}  // namespace

size_t logprobs_scratch(int64_t rows, int64_t vocab, int top) {
  int64_t each;
  const int n = slices_of(rows, vocab, &each);
  if (n == 1) return 0;
  return (size_t)((rows * n + 1) & ~1ll) * sizeof(Stat) + (size_t)rows * n * top * 8;
}

hipError_t launch_token_logprobs(const LogprobArgs &a, int dtype, hipStream_t s) {
  int64_t each;
  const int n = slices_of(a.rows, a.vocab, &each);
  if (dtype == 0)
    logprobs_of<0>(a, n, each, s);
  else
    logprobs_of<1>(a, n, each, s);
  return hipGetLastError();
}

// Slices of the distillation loss: a block a row from a block a CU on, where registers hold a row
// (512 x 50257 bf16 with the gradient: 48 us in two slices, 32 us so).  The loss alone takes the
// same way, so that it has the same bits (a stream would be faster: 4096 x 50257 bf16, 91 us
// against 107).
int distill_slices(int64_t rows, int64_t vocab, int dtype, int64_t *each) {
  return slices_of(rows, vocab, each, row_held(1, rows, vocab, dtype) ? 256 : kFill);
}

size_t distill_scratch(int64_t rows, int64_t vocab, int dtype) {
  int64_t each;
  const int n = distill_slices(rows, vocab, dtype, &each);
  return row_held(n, rows, vocab, dtype) ? 0 : (((size_t)rows * n * sizeof(Stat) + 15) & ~(size_t)15) + (size_t)rows * 16;
}

hipError_t launch_distill_loss(const DistillArgs &a, int dtype, hipStream_t s) {
  int64_t each;
  const int n = distill_slices(a.rows, a.vocab, dtype, &each);
  if (dtype == 0)
    a.tail ? distill_of<0, true>(a, n, each, s) : distill_of<0, false>(a, n, each, s);
  else
    a.tail ? distill_of<1, true>(a, n, each, s) : distill_of<1, false>(a, n, each, s);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const DistillArgs &a, int dtype, hipStream_t s) {
  int64_t each;
  const int n = slices_of(a.rows, a.vocab, &each);
  const unsigned blocks = (unsigned)(a.rows * n);
  if (dtype == 0)
    k_distill_grad<0, false, false><<<blocks, kThreads, 0, s>>>(a, n, each);
  else
    k_distill_grad<1, false, false><<<blocks, kThreads, 0, s>>>(a, n, each);
  return hipGetLastError();
}

}  // namespace gq
