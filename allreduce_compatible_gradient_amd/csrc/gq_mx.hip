// gq_mx.hip -- gfx950 kernels of microscaled 4-bit floating point: quantisation of a matrix by
// rows and by columns, decoding, and the product of two packed matrices.
//
// Format.  A row is cut into blocks of 32; a block holds one scale 2^(s - 127), s a byte, and 32
// codes of 4 bits: a sign and a magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6}.  Element 2t of a row
// sits in the low nibble of its byte t.  s = 255 makes the whole block NaN.  Rows are padded to
// a multiple of 256 elements (8 blocks) with zero codes and zero scales, which stand for zeros,
// so the product's K loop has no tail.
#include <math.h>

#include <type_traits>

#include "gq_device.h"
#include "gq_lm.h"

namespace gq {
namespace {


// ---------------------------------------------------------------- one block's encoding
// Scale byte of a block whose largest magnitude has the bits `top` (sign cleared).  To nearest:
// floor(log2 a) - 2, so that a lies in [4, 8) scales and what exceeds 6 saturates.  Stochastic:
// the least scale with a <= 6 scales, so that nothing saturates and the rounding is unbiased:
// one more where the mantissa is above 1.5.  Both are clamped at 2^-127 (byte 0).
template <bool STOCH>
__device__ __forceinline__ int scale_byte(uint32_t top) {
  int s = (int)(top >> 23) - 2;
  if (STOCH) s += (top & 0x7FFFFFu) > 0x400000u;
  return s < 0 ? 0 : s;
}

__device__ __forceinline__ float inverse_scale(int s) {
  return __uint_as_float((uint32_t)(254 - s) << 23);
}

// 2^(s - 127); 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 0 ? __uint_as_float(0x00400000u) : s == 255 ? __uint_as_float(0x7FC00000u)
                                                           : __uint_as_float(s << 23);
}

// Stochastic code of x (|x| * inv <= 6), 254 too large: the grid's spacing is 1/2 below 2, 1 below
// 4, 2 above, i.e. 2^(e - 1) with e the exponent of max(v, 1).  In units of it v has an exact
// whole part and fraction p, and the code goes up if fp32(h) < p * 2^32.  Codes are packed by
// adding shifted words, so the 254s are taken off once a word (kCodeBias).
constexpr uint32_t kCodeBias = 254u * 0x11111111u;
__device__ __forceinline__ uint32_t stochastic_code(float x, float inv, uint32_t h) {
  const float v = fabsf(x) * inv;
  const uint32_t e = __float_as_uint(fmaxf(v, 1.0f)) & 0x7F800000u;
  const float w = v * __uint_as_float(0x7F800000u - e);
  const uint32_t up = (float)h < __builtin_amdgcn_fractf(w) * 4294967296.0f;
  return (uint32_t)w + (e >> 22) + up;
}

__device__ __forceinline__ uint32_t sign_bit(float x) { return __float_as_uint(x) >> 31; }

// Eight codes of x * inv to nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t nearest_codes(const float *x, float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * inv, x[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * inv, x[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * inv, x[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * inv, x[7] * inv, 1.0f, 3);
  return w;
}

// ---------------------------------------------------------------- quantisation
// Largest over the lane's neighbours: quads, then 16 lanes (a block's lanes in the two kernels).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // [2,3,0,1]
}

// Four values at a time: a step of one needs two cycles' distance from its last.
__device__ __forceinline__ void row_max(uint32_t (&v)[4]) {
#define GQ_DPP_MAX(CTRL)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) v[i] =                                          \
      max(v[i], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[i], CTRL, 0xF, 0xF, true));
  GQ_DPP_MAX(0xB1)   // quad [1,0,3,2]
  GQ_DPP_MAX(0x4E)   // quad [2,3,0,1]
  GQ_DPP_MAX(0x141)  // half mirror
  GQ_DPP_MAX(0x140)  // mirror
#undef GQ_DPP_MAX
}

// By rows: a lane holds eight elements (one 16-byte load of bf16), four lanes a block, so a block's
// maximum takes two steps and its codes leave as one word a lane.  Threads run over the words of a
// packed row, padding included.  333 x 768 bf16, an operand of a product, takes 4.8 us and
// 1 x 4096 1.8 us: a launch's latency.  At size, to nearest it is bound by its bytes: 4096 x 11008
// fp32 37 us (204 MB, 5.5 TB/s), 2047 x 50257 bf16 50 us (5.2 TB/s); stochastic by the draws: 42 and
// 77 us.
template <int DT, bool STOCH>
__global__ __launch_bounds__(256) void k_mx_rows(const MxQuantArgs a, int pitch) {
  const int64_t row = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
  const int word = blockIdx.x * blockDim.x + threadIdx.x;
  if (row >= a.rows || word >= pitch * 4) return;  // whole quads
  const int64_t first = (int64_t)word * 8;
  float x[8];
  load_word<DT>(a.x, row * a.ld, first, a.cols, x);
  const uint32_t top = quad_max(top_of(x));
  const int s = scale_byte<STOCH>(top);
  const float inv = inverse_scale(s);
  uint32_t codes = 0;
  if constexpr (STOCH) {
    const uint32_t counter = a.index_base + (uint32_t)(row * a.cols + first);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      codes += (stochastic_code(x[i], inv, draw(counter + i, a.key_mix)) << (4 * i)) +
               (sign_bit(x[i]) << (4 * i + 3));
    codes -= kCodeBias;
  } else {
    codes = nearest_codes(x, inv);
  }
  const bool bad = top >= 0x7F800000u;
  reinterpret_cast<uint32_t *>(a.codes + row * pitch * 16)[word] = bad ? 0u : codes;
  if ((threadIdx.x & 3) == 0) a.scales[row * pitch + word / 4] = bad ? 255 : (uint8_t)s;
}

// By columns, or both ways (ROWS) in one read.  A block takes 128 rows x 128 columns, a wave 32
// rows of it; a lane holds two neighbouring columns of the 32 rows, so a column's block is a lane's
// own and a row's block lies in 16 lanes.  The draw of an element is shared by its two codes.  Row
// codes (a byte a lane and row) and the scales of both ways are gathered in LDS and leave as
// 16-byte and 4-byte pieces.  Measured both ways: 4096 x 11008 fp32 to nearest 54 us (229 MB, 4.2
// TB/s; codes_t leaves in 64-byte runs, so 71 MB are written for 48), 2047 x 50257 bf16 stochastic
// 127-158 us by the card, bound by the vector ALUs (51 instructions an element, 15 of them the draw,
// the rest two codes' encoding); by columns only 47 and 80 us.  Waves of 64 rows, which write whole
// lines of codes_t, took 59 and 144 us where these took 54 and 132: fewer waves at a time.
template <int DT>
struct Pair;  // two neighbouring elements as loaded
template <>
struct Pair<0> {
  float v[2];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <>
struct Pair<1> {
  uint32_t w;
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i ? w & 0xFFFF0000u : w << 16);
  }
};

template <int DT>
__device__ __forceinline__ Pair<DT> load_pair(const void *p, int i) {
  if constexpr (DT == 0) {
    typedef float f32x2_e4 __attribute__((ext_vector_type(2), aligned(4)));
    const f32x2_e4 v = *reinterpret_cast<const f32x2_e4 *>(static_cast<const float *>(p) + i);
    return Pair<0>{{v.x, v.y}};
  } else {
    typedef uint32_t u32_e2 __attribute__((aligned(2)));
    return Pair<1>{*reinterpret_cast<const u32_e2 *>(static_cast<const uint16_t *>(p) + i)};
  }
}

constexpr int kBothRows = 128, kBothCols = 128;
template <int DT, bool STOCH, bool ROWS>
__global__ __launch_bounds__(256, DT == 0 && !STOCH ? 4 : 3) void k_mx_both(const MxQuantArgs a, int pitch, int pitch_t) {
  __shared__ __align__(16) uint8_t row_codes[ROWS ? 4 : 1][ROWS ? 32 : 1][80];
  __shared__ __align__(16) uint8_t row_scales[ROWS ? 4 : 1][ROWS ? 32 : 1][4];
  __shared__ __align__(16) uint8_t col_scales[kBothCols][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t col0 = (int64_t)blockIdx.x * kBothCols, col = col0 + 2 * lane;
  const bool cols_whole = (int64_t)(blockIdx.x + 1) * kBothCols <= a.cols;
  const int64_t row0 = (int64_t)blockIdx.y * kBothRows + wave * 32;
  const char *tile = static_cast<const char *>(a.x) + (row0 * a.ld + col0) * (DT == 0 ? 4 : 2);
  const int64_t step = a.ld * (DT == 0 ? 4 : 2);  // rows are uniform: scalar addresses
  Pair<DT> x[32];
  if (cols_whole && row0 + 32 <= a.rows) {
#pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = load_pair<DT>(tile + r * step, 2 * lane);
  } else {
#if defined(__HIP_DEVICE_COMPILE__)  // buffer resources are a type of the device only
    // a resource a row, as long as what is there of it: what is outside loads as 0
    constexpr int kBytes = DT == 0 ? 4 : 2;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const bool there = row0 + r < a.rows && col0 < a.cols;
      const auto row = __builtin_amdgcn_make_buffer_rsrc(
          (void *)(there ? tile + r * step : tile), 0, there ? (int)(a.cols - col0) * kBytes : 0, 0x00027000);
      if constexpr (DT == 0)
        x[r] = Pair<0>{{__uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row, lane * 8, 0, 0)),
                        __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row, lane * 8 + 4, 0, 0))}};
      else
        x[r] = Pair<1>{(uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row, lane * 4, 0, 0) |
                       (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row, lane * 4 + 2, 0, 0) << 16};
    }
#endif
  }
  uint32_t top[2] = {0, 0};
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 4) {
    uint32_t row_top[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b0 = __float_as_uint(x[r0 + i].get(0)) & 0x7FFFFFFFu;
      const uint32_t b1 = __float_as_uint(x[r0 + i].get(1)) & 0x7FFFFFFFu;
      top[0] = max(top[0], b0);
      top[1] = max(top[1], b1);
      row_top[i] = max(b0, b1);
    }
    if constexpr (ROWS) {
      row_max(row_top);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        const bool bad = row_top[i] >= 0x7F800000u;
        const int s = scale_byte<STOCH>(row_top[i]);
        if ((lane & 15) == 0) row_scales[wave][r][lane >> 4] = bad ? 255 : (uint8_t)s;
        if constexpr (!STOCH) {
          const float f = inverse_scale(s);
          const uint32_t two = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[r].get(0) * f, x[r].get(1) * f, 1.0f, 0);
          row_codes[wave][r][lane] = bad ? 0 : (uint8_t)two;
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // keeps the live rows' temporaries few
  }
  wave_exchange();
  const int s0 = scale_byte<STOCH>(top[0]), s1 = scale_byte<STOCH>(top[1]);
  const float inv[2] = {inverse_scale(s0), inverse_scale(s1)};
  u32x4 codes[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 8 * q + j;
      uint32_t h[2] = {0, 0};
      if constexpr (STOCH) {
        const uint32_t counter = a.index_base + (uint32_t)((row0 + r) * a.cols + col0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          h[i] = draw(counter + 2 * lane + i, a.key_mix);
          w[i] += (stochastic_code(x[r].get(i), inv[i], h[i]) << (4 * j)) +
                  (sign_bit(x[r].get(i)) << (4 * j + 3));
        }
      } else if (j % 2 == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float lo = x[r].get(i) * inv[i], hi = x[r + 1].get(i) * inv[i];
          if (j == 0) w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], lo, hi, 1.0f, 0);
          if (j == 2) w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], lo, hi, 1.0f, 1);
          if (j == 4) w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], lo, hi, 1.0f, 2);
          if (j == 6) w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], lo, hi, 1.0f, 3);
        }
      }
      if constexpr (ROWS && STOCH) {
        const uint32_t s = row_scales[wave][r][lane >> 4];
        const float f = inverse_scale((int)s);
        const uint32_t two =
            stochastic_code(x[r].get(0), f, h[0]) + (stochastic_code(x[r].get(1), f, h[1]) << 4) +
            (sign_bit(x[r].get(0)) << 3) + (sign_bit(x[r].get(1)) << 7) - 254u * 0x11u;
        row_codes[wave][r][lane] = s == 255 ? 0 : (uint8_t)two;
      }
      if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) codes[i][q] = STOCH ? w[i] - kCodeBias : w[i];
  }
  const int64_t blk = row0 / kMxBlock;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool bad = top[i] >= 0x7F800000u;
    if (bad) codes[i] = u32x4{0, 0, 0, 0};
    if (col + i < a.cols)
      *reinterpret_cast<u32x4 *>(a.codes_t + ((col + i) * pitch_t + blk) * 16) = codes[i];
    col_scales[2 * lane + i][wave] = bad ? 255 : (uint8_t)(i ? s1 : s0);
  }
  if constexpr (ROWS) {
    wave_exchange();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = half * 16 + (lane >> 2);
      const u32x4 v = *reinterpret_cast<const u32x4 *>(&row_codes[wave][r][(lane & 3) * 16]);
      if (row0 + r < a.rows)
        *reinterpret_cast<u32x4 *>(a.codes + ((row0 + r) * pitch + blockIdx.x * 4 + (lane & 3)) * 16) = v;
    }
    if (lane < 32 && row0 + lane < a.rows)
      *reinterpret_cast<uint32_t *>(a.scales + (row0 + lane) * pitch + blockIdx.x * 4) =
          *reinterpret_cast<const uint32_t *>(row_scales[wave][lane]);
    wave_exchange();
  }
  __syncthreads();
  if (threadIdx.x < kBothCols) {
    const int64_t c = (int64_t)blockIdx.x * kBothCols + threadIdx.x;
    if (c < a.cols)
      *reinterpret_cast<uint32_t *>(a.scales_t + c * pitch_t + blockIdx.y * 4) =
          *reinterpret_cast<const uint32_t *>(col_scales[threadIdx.x]);
  }
}

// ---------------------------------------------------------------- decoding
// A thread eight elements: one word of codes, one scale, one 16-byte store of bf16, non-temporal:
// 2047 x 50257 took 59 us with plain stores and takes 39-42 us (261 MB, 6.2-6.7 TB/s), 50257 x 2047
// 64 and 41-52, 4096 x 11008 18.5 and 17.7.  The decoded values are exact in bf16.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const MxDequantArgs a, int pitch) {
  const int word = blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t first = (int64_t)word * 8;
  if (first >= a.cols) return;
  for (int64_t row = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; row < a.rows;
       row += (int64_t)gridDim.y * blockDim.y) {
    const uint32_t c = reinterpret_cast<const uint32_t *>(a.codes + row * pitch * 16)[word];
    const float f = scale_value(a.scales[row * pitch + word / 4]);
    float v[8];
    const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = v0[i] * f;
      v[2 + i] = v1[i] * f;
      v[4 + i] = v2[i] * f;
      v[6 + i] = v3[i] * f;
    }
    const int64_t at = row * a.ld + first;
    if (first + 8 <= a.cols) {
      if constexpr (DT == 0) {
        f32x4_e4 *o = reinterpret_cast<f32x4_e4 *>(static_cast<float *>(a.out) + at);
        __builtin_nontemporal_store(f32x4_e4{v[0], v[1], v[2], v[3]}, o);
        __builtin_nontemporal_store(f32x4_e4{v[4], v[5], v[6], v[7]}, o + 1);
      } else {
        __builtin_nontemporal_store(
            u32x4_e2{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]),
                     to_bf16_pair(v[6], v[7])},
            reinterpret_cast<u32x4_e2 *>(static_cast<uint16_t *>(a.out) + at));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + i < a.cols) {
          if constexpr (DT == 0)
            static_cast<float *>(a.out)[at + i] = v[i];
          else
            static_cast<uint16_t *>(a.out)[at + i] = to_bf16(v[i]);
        }
    }
  }
}

// ---------------------------------------------------------------- products
// Where a product goes: what there is of bias and of the old values is added in fp32, and the sum
// is rounded once.
struct Sink {
  void *out;
  const float *bias;
  int64_t ld, rows, cols;
  int32_t dtype, accumulate;
};

__device__ __forceinline__ Sink sink_of(const MxMatmulArgs &a) {
  return Sink{a.out, a.bias, a.ldo, a.M, a.N, a.out_dtype, a.accumulate};
}

__device__ __forceinline__ void put_one(const Sink &s, int64_t m, int64_t n, float v) {
  if (s.bias) v += s.bias[n];
  const int64_t at = m * s.ld + n;
  if (s.dtype == 0) {
    float *o = static_cast<float *>(s.out) + at;
    *o = s.accumulate ? *o + v : v;
  } else {
    uint16_t *o = static_cast<uint16_t *>(s.out) + at;
    if (s.accumulate) v += __uint_as_float((uint32_t)*o << 16);
    *o = to_bf16(v);
  }
}

// Eight neighbouring elements of a row (16 bytes of bf16, 32 of fp32).
[[maybe_unused]] __device__ __forceinline__ void put_eight(const Sink &s, int64_t m, int64_t n, f32x4 lo, f32x4 hi) {
  if (m >= s.rows || n >= s.cols) return;
  if (n + 8 > s.cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < s.cols) put_one(s, m, n + i, i < 4 ? lo[i & 3] : hi[i & 3]);
    return;
  }
  if (s.bias) {
    const f32x4_e4 *b = reinterpret_cast<const f32x4_e4 *>(s.bias + n);
    lo += b[0];
    hi += b[1];
  }
  const int64_t at = m * s.ld + n;
  if (s.dtype == 0) {
    f32x4_e4 *o = reinterpret_cast<f32x4_e4 *>(static_cast<float *>(s.out) + at);
    if (s.accumulate) {
      lo += o[0];
      hi += o[1];
    }
    o[0] = lo;
    o[1] = hi;
  } else {
    uint16_t *o = static_cast<uint16_t *>(s.out) + at;
    if (s.accumulate) {
      float x[8];
      load_eight<1>(o, 0, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] += x[i];
        hi[i] += x[4 + i];
      }
    }
    *reinterpret_cast<u32x4_e2 *>(o) = u32x4{to_bf16_pair(lo[0], lo[1]), to_bf16_pair(lo[2], lo[3]),
                                             to_bf16_pair(hi[0], hi[1]), to_bf16_pair(hi[2], hi[3])};
  }
}

// Tiled product, C = A B^T on packed operands, for more than kFewRows rows:
// 8192 x 11008 x 4096 takes 190-195 us, 3.8-3.9 PFLOP/s; a step of
// K takes a CU 1.8-1.9 us on random operands and 1.4-1.7 us on zeros, as the card lowers its clock
// (to 1.9 GHz by the counters) under load; a loop of nothing but this instruction reaches 6.6 PFLOP/s
// on random data, 112 us.  The matrix cores are busy 47% of the time, LDS 24%, and waves wait for 31%
// of theirs: one block a CU, so nothing covers a step's barrier and its wait for the next operands,
// nor the first loads and the stores (some 40 us of the whole), and 1376 tiles fill 5.4 of 6 rounds.
// Tried and not faster: 16x16x128 instructions, four waves of 128 x 128 each, operands fetched across
// the barrier.
// A block of WM x WN waves, a wave FM x FN tiles of 32 x 32, K in steps of 256
// (128 bytes of a row).  v_mfma_scale_f32_32x32x64: lane l holds 32 elements of row l mod 32,
// those of block l / 32, and that block's scale; the result has column l mod 32 and rows
// 8 i + 4 (l / 32) + 0..3.  The weights (B) are the first operand, so a lane ends with four
// neighbouring n of one m.
//
// The operands go from memory to LDS without registers (buffer loads with an LDS destination),
// one K step ahead, in two static buffers: the loop body handles two steps, so that every LDS
// access names its buffer and waits only for its own loads.  Row r's 16-byte chunk c is kept at
// chunk c XOR key(r), key(r) = (r XOR r / 8 mod 4) mod 8: 16 rows' reads of one chunk column
// fall on 16 different places of 256 bytes.  A row's scales of two steps are 16 bytes: a thread
// a row brings them to LDS every second step (read by each wave for itself, 8 bytes of 32
// different lines an instruction, they cost as much L2 traffic as the codes).  One permutation
// puts a lane's four scales of a step (every second byte) into a word whose bytes the four
// products of the step select.
[[maybe_unused]] __device__ __forceinline__ int swizzle_key(int r) { return (r ^ (r >> 3 & 3)) & 7; }

template <int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM *WN * 64) void k_mx_matmul(const MxMatmulArgs a, int pitch,
                                                           int tiles_m, int tiles_n,
                                                           int steps_each) {
#if defined(__HIP_DEVICE_COMPILE__)  // buffer resources are a type of the device only
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32, T = WM * WN * 64;
  constexpr int CA = BM * 8 / T, CB = BN * 8 / T;  // 16-byte chunks a thread and step
  __shared__ __align__(1024) uint8_t lds0[(BM + BN) * 128];
  __shared__ __align__(1024) uint8_t lds1[(BM + BN) * 128];
  __shared__ __align__(1024) uint8_t lds_scales[(BM + BN + T - 1) / T * T * 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int bm = blockIdx.x % tiles_m, bn = blockIdx.x / tiles_m;
  const int64_t m0 = (int64_t)bm * BM, n0 = (int64_t)bn * BN;
  const int steps = pitch / 8;
  const int step0 = blockIdx.y * steps_each;
  const int count = min(steps_each, steps - step0);
  const int row_bytes = pitch * 16;
  const int rows_a = (int)min((int64_t)BM, a.M - m0), rows_b = (int)min((int64_t)BN, a.N - n0);
  // resources that end with the tile's last row: nothing outside the matrices is ever read
  const auto ra = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(static_cast<const uint8_t *>(a.a) + m0 * row_bytes), 0, rows_a * row_bytes, 0x00027000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc((void *)(a.b + n0 * row_bytes), 0,
                                                    rows_b * row_bytes, 0x00027000);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc((void *)(a.a_scales + m0 * pitch), 0,
                                                     rows_a * pitch, 0x00027000);
  const auto rsb = __builtin_amdgcn_make_buffer_rsrc((void *)(a.b_scales + n0 * pitch), 0,
                                                     rows_b * pitch, 0x00027000);
  int off_a[CA], off_b[CB];
  {
    const int row = tid >> 3, chunk = ((tid & 7) ^ swizzle_key(row)) << 4;  // T / 8 is a multiple of 32
#pragma unroll
    for (int i = 0; i < CA; ++i) off_a[i] = min(row + i * (T / 8), rows_a - 1) * row_bytes + chunk;
#pragma unroll
    for (int i = 0; i < CB; ++i) off_b[i] = min(row + i * (T / 8), rows_b - 1) * row_bytes + chunk;
  }
  const int r32 = lane & 31, half = lane >> 5;
  int frag[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) frag[j] = r32 * 128 + (((2 * j + half) ^ swizzle_key(r32)) << 4);
  const uint32_t mine = half ? 0x07050301u : 0x06040200u;

  f32x16 acc[FM][FN] = {};
  int pa[2][FM], pb[2][FN];             // scales of two steps, ready for the products
  auto issue = [&](uint8_t *lds, int k) {  // loads of step k
#pragma unroll
    for (int i = 0; i < CA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_PTR void *)(lds + (i * T + wave * 64) * 16),
                                               16, off_a[i], k * 128, 0, 0);
#pragma unroll
    for (int i = 0; i < CB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (LDS_PTR void *)(lds + BM * 128 + (i * T + wave * 64) * 16), 16, off_b[i], k * 128, 0,
          0);
  };
  // Scales of steps k and k + 1, a thread a row (rows of A, then of B; a wave has only one kind).
  auto issue_scales = [&](int k) {
#pragma unroll
    for (int i = 0; i < (BM + BN + T - 1) / T; ++i) {
      const int first = i * T + wave * 64, r = first + lane;
      LDS_PTR void *to = (LDS_PTR void *)(lds_scales + first * 16);
      if (first < BM)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, to, 16, min(r, rows_a - 1) * pitch, k * 8, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, to, 16, min(r - BM, rows_b - 1) * pitch, k * 8,
                                                 0, 0);
    }
  };
  auto pick = [&](uint32_t lo, uint32_t hi) { return (int)__builtin_amdgcn_perm(hi, lo, mine); };
  auto read_scales = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const u32x4 s = *reinterpret_cast<const u32x4 *>(lds_scales + ((wm * FM + i) * 32 + r32) * 16);
      pa[0][i] = pick(s.x, s.y);
      pa[1][i] = pick(s.z, s.w);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const u32x4 s =
          *reinterpret_cast<const u32x4 *>(lds_scales + (BM + (wn * FN + j) * 32 + r32) * 16);
      pb[0][j] = pick(s.x, s.y);
      pb[1][j] = pick(s.z, s.w);
    }
  };
  auto arrive = [&]() {  // every wave's loads so far are in LDS, its reads of the other buffer done
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
  };
  auto multiply = [&](const uint8_t *lds, const int (&sa)[FM], const int (&sb)[FN]) {
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t *la = lds + wm * FM * 32 * 128, *lb = lds + (BM + wn * FN * 32) * 128;
    i32x4 fa[2][FM], fb[2][FN];
    auto fetch = [&](int j) {  // operands of products j, one group ahead of them
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[j & 1][i] = *reinterpret_cast<const i32x4 *>(la + frag[j] + i * 4096);
#pragma unroll
      for (int i = 0; i < FN; ++i)
        fb[j & 1][i] = *reinterpret_cast<const i32x4 *>(lb + frag[j] + i * 4096);
    };
    fetch(0);
#define GQ_MX_STEP(J)                                                                           \
  {                                                                                             \
    if (J < 3) fetch(J + 1);                                                                    \
    __builtin_amdgcn_sched_barrier(0);                                                          \
    _Pragma("unroll") for (int i = 0; i < FM; ++i)                                              \
        _Pragma("unroll") for (int j = 0; j < FN; ++j) {                                        \
      const i32x4 u = fa[J & 1][i], v = fb[J & 1][j];                                           \
      const i32x8 x = __builtin_shufflevector(u, u, 0, 1, 2, 3, -1, -1, -1, -1);                \
      const i32x8 y = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);                \
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(y, x, acc[i][j], 4, 4, J,     \
                                                                  sb[j], J, sa[i]);             \
    }                                                                                           \
    __builtin_amdgcn_sched_barrier(0);                                                          \
  }
    GQ_MX_STEP(0)
    GQ_MX_STEP(1)
    GQ_MX_STEP(2)
    GQ_MX_STEP(3)
#undef GQ_MX_STEP
  };
  const int last = step0 + count - 1;
  int k = step0;
  if (count & 1) {  // an odd count's first step, so that the loop takes two at a time
    issue(lds1, k);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const u32x2 s = __builtin_amdgcn_raw_buffer_load_b64(
          rsa, min((wm * FM + i) * 32 + r32, rows_a - 1) * pitch, k * 8, 0);
      pa[0][i] = pick(s.x, s.y);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const u32x2 s = __builtin_amdgcn_raw_buffer_load_b64(
          rsb, min((wn * FN + j) * 32 + r32, rows_b - 1) * pitch, k * 8, 0);
      pb[0][j] = pick(s.x, s.y);
    }
    arrive();
    issue(lds0, min(k + 1, last));
    if (k < last) issue_scales(k + 1);
    multiply(lds1, pa[0], pb[0]);
    ++k;
  } else {
    issue(lds0, k);
    issue_scales(k);
  }
  for (; k <= last; k += 2) {
    arrive();
    issue(lds1, k + 1);
    read_scales();
    multiply(lds0, pa[0], pb[0]);
    arrive();
    issue(lds0, min(k + 2, last));  // past the end: the last steps again, not multiplied
    issue_scales(min(k + 2, last - 1));
    multiply(lds1, pa[1], pb[1]);
  }
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();  // no load into LDS is in flight when the block ends
  // A wave's 32 rows of an i cross its own part of LDS, so that they leave along n in 16-byte
  // chunks, whole lines a row: lane l has four n of row l mod 32 before.  Chunks are XORed with
  // the row as above.
  Sink sink = sink_of(a);
  if (gridDim.y > 1)
    sink = Sink{a.partial + (int64_t)blockIdx.y * a.M * a.N, nullptr, a.N, a.M, a.N, 0, 0};
  static_assert(WM * WN * 32 * FN * 128 <= (BM + BN) * 128, "the waves' rows fit one buffer");
  uint8_t *own = lds0 + wave * 32 * FN * 128;
  const int64_t wm0 = m0 + wm * FM * 32, wn0 = n0 + wn * FN * 32;
  if (!sink.bias && !sink.accumulate && n0 + BN <= a.N) {
    // Nothing to add and no row cut short.  (With the general way's questions at each store, the
    // stores ran at 2 TB/s: 8192 x 11008 x 4096 193 us so, 216 us with a bias, 234 us where old values
    // are added.)
    // Rows on 128-byte lines are stored non-temporally: every store covers whole lines, and the
    // operands keep their place in the caches (8192 x 11008 x 4096: 225 us with plain stores, 199 us
    // so; rows off the lines lose by it: 4096 x 50257 x 768 205 us plain, 244 us).
    auto leave = [&](auto half_width, auto on_lines) {
      constexpr bool kHalf = decltype(half_width)::value;  // bf16
      constexpr int kCpr = kHalf ? FN * 4 : FN * 8, kRowBytes = kCpr * 16, kElem = kHalf ? 2 : 4;
      const int lrow = lane / kCpr, lchunk = lane % kCpr;
      const int64_t row_bytes = sink.ld * kElem;
      char *out = static_cast<char *>(sink.out) + (wm0 + lrow) * row_bytes + wn0 * kElem + lchunk * 16;
      const int rows = (int)min((int64_t)FM * 32, a.M - wm0) - lrow;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            if constexpr (kHalf) {
              const int chunk = (j * 4 + q) ^ (r32 & (kCpr - 1));
              *reinterpret_cast<u32x2 *>(own + r32 * kRowBytes + chunk * 16 + half * 8) =
                  u32x2{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3])};
            } else {
              const int chunk = (j * 8 + 2 * q + half) ^ (r32 & (kCpr - 1));
              *reinterpret_cast<f32x4 *>(own + r32 * kRowBytes + chunk * 16) = f32x4{v[0], v[1], v[2], v[3]};
            }
          }
        wave_exchange();
#pragma unroll
        for (int p = 0; p < kCpr / 2; ++p) {
          const int row = p * (64 / kCpr) + lrow;
          const u32x4 v = *reinterpret_cast<const u32x4 *>(own + row * kRowBytes + ((lchunk ^ (row & (kCpr - 1))) * 16));
          const int at = i * 32 + p * (64 / kCpr);
          if (at < rows) {
            if constexpr (decltype(on_lines)::value)
              __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(out + at * row_bytes));
            else
              *reinterpret_cast<u32x4_e2 *>(out + at * row_bytes) = v;
          }
        }
        wave_exchange();
      }
    };
    const bool lines = ((reinterpret_cast<uintptr_t>(sink.out) | (uint64_t)sink.ld * (sink.dtype == 0 ? 4 : 2)) & 127) == 0;
    if (sink.dtype == 0)
      lines ? leave(std::false_type{}, std::true_type{}) : leave(std::false_type{}, std::false_type{});
    else
      lines ? leave(std::true_type{}, std::true_type{}) : leave(std::true_type{}, std::false_type{});
    return;
  }
  constexpr int kRow = FN * 128, kChunks = FN * 8;  // bytes and chunks of a row of fp32
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int chunk = (j * 8 + 2 * q + half) ^ (r32 & (kChunks - 1));
        *reinterpret_cast<f32x4 *>(own + r32 * kRow + chunk * 16) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
    wave_exchange();
#pragma unroll 1
    for (int p = 0; p < kChunks / 4; ++p) {
      const int row = p * (128 / kChunks) + lane / (kChunks / 2), c = lane % (kChunks / 2) * 2;
      const f32x4 lo = *reinterpret_cast<const f32x4 *>(own + row * kRow + ((c ^ (row & (kChunks - 1))) * 16));
      const f32x4 hi = *reinterpret_cast<const f32x4 *>(own + row * kRow + (((c + 1) ^ (row & (kChunks - 1))) * 16));
      put_eight(sink, wm0 + i * 32 + row, wn0 + c * 4, lo, hi);
    }
    wave_exchange();
  }
#endif
}

// The partial products of the K splits, added in their order: they are few and small
// where splits are used (64 x 4096 x 11008 in 4: 4 MB), so a launch's latency bounds it.
__global__ __launch_bounds__(256) void k_mx_join(const MxMatmulArgs a, int splits) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.M * a.N) return;
  float v = 0.0f;
  for (int i = 0; i < splits; ++i) v += a.partial[(int64_t)i * a.M * a.N + t];
  put_one(sink_of(a), t / a.N, t % a.N, v);
}

// Few rows of A (M <= 16, one decoded token to a small batch): the weights' bytes bound it (1 x 4096
// by 11008 x 4096, 24 MB: 6.9 us, 3.5 TB/s, a launch and the packing before the first product), so
// each block streams 16 rows of B straight to registers, its waves on interleaved K steps of
// 256, and nothing of B is shared.  v_mfma_scale_f32_16x16x128: lane l holds 32 elements of row
// l mod 16, block l / 16 of the step.  fp32 / bf16 rows are packed by the block into LDS, eight
// elements a lane, while its first weights are on their way (a lane packing its own operand's 32
// elements, with the lanes of absent rows idle, took 12 us in that case).
// The waves' sums meet in LDS, in order.
constexpr int kFewWaves = 8;
// LDS of M packed rows: a row is padded by a chunk, so that 16 rows lie on different banks.
inline size_t few_lds(int64_t M, int64_t pitch) { return (size_t)M * (size_t)(pitch * 17 + 16); }

template <int AT>
__global__ __launch_bounds__(kFewWaves * 64) void k_mx_matmul_few(const MxMatmulArgs a, int pitch) {
  __shared__ f32x4 sums[kFewWaves][64];
  extern __shared__ __align__(16) uint8_t packed[];  // M rows of codes, then of scales
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quarter = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = min(n0 + r16, a.N - 1);
  const uint8_t *b = a.b + n * pitch * 16, *bs = a.b_scales + n * pitch;
  // a wave's step of B, the next one loaded before this one is used
  struct Step {
    i32x4 codes[2];
    u32x2 scales;
  };
  auto load = [&](int blk) {
    Step s;
    s.codes[0] = *reinterpret_cast<const i32x4 *>(b + (int64_t)(blk + quarter) * 16);
    s.codes[1] = *reinterpret_cast<const i32x4 *>(b + (int64_t)(blk + 4 + quarter) * 16);
    s.scales = *reinterpret_cast<const u32x2 *>(bs + blk);
    return s;
  };
  Step now = {}, next = {};
  if (wave * 8 < pitch) now = load(wave * 8);
  const int row_bytes = AT == 2 ? pitch * 16 : pitch * 16 + 16;
  const uint8_t *rows = static_cast<const uint8_t *>(a.a), *scales = a.a_scales;
  if constexpr (AT != 2) {
    uint8_t *out_scales = packed + (int)a.M * row_bytes;
    const int words = pitch * 4;
    for (int i = threadIdx.x; i < (int)a.M * words; i += kFewWaves * 64) {
      const int m = i / words, word = i % words;
      float x[8];
      load_word<AT>(a.a, m * a.lda, (int64_t)word * 8, a.K, x);
      const uint32_t top = quad_max(top_of(x));
      const int s = scale_byte<false>(top);
      const uint32_t codes = nearest_codes(x, inverse_scale(s));
      const bool bad = top >= 0x7F800000u;
      reinterpret_cast<uint32_t *>(packed + m * row_bytes)[word] = bad ? 0u : codes;
      if ((word & 3) == 0) out_scales[m * pitch + word / 4] = bad ? 255 : (uint8_t)s;
    }
    rows = packed;
    scales = out_scales;
    __syncthreads();
  }
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int blk = wave * 8; blk < pitch; blk += kFewWaves * 8) {
    if (blk + kFewWaves * 8 < pitch) next = load(blk + kFewWaves * 8);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = blk + 4 * h + quarter;
      const i32x4 fb = now.codes[h];
      const int sb = (int)(now.scales[h] >> (8 * quarter));
      i32x4 fa = {0, 0, 0, 0};
      int sa = 0;
      if (r16 < a.M) {
        fa = *reinterpret_cast<const i32x4 *>(rows + (int64_t)r16 * row_bytes + at * 16);
        sa = scales[(int64_t)r16 * pitch + at];
      }
      const i32x8 x = __builtin_shufflevector(fa, fa, 0, 1, 2, 3, -1, -1, -1, -1);
      const i32x8 y = __builtin_shufflevector(fb, fb, 0, 1, 2, 3, -1, -1, -1, -1);
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, acc, 4, 4, 0, sb, 0, sa);
    }
    now = next;
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int from = threadIdx.x >> 2, e = threadIdx.x & 3;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += sums[w][from][e];
    const int64_t m = from & 15, col = n0 + 4 * (from >> 4) + e;
    if (m < a.M && col < a.N) put_one(sink_of(a), m, col, v);
  }
}

constexpr int kCus = 256;

struct MatmulPlan {
  int bm, bn;          // tile
  int splits, each;    // K splits and steps of each
};

// Tile and K splits of a product of more than kFewRows rows.  The tile is the one of the least
// expected time: with n blocks on the fullest CU, n (step K / 256 + rest) + wait K / 256, the three
// constants of each tile (in us) fitted to 260 sizes (M 17 to 8192, N 768 to 51200, K 256 to
// 11008; the operands not in L2), where the tile so chosen takes 1.03 times the best one's time in
// the mean; bounds on the numbers of tiles took 1.06 (248 x 36032 x 4561: 256 x 256 31.6 us, 128 x
// 128 44.3; 333 x 50257 x 768: 27.6 and 30.4; 128 x 4096 x 4096: 64 x 128 8.7, 128 x 128 11.9).
// Splits only where tiles are few and K is long: partial products cost a second kernel and
// their bytes (64 x 4096 x 11008: 17 us whole, 13.2 in 4; 64 x 4096 x 4096 is no faster in 2).
MatmulPlan plan_matmul(int64_t M, int64_t N, int64_t K) {
  struct Tile {
    int bm, bn;
    float step, rest, wait;
  };
  constexpr Tile kTiles[3] = {
      {256, 256, 1.8f, 3.5f, 0.0f}, {128, 128, 0.54f, 1.7f, 0.47f}, {64, 128, 0.44f, 2.2f, 0.45f}};
  MatmulPlan p = {};
  const int64_t steps = mx_pitch(K) / 8;
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  float least = INFINITY;
  for (const Tile &t : kTiles) {
    const float each = (float)((tiles(t.bm, t.bn) + kCus - 1) / kCus);
    const float us = each * ((float)steps * t.step + t.rest) + (float)steps * t.wait;
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

constexpr int64_t kFewRows = 16;

template <int WM, int WN, int FM, int FN>
void matmul_tiles(const MxMatmulArgs &a, const MatmulPlan &p, hipStream_t s) {
  const int tm = (int)((a.M + p.bm - 1) / p.bm), tn = (int)((a.N + p.bn - 1) / p.bn);
  k_mx_matmul<WM, WN, FM, FN><<<dim3((unsigned)((int64_t)tm * tn), p.splits), WM * WN * 64, 0, s>>>(
      a, (int)mx_pitch(a.K), tm, tn, p.each);
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

// Threads over the words of a row, the rest of a block of 256 over rows.
struct RowGrid {
  dim3 grid, block;
};
RowGrid row_grid(int64_t rows, int64_t words, int64_t most_rows) {
  const unsigned bx = words > 64 ? 256 : words > 16 ? 64 : 16;
  const int64_t by = 256 / bx, gy = (rows + by - 1) / by;
  return RowGrid{dim3((unsigned)((words + bx - 1) / bx), (unsigned)(gy < most_rows ? gy : most_rows)),
                 dim3(bx, (unsigned)by)};
}

template <int DT, bool STOCH>
void quantize_of(const MxQuantArgs &a, hipStream_t s) {
  const int pitch = (int)mx_pitch(a.cols), pitch_t = (int)mx_pitch(a.rows);
  const dim3 grid((unsigned)(pitch / 4), (unsigned)(pitch_t / 4));
  if (a.codes && a.codes_t) {
    k_mx_both<DT, STOCH, true><<<grid, 256, 0, s>>>(a, pitch, pitch_t);
  } else if (a.codes_t) {
    k_mx_both<DT, STOCH, false><<<grid, 256, 0, s>>>(a, pitch, pitch_t);
  } else {
    MxQuantArgs part = a;  // a grid is at most 65535 blocks high
    const int64_t most = 65535;
    for (int64_t r = 0; r < a.rows; r += most) {
      part.x = static_cast<const char *>(a.x) + r * a.ld * (DT == 0 ? 4 : 2);
      part.codes = a.codes + r * pitch * 16;
      part.scales = a.scales + r * pitch;
      part.rows = a.rows - r < most ? a.rows - r : most;
      part.index_base = a.index_base + (uint32_t)(r * a.cols);
      const RowGrid g = row_grid(part.rows, pitch * 4ll, most);
      k_mx_rows<DT, STOCH><<<g.grid, g.block, 0, s>>>(part, pitch);
    }
  }
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs &a, int dtype, hipStream_t s) {
  if (dtype == 0)
    a.stochastic ? quantize_of<0, true>(a, s) : quantize_of<0, false>(a, s);
  else
    a.stochastic ? quantize_of<1, true>(a, s) : quantize_of<1, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxDequantArgs &a, int out_dtype, hipStream_t s) {
  const int pitch = (int)mx_pitch(a.cols);
  const RowGrid g = row_grid(a.rows, (a.cols + 7) / 8, 65535);
  if (out_dtype == 0)
    k_mx_dequantize<0><<<g.grid, g.block, 0, s>>>(a, pitch);
  else
    k_mx_dequantize<1><<<g.grid, g.block, 0, s>>>(a, pitch);
  return hipGetLastError();
}

bool mx_matmul_packs_rows(int64_t M, int64_t K) {
  return M <= kFewRows && few_lds(M, mx_pitch(K)) <= 49152;
}

size_t mx_matmul_scratch(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewRows) return 0;
  const MatmulPlan p = plan_matmul(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s) {
  const int pitch = (int)mx_pitch(a.K);
  if (a.M <= kFewRows) {
    const unsigned blocks = (unsigned)((a.N + 15) / 16);
    const size_t lds = few_lds(a.M, pitch);
    if (a.a_dtype == 0)
      k_mx_matmul_few<0><<<blocks, kFewWaves * 64, lds, s>>>(a, pitch);
    else if (a.a_dtype == 1)
      k_mx_matmul_few<1><<<blocks, kFewWaves * 64, lds, s>>>(a, pitch);
    else
      k_mx_matmul_few<2><<<blocks, kFewWaves * 64, 0, s>>>(a, pitch);
    return hipGetLastError();
  }
  const MatmulPlan p = plan_matmul(a.M, a.N, a.K);
  if (p.bm == 256)
    matmul_tiles<2, 4, 4, 2>(a, p, s);
  else if (p.bm == 128)
    matmul_tiles<2, 2, 2, 2>(a, p, s);
  else
    matmul_tiles<1, 4, 2, 1>(a, p, s);
  if (p.splits > 1) k_mx_join<<<blocks_of(a.M * a.N), 256, 0, s>>>(a, p.splits);
  return hipGetLastError();
}

}  // namespace gq
