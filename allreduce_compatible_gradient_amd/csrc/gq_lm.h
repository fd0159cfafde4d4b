// gq_lm.h -- internal interface of the language-model kernels (gq_mx.hip: microscaled 4-bit
// quantisation and products; gq_vocab.hip: passes over rows of logits) used by gq_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {

// ---------------------------------------------------------------- microscaled 4-bit matrices
constexpr int kMxBlock = 32;            // elements that share a scale
constexpr int64_t kMxMaxDim = 1 << 23;  // rows and columns of a matrix: a tile of 256 rows stays below 2^31 bytes

// Blocks per packed row: the row's blocks rounded up to 8 (256 elements, one K tile of the
// product), so that no K loop has a tail.
inline int64_t mx_pitch(int64_t cols) { return (cols + 255) / 256 * 8; }

struct MxQuantArgs {
  const void *x;
  int64_t rows, cols, ld;
  uint8_t *codes, *scales;      // by rows, or null
  uint8_t *codes_t, *scales_t;  // by columns, or null
  int32_t stochastic;
  uint32_t key_mix;             // key ^ (key >> 16)
  uint32_t index_base;
};

struct MxDequantArgs {
  const uint8_t *codes, *scales;
  int64_t rows, cols, ld;
  void *out;
};

struct MxMatmulArgs {
  const void *a;                // M x K: packed codes, or fp32 / bf16 rows (a_dtype)
  const uint8_t *a_scales;
  const uint8_t *b, *b_scales;  // N x K packed
  const float *bias;            // N, or null
  void *out;                    // M x N, row stride ldo
  float *partial;               // splits x M x N (scratch) where splits > 1
  int64_t M, N, K, lda, ldo;
  int32_t a_dtype;              // 0 fp32, 1 bf16, 2 packed
  int32_t out_dtype;
  int32_t accumulate;
};

hipError_t launch_mx_quantize(const MxQuantArgs &a, int dtype, hipStream_t s);
hipError_t launch_mx_dequantize(const MxDequantArgs &a, int out_dtype, hipStream_t s);
// Whether the product of these sizes quantises fp32 / bf16 rows of A by itself; otherwise the
// caller packs them first.
bool mx_matmul_packs_rows(int64_t M, int64_t K);
// Bytes of scratch for partial products (0: none).
size_t mx_matmul_scratch(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s);

// ---------------------------------------------------------------- rows of logits
constexpr int kVocabTop = 128;            // alternatives of a token, at most
constexpr int64_t kVocabMax = 1 << 30;    // entries of a row
constexpr int64_t kVocabRows = (1 << 24) - 1;  // rows of a call: 256 threads each, of a launch's 2^32 - 1

struct LogprobArgs {
  const void *logits;
  int64_t rows, vocab, ld;
  const int64_t *tokens;
  float inv_t;                // 1 / temperature
  int32_t top;
  float *logprob, *entropy;   // rows
  int32_t *top_ids;           // rows x top
  float *top_logprobs;        // rows x top
  void *scratch;
};

struct DistillArgs {
  const void *logits;
  int64_t rows, vocab, ld;
  const int32_t *top_ids;     // rows x top
  const float *top_logprobs;  // rows x top
  int32_t top;
  float temperature, inv_t;
  int32_t tail;
  const float *weight;        // rows, or null: the gradient's factor of each row
  float *loss;                // rows
  float *stats;               // rows x 4, or null
  void *grad;                 // rows x vocab, row stride ldg, or null
  int64_t ldg;
  void *scratch;
};

size_t logprobs_scratch(int64_t rows, int64_t vocab, int top);
hipError_t launch_token_logprobs(const LogprobArgs &a, int dtype, hipStream_t s);
size_t distill_scratch(int64_t rows, int64_t vocab, int dtype);
hipError_t launch_distill_loss(const DistillArgs &a, int dtype, hipStream_t s);
hipError_t launch_distill_grad(const DistillArgs &a, int dtype, hipStream_t s);

}  // namespace gq
