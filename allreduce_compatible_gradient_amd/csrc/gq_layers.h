// gq_layers.h -- internal interface of the kernels around a language model's layers (gq_i8.hip:
// 8-bit quantisation by rows and its products; gq_embed.hip: token embeddings; gq_ortho.hip: the
// orthogonalised update) used by gq_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_plans.h"

namespace gq {

// ---------------------------------------------------------------- 8-bit matrices
constexpr int64_t kI8MaxRows = 1 << 23;
constexpr int64_t kI8MaxCols = 1 << 17;  // 2^17 * 127 * 127 < 2^31: a row's sum of products fits

struct I8QuantArgs {
  const void *x;
  int64_t rows, cols, ld;
  int8_t *codes;           // rows x pitch, or null
  float *scales;           // rows
  int8_t *codes_t;         // cols x pitch_t, or null
  float *scales_t;         // cols
  int32_t stochastic;
  uint32_t key_mix;        // key ^ (key >> 16)
  uint32_t index_base;
  uint32_t *tops;          // scratch: parts' largest magnitudes (bits), where codes_t is wanted
};

struct I8MatmulArgs {
  const void *a;           // M x K: codes, or fp32 / bf16 rows (a_dtype)
  const float *a_scales;
  const int8_t *b;         // N x K codes
  const float *b_scales;
  const float *bias;       // N, or null
  void *out;               // M x N, row stride ldo
  int32_t *partial;        // splits x M x N (scratch) where splits > 1
  int64_t M, N, K, lda, ldo;
  int32_t a_dtype;         // 0 fp32, 1 bf16, 3 codes
  int32_t out_dtype;
  int32_t accumulate;
};

size_t i8_quantize_scratch(int64_t rows, int64_t cols, bool by_cols);
hipError_t launch_i8_quantize(const I8QuantArgs &a, int dtype, hipStream_t s);
// Whether the product of these sizes quantises fp32 / bf16 rows of A by itself; otherwise the
// caller packs them first.
bool i8_matmul_packs_rows(int64_t M, int64_t K);
// Bytes of scratch for partial products (0: none).
size_t i8_matmul_scratch(int64_t M, int64_t N, int64_t K);
hipError_t launch_i8_matmul(const I8MatmulArgs &a, hipStream_t s);

// ---------------------------------------------------------------- token embeddings
constexpr int64_t kEmbedMaxTokens = 1 << 24;
constexpr int64_t kEmbedMaxVocab = 1 << 23;
constexpr int64_t kEmbedMaxDim = 1 << 20;

struct EmbedArgs {
  const void *table;      // vocab x dim, row stride ld_table
  const int64_t *ids;     // tokens
  int64_t tokens, vocab, dim, ld_table, ld_out;
  float scale;
  void *out;              // tokens x dim, row stride ld_out
};

struct EmbedGradArgs {
  const void *dout;       // tokens x dim, row stride ld_dout
  const int64_t *ids;     // tokens
  int64_t tokens, vocab, dim, ld_dout, ld_out;
  float scale;
  int32_t accumulate;
  void *out;              // vocab x dim, row stride ld_out
  void *scratch;
};

hipError_t launch_embed(const EmbedArgs &a, int dtype, int out_dtype, hipStream_t s);
size_t embed_grad_scratch(int64_t tokens, int64_t vocab, int64_t dim);
hipError_t launch_embed_grad(const EmbedGradArgs &a, int dtype, int out_dtype, hipStream_t s);

// ---------------------------------------------------------------- orthogonalised update
constexpr int64_t kOrthoMaxDim = 1 << 16;

struct OrthoArgs {
  const void *g;            // batch matrices of rows x cols, row stride ldg, stride_g apart
  int64_t batch, rows, cols, ldg, stride_g;
  int32_t steps;
  float a, b, c;
  void *out;                // bf16, row stride ldo, stride_o apart
  int64_t ldo, stride_o;
  void *scratch;
};

// Matrices that one group of launches takes, and the scratch it needs.
int64_t ortho_group(int64_t batch, int64_t rows, int64_t cols);
size_t ortho_scratch(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_orthogonalise(const OrthoArgs &a, int dtype, hipStream_t s);

}  // namespace gq
