// Sampling and sampled verification (verify.cu), as cache_api.cu launches them.
#pragma once

#include "cache.h"

namespace dflash {

constexpr int kVocabMost = 327680;     // a block of a cluster of 8 holds 20 tiles of a row
constexpr int kVerifyRows = 65536;     // rows of logits of one call

// Rows of logits, f32 or bf16.
struct Logits {
  const char* at;
  int64_t ld;                  // bytes
  int rows, el;
  const float* temperature;    // [rows], null: 1
};

// A row's probabilities: p_i = 2^(x_i s - m) / z.  z -1: all on `arg` (a target of temperature 0)
// or not needed (a drafter's); NaN: not a distribution.
struct RowStats {
  double z;
  int m, arg;
};

struct VerifyParams {
  RowView rows;
  int V;
  Logits target, draft;        // draft.at null: tokens drafted with certainty
  const int32_t *parents, *tokens, *draft_row;
  const float *uniform, *noise;
  int64_t noise_ld;            // elements
  RowStats* stats;             // [T + draft rows]
  int32_t* path;
  int max_path;
  int32_t *n_path, *id_last;
  unsigned* status;
};
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t st);

struct SampleParams {
  int T, V, n_rows;
  Logits logits;               // temperature: [T]
  const int32_t* rows;         // null: row t
  const char* noise;
  int64_t noise_ld;            // bytes
  int32_t* tokens;
  unsigned* status;
};
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st);
cudaError_t configure_verify();

}  // namespace dflash
