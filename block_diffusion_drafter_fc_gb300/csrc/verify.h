// Sampling and sampled verification (verify.cu), as cache_api.cu launches them.
#pragma once

#include "cache.h"

namespace dflash {

constexpr int kVocabMost = 327680;     // a block of a cluster of 8 holds an eighth of a row in fp32
constexpr int kVerifyRows = 65536;     // rows of logits of one call, and pieces of them

// Rows of logits, f32 or bf16.
struct Logits {
  const char* at;
  int64_t ld;                  // bytes
  int rows, el;
  const float* temperature;    // [rows], null: 1
};

// A piece of a row: z 2^-40 is the sum of 2^(x s - m).  kGreedyPiece: its largest logit is at
// `arg`, m its bits in their order (a target of temperature 0), or not needed (a drafter's);
// kNoPiece: no distribution.
constexpr long long kGreedyPiece = -1, kNoPiece = -2;
struct Piece {
  long long z;
  int m, arg;
};

struct VerifyParams {
  RowView rows;
  int V;
  Logits target, draft;        // draft.at null: tokens drafted with certainty
  const int32_t *parents, *tokens, *draft_row;
  const float *uniform, *noise;
  int64_t noise_ld;            // elements
  Piece* stats;                // [T + draft rows][pieces]
  int pieces, rest;            // (set by launch_verify: pieces of a row, a block's share of a rest)
  int32_t* path;
  int max_path;
  int32_t *n_path, *id_last;
  unsigned* status;
};
cudaError_t launch_verify(VerifyParams p, cudaStream_t st);

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
