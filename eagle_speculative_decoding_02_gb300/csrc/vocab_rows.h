// Host-side launchers of the operators on vocabulary rows (logits [rows][ld],
// the first `vocab` entries of a row count): token log probabilities with
// entropy and alternatives, and distillation from a teacher's top tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace eg {

constexpr int kMaxAlternatives = 64;  // k of token_logprobs
constexpr int kMaxTeacher = 64;       // teacher entries per row

struct VocabRows {
  const void* z;   // logits
  int dtype;       // eagle_dtype of the logits and of their gradient
  int rows, vocab;
  int64_t ld;      // elements from one row to the next
  float temperature;
};

struct TokenLogprobs {
  const int* tok;  // [rows] or NULL
  int k;
  float* logprob;  // [rows], set when tok is
  float* entropy;  // [rows] or NULL
  float* lse;      // [rows] or NULL
  int* idx;        // [rows][k] when k > 0
  float* val;
};

struct Distill {
  int k;
  const int* t_idx;   // [rows][k]
  const float* t_lp;  // [rows][k]
  int tail;           // 1: the teacher's other tokens as one outcome; 0: its k tokens renormalised
  float* loss;        // [rows] (loss passes)
  float* stats;       // [rows][4]: max and log of the sum, of all entries and of the unlisted (see eagle.h)
  const float* g;     // [rows] (gradient passes)
  void* dz;           // [rows][ld_dz]
  int64_t ld_dz;
};

cudaError_t token_logprobs(const VocabRows& r, const TokenLogprobs& t, cudaStream_t s);
cudaError_t distill_loss(const VocabRows& r, const Distill& d, cudaStream_t s);
cudaError_t distill_grad(const VocabRows& r, const Distill& d, cudaStream_t s);
cudaError_t distill_loss_grad(const VocabRows& r, const Distill& d, cudaStream_t s);

// Limit of the kernels' waits in later calls from this host thread, for tests; below 0: 2 s as by default.
void set_vocab_wait(int64_t ns);

}  // namespace eg
