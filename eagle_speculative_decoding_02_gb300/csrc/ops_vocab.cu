// C entry points of the operators on vocabulary rows (eagle_op_token_logprobs,
// eagle_op_distill_*): argument checks, then the launchers of vocab_rows.h.
#include "../../include/eagle.h"
#include "vocab_rows.h"

using namespace eg;

namespace {

int esize(int dtype) {
  return dtype == EAGLE_DTYPE_F32 ? 4 : dtype == EAGLE_DTYPE_BF16 || dtype == EAGLE_DTYPE_F16 ? 2 : 0;
}

// Arrays of 4-byte elements, aligned to them (NULL is).
template <typename... P> bool words_ok(const P*... p) { return (((uintptr_t)p % 4 == 0) && ...); }

// A row-major matrix of `size`-byte elements: aligned to them, rows that do not overlap.
bool matrix_ok(const void* p, int size, int32_t rows, int32_t vocab, int64_t ld) {
  return p && (uintptr_t)p % size == 0 && ld >= vocab && ld <= INT64_MAX / 8 / rows;
}

// The gradient may take the logits' place; otherwise no row of one may reach into a row of the other.
bool apart(const void* z, int64_t ld, const void* dz, int64_t ld_dz, int32_t rows, int32_t vocab, int size) {
  if (z == dz && (ld == ld_dz || rows == 1)) return true;
  const int64_t diff = (intptr_t)dz - (intptr_t)z;  // bytes
  const int64_t row = (int64_t)vocab * size;
  if (diff >= (rows - 1) * ld * size + row || -diff >= (rows - 1) * ld_dz * size + row) return true;
  if (ld != ld_dz) return false;
  const int64_t at = ((diff % (ld * size)) + ld * size) % (ld * size);  // of a gradient row after a row of logits
  return at >= row && ld * size - at >= row;
}

// Whether the gradient's rows leave an array (NULL: none) of `bytes` bytes alone; it may lie between them.
bool clear_of(const void* dz, int64_t ld, int32_t rows, int32_t vocab, int size, const void* p, int64_t bytes) {
  const int64_t at = (intptr_t)p - (intptr_t)dz, pitch = ld * size, row = (int64_t)vocab * size;
  if (!p || at + bytes <= 0) return true;
  const int64_t first = at < row ? 0 : (at - row) / pitch + 1;  // the first row that ends after the array begins
  return first >= rows || first * pitch >= at + bytes;
}

bool grad_ok(int32_t rows, int32_t vocab, int size, const void* z, int64_t ld, const Distill& d) {
  auto clear = [&](const void* p, int64_t each) { return clear_of(d.dz, d.ld_dz, rows, vocab, size, p, rows * each); };
  return d.g && words_ok(d.g, d.stats, d.loss) && matrix_ok(d.dz, size, rows, vocab, d.ld_dz) && apart(z, ld, d.dz, d.ld_dz, rows, vocab, size) &&
         clear(d.t_idx, 4 * d.k) && clear(d.t_lp, 4 * d.k) && clear(d.g, 4) && clear(d.stats, 16) && clear(d.loss, 4);
}

bool rows_ok(int32_t dtype, int32_t rows, int32_t vocab, int64_t ld, const void* z, float temperature) {
  return esize(dtype) && rows >= 0 && vocab >= 1 && temperature >= 1e-6f && temperature <= 1e6f &&
         (rows == 0 || matrix_ok(z, esize(dtype), rows, vocab, ld));
}

bool teacher_ok(int32_t rows, int32_t k, const int32_t* idx, const float* lp, int32_t tail) {
  return k >= 1 && k <= EAGLE_MAX_TEACHER && (tail == 0 || tail == 1) && (rows == 0 || (idx && lp && words_ok(idx, lp)));
}

// What a launch says; nothing is thrown through the C entry points.
template <typename F> eagle_status launched(F f) {
  try {
    return f() == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
  } catch (...) {
    return EAGLE_ERR_CUDA;
  }
}

}  // namespace

static_assert(kMaxAlternatives == EAGLE_MAX_ALTERNATIVES && kMaxTeacher == EAGLE_MAX_TEACHER, "limits");

extern "C" {

eagle_status eagle_op_token_logprobs(int32_t dtype, int32_t rows, int32_t vocab, int64_t ld, const void* d_logits,
                                     const int32_t* d_tokens, float temperature, int32_t k, float* d_logprob,
                                     float* d_entropy, float* d_lse, int32_t* d_idx, float* d_val, void* stream) {
  if (!rows_ok(dtype, rows, vocab, ld, d_logits, temperature) || k < 0 || k > EAGLE_MAX_ALTERNATIVES ||
      !d_tokens != !d_logprob)
    return EAGLE_ERR_INVALID_ARG;
  if (rows == 0) return EAGLE_OK;
  if ((k > 0 && (!d_idx || !d_val)) || !words_ok(d_tokens, d_logprob, d_entropy, d_lse, d_idx, d_val))
    return EAGLE_ERR_INVALID_ARG;
  const VocabRows r{d_logits, dtype, rows, vocab, ld, temperature};
  const TokenLogprobs t{d_tokens, k, d_logprob, d_entropy, d_lse, d_idx, d_val};
  return launched([&] { return token_logprobs(r, t, (cudaStream_t)stream); });
}

eagle_status eagle_op_distill_loss(int32_t dtype, int32_t rows, int32_t vocab, int64_t ld, const void* d_logits,
                                   int32_t k, const int32_t* d_t_idx, const float* d_t_logp, float temperature,
                                   int32_t tail, float* d_loss, float* d_stats, void* stream) {
  if (!rows_ok(dtype, rows, vocab, ld, d_logits, temperature) || !teacher_ok(rows, k, d_t_idx, d_t_logp, tail))
    return EAGLE_ERR_INVALID_ARG;
  if (rows == 0) return EAGLE_OK;
  if (!d_loss || !d_stats || !words_ok(d_loss, d_stats)) return EAGLE_ERR_INVALID_ARG;
  const VocabRows r{d_logits, dtype, rows, vocab, ld, temperature};
  const Distill d{k, d_t_idx, d_t_logp, tail, d_loss, d_stats, nullptr, nullptr, 0};
  return launched([&] { return distill_loss(r, d, (cudaStream_t)stream); });
}

eagle_status eagle_op_distill_grad(int32_t dtype, int32_t rows, int32_t vocab, int64_t ld, const void* d_logits,
                                   int32_t k, const int32_t* d_t_idx, const float* d_t_logp, float temperature,
                                   int32_t tail, const float* d_stats, const float* d_g, int64_t ld_out,
                                   void* d_dlogits, void* stream) {
  if (!rows_ok(dtype, rows, vocab, ld, d_logits, temperature) || !teacher_ok(rows, k, d_t_idx, d_t_logp, tail))
    return EAGLE_ERR_INVALID_ARG;
  if (rows == 0) return EAGLE_OK;
  const VocabRows r{d_logits, dtype, rows, vocab, ld, temperature};
  const Distill d{k, d_t_idx, d_t_logp, tail, nullptr, const_cast<float*>(d_stats), d_g, d_dlogits, ld_out};
  if (!d_stats || !grad_ok(rows, vocab, esize(dtype), d_logits, ld, d)) return EAGLE_ERR_INVALID_ARG;
  return launched([&] { return distill_grad(r, d, (cudaStream_t)stream); });
}

eagle_status eagle_op_distill_loss_grad(int32_t dtype, int32_t rows, int32_t vocab, int64_t ld, const void* d_logits,
                                        int32_t k, const int32_t* d_t_idx, const float* d_t_logp, float temperature,
                                        int32_t tail, const float* d_g, float* d_loss, float* d_stats, int64_t ld_out,
                                        void* d_dlogits, void* stream) {
  if (!rows_ok(dtype, rows, vocab, ld, d_logits, temperature) || !teacher_ok(rows, k, d_t_idx, d_t_logp, tail))
    return EAGLE_ERR_INVALID_ARG;
  if (rows == 0) return EAGLE_OK;
  const VocabRows r{d_logits, dtype, rows, vocab, ld, temperature};
  const Distill d{k, d_t_idx, d_t_logp, tail, d_loss, d_stats, d_g, d_dlogits, ld_out};
  if (!d_loss || (!d_stats && (int64_t)vocab * esize(dtype) > EAGLE_DISTILL_ONE_PASS_BYTES) ||
      !grad_ok(rows, vocab, esize(dtype), d_logits, ld, d))
    return EAGLE_ERR_INVALID_ARG;
  return launched([&] { return distill_loss_grad(r, d, (cudaStream_t)stream); });
}

eagle_status eagle_selftest_vocab_wait(int64_t ns) {
  set_vocab_wait(ns);
  return EAGLE_OK;
}

}  // extern "C"
