// Logits of a batch's rows under penalties, biases and masks, and the token
// counts they read (logits.cu).
#pragma once

#include "ts_common.cuh"

namespace ts {

struct LogitsArgs {
  const void* logits;              // n rows of V values, row_stride apart
  int64_t row_stride, out_stride;
  int n, V, n_seq;
  const int32_t* cu_q;             // [n_seq + 1]
  const int32_t *tokens, *parents; // [n] or NULL
  const int32_t *counts, *seen;    // [n_seq, V], [n_seq, words] or NULL
  const float *repetition, *frequency, *presence;   // [n_seq] or NULL
  const int32_t* bias_ids;         // [n_seq, n_bias]
  const float* bias;
  int n_bias;
  const int32_t *mask, *mask_rows; // [n_masks, words], [n] or NULL
  int n_masks;
  float masked_value;
  float* out;
};
// type: 0 fp32, 1 bf16, 2 fp16
int launch_logits(const LogitsArgs& a, int type, int32_t* status, cudaStream_t st);

int launch_token_counts(const int32_t* tokens, const int32_t* lens, int n_seq, int stride, int V,
                        int32_t* counts, int32_t* seen, bool reset, bool prompt, int32_t* status,
                        cudaStream_t st);

}  // namespace ts
