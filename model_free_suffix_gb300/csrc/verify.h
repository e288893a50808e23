// verify.h -- the verification of drafts as its kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sgd {

struct VerifyArgs {
  const void *logits;
  long long stride, rows;
  const int32_t *row_start, *drafts, *num_valid;
  const uint8_t *active;
  int B, V, k;
  const float *temp, *uniform, *noise;
  long long noise_stride;
  const float *q;  // draft probabilities, or null
  long long q_stride;
  int32_t *sampled, *accepted;
  float *logprobs;
  uint32_t *err;
  // workspace (verify_layout)
  float4 *stat;  // [B][k + 1] {m, Z, argmax}
  int *stop;     // [B] first position not accepted; 2^31 - 1 between calls
  int splits, draw_splits;  // CTAs of a position, of a row's draw
};
struct VerifyLayout {
  size_t stat, stop, bytes;
};
VerifyLayout verify_layout(int max_batch, int k);
// dtype: SGD_F32, SGD_F16 or SGD_BF16
cudaError_t launch_verify(const VerifyArgs &a, int dtype, cudaStream_t st);

}  // namespace sgd
