// Launch interface of the sampling kernel (msm_sample.cu), shared with the host side (msm_paged_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "msm.h"

namespace msm {

struct SampleArgs {
  const void* logits;
  int64_t stride;  // elements between rows
  const float *temperature, *top_p, *min_p, *random;
  const int32_t* top_k;
  int32_t *tokens, *kept;
  float* probs;
  int n_rows, vocab;
  int slice, room;  // set by the launch: logits of a block, and 16-byte pieces of them in shared memory
};
constexpr int kSampleVocab = 1 << 20;  // most logits of a row (their weights' sum has 62 bits)
cudaError_t launch_sample(const SampleArgs& p, int dtype, int sms, cudaStream_t s);

}  // namespace msm
