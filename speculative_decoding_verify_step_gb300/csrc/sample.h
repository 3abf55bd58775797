// Host-side launcher of the standalone sampler (sample.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace spec {

struct SampleParams {
  const void* logits;        // [rows, V], rows row_stride elements apart
  long long row_stride;
  int rows, V, dtype;        // dtype: spec_dtype
  const float* u;            // [rows]
  float temperature_all;     // where temperature is null
  const float* temperature;  // [settings] or null; row r has setting r / rows_per_setting
  const int32_t* top_k;      // null: off
  const float* top_p;
  const float* min_p;
  int rows_per_setting;
  int32_t* tokens;           // [rows]
  float* probs;              // [rows, V] or null
  int sm_count;              // launch shape only
};
bool sample_temperature_ok(float t);
int sample_max_vocab();
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st);

}  // namespace spec
