// The gated delta rule.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace hyb {

struct DeltaParams {
  float* state;  // [n_slots][Hv][DK][DV]
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* g;     // [n_new][Hv]
  const float* beta;  // [n_new][Hv]
  uint16_t* out;
  const int32_t* cu;     // [B + 1]
  const int32_t* slots;  // [B] or null
  int64_t q_stride, k_stride, v_stride, out_stride;
  int32_t B, n_new, max_new, n_slots, Hk, Hv, DK, DV;
  float scale;
  uint32_t* status;
};

cudaError_t launch_delta_steps(const DeltaParams& p, cudaStream_t s);
cudaError_t launch_delta_chunks(const DeltaParams& p, cudaStream_t s);

}  // namespace hyb
