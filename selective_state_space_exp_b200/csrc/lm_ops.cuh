// lm_ops.cuh -- internal declarations of the operators between the layer and
// a language model's tokens: the grouped norm with its activation
// (group_norm.cu), the head's cross entropy (linear_xent.cu) and the products
// with 4-bit weights (linear_w4.cu).  lm_api.cu holds their C entry points.
#pragma once

#include "m3_internal.cuh"

namespace m3 {

// The plans (grid splits, workspace sizes) are made for this many SMs, so that
// sizing a workspace needs no device.
constexpr int kPlanSms = 148;

// Device address of the library's error word (m3_api.cu).
int device_status_word(int** out);

struct NormArgs {
  int64_t batch, seqlen, channels, groups, cg;  // cg = channels / groups
  bool bf16;
  int act;  // M3_ACT_*
  float eps;
  const int32_t* cu_seqlens;  // packed batch, or nullptr
  int64_t total_tokens;       // rows of x
  const void* x;
  const float* w;  // [channels] or nullptr (1)
  const float* b;  // [channels] or nullptr (0)
  const void* z;   // the gate (M3_ACT_GATE)
  void* y;
  float* mean;     // [batch][groups]
  float* rstd;
  // backward
  const void* dy;
  void* dx;
  void* dz;
  float* dw;
  float* db;
  char* ws;
  int* status;
};

size_t group_norm_workspace(const NormArgs& a, bool backward);
cudaError_t group_norm_fwd_launch(const NormArgs& a, cudaStream_t s);
cudaError_t group_norm_bwd_launch(const NormArgs& a, cudaStream_t s);

}  // namespace m3
