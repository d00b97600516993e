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

// The kernels of one call follow each other as programmatic dependents: each
// lets the next one start (its blocks set up on SMs that are free), and waits for
// the one before to be complete, and its writes visible, before it touches global
// memory.  Every kernel of a call does both, so the order is that of the stream.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(on));
  return on != 0;
}

// Launches a kernel; dependent: as a programmatic dependent of the kernel before
// it in the stream (one of the same call); cluster: blocks of a cluster along x.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                          bool dependent, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

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
  float* part_w;   // rows of partial sums of dw and db (or dw and db themselves), or nullptr
  float* part_b;
  char* ws;
  int* status;
};

// Whether a grid holds the call's blocks (one or more a sample and tile of channels).
bool group_norm_fits(const NormArgs& a);
size_t group_norm_workspace(const NormArgs& a, bool backward);
cudaError_t group_norm_fwd_launch(const NormArgs& a, cudaStream_t s);
cudaError_t group_norm_bwd_launch(const NormArgs& a, cudaStream_t s);

// Softmax cross entropy of logits = h W^T, never stored: M tokens, V classes,
// width K.
struct XentArgs {
  int64_t M, V, K;
  const void* h;  // [M][K] bf16
  const void* W;  // [V][K] bf16
  const int64_t* targets;
  int64_t ignore;
  float* loss;       // [M] (forward)
  float* lse;        // [M] (written by the forward, read by the backward)
  const float* dloss;  // [M]
  void* dh;          // [M][K] bf16 or nullptr
  void* dW;          // [V][K] bf16 or nullptr
  char* ws;
  int* status;
};
// The backward's depends on which of dh and dW are set.
size_t xent_workspace(const XentArgs& a, bool backward);
cudaError_t xent_fwd_launch(const XentArgs& a, cudaStream_t s);
cudaError_t xent_bwd_launch(const XentArgs& a, cudaStream_t s);

// out = A Wq^T (+ bias) with 4-bit weights: M tokens, N outputs, K inputs.
struct W4Args {
  int64_t M, N, K;
  int group;
  const void* A;          // [M][K] bf16
  const uint8_t* codes;   // [N][K / 2], the even input low
  const void* scales;     // [N][K / group] bf16
  const uint8_t* zeros;   // [N][K / group] or nullptr (8)
  const float* bias;      // [N] or nullptr
  void* out;              // [M][N]
  bool out_f32;
  int* status;
};
cudaError_t w4_launch(const W4Args& a, cudaStream_t s);
cudaError_t w4_quantize_launch(int64_t N, int64_t K, int group, bool bf16, const void* W,
                               uint8_t* codes, void* scales, uint8_t* zeros, cudaStream_t s);

}  // namespace m3
