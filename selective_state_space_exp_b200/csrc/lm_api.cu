// lm_api.cu -- C entry points of the operators between the layer and a language
// model's tokens (declared in include/m3.h): argument checks, workspace sizing
// and dispatch.  Conventions as in m3_api.cu: every argument error is found
// here, before any launch.
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstring>
#include <initializer_list>

#include "lm_ops.cuh"

namespace m3 {
namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
  const void* p;
  size_t n;
};

// Whether the two byte ranges share a byte (an absent one shares none).
bool overlap(const Span& a, const Span& b) {
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
}

// Extents are limited so that every product of them stays far inside int64.
constexpr int64_t kMaxExtent = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 46;

int check_norm(const m3_norm_shape* s) {
  if (!s) return M3_ERR_INVALID_ARGUMENT;
  if (s->batch < 1 || s->seqlen < 0 || s->channels < 1 || s->groups < 1 ||
      s->channels % s->groups != 0)
    return M3_ERR_INVALID_ARGUMENT;
  if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARGUMENT;
  if (s->act != M3_ACT_NONE && s->act != M3_ACT_SILU && s->act != M3_ACT_GATE)
    return M3_ERR_INVALID_ARGUMENT;
  if (!(s->eps >= 0.f) || !(s->eps < 1e30f)) return M3_ERR_INVALID_ARGUMENT;
  if (s->batch >= kMaxExtent || s->seqlen >= kMaxExtent || s->channels >= kMaxExtent ||
      s->batch * s->groups >= kMaxExtent)
    return M3_ERR_UNSUPPORTED;
  if (s->seqlen > 0 && s->batch > kMaxElems / s->seqlen / s->channels) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

NormArgs norm_args(const m3_norm_shape* s) {
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.batch = s->batch;
  a.seqlen = s->seqlen;
  a.channels = s->channels;
  a.groups = s->groups;
  a.cg = s->channels / s->groups;
  a.bf16 = s->io_dtype == M3_BF16;
  a.act = s->act;
  a.eps = s->eps;
  a.total_tokens = s->batch * s->seqlen;
  return a;
}

struct NormIo {
  const void *x, *z, *dy;
  const float *w, *b;
  void *y, *dx, *dz;
  float *mean, *rstd, *dw, *db;
};

int norm_call(const m3_norm_shape* s, const int32_t* cu, int64_t tokens, bool varlen,
              const NormIo& io, bool backward, void* ws, size_t ws_bytes, m3_stream_t stream) {
  int st = check_norm(s);
  if (st != M3_OK) return st;
  if (varlen && (!cu || tokens < 0 || !is_aligned(cu, 4))) return M3_ERR_INVALID_ARGUMENT;
  if (varlen && (tokens >= kMaxExtent || tokens > kMaxElems / s->channels))
    return M3_ERR_UNSUPPORTED;
  NormArgs a = norm_args(s);
  if (varlen) {
    a.cu_seqlens = cu;
    a.total_tokens = tokens;
  }
  const bool empty = a.total_tokens == 0 || s->seqlen == 0;
  const bool gate = s->act == M3_ACT_GATE;
  if (!gate && (io.z || io.dz)) return M3_ERR_INVALID_ARGUMENT;
  if (!empty) {
    if (!io.x || (gate && !io.z)) return M3_ERR_INVALID_ARGUMENT;
    if (backward ? (!io.dy || !io.mean || !io.rstd) : !io.y) return M3_ERR_INVALID_ARGUMENT;
  }
  for (const void* p : {io.x, io.z, io.dy, (const void*)io.y, (const void*)io.dx, (const void*)io.dz})
    if (p && !is_aligned(p, 16)) return M3_ERR_ALIGNMENT;
  for (const void* p : {(const void*)io.w, (const void*)io.b, (const void*)io.mean,
                        (const void*)io.rstd, (const void*)io.dw, (const void*)io.db})
    if (p && !is_aligned(p, 4)) return M3_ERR_ALIGNMENT;
  const size_t nx = (size_t)a.total_tokens * s->channels * (a.bf16 ? 2 : 4);
  const size_t nc = (size_t)s->channels * 4, ns = (size_t)s->batch * s->groups * 4;
  const Span in[] = {{io.x, nx}, {io.z, nx}, {io.dy, nx}, {io.w, nc}, {io.b, nc},
                     {backward ? io.mean : nullptr, ns}, {backward ? io.rstd : nullptr, ns},
                     {cu, varlen ? (size_t)(s->batch + 1) * 4 : 0}};
  const Span out[] = {{io.y, nx}, {io.dx, nx}, {io.dz, nx}, {io.dw, nc}, {io.db, nc},
                      {backward ? nullptr : io.mean, ns}, {backward ? nullptr : io.rstd, ns},
                      {ws, ws_bytes}};
  for (const Span& o : out) {
    const bool is_y = io.y && o.p == io.y;  // may be x or z itself
    for (const Span& i : in)
      if (overlap(o, i) && !(is_y && i.p == o.p && (i.p == io.x || i.p == io.z)))
        return M3_ERR_INVALID_ARGUMENT;
    for (const Span& q : out)
      if (&o != &q && overlap(o, q)) return M3_ERR_INVALID_ARGUMENT;
  }
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (empty) {  // no position: statistics and parameter gradients are zero
    float* const zero[] = {backward ? nullptr : io.mean, backward ? nullptr : io.rstd, io.dw, io.db};
    const size_t n[] = {ns, ns, nc, nc};
    for (int i = 0; i < 4; ++i)
      if (zero[i] && cudaMemsetAsync(zero[i], 0, n[i], cs) != cudaSuccess) return M3_ERR_CUDA;
    return M3_OK;
  }
  if (!group_norm_fits(a)) return M3_ERR_UNSUPPORTED;
  const size_t need = group_norm_workspace(a, backward);
  if (need > 0 && (!ws || ws_bytes < need || !is_aligned(ws, 256))) return M3_ERR_WORKSPACE;
  a.x = io.x; a.z = io.z; a.dy = io.dy; a.w = io.w; a.b = io.b;
  a.y = io.y; a.dx = io.dx; a.dz = io.dz; a.mean = io.mean; a.rstd = io.rstd;
  a.dw = io.dw; a.db = io.db;
  a.ws = static_cast<char*>(ws);
  if (device_status_word(&a.status) != M3_OK) return M3_ERR_CUDA;
  const cudaError_t e = backward ? group_norm_bwd_launch(a, cs) : group_norm_fwd_launch(a, cs);
  return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

int check_xent(int64_t M, int64_t V, int64_t K) {
  if (M < 0 || V < 1 || K < 8) return M3_ERR_INVALID_ARGUMENT;
  const int64_t most = kMaxExtent - 256;
  if (K % 8 != 0 || M >= most || V >= most || K >= most) return M3_ERR_UNSUPPORTED;
  if (M > kMaxElems / V || M > kMaxElems / K || V > kMaxElems / K) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

int xent_size(int64_t M, int64_t V, int64_t K, bool backward, bool dh, bool dW, size_t* bytes) {
  int st = check_xent(M, V, K);
  if (st != M3_OK) return st;
  if (!bytes) return M3_ERR_INVALID_ARGUMENT;
  XentArgs a;
  memset(&a, 0, sizeof(a));
  a.M = M; a.V = V; a.K = K;
  a.dh = dh ? bytes : nullptr;  // whether they are set counts
  a.dW = dW ? bytes : nullptr;
  *bytes = xent_workspace(a, backward);
  return M3_OK;
}

int xent_call(XentArgs a, void* ws, size_t ws_bytes, bool backward, m3_stream_t stream) {
  int st = check_xent(a.M, a.V, a.K);
  if (st != M3_OK) return st;
  const int64_t M = a.M, V = a.V, K = a.K;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (!a.h && M > 0) return M3_ERR_INVALID_ARGUMENT;
  if (M > 0 && (!a.W || !a.targets)) return M3_ERR_INVALID_ARGUMENT;
  if (M > 0 && backward && (!a.lse || !a.dloss)) return M3_ERR_INVALID_ARGUMENT;
  for (const void* p : {a.h, a.W, (const void*)a.dh, (const void*)a.dW})
    if (p && !is_aligned(p, 16)) return M3_ERR_ALIGNMENT;
  if (a.targets && !is_aligned(a.targets, 8)) return M3_ERR_ALIGNMENT;
  for (const void* p : {(const void*)a.loss, (const void*)a.lse, (const void*)a.dloss})
    if (p && !is_aligned(p, 4)) return M3_ERR_ALIGNMENT;
  const size_t nh = (size_t)M * K * 2, nw = (size_t)V * K * 2, nt = (size_t)M * 4;
  const Span in[] = {{a.h, nh}, {a.W, nw}, {a.targets, (size_t)M * 8}, {a.dloss, nt},
                     {backward ? a.lse : nullptr, nt}};
  const Span out[] = {{a.loss, nt}, {backward ? nullptr : a.lse, nt}, {a.dh, nh}, {a.dW, nw},
                      {ws, ws_bytes}};
  for (const Span& o : out) {
    for (const Span& i : in)
      if (overlap(o, i)) return M3_ERR_INVALID_ARGUMENT;
    for (const Span& q : out)
      if (&o != &q && overlap(o, q)) return M3_ERR_INVALID_ARGUMENT;
  }
  if (M == 0) {  // no token: the weights' gradient is zero
    if (a.dW && cudaMemsetAsync(a.dW, 0, nw, cs) != cudaSuccess) return M3_ERR_CUDA;
    return M3_OK;
  }
  if (backward ? (!a.dh && !a.dW) : (!a.loss && !a.lse)) return M3_OK;
  const size_t need = xent_workspace(a, backward);
  if (!ws || ws_bytes < need || !is_aligned(ws, 256)) return M3_ERR_WORKSPACE;
  a.ws = static_cast<char*>(ws);
  if (device_status_word(&a.status) != M3_OK) return M3_ERR_CUDA;
  const cudaError_t e = backward ? xent_bwd_launch(a, cs) : xent_fwd_launch(a, cs);
  return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

int check_w4(int64_t M, int64_t N, int64_t K, int32_t group) {
  if (M < 0 || N < 1 || K < 1 || group < 1) return M3_ERR_INVALID_ARGUMENT;
  if (group != 32 && group != 64 && group != 128) return M3_ERR_UNSUPPORTED;
  if (K % group != 0) return M3_ERR_INVALID_ARGUMENT;
  const int64_t most = kMaxExtent / 2;
  if (M >= most || N >= most || K >= most) return M3_ERR_UNSUPPORTED;
  if (N > kMaxElems / K || M > kMaxElems / K || M > kMaxElems / N) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

M3_API int m3_group_norm_workspace_size(const m3_norm_shape* s, int backward, int packed,
                                        size_t* bytes) {
  int st = check_norm(s);
  if (st != M3_OK) return st;
  if (!bytes) return M3_ERR_INVALID_ARGUMENT;
  NormArgs a = norm_args(s);
  const int32_t some = 0;  // which kernels a call takes depends on whether it is packed
  if (packed) a.cu_seqlens = &some;
  if (s->seqlen > 0 && !group_norm_fits(a)) return M3_ERR_UNSUPPORTED;
  *bytes = s->seqlen == 0 ? 0 : group_norm_workspace(a, backward != 0);
  return M3_OK;
}

M3_API int m3_group_norm_fwd(const m3_norm_shape* s, const void* x, const float* weight,
                             const float* bias, const void* z, void* y, float* mean, float* rstd,
                             void* workspace, size_t workspace_bytes, m3_stream_t stream) {
  m3::Range range_("m3_group_norm_fwd");
  const NormIo io{x, z, nullptr, weight, bias, y, nullptr, nullptr, mean, rstd, nullptr, nullptr};
  return norm_call(s, nullptr, 0, false, io, false, workspace, workspace_bytes, stream);
}

M3_API int m3_group_norm_fwd_varlen(const m3_norm_shape* s, const int32_t* cu_seqlens,
                                    int64_t total_tokens, const void* x, const float* weight,
                                    const float* bias, const void* z, void* y, float* mean,
                                    float* rstd, void* workspace, size_t workspace_bytes,
                                    m3_stream_t stream) {
  m3::Range range_("m3_group_norm_fwd_varlen");
  const NormIo io{x, z, nullptr, weight, bias, y, nullptr, nullptr, mean, rstd, nullptr, nullptr};
  return norm_call(s, cu_seqlens, total_tokens, true, io, false, workspace, workspace_bytes,
                   stream);
}

M3_API int m3_group_norm_bwd(const m3_norm_shape* s, const void* x, const float* weight,
                             const float* bias, const void* z, const float* mean,
                             const float* rstd, const void* dy, void* dx, float* dweight,
                             float* dbias, void* dz, void* workspace, size_t workspace_bytes,
                             m3_stream_t stream) {
  m3::Range range_("m3_group_norm_bwd");
  const NormIo io{x, z, dy, weight, bias, nullptr, dx, dz, const_cast<float*>(mean),
                  const_cast<float*>(rstd), dweight, dbias};
  return norm_call(s, nullptr, 0, false, io, true, workspace, workspace_bytes, stream);
}

M3_API int m3_group_norm_bwd_varlen(const m3_norm_shape* s, const int32_t* cu_seqlens,
                                    int64_t total_tokens, const void* x, const float* weight,
                                    const float* bias, const void* z, const float* mean,
                                    const float* rstd, const void* dy, void* dx, float* dweight,
                                    float* dbias, void* dz, void* workspace,
                                    size_t workspace_bytes, m3_stream_t stream) {
  m3::Range range_("m3_group_norm_bwd_varlen");
  const NormIo io{x, z, dy, weight, bias, nullptr, dx, dz, const_cast<float*>(mean),
                  const_cast<float*>(rstd), dweight, dbias};
  return norm_call(s, cu_seqlens, total_tokens, true, io, true, workspace, workspace_bytes,
                   stream);
}

M3_API int m3_linear_xent_fwd_workspace_size(int64_t tokens, int64_t vocab, int64_t width,
                                             size_t* bytes) {
  return xent_size(tokens, vocab, width, false, false, false, bytes);
}

M3_API int m3_linear_xent_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t width,
                                             size_t* bytes) {
  return xent_size(tokens, vocab, width, true, true, true, bytes);
}

M3_API int m3_linear_xent_bwd_workspace_size_for(int64_t tokens, int64_t vocab, int64_t width,
                                                 int want_dh, int want_dW, size_t* bytes) {
  return xent_size(tokens, vocab, width, true, want_dh != 0, want_dW != 0, bytes);
}

M3_API int m3_linear_xent_fwd(int64_t tokens, int64_t vocab, int64_t width, const void* h,
                              const void* W, const int64_t* targets, int64_t ignore_index,
                              float* loss, float* lse, void* workspace, size_t workspace_bytes,
                              m3_stream_t stream) {
  m3::Range range_("m3_linear_xent_fwd");
  XentArgs a;
  memset(&a, 0, sizeof(a));
  a.M = tokens; a.V = vocab; a.K = width;
  a.h = h; a.W = W; a.targets = targets; a.ignore = ignore_index;
  a.loss = loss; a.lse = lse;
  return xent_call(a, workspace, workspace_bytes, false, stream);
}

M3_API int m3_linear_xent_bwd(int64_t tokens, int64_t vocab, int64_t width, const void* h,
                              const void* W, const int64_t* targets, int64_t ignore_index,
                              const float* lse, const float* dloss, void* dh, void* dW,
                              void* workspace, size_t workspace_bytes, m3_stream_t stream) {
  m3::Range range_("m3_linear_xent_bwd");
  XentArgs a;
  memset(&a, 0, sizeof(a));
  a.M = tokens; a.V = vocab; a.K = width;
  a.h = h; a.W = W; a.targets = targets; a.ignore = ignore_index;
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss; a.dh = dh; a.dW = dW;
  return xent_call(a, workspace, workspace_bytes, true, stream);
}

M3_API int m3_linear_w4(int64_t M, int64_t N, int64_t K, int32_t group, const void* A,
                        const uint8_t* codes, const void* scales, const uint8_t* zeros,
                        const float* bias, void* out, int32_t out_dtype, m3_stream_t stream) {
  m3::Range range_("m3_linear_w4");
  int st = check_w4(M, N, K, group);
  if (st != M3_OK) return st;
  if (out_dtype != M3_BF16 && out_dtype != M3_F32) return M3_ERR_INVALID_ARGUMENT;
  if (M == 0) return M3_OK;
  if (!A || !codes || !scales || !out) return M3_ERR_INVALID_ARGUMENT;
  if (!is_aligned(A, 16) || !is_aligned(codes, 16) || !is_aligned(out, 16) ||
      !is_aligned(scales, 16) || !is_aligned(zeros, 16) || !is_aligned(bias, 4))
    return M3_ERR_ALIGNMENT;
  const size_t groups = (size_t)N * (K / group);
  const Span o{out, (size_t)M * N * (out_dtype == M3_F32 ? 4 : 2)};
  for (const Span& i : {Span{A, (size_t)M * K * 2}, Span{codes, (size_t)N * (K / 2)},
                        Span{scales, groups * 2}, Span{zeros, groups}, Span{bias, (size_t)N * 4}})
    if (overlap(o, i)) return M3_ERR_INVALID_ARGUMENT;
  W4Args a;
  a.M = M; a.N = N; a.K = K; a.group = group;
  a.A = A; a.codes = codes; a.scales = scales; a.zeros = zeros; a.bias = bias;
  a.out = out; a.out_f32 = out_dtype == M3_F32;
  if (device_status_word(&a.status) != M3_OK) return M3_ERR_CUDA;
  const cudaError_t e = w4_launch(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

M3_API int m3_w4_quantize(int64_t N, int64_t K, int32_t group, int32_t w_dtype, const void* W,
                          uint8_t* codes, void* scales, uint8_t* zeros, m3_stream_t stream) {
  m3::Range range_("m3_w4_quantize");
  int st = check_w4(1, N, K, group);
  if (st != M3_OK) return st;
  if (w_dtype != M3_BF16 && w_dtype != M3_F32) return M3_ERR_INVALID_ARGUMENT;
  if (!W || !codes || !scales) return M3_ERR_INVALID_ARGUMENT;
  if (!is_aligned(W, 4) || !is_aligned(codes, 16) || !is_aligned(scales, 16) ||
      !is_aligned(zeros, 16))
    return M3_ERR_ALIGNMENT;
  const size_t groups = (size_t)N * (K / group);
  const Span w{W, (size_t)N * K * (w_dtype == M3_F32 ? 4 : 2)};
  const Span out[] = {{codes, (size_t)N * (K / 2)}, {scales, groups * 2}, {zeros, groups}};
  for (const Span& o : out) {
    if (overlap(o, w)) return M3_ERR_INVALID_ARGUMENT;
    for (const Span& q : out)
      if (&o != &q && overlap(o, q)) return M3_ERR_INVALID_ARGUMENT;
  }
  const cudaError_t e = w4_quantize_launch(N, K, group, w_dtype == M3_BF16, W, codes, scales,
                                           zeros, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
