// group_norm.cu -- grouped normalisation with an activation, channels last: the
// norm on the layer's output, before or together with the block's gate.
//
//   over one sample's positions p and one group's channels c (n = S * C / G):
//     mean = sum x / n,   rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//     xh = (x - mean) rstd,   u = xh w + b
//     y = u,  u sigma(u) (SiLU),  or  u z sigma(z) (the gate)
//   backward, from dy:
//     g = dy,  dy sigma(u) (1 + u (1 - sigma(u))),  or  dy z sigma(z)
//     dz = dy u sigma(z) (1 + z (1 - sigma(z)))
//     dw = sum_{samples, p} g xh,   db = sum_{samples, p} g
//     dx = rstd (g w - mean_n(g w) - xh mean_n(g w xh))
//
// All of it is bound by HBM: the floor is one read of each input and one write
// of each output.  Two forms, chosen by what one (sample, group) slice is:
//   unit kernels   one position per sample (every token its own sample): a
//                  slice is C / G contiguous values, held in the registers of
//                  up to 32 lanes, so statistics and result take one read.
//                  A thread keeps its channels over all the rows it visits, so
//                  w, b and the sums for dw, db stay in registers.
//   slice kernels  everything else: partial statistics over splits of a
//                  slice's positions, then a second pass that applies them
//                  (its reads come from L2 where the tensor fits there).
// Statistics are fp32: in the unit kernels the mean first, then the deviations
// from it (whose own mean corrects it) and their squares; in the slice kernels
// per-vector means and deviations merged pairwise (Chan, Golub and LeVeque), so
// a large common offset is not squared.  No atomics: dw and db are partial sums in the workspace, added in
// a fixed order.
#include "lm_ops.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxLaneElems = 32;  // values one lane of a unit kernel may hold

template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = uint16_t; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };

// V elements of the io type as one aligned access.
template <bool BF16, int V>
struct Io {
  static constexpr int ES = BF16 ? 2 : 4;
  using R = typename Raw<V * ES>::T;
  __device__ static R load(const void* p, int64_t i) {
    return *reinterpret_cast<const R*>(static_cast<const char*>(p) + i * ES);
  }
  __device__ static void unpack(const R& r, float (&f)[V]) {
    if constexpr (BF16) {
      const __nv_bfloat16* h = reinterpret_cast<const __nv_bfloat16*>(&r);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = __bfloat162float(h[e]);
    } else {
      const float* h = reinterpret_cast<const float*>(&r);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = h[e];
    }
  }
  __device__ static void store(void* p, int64_t i, const float (&f)[V]) {
    R r;
    if constexpr (BF16) {
      __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(&r);
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = __float2bfloat16_rn(f[e]);
    } else {
      float* h = reinterpret_cast<float*>(&r);
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = f[e];
    }
    *reinterpret_cast<R*>(static_cast<char*>(p) + i * ES) = r;
  }
};

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// 1 / (1 + e^-v) with the quotient's edge cases: __fdividef gives 0 for a
// divisor beyond 2^126, which is sigma's limit there.
__device__ __forceinline__ float activate(int act, float u, float z) {
  if (act == M3_ACT_SILU) return u * sigmoid(u);
  if (act == M3_ACT_GATE) return u * z * sigmoid(z);
  return u;
}

// g = dL/du, and dz for the gate
__device__ __forceinline__ float act_grad(int act, float u, float z, float dy, float& dz) {
  if (act == M3_ACT_SILU) {
    const float s = sigmoid(u);
    return dy * s * fmaf(u, 1.f - s, 1.f);
  }
  if (act == M3_ACT_GATE) {
    const float s = sigmoid(z);
    dz = dy * u * s * fmaf(z, 1.f - s, 1.f);
    return dy * z * s;
  }
  return dy;
}

// ---- unit kernels: one position per sample -----------------------------------
// A block covers `ub` units (groups) of a row with `L` lanes each, and `ty`
// rows at a time; blockIdx.x picks the units, blockIdx.y the rows.

struct UnitPlan {
  int V, L, NV, ub, ty, xb, yb;  // vector elements, lanes, vectors a lane, units, row slots, grid
};

__device__ __forceinline__ float lane_sum(float v, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool BF16, int V, int NV>
__global__ void __launch_bounds__(kThreads) unit_fwd_kernel(const NormArgs a, const UnitPlan p) {
  using X = Io<BF16, V>;
  const int lane = threadIdx.x % p.L, slot = threadIdx.x / p.L;
  const int unit = slot % p.ub, ry = slot / p.ub;
  const int64_t g = (int64_t)blockIdx.x * p.ub + unit;
  const bool mine = ry < p.ty && g < a.groups;
  const int nvec = (int)(a.cg / V);
  float w[NV][V], b[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = k * p.L + lane;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const bool in = mine && v < nvec;
      const int64_t c = g * a.cg + (int64_t)v * V + e;
      w[k][e] = in && a.w ? __ldg(a.w + c) : 1.f;
      b[k][e] = in && a.b ? __ldg(a.b + c) : 0.f;
    }
  }
  const float inv_n = 1.f / (float)a.cg;
  for (int64_t r0 = (int64_t)blockIdx.y * p.ty; r0 < a.batch; r0 += (int64_t)gridDim.y * p.ty) {
    const int64_t row = r0 + ry;
    const bool on = mine && row < a.batch;
    const int64_t base = row * a.channels + g * a.cg;
    float x[NV][V], z[NV][V];
    typename X::R xr[NV], zr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (on && v < nvec) {
        xr[k] = X::load(a.x, base + (int64_t)v * V);
        if (a.act == M3_ACT_GATE) zr[k] = X::load(a.z, base + (int64_t)v * V);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (on && k * p.L + lane < nvec) {
        X::unpack(xr[k], x[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += x[k][e];
      }
    }
    // deviations from the rounded mean; their own mean `off` corrects it
    const float mean0 = lane_sum(sum, p.L) * inv_n;
    float sq = 0.f, dev = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (on && k * p.L + lane < nvec) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[k][e] -= mean0;
          dev += x[k][e];
          sq = fmaf(x[k][e], x[k][e], sq);
        }
      }
    }
    const float off = lane_sum(dev, p.L) * inv_n;
    const float var = fmaf(-off, off, lane_sum(sq, p.L) * inv_n);
    const float mean = mean0 + off, rstd = 1.f / sqrtf(var + a.eps);
    if (!on) continue;
    if (lane == 0 && M3_IN(row * a.groups + g, a.batch * a.groups, a.status)) {
      if (a.mean) a.mean[row * a.groups + g] = mean;
      if (a.rstd) a.rstd[row * a.groups + g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (v >= nvec) continue;
      if (a.act == M3_ACT_GATE) X::unpack(zr[k], z[k]);
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = activate(a.act, fmaf((x[k][e] - off) * rstd, w[k][e], b[k][e]), z[k][e]);
      if (M3_IN(base + (int64_t)v * V + V - 1, a.batch * a.channels, a.status))
        X::store(a.y, base + (int64_t)v * V, o);
    }
  }
}

template <bool BF16, int V, int NV>
__global__ void __launch_bounds__(kThreads) unit_bwd_kernel(const NormArgs a, const UnitPlan p) {
  using X = Io<BF16, V>;
  const int lane = threadIdx.x % p.L, slot = threadIdx.x / p.L;
  const int unit = slot % p.ub, ry = slot / p.ub;
  const int64_t g = (int64_t)blockIdx.x * p.ub + unit;
  const bool mine = ry < p.ty && g < a.groups;
  const int nvec = (int)(a.cg / V);
  float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = k * p.L + lane;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const bool in = mine && v < nvec;
      const int64_t c = g * a.cg + (int64_t)v * V + e;
      w[k][e] = in && a.w ? __ldg(a.w + c) : 1.f;
      b[k][e] = in && a.b ? __ldg(a.b + c) : 0.f;
      dw[k][e] = db[k][e] = 0.f;
    }
  }
  const float inv_n = 1.f / (float)a.cg;
  for (int64_t r0 = (int64_t)blockIdx.y * p.ty; r0 < a.batch; r0 += (int64_t)gridDim.y * p.ty) {
    const int64_t row = r0 + ry;
    const bool on = mine && row < a.batch;
    const int64_t base = row * a.channels + g * a.cg;
    typename X::R xr[NV], yr[NV], zr[NV];
    float mean = 0.f, rstd = 0.f;
    if (on) {
      mean = __ldg(a.mean + row * a.groups + g);
      rstd = __ldg(a.rstd + row * a.groups + g);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (on && v < nvec) {
        xr[k] = X::load(a.x, base + (int64_t)v * V);
        yr[k] = X::load(a.dy, base + (int64_t)v * V);
        if (a.act == M3_ACT_GATE) zr[k] = X::load(a.z, base + (int64_t)v * V);
      }
    }
    float xh[NV][V], gw[NV][V], c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (!(on && v < nvec)) continue;
      float dy[V], z[V], dz[V];
      X::unpack(xr[k], xh[k]);
      X::unpack(yr[k], dy);
      if (a.act == M3_ACT_GATE) X::unpack(zr[k], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[k][e] = (xh[k][e] - mean) * rstd;
        const float u = fmaf(xh[k][e], w[k][e], b[k][e]);
        const float gr = act_grad(a.act, u, z[e], dy[e], dz[e]);
        dw[k][e] = fmaf(gr, xh[k][e], dw[k][e]);
        db[k][e] += gr;
        gw[k][e] = gr * w[k][e];
        c1 += gw[k][e];
        c2 = fmaf(gw[k][e], xh[k][e], c2);
      }
      if (a.act == M3_ACT_GATE && a.dz &&
          M3_IN(base + (int64_t)v * V + V - 1, a.batch * a.channels, a.status))
        X::store(a.dz, base + (int64_t)v * V, dz);
    }
    c1 = lane_sum(c1, p.L) * inv_n;
    c2 = lane_sum(c2, p.L) * inv_n;
    if (!on || !a.dx) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (v >= nvec) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = rstd * (gw[k][e] - c1 - xh[k][e] * c2);
      if (M3_IN(base + (int64_t)v * V + V - 1, a.batch * a.channels, a.status))
        X::store(a.dx, base + (int64_t)v * V, o);
    }
  }
  if (!a.ws) return;
  // the block's sums over its rows: row slots are added in shared memory
  extern __shared__ float s_sum[];  // [ty][ub * cg] twice
  const int width = p.ub * (int)a.cg;
  if (ry < p.ty) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * p.L + lane;
      if (v >= nvec) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int at = ry * width + unit * (int)a.cg + v * V + e;
        s_sum[at] = dw[k][e];
        s_sum[p.ty * width + at] = db[k][e];
      }
    }
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(a.ws);  // [2][gridDim.y][channels]
  for (int i = threadIdx.x; i < width; i += kThreads) {
    const int64_t c = (int64_t)blockIdx.x * width + i;
    if (c >= a.channels) break;
    float tw = 0.f, tb = 0.f;
    for (int r = 0; r < p.ty; ++r) {
      tw += s_sum[r * width + i];
      tb += s_sum[(p.ty + r) * width + i];
    }
    part[(int64_t)blockIdx.y * a.channels + c] = tw;
    part[((int64_t)gridDim.y + blockIdx.y) * a.channels + c] = tb;
  }
}

// ---- slice kernels: any number of positions per sample -----------------------
// blockIdx.x = sample * groups + group, blockIdx.y = split of the positions.
// tx threads along the channels (vectors), ty along the positions.

struct SlicePlan {
  int V, tx, ty, splits;
};

// Positions of sample i in the token dimension (the checks of chain_of).
__device__ __forceinline__ Chain rows_of(const NormArgs& a, int64_t i) {
  if (!a.cu_seqlens) return Chain{i * a.seqlen, a.seqlen};
  const int64_t s0 = __ldg(a.cu_seqlens + i), s1 = __ldg(a.cu_seqlens + i + 1);
  if (s0 >= 0 && s1 >= s0 && s1 <= a.total_tokens && s1 - s0 <= a.seqlen) return Chain{s0, s1 - s0};
  if (a.status) atomicCAS(a.status, 0, (int)M3_ERR_INVALID_ARGUMENT);
  return Chain{0, 0};
}

// A running (count, mean, sum of squared deviations), merged pairwise.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments merge(const Moments& p, const Moments& q) {
  const float n = p.n + q.n;
  if (n == 0.f) return Moments{0.f, 0.f, 0.f};
  const float d = q.mean - p.mean, f = q.n / n;
  return Moments{n, fmaf(d, f, p.mean), p.m2 + q.m2 + d * d * p.n * f};
}
__device__ __forceinline__ Moments shfl_merge(const Moments& m) {
  Moments r = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Moments q{__shfl_xor_sync(0xffffffffu, r.n, o), __shfl_xor_sync(0xffffffffu, r.mean, o),
                    __shfl_xor_sync(0xffffffffu, r.m2, o)};
    // both lanes of a pair merge in the same order, so they agree bit for bit
    r = (threadIdx.x & o) ? merge(q, r) : merge(r, q);
  }
  return r;
}

__device__ __forceinline__ void split_rows(const Chain& c, int splits, int64_t& r0, int64_t& r1) {
  const int64_t per = (c.len + splits - 1) / splits;
  r0 = per * blockIdx.y < c.len ? per * blockIdx.y : c.len;
  r1 = r0 + per < c.len ? r0 + per : c.len;
}

template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads) slice_stats_kernel(const NormArgs a, const SlicePlan p) {
  using X = Io<BF16, V>;
  const int64_t sample = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const Chain ch = rows_of(a, sample);
  int64_t r0, r1;
  split_rows(ch, p.splits, r0, r1);
  const int tx = threadIdx.x % p.tx, ty = threadIdx.x / p.tx;
  const int64_t nvec = a.cg / V;
  Moments m{0.f, 0.f, 0.f};
  if (ty < p.ty) {
    for (int64_t v = tx; v < nvec; v += p.tx) {
      for (int64_t r = r0 + ty; r < r1; r += p.ty) {
        const typename X::R raw = X::load(a.x, (ch.base + r) * a.channels + g * a.cg + v * V);
        float f[V];
        X::unpack(raw, f);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) s += f[e];
        Moments q{(float)V, s * (1.f / V), 0.f};
#pragma unroll
        for (int e = 0; e < V; ++e) q.m2 = fmaf(f[e] - q.mean, f[e] - q.mean, q.m2);
        m = merge(m, q);
      }
    }
  }
  __shared__ Moments s_m[kThreads / 32];
  m = shfl_merge(m);
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = merge(m, s_m[i]);
    Moments* out = reinterpret_cast<Moments*>(a.ws);
    out[(int64_t)blockIdx.x * p.splits + blockIdx.y] = m;
  }
}

template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads) slice_apply_kernel(const NormArgs a, const SlicePlan p) {
  using X = Io<BF16, V>;
  const int64_t sample = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const Chain ch = rows_of(a, sample);
  int64_t r0, r1;
  split_rows(ch, p.splits, r0, r1);
  __shared__ float s_stat[2];
  if (threadIdx.x < 32) {  // the splits' moments, merged in the same order by every block
    const Moments* in = reinterpret_cast<const Moments*>(a.ws) + (int64_t)blockIdx.x * p.splits;
    Moments m{0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < p.splits; i += 32) m = merge(m, in[i]);
    m = shfl_merge(m);
    if (threadIdx.x == 0) {
      const float rstd = m.n > 0.f ? 1.f / sqrtf(m.m2 / m.n + a.eps) : 0.f;
      s_stat[0] = m.mean;
      s_stat[1] = rstd;
      if (blockIdx.y == 0) {
        if (a.mean) a.mean[blockIdx.x] = m.mean;
        if (a.rstd) a.rstd[blockIdx.x] = rstd;
      }
    }
  }
  __syncthreads();
  const float mean = s_stat[0], rstd = s_stat[1];
  const int tx = threadIdx.x % p.tx, ty = threadIdx.x / p.tx;
  const int64_t nvec = a.cg / V;
  if (ty >= p.ty) return;
  for (int64_t v = tx; v < nvec; v += p.tx) {
    float w[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = a.w ? __ldg(a.w + g * a.cg + v * V + e) : 1.f;
      b[e] = a.b ? __ldg(a.b + g * a.cg + v * V + e) : 0.f;
    }
    for (int64_t r = r0 + ty; r < r1; r += p.ty) {
      const int64_t at = (ch.base + r) * a.channels + g * a.cg + v * V;
      float x[V], z[V], o[V];
      X::unpack(X::load(a.x, at), x);
      if (a.act == M3_ACT_GATE) X::unpack(X::load(a.z, at), z);
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = activate(a.act, fmaf((x[e] - mean) * rstd, w[e], b[e]), z[e]);
      if (M3_IN(at + V - 1, a.total_tokens * a.channels, a.status)) X::store(a.y, at, o);
    }
  }
}

// Backward, first pass: the slice's two sums (one partial per split) and the
// block's share of dw, db (one row of partials per sample and split), and dz.
template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads)
slice_sums_kernel(const NormArgs a, const SlicePlan p, float2* csum, float* part) {
  using X = Io<BF16, V>;
  const int64_t sample = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const Chain ch = rows_of(a, sample);
  int64_t r0, r1;
  split_rows(ch, p.splits, r0, r1);
  const int tx = threadIdx.x % p.tx, ty = threadIdx.x / p.tx;
  const int64_t nvec = a.cg / V;
  const float mean = __ldg(a.mean + blockIdx.x), rstd = __ldg(a.rstd + blockIdx.x);
  const int64_t prow = sample * p.splits + blockIdx.y, prows = a.batch * p.splits;
  extern __shared__ float s_col[];  // [2][ty][tx * V]
  float c1 = 0.f, c2 = 0.f;
  for (int64_t v0 = 0; v0 < nvec; v0 += p.tx) {
    const int64_t v = v0 + tx;
    const bool on = ty < p.ty && v < nvec;
    float dw[V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
    if (on) {
      float w[V], b[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = a.w ? __ldg(a.w + g * a.cg + v * V + e) : 1.f;
        b[e] = a.b ? __ldg(a.b + g * a.cg + v * V + e) : 0.f;
      }
      for (int64_t r = r0 + ty; r < r1; r += p.ty) {
        const int64_t at = (ch.base + r) * a.channels + g * a.cg + v * V;
        float x[V], dy[V], z[V], dz[V];
        X::unpack(X::load(a.x, at), x);
        X::unpack(X::load(a.dy, at), dy);
        if (a.act == M3_ACT_GATE) X::unpack(X::load(a.z, at), z);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (x[e] - mean) * rstd;
          const float gr = act_grad(a.act, fmaf(xh, w[e], b[e]), z[e], dy[e], dz[e]);
          dw[e] = fmaf(gr, xh, dw[e]);
          db[e] += gr;
          c1 = fmaf(gr, w[e], c1);
          c2 = fmaf(gr * w[e], xh, c2);
        }
        if (a.act == M3_ACT_GATE && a.dz && M3_IN(at + V - 1, a.total_tokens * a.channels, a.status))
          X::store(a.dz, at, dz);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s_col[(ty * p.tx + tx) * V + e] = dw[e];
        s_col[((p.ty + ty) * p.tx + tx) * V + e] = db[e];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.tx * V; i += kThreads) {
      const int64_t c = v0 * V + i;
      if (c >= a.cg) break;
      float tw = 0.f, tb = 0.f;
      for (int r = 0; r < p.ty; ++r) {
        tw += s_col[r * p.tx * V + i];
        tb += s_col[(p.ty + r) * p.tx * V + i];
      }
      part[prow * a.channels + g * a.cg + c] = tw;
      part[(prows + prow) * a.channels + g * a.cg + c] = tb;
    }
    __syncthreads();
  }
  __shared__ float2 s_c[kThreads / 32];
  c1 = lane_sum(c1, 32);
  c2 = lane_sum(c2, 32);
  if ((threadIdx.x & 31) == 0) s_c[threadIdx.x >> 5] = make_float2(c1, c2);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) {
      c1 += s_c[i].x;
      c2 += s_c[i].y;
    }
    csum[(int64_t)blockIdx.x * p.splits + blockIdx.y] = make_float2(c1, c2);
  }
}

// Backward, second pass: dx.
template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads)
slice_dx_kernel(const NormArgs a, const SlicePlan p, const float2* csum) {
  using X = Io<BF16, V>;
  const int64_t sample = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const Chain ch = rows_of(a, sample);
  int64_t r0, r1;
  split_rows(ch, p.splits, r0, r1);
  __shared__ float2 s_c;
  if (threadIdx.x < 32) {
    float c1 = 0.f, c2 = 0.f;
    for (int i = threadIdx.x; i < p.splits; i += 32) {
      const float2 c = csum[(int64_t)blockIdx.x * p.splits + i];
      c1 += c.x;
      c2 += c.y;
    }
    c1 = lane_sum(c1, 32);
    c2 = lane_sum(c2, 32);
    const float n = (float)((double)ch.len * (double)a.cg);
    if (threadIdx.x == 0) s_c = make_float2(c1 / n, c2 / n);
  }
  __syncthreads();
  const float c1 = s_c.x, c2 = s_c.y;
  const float mean = __ldg(a.mean + blockIdx.x), rstd = __ldg(a.rstd + blockIdx.x);
  const int tx = threadIdx.x % p.tx, ty = threadIdx.x / p.tx;
  const int64_t nvec = a.cg / V;
  if (ty >= p.ty) return;
  for (int64_t v = tx; v < nvec; v += p.tx) {
    float w[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = a.w ? __ldg(a.w + g * a.cg + v * V + e) : 1.f;
      b[e] = a.b ? __ldg(a.b + g * a.cg + v * V + e) : 0.f;
    }
    for (int64_t r = r0 + ty; r < r1; r += p.ty) {
      const int64_t at = (ch.base + r) * a.channels + g * a.cg + v * V;
      float x[V], dy[V], z[V], o[V], dz;
      X::unpack(X::load(a.x, at), x);
      X::unpack(X::load(a.dy, at), dy);
      if (a.act == M3_ACT_GATE) X::unpack(X::load(a.z, at), z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (x[e] - mean) * rstd;
        const float gr = act_grad(a.act, fmaf(xh, w[e], b[e]), z[e], dy[e], dz);
        o[e] = rstd * (gr * w[e] - c1 - xh * c2);
      }
      if (M3_IN(at + V - 1, a.total_tokens * a.channels, a.status)) X::store(a.dx, at, o);
    }
  }
}

// dw, db: the rows of partials added in a fixed order.  32 channels a block.
__global__ void __launch_bounds__(1024)
param_reduce_kernel(const float* part, int64_t rows, int64_t channels, float* dw, float* db) {
  __shared__ float s[2][32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cx;
  float tw = 0.f, tb = 0.f;
  if (c < channels) {
    for (int64_t r = ry; r < rows; r += 32) {
      tw += part[r * channels + c];
      tb += part[(rows + r) * channels + c];
    }
  }
  s[0][ry][cx] = tw;
  s[1][ry][cx] = tb;
  __syncthreads();
  if (ry < 2) {  // warp 0 adds dw's column sums, warp 1 db's
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += s[ry][r][cx];
    float* out = ry == 0 ? dw : db;
    if (out && c < channels) out[c] = t;
  }
}

// ---- plans ---------------------------------------------------------------------

// Widest aligned vector that divides a group's channels (base pointers and rows
// are then aligned to it: rows are whole groups).
int vec_elems(const NormArgs& a) {
  const int es = a.bf16 ? 2 : 4;
  for (int bytes = 16; bytes > es; bytes >>= 1)
    if ((a.cg * es) % bytes == 0) return bytes / es;
  return 1;
}

int round_nv(int64_t n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 16; }

bool unit_plan(const NormArgs& a, bool backward, UnitPlan* p) {
  if (a.seqlen != 1 || a.cu_seqlens) return false;
  p->V = vec_elems(a);
  const int64_t nvec = a.cg / p->V;
  int L = 1;
  while (L < 32 && L < nvec) L <<= 1;
  const int64_t nv = (nvec + L - 1) / L;
  if (nv > 16 || round_nv(nv) * p->V > kMaxLaneElems) return false;
  p->L = L;
  p->NV = round_nv(nv);
  const int slots = kThreads / L;
  p->ub = (int)(a.groups < slots ? a.groups : slots);
  p->ty = slots / p->ub;
  p->xb = (int)((a.groups + p->ub - 1) / p->ub);
  // rows: enough blocks to fill the SMs; the backward keeps them few, since
  // each leaves a row of partial sums
  const int64_t want = (int64_t)kPlanSms * (backward ? 4 : 8);
  int64_t yb = (want + p->xb - 1) / p->xb;
  const int64_t most = (a.batch + p->ty - 1) / p->ty;
  if (yb > most) yb = most;
  if (yb > 65535) yb = 65535;
  p->yb = (int)(yb < 1 ? 1 : yb);
  return true;
}

SlicePlan slice_plan(const NormArgs& a) {
  SlicePlan p;
  p.V = vec_elems(a);
  const int64_t nvec = a.cg / p.V;
  p.tx = (int)(nvec < kThreads ? nvec : kThreads);
  p.ty = kThreads / p.tx;
  const int64_t slices = a.batch * a.groups;
  int64_t s = ((int64_t)kPlanSms * 8 + slices - 1) / slices;
  const int64_t most = (a.seqlen + 4 * p.ty - 1) / (4 * p.ty);  // at least four rows a thread
  if (s > most) s = most;
  if (s > 1024) s = 1024;
  p.splits = (int)(s < 1 ? 1 : s);
  return p;
}

size_t unit_bwd_bytes(const NormArgs& a, const UnitPlan& p) {
  return (size_t)2 * p.yb * a.channels * 4;
}

size_t slice_csum_bytes(const NormArgs& a, const SlicePlan& p) {
  return align_up((size_t)a.batch * a.groups * p.splits * sizeof(float2), 256);
}

#define M3_NORM_V(KERNEL, V, ...)                                \
  do {                                                           \
    if (a.bf16) {                                                \
      switch (V) {                                               \
        case 8: KERNEL<true, 8> __VA_ARGS__; break;              \
        case 4: KERNEL<true, 4> __VA_ARGS__; break;              \
        case 2: KERNEL<true, 2> __VA_ARGS__; break;              \
        default: KERNEL<true, 1> __VA_ARGS__; break;             \
      }                                                          \
    } else {                                                     \
      switch (V) {                                               \
        case 4: KERNEL<false, 4> __VA_ARGS__; break;             \
        case 2: KERNEL<false, 2> __VA_ARGS__; break;             \
        default: KERNEL<false, 1> __VA_ARGS__; break;            \
      }                                                          \
    }                                                            \
  } while (0)

template <bool BF16, int V, int NV>
cudaError_t unit_launch_nv(const NormArgs& a, const UnitPlan& p, bool backward, cudaStream_t s) {
  const dim3 grid((unsigned)p.xb, (unsigned)p.yb);
  if constexpr (V * NV <= kMaxLaneElems) {
    if (backward) {
      const size_t smem = a.ws ? (size_t)2 * p.ty * p.ub * a.cg * 4 : 0;
      if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(unit_bwd_kernel<BF16, V, NV>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
      }
      unit_bwd_kernel<BF16, V, NV><<<grid, kThreads, smem, s>>>(a, p);
    } else {
      unit_fwd_kernel<BF16, V, NV><<<grid, kThreads, 0, s>>>(a, p);
    }
  }
  return cudaGetLastError();
}

template <bool BF16, int V>
cudaError_t unit_launch_v(const NormArgs& a, const UnitPlan& p, bool backward, cudaStream_t s) {
  switch (p.NV) {
    case 1: return unit_launch_nv<BF16, V, 1>(a, p, backward, s);
    case 2: return unit_launch_nv<BF16, V, 2>(a, p, backward, s);
    case 4: return unit_launch_nv<BF16, V, 4>(a, p, backward, s);
    case 8: return unit_launch_nv<BF16, V, 8>(a, p, backward, s);
    default: return unit_launch_nv<BF16, V, 16>(a, p, backward, s);
  }
}

cudaError_t unit_launch(const NormArgs& a, const UnitPlan& p, bool backward, cudaStream_t s) {
  if (a.bf16) {
    switch (p.V) {
      case 8: return unit_launch_v<true, 8>(a, p, backward, s);
      case 4: return unit_launch_v<true, 4>(a, p, backward, s);
      case 2: return unit_launch_v<true, 2>(a, p, backward, s);
      default: return unit_launch_v<true, 1>(a, p, backward, s);
    }
  }
  switch (p.V) {
    case 4: return unit_launch_v<false, 4>(a, p, backward, s);
    case 2: return unit_launch_v<false, 2>(a, p, backward, s);
    default: return unit_launch_v<false, 1>(a, p, backward, s);
  }
}

}  // namespace

size_t group_norm_workspace(const NormArgs& a, bool backward) {
  UnitPlan u;
  if (unit_plan(a, backward, &u)) return backward ? unit_bwd_bytes(a, u) : 0;
  const SlicePlan p = slice_plan(a);
  const size_t slices = (size_t)a.batch * a.groups * p.splits;
  if (!backward) return slices * sizeof(Moments);
  return slice_csum_bytes(a, p) + (size_t)2 * a.batch * p.splits * a.channels * 4;
}

cudaError_t group_norm_fwd_launch(const NormArgs& a, cudaStream_t s) {
  UnitPlan u;
  if (unit_plan(a, false, &u)) return unit_launch(a, u, false, s);
  const SlicePlan p = slice_plan(a);
  const dim3 grid((unsigned)(a.batch * a.groups), (unsigned)p.splits);
  M3_NORM_V(slice_stats_kernel, p.V, <<<grid, kThreads, 0, s>>>(a, p));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  M3_NORM_V(slice_apply_kernel, p.V, <<<grid, kThreads, 0, s>>>(a, p));
  return cudaGetLastError();
}

cudaError_t group_norm_bwd_launch(const NormArgs& a0, cudaStream_t s) {
  NormArgs a = a0;
  UnitPlan u;
  const bool params = a.dw || a.db;
  if (unit_plan(a, true, &u)) {
    char* ws = a.ws;
    if (!params) a.ws = nullptr;
    cudaError_t e = unit_launch(a, u, true, s);
    if (e != cudaSuccess || !params) return e;
    param_reduce_kernel<<<(unsigned)((a.channels + 31) / 32), 1024, 0, s>>>(
        reinterpret_cast<const float*>(ws), u.yb, a.channels, a.dw, a.db);
    return cudaGetLastError();
  }
  const SlicePlan p = slice_plan(a);
  const dim3 grid((unsigned)(a.batch * a.groups), (unsigned)p.splits);
  float2* csum = reinterpret_cast<float2*>(a.ws);
  float* part = reinterpret_cast<float*>(a.ws + slice_csum_bytes(a, p));
  const size_t smem = (size_t)2 * p.ty * p.tx * p.V * 4;
  M3_NORM_V(slice_sums_kernel, p.V, <<<grid, kThreads, smem, s>>>(a, p, csum, part));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.dx) {
    M3_NORM_V(slice_dx_kernel, p.V, <<<grid, kThreads, 0, s>>>(a, p, csum));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (params) {
    param_reduce_kernel<<<(unsigned)((a.channels + 31) / 32), 1024, 0, s>>>(
        part, a.batch * p.splits, a.channels, a.dw, a.db);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace m3
