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
//                  some lanes (or warps), so statistics and result take one read.
//                  A thread keeps its channels over all the rows it visits, so
//                  w, b and the sums for dw, db stay in registers.
//   slice kernels  everything else: partial sums over splits of a sample's
//                  positions, joined by a small kernel, then a second pass that
//                  applies them (from HBM again where the batch is larger than
//                  L2: each pass goes over all of it).  Blocks cover whole rows,
//                  so that what runs at one time reads neighbouring memory.
//                  (Slices held in the shared memory of clusters, read once,
//                  measured slower: 56 against 54 us forward and 169 against 100
//                  us backward at 8 x 2048 x 2048, for the clusters leave SMs
//                  idle between them.)  Short samples: one block makes both passes.
// Measured in bf16: 16384 tokens x 4096 channels, 64 groups, with the gate 77 us
// forward (5.2 TB/s) and 129 us backward (5.2 TB/s, 6 us of it the sums of dw and db);
// 8 sequences x 2048 x 2048, 32 groups, SiLU 44 us forward and 83 us backward (each
// of their four passes at 4.5 to 5 TB/s, two joining launches at about 5 us).
// Statistics are fp32: in the unit kernels the mean first, then the deviations
// from it (whose own mean corrects it) and their squares; in the others sums about a
// reference that follows each thread's mean, joined as counts, means and squared
// deviations (Chan, Golub and LeVeque): neither a large common offset nor an outlier among
// the first values costs the others their squares.  No atomics: dw and db are
// partial sums in the workspace, added in a fixed order.  y, dx and dz are rounded to
// the io type once, at their store.
#include <type_traits>

#include "lm_ops.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 256;
// Values one lane of a unit kernel may hold: its weights, biases and their sums
// are as many registers each.
constexpr int kMaxLaneElems = 16;

template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = uint16_t; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };

// V elements of the io type as one aligned access, held as pairs of fp32 (one
// packed instruction does a pair's arithmetic); with V = 1 the pair's second
// half is 0 and not stored.
template <bool BF16, int V>
struct Io {
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int P = (V + 1) / 2;  // pairs
  using R = typename Raw<V * ES>::T;
  __device__ static R load(const void* p, int64_t i) {
    return *reinterpret_cast<const R*>(static_cast<const char*>(p) + i * ES);
  }
  __device__ static void unpack(const R& r, float2 (&f)[P]) {
    if constexpr (V == 1) {
      f[0].x = BF16 ? __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(&r) << 16)
                    : *reinterpret_cast<const float*>(&r);
      f[0].y = 0.f;
    } else if constexpr (BF16) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
      for (int e = 0; e < P; ++e)
        f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    } else {
      const float* h = reinterpret_cast<const float*>(&r);
#pragma unroll
      for (int e = 0; e < P; ++e) f[e] = make_float2(h[2 * e], h[2 * e + 1]);
    }
  }
  __device__ static void store(void* p, int64_t i, const float2 (&f)[P]) {
    R r;
    if constexpr (V == 1) {
      if constexpr (BF16)
        *reinterpret_cast<__nv_bfloat16*>(&r) = __float2bfloat16_rn(f[0].x);
      else
        *reinterpret_cast<float*>(&r) = f[0].x;
    } else if constexpr (BF16) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
      for (int e = 0; e < P; ++e) w[e] = tc::pack_bf16(f[e].x, f[e].y);
    } else {
      float* h = reinterpret_cast<float*>(&r);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        h[2 * e] = f[e].x;
        h[2 * e + 1] = f[e].y;
      }
    }
    *reinterpret_cast<R*>(static_cast<char*>(p) + i * ES) = r;
  }
};

using tc::ffma2;
using tc::fmul2;
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 / (1 + e^-v) of a pair; beyond the exponential's range the quotient is 0,
// sigma's limit.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = fmul2(v, both(-1.4426950408889634f));
  const float2 d = fadd2(make_float2(tc::ex2(t.x), tc::ex2(t.y)), both(1.f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}

template <int ACT>
__device__ __forceinline__ float2 activate(float2 u, float2 z) {
  if constexpr (ACT == M3_ACT_SILU) return fmul2(u, sigmoid2(u));
  if constexpr (ACT == M3_ACT_GATE) return fmul2(u, fmul2(z, sigmoid2(z)));
  return u;
}

// g = dL/du, and dz for the gate
template <int ACT>
__device__ __forceinline__ float2 act_grad(float2 u, float2 z, float2 dy, float2& dz) {
  if constexpr (ACT == M3_ACT_SILU) {
    const float2 s = sigmoid2(u);
    return fmul2(fmul2(dy, s), ffma2(u, ffma2(s, both(-1.f), both(1.f)), both(1.f)));
  }
  if constexpr (ACT == M3_ACT_GATE) {
    const float2 s = sigmoid2(z), ds = fmul2(dy, s);
    dz = fmul2(fmul2(ds, u), ffma2(z, ffma2(s, both(-1.f), both(1.f)), both(1.f)));
    return fmul2(ds, z);
  }
  return dy;
}

// A group's weights and biases from channel c on (1 and 0 where there are none;
// 0 and 0 in the unused half of V = 1, which keeps it out of every sum).
template <int V>
__device__ __forceinline__ void load_params(const NormArgs& a, int64_t c, bool in,
                                            float2 (&w)[(V + 1) / 2], float2 (&b)[(V + 1) / 2]) {
  float fw[V + 1], fb[V + 1];
  fw[V] = fb[V] = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    fw[e] = in && a.w ? __ldg(a.w + c + e) : 1.f;
    fb[e] = in && a.b ? __ldg(a.b + c + e) : 0.f;
  }
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) {
    w[e] = make_float2(fw[2 * e], fw[2 * e + 1]);
    b[e] = make_float2(fb[2 * e], fb[2 * e + 1]);
  }
}

// x - m of a pair; the unused half of V = 1 stays 0.
template <int V>
__device__ __forceinline__ float2 minus(float2 x, float m) {
  const float2 d = fadd2(x, make_float2(-m, -m));
  return V == 1 ? make_float2(d.x, 0.f) : d;
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

// Sums of two values over a unit's lanes.  LANES: their number where it is known
// at compile time, 0 where it is at most 32, -1 where a unit is several warps
// (which add up in shared memory; every thread of the block takes part).
template <int LANES>
__device__ __forceinline__ float2 unit_sum(float2 v, int L, float2* s_red) {
  if constexpr (LANES > 0) {
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1)
      v = fadd2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                               __shfl_xor_sync(0xffffffffu, v.y, o)));
  } else if constexpr (LANES == 0) {
    v = make_float2(lane_sum(v.x, L), lane_sum(v.y, L));
  } else {
    v = make_float2(lane_sum(v.x, 32), lane_sum(v.y, 32));
    const int warp = threadIdx.x >> 5, per = L >> 5, first = warp / per * per;
    if ((threadIdx.x & 31) == 0) s_red[warp] = v;
    __syncthreads();
    v = s_red[first];
    for (int i = 1; i < per; ++i) v = fadd2(v, s_red[first + i]);
    __syncthreads();
  }
  return v;
}

// What a thread of the unit kernels walks over: its vectors of the rows ry, ry +
// step, ... of a column of units.
struct Walk {
  int lane, unit, ry, rows;  // rows: how many it has
  int64_t first, step;       // elements: its first vector of its first row, and a row on
  int64_t stat, sstep;       // the same in [samples][groups]
  int64_t col;               // first channel of its first vector
  bool any;                  // whether it has a unit
};
__device__ __forceinline__ Walk walk_of(const NormArgs& a, const UnitPlan& p, int L, int V) {
  Walk o;
  o.lane = threadIdx.x % L;
  const int slot = threadIdx.x / L;
  o.unit = slot % p.ub;
  o.ry = slot / p.ub;
  const int64_t g = (int64_t)blockIdx.x * p.ub + o.unit;
  const int64_t row = (int64_t)blockIdx.y * p.ty + o.ry, step = (int64_t)gridDim.y * p.ty;
  o.any = o.ry < p.ty && g < a.groups;
  o.rows = o.any && row < a.batch ? (int)((a.batch - row + step - 1) / step) : 0;
  o.col = g * a.cg + o.lane * V;
  o.first = row * a.channels + o.col;
  o.step = step * a.channels;
  o.stat = row * a.groups + g;
  o.sstep = step * a.groups;
  return o;
}
// Rows that any thread of the block has: all take part in a unit's sums.
__device__ __forceinline__ int most_rows(const NormArgs& a, const UnitPlan& p) {
  const int64_t row = (int64_t)blockIdx.y * p.ty, step = (int64_t)gridDim.y * p.ty;
  return row < a.batch ? (int)((a.batch - row + step - 1) / step) : 0;
}

template <bool BF16, int V, int NV, int LANES, int ACT>
__global__ void __launch_bounds__(kThreads) unit_fwd_kernel(const NormArgs a, const UnitPlan p) {
  let_next_start();
  wait_for_previous();
  using X = Io<BF16, V>;
  using R = typename X::R;
  constexpr int P = X::P;
  __shared__ float2 s_red[kThreads / 32];
  const int L = LANES > 0 ? LANES : p.L;
  const Walk o = walk_of(a, p, L, V);
  const int nvec = (int)(a.cg / V);
  const int gap = L * V * X::ES;  // bytes between a lane's vectors
  float2 w[NV][P], b[NV][P];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    load_params<V>(a, o.col + (int64_t)k * L * V, o.any && k * L + o.lane < nvec, w[k], b[k]);
  const float inv_n = 1.f / (float)a.cg;
  const char* px = static_cast<const char*>(a.x) + o.first * X::ES;
  const char* pz = static_cast<const char*>(a.z) + o.first * X::ES;
  char* py = static_cast<char*>(a.y) + o.first * X::ES;
  const int64_t step = o.step * X::ES;
  int64_t stat = o.stat;
  R xn[NV], zn[NV];  // the next row, on its way while this one is worked on
  auto fetch = [&] {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (k * L + o.lane >= nvec) break;
      xn[k] = *reinterpret_cast<const R*>(px + k * gap);
      if constexpr (ACT == M3_ACT_GATE) zn[k] = *reinterpret_cast<const R*>(pz + k * gap);
    }
    px += step;
    pz += step;
  };
  if (o.rows > 0) fetch();
  const int most = most_rows(a, p);
  for (int r = 0; r < most; ++r) {
    float2 x[NV][P];
    R z0[NV];
    float2 sum = both(0.f);
    const bool on = r < o.rows;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!on || k * L + o.lane >= nvec) break;
      X::unpack(xn[k], x[k]);
      if constexpr (ACT == M3_ACT_GATE) z0[k] = zn[k];
#pragma unroll
      for (int e = 0; e < P; ++e) sum = fadd2(sum, x[k][e]);
    }
    if (r + 1 < o.rows) fetch();
    // deviations from the rounded mean; their own mean `off` corrects it
    const float mean0 = unit_sum<LANES>(make_float2(sum.x + sum.y, 0.f), L, s_red).x * inv_n;
    float2 sq = both(0.f), dev = both(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!on || k * L + o.lane >= nvec) break;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        x[k][e] = minus<V>(x[k][e], mean0);
        dev = fadd2(dev, x[k][e]);
        sq = ffma2(x[k][e], x[k][e], sq);
      }
    }
    const float2 t = unit_sum<LANES>(make_float2(dev.x + dev.y, sq.x + sq.y), L, s_red);
    if (on) {
      const float off = t.x * inv_n;
      const float rstd = rsqrtf(fmaf(-off, off, t.y * inv_n) + a.eps);
      if (o.lane == 0 && M3_IN(stat, a.batch * a.groups, a.status)) {
        if (a.mean) a.mean[stat] = mean0 + off;
        if (a.rstd) a.rstd[stat] = rstd;
      }
      const float2 scale = both(rstd), shift = both(-off * rstd);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k * L + o.lane >= nvec) break;
        float2 z[P], y[P];
        if constexpr (ACT == M3_ACT_GATE) X::unpack(z0[k], z);
#pragma unroll
        for (int e = 0; e < P; ++e)
          y[e] = activate<ACT>(ffma2(ffma2(x[k][e], scale, shift), w[k][e], b[k][e]), z[e]);
        if (M3_IN((py - static_cast<char*>(a.y)) + k * gap + V * X::ES - 1, a.batch * a.channels * X::ES, a.status))
          X::store(py + k * gap, 0, y);
      }
    }
    py += step;
    stat += o.sstep;
  }
}

constexpr int kUnitRows = 2;  // rows whose loads are in flight together
// Rows of a row slot that one block takes alone in the backward: it then leaves dw
// and db themselves (8 x 4096, 64 groups: 8.0 us for 8 rows by one block, against
// 6.1 us by several and a second kernel that adds their sums; 2 rows: 2.7 us).
constexpr int kOneBlockRows = 4;

template <bool BF16, int V, int NV, int LANES, int ACT>
__global__ void __launch_bounds__(kThreads) unit_bwd_kernel(const NormArgs a, const UnitPlan p) {
  let_next_start();
  wait_for_previous();
  using X = Io<BF16, V>;
  constexpr int P = X::P;
  __shared__ float2 s_red[kThreads / 32];
  const int L = LANES > 0 ? LANES : p.L;
  const Walk o = walk_of(a, p, L, V);
  const int nvec = (int)(a.cg / V);
  const int gap = L * V * X::ES;  // bytes between a lane's vectors
  float2 w[NV][P], b[NV][P], dw[NV][P], db[NV][P];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    load_params<V>(a, o.col + (int64_t)k * L * V, o.any && k * L + o.lane < nvec, w[k], b[k]);
#pragma unroll
    for (int e = 0; e < P; ++e) dw[k][e] = db[k][e] = both(0.f);
  }
  const float inv_n = 1.f / (float)a.cg;
  const int64_t step = o.step * X::ES;
  int64_t at = o.first * X::ES, stat = o.stat;
  const char *px = static_cast<const char*>(a.x), *pd = static_cast<const char*>(a.dy),
             *pz = static_cast<const char*>(a.z);
  char *dx = static_cast<char*>(a.dx), *dz = static_cast<char*>(a.dz);
  const int most = most_rows(a, p);
  for (int r = 0; r < most; r += kUnitRows) {
    typename X::R xr[kUnitRows][NV], yr[kUnitRows][NV], zr[kUnitRows][NV];
    float mean[kUnitRows], rstd[kUnitRows];
#pragma unroll
    for (int u = 0; u < kUnitRows; ++u) {
      if (r + u >= o.rows) break;
      mean[u] = __ldg(a.mean + stat + u * o.sstep);
      rstd[u] = __ldg(a.rstd + stat + u * o.sstep);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k * L + o.lane >= nvec) break;
        const int64_t i = at + u * step + k * gap;
        xr[u][k] = *reinterpret_cast<const typename X::R*>(px + i);
        yr[u][k] = *reinterpret_cast<const typename X::R*>(pd + i);
        if constexpr (ACT == M3_ACT_GATE) zr[u][k] = *reinterpret_cast<const typename X::R*>(pz + i);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnitRows; ++u) {
      const bool on = r + u < o.rows;
      float2 xh[NV][P], gw[NV][P], c1 = both(0.f), c2 = both(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!on || k * L + o.lane >= nvec) break;
        float2 dy[P], z[P], d[P];
        X::unpack(xr[u][k], xh[k]);
        X::unpack(yr[u][k], dy);
        if constexpr (ACT == M3_ACT_GATE) X::unpack(zr[u][k], z);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          xh[k][e] = fmul2(minus<V>(xh[k][e], mean[u]), both(rstd[u]));
          const float2 gr = act_grad<ACT>(ffma2(xh[k][e], w[k][e], b[k][e]), z[e], dy[e], d[e]);
          dw[k][e] = ffma2(gr, xh[k][e], dw[k][e]);
          db[k][e] = fadd2(db[k][e], gr);
          gw[k][e] = fmul2(gr, w[k][e]);
          c1 = fadd2(c1, gw[k][e]);
          c2 = ffma2(gw[k][e], xh[k][e], c2);
        }
        if (ACT == M3_ACT_GATE && dz &&
            M3_IN(at + u * step + k * gap + V * X::ES - 1, a.batch * a.channels * X::ES, a.status))
          X::store(dz + at + u * step + k * gap, 0, d);
      }
      const float2 c = unit_sum<LANES>(make_float2(c1.x + c1.y, c2.x + c2.y), L, s_red);
      if (on && dx) {
        const float2 s = both(rstd[u]), k1 = both(-c.x * inv_n * rstd[u]), k2 = both(-c.y * inv_n * rstd[u]);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (k * L + o.lane >= nvec) break;
          float2 d[P];
#pragma unroll
          for (int e = 0; e < P; ++e) d[e] = ffma2(gw[k][e], s, ffma2(xh[k][e], k2, k1));
          if (M3_IN(at + u * step + k * gap + V * X::ES - 1, a.batch * a.channels * X::ES, a.status))
            X::store(dx + at + u * step + k * gap, 0, d);
        }
      }
    }
    at += kUnitRows * step;
    stat += kUnitRows * o.sstep;
  }
  if (!a.part_w && !a.part_b) return;
  // the block's sums over its rows: row slots are added in shared memory
  extern __shared__ float s_sum[];  // [ty][ub * cg] twice
  const int width = p.ub * (int)a.cg;
  if (o.ry < p.ty) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * L + o.lane;
      if (v >= nvec) break;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = o.ry * width + o.unit * (int)a.cg + v * V + e;
        s_sum[i] = (e & 1) ? dw[k][e / 2].y : dw[k][e / 2].x;
        s_sum[p.ty * width + i] = (e & 1) ? db[k][e / 2].y : db[k][e / 2].x;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += kThreads) {
    const int64_t c = (int64_t)blockIdx.x * width + i;
    if (c >= a.channels) break;
    float tw = 0.f, tb = 0.f;
    for (int r = 0; r < p.ty; ++r) {
      tw += s_sum[r * width + i];
      tb += s_sum[(p.ty + r) * width + i];
    }
    const int64_t at = (int64_t)blockIdx.y * a.channels + c;
    if (!M3_IN(at, (int64_t)p.yb * a.channels, a.status)) continue;
    if (a.part_w) a.part_w[at] = tw;
    if (a.part_b) a.part_b[at] = tb;
  }
}

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
  if (p.n == 0.f) return q;  // a quotient of equal counts need not come out as 1
  const float d = q.mean - p.mean, f = __fdividef(q.n, n);
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

// ---- two passes over whole rows -------------------------------------------------
// A block takes some positions of one sample (blockIdx.y = split) and a tile of
// channels: as many whole groups as fit its threads, or a piece of one group
// (blockIdx.x = sample and tile).  tx threads along the channels, one vector
// each, ty along the positions: neighbouring threads read neighbouring memory.

struct SlicePlan {
  int V, tx, ty;
  int gpt;     // groups of a tile
  int pieces;  // tiles of a group, where one does not fit a block
  int tiles;   // of a row
  int splits;
  bool whole;  // a block takes all rows of its sample and makes both passes
};

// Rows whose loads are in flight together; fewer in the backward, where three
// blocks an SM do better than two (both passes 79 us against 85 at 8 x 2048 x 2048).
constexpr int kRowsAhead = 4, kBwdRowsAhead = 2;

// A block makes both passes over all rows of its sample where a thread has at most
// this many: one launch and no partial sums, but fewer blocks.  Forward / backward
// with SiLU, us, this form against splits: 4 x 128 x 2048 in bf16 (8 rows a thread)
// 4.6 / 7.7 against 9.6 / 16.3; 16 x 256 x 2048 (32) 11.8 / 20.8 against 18.9 / 30.7;
// 64 x 256 x 2048 (128) 51.8 / 110 against 45.5 / 88.5.  Between them it depends on the
// blocks: 16 x 512 x 2048 (64, 128 blocks) 20.1 / 45.9 against 23.8 / 47.4, 6 x 160 x 2400
// (54, 48 blocks) 12.0 / 19.5 against 10.4 / 17.1; splits are taken there.  More rows are in
// flight than above, for the blocks are few.
constexpr int kWholeRows = 32;
constexpr int kWholeAhead = 8, kWholeBwdAhead = 4;

__device__ __forceinline__ void split_rows(const Chain& c, int splits, int64_t& r0, int64_t& r1) {
  const int64_t per = ((uint32_t)c.len + (uint32_t)splits - 1) / (uint32_t)splits;
  r0 = per * blockIdx.y < c.len ? per * blockIdx.y : c.len;
  r1 = r0 + per < c.len ? r0 + per : c.len;
}

// Where a thread stands.
struct Place {
  int64_t sample, base, r0, r1, col;  // first row of the sample; its split; its vector's first channel
  int tile, group, piece, tx, ty;     // group: of the tile (gpt: none)
  bool on;
};
__device__ __forceinline__ Place place_of(const NormArgs& a, const SlicePlan& p) {
  Place o;
  o.sample = blockIdx.x / (unsigned)p.tiles;
  o.tile = (int)(blockIdx.x % (unsigned)p.tiles);
  const Chain ch = rows_of(a, o.sample);
  o.base = ch.base;
  split_rows(ch, p.splits, o.r0, o.r1);
  o.tx = threadIdx.x % p.tx;
  o.ty = threadIdx.x / p.tx;
  const int nvec = (int)(a.cg / p.V);
  if (p.pieces > 1) {
    o.group = 0;
    o.piece = o.tile % p.pieces;
    const int v = o.piece * p.tx + o.tx;
    o.col = (int64_t)(o.tile / p.pieces) * a.cg + (int64_t)v * p.V;
    o.on = o.ty < p.ty && v < nvec;
  } else {
    o.group = o.tx / nvec;
    o.piece = 0;
    o.col = (int64_t)o.tile * p.gpt * a.cg + (int64_t)o.tx * p.V;
    o.on = o.ty < p.ty && o.col < a.channels;
  }
  return o;
}
// Group `i` of the tile, among all (a.groups: none).
__device__ __forceinline__ int64_t group_of(const NormArgs& a, const SlicePlan& p, const Place& o, int i) {
  return p.pieces > 1 ? o.tile / p.pieces : (int64_t)o.tile * p.gpt + i;
}

// Place of the block's partial sums of group g among all.
__device__ __forceinline__ int64_t part_of(const NormArgs& a, const SlicePlan& p, const Place& o, int64_t g) {
  return ((o.sample * a.groups + g) * p.splits + blockIdx.y) * p.pieces + o.piece;
}

// Rows of a thread.
__device__ __forceinline__ int rows_of_thread(const SlicePlan& p, const Place& o) {
  return o.r0 + o.ty < o.r1 ? ((int)(o.r1 - o.r0) - o.ty + p.ty - 1) / p.ty : 0;
}

// The rows of a thread, AHEAD at a time: load(u, at) of all of them, use(u, at) of
// each, then pause(rows so far).  at: element of the thread's vector.
template <int AHEAD, typename Load, typename Use, typename Pause>
__device__ __forceinline__ void over_rows(const NormArgs& a, const SlicePlan& p, const Place& o,
                                          Load&& load, Use&& use, Pause&& pause) {
  const int64_t next = p.ty * a.channels;
  int64_t at = (o.base + o.r0 + o.ty) * a.channels + o.col;
  const int rows = rows_of_thread(p, o);
  int left = rows;
  for (; left >= AHEAD; left -= AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(u, at + u * next);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) use(u, at + u * next);
    at += AHEAD * next;
    pause(rows - left + AHEAD);
  }
#pragma unroll
  for (int u = 0; u < AHEAD - 1; ++u)
    if (u < left) load(u, at + u * next);
#pragma unroll
  for (int u = 0; u < AHEAD - 1; ++u)
    if (u < left) use(u, at + u * next);
}
template <int AHEAD, typename Load, typename Use>
__device__ __forceinline__ void over_rows(const NormArgs& a, const SlicePlan& p, const Place& o,
                                          Load&& load, Use&& use) {
  over_rows<AHEAD>(a, p, o, load, use, [](int) {});
}

// Sums over the threads of each group of the tile, a warp a group: f(group, sum).
template <typename F>
__device__ __forceinline__ void tile_sums(const SlicePlan& p, float2 c, float2* s_c, F&& f) {
  s_c[threadIdx.x] = c;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wide = p.tx / p.gpt, count = wide * p.ty;
  for (int i = warp; i < p.gpt; i += kThreads / 32) {
    c = both(0.f);
    if (p.ty == 1) {
      for (int k = lane; k < wide; k += 32) c = fadd2(c, s_c[i * wide + k]);
    } else {
      for (int k = lane; k < count; k += 32) c = fadd2(c, s_c[(k / wide) * p.tx + i * wide + k % wide]);
    }
    c = make_float2(lane_sum(c.x, 32), lane_sum(c.y, 32));
    if (lane == 0) f(i, c);
  }
}

// The moments of the threads of each group of the tile joined, a warp a group: f(group,
// moments).  The means' mean first, then what is left about it: all of it positive.
template <typename F>
__device__ __forceinline__ void tile_moments(const SlicePlan& p, const Moments& m, Moments* s_m, F&& f) {
  s_m[threadIdx.x] = m;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wide = p.tx / p.gpt, count = wide * p.ty;
  for (int i = warp; i < p.gpt; i += kThreads / 32) {
    const Moments* at = s_m + i * wide;
    auto of = [&](int k) -> const Moments& {  // neighbours where a group has all threads, or all of a row
      return p.ty == 1 || p.gpt == 1 ? at[k] : at[(k / wide) * p.tx + k % wide];
    };
    const float first = at->mean;  // that thread has rows if any has
    float n = 0.f, e = 0.f;
    for (int k = lane; k < count; k += 32) {
      const Moments& q = of(k);
      n += q.n;
      e = fmaf(q.n, q.mean - first, e);
    }
    n = lane_sum(n, 32);
    e = lane_sum(e, 32);
    if (n == 0.f) {
      if (lane == 0) f(i, Moments{0.f, 0.f, 0.f});
      continue;
    }
    const float mean = first + __fdividef(e, n);
    e = 0.f;
    float m2 = 0.f;
    for (int k = lane; k < count; k += 32) {
      const Moments& q = of(k);
      const float d = q.mean - mean, nd = q.n * d;
      e += nd;
      m2 += fmaf(nd, d, q.m2);
    }
    e = lane_sum(e, 32);
    m2 = lane_sum(m2, 32);
    const float d = __fdividef(e, n);
    if (lane == 0) f(i, Moments{n, mean + d, fmaf(-d, e, m2)});
  }
}

// The moments of each group of the tile over the block's rows: f(group of the tile,
// group, moments).
//
// A thread sums deviations and their squares about a reference that follows its mean:
// the mean of its first vector, and whenever it has seen as many rows again the mean so
// far.  What a sum then loses is a part of the values' own squares, wherever an outlier
// stands among them: with n values about the old reference and n more, whose means differ
// by 2 d, the squares hold at least 4 n d^2 and the move takes 2 n d^2 off.  Sums about the
// group's first value (one pivot for the block) lost 1e-4 to 1e-3 of rstd where that value
// was 300 deviations out, in an emulation of their order.  Forward in bf16 against them:
// 8 x 2048 x 2048 44.0 us, as before; 16 x 256 x 2048 11.8 against 11.3.
template <bool BF16, int V, int AHEAD, typename F>
__device__ __forceinline__ void stats_pass(const NormArgs& a, const SlicePlan& p, const Place& o, F&& f) {
  using X = Io<BF16, V>;
  const int rows = o.on ? rows_of_thread(p, o) : 0;
  Moments m{0.f, 0.f, 0.f};
  if (rows > 0) {
    float2 s1 = both(0.f), s2 = both(0.f), v[X::P];
    X::unpack(X::load(a.x, (o.base + o.r0 + o.ty) * a.channels + o.col), v);
#pragma unroll
    for (int e = 0; e < X::P; ++e) s1 = fadd2(s1, minus<V>(v[e], v[0].x));
    float ref = fmaf(s1.x + s1.y, 1.f / V, v[0].x);  // of equal values the value itself
    s1 = both(0.f);
    float sq = 0.f;     // s2 of the rows before the last pause: short sums, then their sum
    int moved = AHEAD;  // rows at which the reference moves next
    typename X::R raw[AHEAD];
    over_rows<AHEAD>(a, p, o, [&](int u, int64_t at) { raw[u] = X::load(a.x, at); },
                     [&](int u, int64_t) {
                       X::unpack(raw[u], v);
#pragma unroll
                       for (int e = 0; e < X::P; ++e) {
                         const float2 d = minus<V>(v[e], ref);
                         s1 = fadd2(s1, d);
                         s2 = ffma2(d, d, s2);
                       }
                     },
                     [&](int seen) {
                       sq += s2.x + s2.y;
                       s2 = both(0.f);
                       if (seen != moved) return;
                       moved = 2 * seen;
                       const float n = (float)seen * V, e = s1.x + s1.y;
                       const float to = ref + __fdividef(e, n), d = to - ref;
                       const float left = fmaf(-n, d, e);  // of the sum about the new one
                       sq = fmaf(-d, e + left, sq);
                       s1 = make_float2(left, 0.f);
                       ref = to;
                     });
    const float n = (float)rows * V, e = s1.x + s1.y, d = __fdividef(e, n);
    const float m2 = fmaf(-d, e, sq + (s2.x + s2.y));
    m = Moments{n, ref + d, m2 < 0.f ? 0.f : m2};
  }
  __shared__ Moments s_m[kThreads];
  tile_moments(p, m, s_m, [&](int i, const Moments& t) {
    const int64_t g = group_of(a, p, o, i);
    if (g < a.groups) f(i, g, t);
  });
}

// A slice's mean and 1 / deviation, also for the caller.
__device__ __forceinline__ float2 finish_stats(const NormArgs& a, int64_t slice, const Moments& m) {
  const float rstd = m.n > 0.f ? rsqrtf(m.m2 / m.n + a.eps) : 0.f;
  if (!M3_IN(slice, a.batch * a.groups, a.status)) return make_float2(0.f, 0.f);
  if (a.mean) a.mean[slice] = m.mean;
  if (a.rstd) a.rstd[slice] = rstd;
  return make_float2(m.mean, rstd);
}

template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads, 4) slice_stats_kernel(const NormArgs a, const SlicePlan p) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  Moments* out = reinterpret_cast<Moments*>(a.ws);
  stats_pass<BF16, V, kRowsAhead>(a, p, o, [&](int, int64_t g, const Moments& m) {
    const int64_t at = part_of(a, p, o, g);
    if (M3_IN(at, a.batch * a.groups * p.splits * p.pieces, a.status)) out[at] = m;
  });
}

// A slice's mean and 1 / deviation from its partial moments, a warp each.
__global__ void __launch_bounds__(kThreads)
slice_finish_kernel(const NormArgs a, int parts, int64_t slices, float2* stat) {
  let_next_start();
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= slices) return;
  const Moments* in = reinterpret_cast<const Moments*>(a.ws) + i * parts;
  Moments m{0.f, 0.f, 0.f};
  for (int k = lane; k < parts; k += 32) m = merge(m, in[k]);
  m = shfl_merge(m);
  if (lane == 0) stat[i] = finish_stats(a, i, m);
}

// y of the block's rows, st: the mean and 1 / deviation of the thread's group.
template <bool BF16, int V, int ACT, int AHEAD>
__device__ __forceinline__ void apply_pass(const NormArgs& a, const SlicePlan& p, const Place& o,
                                           const float2 st) {
  using X = Io<BF16, V>;
  const float mean = st.x;
  float2 w[X::P], b[X::P];
  load_params<V>(a, o.col, true, w, b);
#pragma unroll
  for (int e = 0; e < X::P; ++e) w[e] = fmul2(w[e], both(st.y));
  typename X::R xr[AHEAD], zr[AHEAD];
  over_rows<AHEAD>(a, p, o,
            [&](int u, int64_t at) {
              xr[u] = X::load(a.x, at);
              if constexpr (ACT == M3_ACT_GATE) zr[u] = X::load(a.z, at);
            },
            [&](int u, int64_t at) {
              float2 x[X::P], z[X::P], y[X::P];
              X::unpack(xr[u], x);
              if constexpr (ACT == M3_ACT_GATE) X::unpack(zr[u], z);
#pragma unroll
              for (int e = 0; e < X::P; ++e)
                y[e] = activate<ACT>(ffma2(minus<V>(x[e], mean), w[e], b[e]), z[e]);
              if (M3_IN(at + V - 1, a.total_tokens * a.channels, a.status)) X::store(a.y, at, y);
            });
}

template <bool BF16, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4)
slice_apply_kernel(const NormArgs a, const SlicePlan p, const float2* stat) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  if (o.on) apply_pass<BF16, V, ACT, kRowsAhead>(a, p, o, stat[o.sample * a.groups + group_of(a, p, o, o.group)]);
}

// Both passes by one block a tile, for samples of few rows.
template <bool BF16, int V, int ACT>
__global__ void __launch_bounds__(kThreads) whole_fwd_kernel(const NormArgs a, const SlicePlan p) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  __shared__ float2 s_stat[kThreads];
  stats_pass<BF16, V, kWholeAhead>(a, p, o, [&](int i, int64_t g, const Moments& m) {
    s_stat[i] = finish_stats(a, o.sample * a.groups + g, m);
  });
  __syncthreads();
  if (o.on) apply_pass<BF16, V, ACT, kWholeAhead>(a, p, o, s_stat[o.group]);
}

// Backward, first pass: the groups' two sums over the block's rows (f(group of the
// tile, group, sums)), the block's share of dw, db (one row of partials per sample
// and split), and dz.
template <bool BF16, int V, int ACT, int AHEAD, typename F>
__device__ __forceinline__ void sums_pass(const NormArgs& a, const SlicePlan& p, const Place& o, F&& f) {
  using X = Io<BF16, V>;
  float2 c = both(0.f), dw[X::P], db[X::P];
#pragma unroll
  for (int e = 0; e < X::P; ++e) dw[e] = db[e] = both(0.f);
  if (o.on) {
    const int64_t g = o.sample * a.groups + group_of(a, p, o, o.group);
    const float mean = __ldg(a.mean + g), rstd = __ldg(a.rstd + g);
    float2 w[X::P], b[X::P];
    load_params<V>(a, o.col, true, w, b);
    typename X::R xr[AHEAD], yr[AHEAD], zr[AHEAD];
    over_rows<AHEAD>(a, p, o,
              [&](int u, int64_t at) {
                xr[u] = X::load(a.x, at);
                yr[u] = X::load(a.dy, at);
                if constexpr (ACT == M3_ACT_GATE) zr[u] = X::load(a.z, at);
              },
              [&](int u, int64_t at) {
                float2 x[X::P], dy[X::P], z[X::P], dz[X::P];
                X::unpack(xr[u], x);
                X::unpack(yr[u], dy);
                if constexpr (ACT == M3_ACT_GATE) X::unpack(zr[u], z);
#pragma unroll
                for (int e = 0; e < X::P; ++e) {
                  const float2 xh = fmul2(minus<V>(x[e], mean), both(rstd));
                  const float2 gr = act_grad<ACT>(ffma2(xh, w[e], b[e]), z[e], dy[e], dz[e]);
                  dw[e] = ffma2(gr, xh, dw[e]);
                  db[e] = fadd2(db[e], gr);
                }
                if (ACT == M3_ACT_GATE && a.dz &&
                    M3_IN(at + V - 1, a.total_tokens * a.channels, a.status))
                  X::store(a.dz, at, dz);
              });
    // a channel's weight is the same in all its rows
#pragma unroll
    for (int e = 0; e < X::P; ++e) {
      c.x += db[e].x * w[e].x + db[e].y * w[e].y;
      c.y += dw[e].x * w[e].x + dw[e].y * w[e].y;
    }
  }
  __shared__ float2 s_c[kThreads];
  extern __shared__ float s_col[];  // [2][ty][tx * V], for dw and db
  const int width = p.tx * V;
  const bool params = a.part_w || a.part_b;
  if (params && o.ty < p.ty) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s_col[o.ty * width + o.tx * V + e] = (e & 1) ? dw[e / 2].y : dw[e / 2].x;
      s_col[(p.ty + o.ty) * width + o.tx * V + e] = (e & 1) ? db[e / 2].y : db[e / 2].x;
    }
  }
  tile_sums(p, c, s_c, [&](int i, float2 v) {
    const int64_t g = group_of(a, p, o, i);
    if (g < a.groups) f(i, g, v);
  });
  if (!params) return;
  // columns of the tile: the first of its channels, and how many there are
  const int64_t c0 = o.col - (int64_t)o.tx * V;
  const int64_t end = p.pieces > 1 ? (o.tile / p.pieces + 1) * a.cg : a.channels;
  const int64_t prow = o.sample * p.splits + blockIdx.y;
  for (int i = threadIdx.x; i < 2 * width; i += kThreads) {
    const int which = i >= width, j = i - which * width;
    float* part = which ? a.part_b : a.part_w;
    if (!part || c0 + j >= end) continue;
    float v = 0.f;
    for (int r = 0; r < p.ty; ++r) v += s_col[(which * p.ty + r) * width + j];
    if (M3_IN(prow * a.channels + c0 + j, a.batch * p.splits * a.channels, a.status))
      part[prow * a.channels + c0 + j] = v;
  }
}

template <bool BF16, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 3)
slice_sums_kernel(const NormArgs a, const SlicePlan p, float2* csum) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  sums_pass<BF16, V, ACT, kBwdRowsAhead>(a, p, o, [&](int, int64_t g, float2 c) {
    const int64_t at = part_of(a, p, o, g);
    if (M3_IN(at, a.batch * a.groups * p.splits * p.pieces, a.status)) csum[at] = c;
  });
}

// Values of a slice of `rows` positions.
__device__ __forceinline__ float values_of(const NormArgs& a, int64_t rows) {
  return (float)((double)rows * (double)a.cg);
}

// A slice's two means from its partial sums, a warp each.
__global__ void __launch_bounds__(kThreads)
slice_means_kernel(const NormArgs a, int parts, int64_t slices, const float2* csum, float2* means) {
  let_next_start();
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= slices) return;
  float2 c = both(0.f);
  for (int k = lane; k < parts; k += 32) c = fadd2(c, csum[i * parts + k]);
  c = make_float2(lane_sum(c.x, 32), lane_sum(c.y, 32));
  const float n = values_of(a, rows_of(a, i / a.groups).len);
  if (lane == 0) means[i] = make_float2(c.x / n, c.y / n);
}

// Backward, second pass: dx of the block's rows, c: the two means of the thread's group.
template <bool BF16, int V, int ACT, int AHEAD>
__device__ __forceinline__ void dx_pass(const NormArgs& a, const SlicePlan& p, const Place& o,
                                        const float2 c) {
  using X = Io<BF16, V>;
  const int64_t g = o.sample * a.groups + group_of(a, p, o, o.group);
  const float mean = __ldg(a.mean + g), rstd = __ldg(a.rstd + g);
  const float2 k1 = both(-c.x * rstd), k2 = both(-c.y * rstd);
  float2 w[X::P], b[X::P];
  load_params<V>(a, o.col, true, w, b);
  typename X::R xr[AHEAD], yr[AHEAD], zr[AHEAD];
  over_rows<AHEAD>(a, p, o,
            [&](int u, int64_t at) {
              xr[u] = X::load(a.x, at);
              yr[u] = X::load(a.dy, at);
              if constexpr (ACT == M3_ACT_GATE) zr[u] = X::load(a.z, at);
            },
            [&](int u, int64_t at) {
              float2 x[X::P], dy[X::P], z[X::P], dx[X::P], dz;
              X::unpack(xr[u], x);
              X::unpack(yr[u], dy);
              if constexpr (ACT == M3_ACT_GATE) X::unpack(zr[u], z);
#pragma unroll
              for (int e = 0; e < X::P; ++e) {
                const float2 xh = fmul2(minus<V>(x[e], mean), both(rstd));
                const float2 gr = act_grad<ACT>(ffma2(xh, w[e], b[e]), z[e], dy[e], dz);
                dx[e] = ffma2(fmul2(gr, w[e]), both(rstd), ffma2(xh, k2, k1));
              }
              if (M3_IN(at + V - 1, a.total_tokens * a.channels, a.status)) X::store(a.dx, at, dx);
            });
}

template <bool BF16, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 3)
slice_dx_kernel(const NormArgs a, const SlicePlan p, const float2* means) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  if (o.on) dx_pass<BF16, V, ACT, kBwdRowsAhead>(a, p, o, means[o.sample * a.groups + group_of(a, p, o, o.group)]);
}

// Both passes by one block a tile.
template <bool BF16, int V, int ACT>
__global__ void __launch_bounds__(kThreads) whole_bwd_kernel(const NormArgs a, const SlicePlan p) {
  let_next_start();
  wait_for_previous();
  const Place o = place_of(a, p);
  const float n = values_of(a, o.r1);
  __shared__ float2 s_mean[kThreads];
  sums_pass<BF16, V, ACT, kWholeBwdAhead>(a, p, o, [&](int i, int64_t, float2 c) {
    s_mean[i] = make_float2(c.x / n, c.y / n);
  });
  __syncthreads();
  if (o.on && a.dx) dx_pass<BF16, V, ACT, kWholeBwdAhead>(a, p, o, s_mean[o.group]);
}

// dw (blockIdx.y = 0) or db: the rows of partials added in a fixed order, 32
// channels a block.
__global__ void __launch_bounds__(1024)
param_reduce_kernel(const float* part, int rows, int64_t channels, float* dw, float* db) {
  let_next_start();
  wait_for_previous();
  __shared__ float s[32][33];
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cx;
  float t = 0.f;
  if (c < channels) {
    const float* p = part + ((int64_t)blockIdx.y * rows + ry) * channels + c;
#pragma unroll 8
    for (int r = ry; r < rows; r += 32, p += 32 * channels) t += *p;
  }
  s[ry][cx] = t;
  __syncthreads();
  if (ry == 0 && c < channels) {
    t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += s[r][cx];
    out[c] = t;
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
  // up to 32 lanes a vector each, then several vectors a lane, then several warps
  int L = 1;
  while (L < 32 && L < nvec) L <<= 1;
  auto fits = [&](int lanes) {
    const int64_t n = (nvec + lanes - 1) / lanes;
    return n <= 16 && round_nv(n) * p->V <= kMaxLaneElems;
  };
  while (L < kThreads && !fits(L)) L <<= 1;
  if (!fits(L)) return false;
  const int64_t nv = (nvec + L - 1) / L;
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
  // a few rows: by one block, whose sums are dw and db
  if (backward && a.batch <= kOneBlockRows * p->ty) yb = 1;
  const int64_t most = (a.batch + p->ty - 1) / p->ty;
  if (yb > most) yb = most;
  if (yb > 65535) yb = 65535;
  p->yb = (int)(yb < 1 ? 1 : yb);
  return true;
}

int64_t rows_a_thread(const NormArgs& a, const SlicePlan& p) { return (a.seqlen + p.ty - 1) / p.ty; }

SlicePlan slice_plan(const NormArgs& a, bool backward) {
  SlicePlan p;
  p.whole = false;
  p.V = vec_elems(a);
  const int64_t nvec = a.cg / p.V;
  p.pieces = (int)((nvec + kThreads - 1) / kThreads);
  if (p.pieces > 1) {
    p.gpt = 1;
    p.tx = kThreads;
    p.tiles = (int)(a.groups * p.pieces);
  } else {
    const int64_t fit = kThreads / nvec;
    p.tiles = (int)((a.groups + fit - 1) / fit);
    p.gpt = (int)((a.groups + p.tiles - 1) / p.tiles);
    p.tx = (int)(p.gpt * nvec);
    p.tiles = (int)((a.groups + p.gpt - 1) / p.gpt);
  }
  p.ty = kThreads / p.tx;
  const int64_t blocks = a.batch * p.tiles;
  // as many blocks as run at one time (three an SM in the backward, whose threads
  // hold more), so that each has many rows to spread its start and end over
  int64_t s = (int64_t)kPlanSms * (backward ? 3 : 4) / blocks;
  const int64_t most = (a.seqlen + kRowsAhead * p.ty - 1) / (kRowsAhead * p.ty);
  if (s > most) s = most;
  if (s > 1024) s = 1024;
  p.splits = (int)(s < 1 ? 1 : s);
  if (p.pieces > 1) return p;
  // a block for a tile of a whole sample: fewer groups a tile while SMs are idle
  SlicePlan w = p;
  w.splits = 1;
  while (w.gpt > 1 && rows_a_thread(a, w) > kRowsAhead && a.batch * w.tiles * 2 <= kPlanSms) {
    w.gpt = (w.gpt + 1) / 2;
    w.tx = (int)(w.gpt * nvec);
    w.ty = kThreads / w.tx;
    w.tiles = (int)((a.groups + w.gpt - 1) / w.gpt);
  }
  w.whole = true;
  return rows_a_thread(a, w) <= kWholeRows ? w : p;
}

// Rows of partial sums for dw and db; a single row is dw and db themselves.
size_t part_bytes(const NormArgs& a, int64_t rows) {
  return rows > 1 ? (size_t)2 * rows * a.channels * 4 : 0;
}
void set_parts(NormArgs* a, int64_t rows, char* ws) {
  if (!a->dw && !a->db) return;
  a->part_w = rows > 1 ? reinterpret_cast<float*>(ws) : a->dw;
  a->part_b = rows > 1 ? a->part_w + rows * a->channels : a->db;
}

size_t slice_stat_bytes(const NormArgs& a) {
  return align_up((size_t)a.batch * a.groups * sizeof(float2), 256);
}

size_t slice_csum_bytes(const NormArgs& a, const SlicePlan& p) {
  return align_up((size_t)a.batch * a.groups * p.splits * p.pieces * sizeof(float2), 256);
}

// f(bf16, vector elements, activation) as compile-time constants
template <typename F>
cudaError_t with_shape(const NormArgs& a, int V, F&& f) {
  auto act = [&](auto bf16, auto v) {
    switch (a.act) {
      case M3_ACT_SILU: return f(bf16, v, std::integral_constant<int, M3_ACT_SILU>());
      case M3_ACT_GATE: return f(bf16, v, std::integral_constant<int, M3_ACT_GATE>());
      default: return f(bf16, v, std::integral_constant<int, M3_ACT_NONE>());
    }
  };
  if (a.bf16) {
    switch (V) {
      case 8: return act(std::true_type(), std::integral_constant<int, 8>());
      case 4: return act(std::true_type(), std::integral_constant<int, 4>());
      case 2: return act(std::true_type(), std::integral_constant<int, 2>());
      default: return act(std::true_type(), std::integral_constant<int, 1>());
    }
  }
  switch (V) {
    case 4: return act(std::false_type(), std::integral_constant<int, 4>());
    case 2: return act(std::false_type(), std::integral_constant<int, 2>());
    default: return act(std::false_type(), std::integral_constant<int, 1>());
  }
}

// smem: of the backward's sums, 32 KB at most (two of every value that the block's threads hold).
template <typename K, typename... Args>
cudaError_t launch(K kernel, dim3 grid, size_t smem, cudaStream_t s, bool dependent, Args... args) {
  return launch_kernel(kernel, grid, kThreads, smem, s, dependent, 1, args...);
}

// The lanes of a unit are a compile-time number where the vectors are whole
// 16 bytes of 64 or 128 channels (8 or 16 lanes) and where there are 32.
template <bool BF16, int V, int NV, int ACT>
cudaError_t unit_launch_nv(const NormArgs& a, const UnitPlan& p, bool backward, cudaStream_t s) {
  const dim3 grid((unsigned)p.xb, (unsigned)p.yb);
  if constexpr (V * NV > kMaxLaneElems) return cudaErrorInvalidValue;
  else {
    const size_t smem = backward && (a.part_w || a.part_b) ? (size_t)2 * p.ty * p.ub * a.cg * 4 : 0;
    constexpr int wide = V * (BF16 ? 2 : 4) == 16;
    auto go = [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      return backward ? launch(unit_bwd_kernel<BF16, V, NV, L, ACT>, grid, smem, s, false, a, p)
                      : launch(unit_fwd_kernel<BF16, V, NV, L, ACT>, grid, 0, s, false, a, p);
    };
    if (p.L == 32) return go(std::integral_constant<int, 32>());
    if constexpr (V * NV > kMaxLaneElems / 4) {  // more lanes only where fewer would hold too much
      if (p.L > 32) return go(std::integral_constant<int, -1>());
    }
    if constexpr (NV == 1) {
      if constexpr (wide) {
        if (p.L == 8) return go(std::integral_constant<int, 8>());
        if (p.L == 16) return go(std::integral_constant<int, 16>());
      }
      return go(std::integral_constant<int, 0>());
    }
    return cudaErrorInvalidValue;  // several vectors a lane only with 32 lanes
  }
}

cudaError_t unit_launch(const NormArgs& a, const UnitPlan& p, bool backward, cudaStream_t s) {
  return with_shape(a, p.V, [&](auto bf16, auto v, auto act) {
    constexpr bool B = decltype(bf16)::value;
    constexpr int V = decltype(v)::value, A = decltype(act)::value;
    switch (p.NV) {
      case 1: return unit_launch_nv<B, V, 1, A>(a, p, backward, s);
      case 2: return unit_launch_nv<B, V, 2, A>(a, p, backward, s);
      case 4: return unit_launch_nv<B, V, 4, A>(a, p, backward, s);
      case 8: return unit_launch_nv<B, V, 8, A>(a, p, backward, s);
      default: return unit_launch_nv<B, V, 16, A>(a, p, backward, s);
    }
  });
}

cudaError_t param_reduce(const NormArgs& a, int64_t rows, cudaStream_t s) {
  if (rows == 1 || !a.part_w) return cudaSuccess;
  return launch_kernel(param_reduce_kernel, dim3((unsigned)((a.channels + 31) / 32), 2), 1024, 0, s, true, 1,
                       (const float*)a.part_w, (int)rows, a.channels, a.dw, a.db);
}

}  // namespace

size_t group_norm_workspace(const NormArgs& a, bool backward) {
  UnitPlan u;
  if (unit_plan(a, backward, &u)) return backward ? part_bytes(a, u.yb) : 0;
  const SlicePlan p = slice_plan(a, backward);
  if (!backward)
    return p.whole ? 0 : slice_stat_bytes(a) + (size_t)a.batch * a.groups * p.splits * p.pieces * sizeof(Moments);
  return (p.whole ? 0 : slice_stat_bytes(a) + slice_csum_bytes(a, p)) + part_bytes(a, a.batch * p.splits);
}

bool group_norm_fits(const NormArgs& a) {
  if (a.cg <= kThreads) return true;  // no more tiles than groups
  UnitPlan u;
  return unit_plan(a, false, &u) || a.batch * slice_plan(a, false).tiles <= INT32_MAX;
}

cudaError_t group_norm_fwd_launch(const NormArgs& a0, cudaStream_t s) {
  NormArgs a = a0;
  UnitPlan u;
  if (unit_plan(a, false, &u)) return unit_launch(a, u, false, s);
  const SlicePlan p = slice_plan(a, false);
  const dim3 grid((unsigned)(a.batch * p.tiles), (unsigned)p.splits);
  if (p.whole)
    return with_shape(a, p.V, [&](auto bf16, auto v, auto act) {
      return launch(whole_fwd_kernel<decltype(bf16)::value, decltype(v)::value, decltype(act)::value>,
                    grid, 0, s, false, a, p);
    });
  const int64_t slices = a.batch * a.groups;
  float2* stat = reinterpret_cast<float2*>(a.ws);
  a.ws += slice_stat_bytes(a);
  return with_shape(a, p.V, [&](auto bf16, auto v, auto act) {
    constexpr bool B = decltype(bf16)::value;
    constexpr int V = decltype(v)::value, A = decltype(act)::value;
    cudaError_t e = launch(slice_stats_kernel<B, V>, grid, 0, s, false, a, p);
    if (e == cudaSuccess)
      e = launch(slice_finish_kernel, dim3((unsigned)((slices + kThreads / 32 - 1) / (kThreads / 32))), 0, s,
                 true, a, p.splits * p.pieces, slices, stat);
    return e != cudaSuccess ? e : launch(slice_apply_kernel<B, V, A>, grid, 0, s, true, a, p, (const float2*)stat);
  });
}

cudaError_t group_norm_bwd_launch(const NormArgs& a0, cudaStream_t s) {
  NormArgs a = a0;
  UnitPlan u;
  const bool params = a.dw || a.db;
  if (unit_plan(a, true, &u)) {
    set_parts(&a, u.yb, a.ws);
    const cudaError_t e = unit_launch(a, u, true, s);
    return e != cudaSuccess ? e : param_reduce(a, u.yb, s);
  }
  const SlicePlan p = slice_plan(a, true);
  const dim3 grid((unsigned)(a.batch * p.tiles), (unsigned)p.splits);
  const int64_t slices = a.batch * a.groups;
  float2* means = reinterpret_cast<float2*>(a.ws);
  float2* csum = reinterpret_cast<float2*>(a.ws + slice_stat_bytes(a));
  set_parts(&a, a.batch * p.splits, p.whole ? a.ws : a.ws + slice_stat_bytes(a) + slice_csum_bytes(a, p));
  const size_t smem = params ? (size_t)2 * p.ty * p.tx * p.V * 4 : 0;
  const cudaError_t e = with_shape(a, p.V, [&](auto bf16, auto v, auto act) {
    constexpr bool B = decltype(bf16)::value;
    constexpr int V = decltype(v)::value, A = decltype(act)::value;
    if (p.whole) return launch(whole_bwd_kernel<B, V, A>, grid, smem, s, false, a, p);
    cudaError_t r = launch(slice_sums_kernel<B, V, A>, grid, smem, s, false, a, p, csum);
    if (r != cudaSuccess || !a.dx) return r;
    r = launch(slice_means_kernel, dim3((unsigned)((slices + kThreads / 32 - 1) / (kThreads / 32))), 0, s, true, a,
               p.splits * p.pieces, slices, (const float2*)csum, means);
    return r != cudaSuccess ? r : launch(slice_dx_kernel<B, V, A>, grid, 0, s, true, a, p, (const float2*)means);
  });
  return e != cudaSuccess ? e : param_reduce(a, a.batch * p.splits, s);
}

}  // namespace m3
