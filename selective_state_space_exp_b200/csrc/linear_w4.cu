// linear_w4.cu -- products with 4-bit weights and group scales, the projections
// and the head while serving:
//   out[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] (q[n][k] - z[n][g])  (+ bias[n])
// with q in 0..15, z in 0..15 (8 where there are no zero points), s bf16.
//
// Bound by HBM for a few tokens: N K / 2 bytes of codes once.  The weights are
// never scaled before they are multiplied: q - z is a small integer, exact in
// bf16, so a group's sum on the tensor cores (mma m16n8k16, fp32 accumulation)
// loses nothing to rounded weights, and its scale is applied to the fp32 sum.
//
// A warp takes 16 outputs and a range of the inputs in chunks of 128.  The codes
// go straight from global memory to the registers that hold them as the
// product's A operand: which input a fragment's slot stands for is free as long
// as both operands agree, so each lane takes the consecutive inputs of one wide
// load, and the tokens' values are laid out in shared memory in that order once
// per block.  A word of eight codes becomes four bf16 pairs: the codes of a pair
// (e, e + 4) are masked into the low mantissa bits of 128 (0x4300), which makes
// the number 128 + q, and 128 + z is taken off, both exactly.
#include "lm_ops.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

using tc::pack_bf16;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 128;             // inputs a warp takes at a time
constexpr int kXChunk = 4 * 32 * 16;    // bytes of eight tokens' values of one chunk
constexpr int kSmemMost = 200 * 1024;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Input of word w (0..3), code e (0..7) of lane column c (0..3) in a chunk: per
// group a lane has group / 4 consecutive inputs, eight a word.
template <int G>
__device__ __forceinline__ int input_of(int w, int c) {
  constexpr int words = G / 32;  // words of one group in a lane
  return (w / words) * G + c * (G / 4) + (w % words) * 8;
}

// What a lane holds of one chunk: the codes of its two rows, and per group the
// scale and the zero point of each.
template <int G>
struct Chunk {
  static constexpr int NG = kChunk / G;
  uint32_t q[2][4];
  float s[2][NG];
  uint32_t z[2][NG];  // 128 + z, twice
};

template <int G, bool ZEROS>
__device__ __forceinline__ void load_chunk(const W4Args& a, int64_t row0, int64_t k0, int lane,
                                           Chunk<G>& o) {
  constexpr int NG = Chunk<G>::NG;
  const int c = lane & 3;
  const int64_t kg = a.K / G;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = row0 + (lane >> 2) + 8 * h;
    const bool on = row < a.N;
    const uint8_t* p = a.codes + row * (a.K >> 1) + (k0 >> 1);
#pragma unroll
    for (int w = 0; w < 4; ++w) o.q[h][w] = 0;
#pragma unroll
    for (int i = 0; i < NG; ++i) {  // a group is whole or absent: K is a multiple of it
      const bool in = on && k0 + i * G < a.K;
      o.s[h][i] = 0.f;
      uint32_t z = 8;
      if (in) {
        const uint8_t* g = p + i * (G / 2) + c * (G / 8);
        if constexpr (G == 128) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(g));
          o.q[h][0] = v.x; o.q[h][1] = v.y; o.q[h][2] = v.z; o.q[h][3] = v.w;
        } else if constexpr (G == 64) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(g));
          o.q[h][2 * i] = v.x; o.q[h][2 * i + 1] = v.y;
        } else {
          o.q[h][i] = __ldg(reinterpret_cast<const uint32_t*>(g));
        }
        const int64_t at = row * kg + k0 / G + i;
        o.s[h][i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.scales)[at]);
        if constexpr (ZEROS) z = __ldg(a.zeros + at) & 15u;
      }
      o.z[h][i] = 0x43004300u + z * 0x00010001u;
    }
  }
}

// One chunk's products, group by group, added to acc with the groups' scales.
template <int G, int NT>
__device__ __forceinline__ void chunk_products(const Chunk<G>& q, const uint8_t* xs, int xstride,
                                               int lane, float (&acc)[NT][4]) {
  constexpr int words = G / 32;
#pragma unroll
  for (int i = 0; i < Chunk<G>::NG; ++i) {
    float d[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.f;
#pragma unroll
    for (int j = 0; j < words; ++j) {
      const int w = i * words + j;
      uint32_t f[2][4];  // pairs (e, e + 4), e = 0..3, of the two rows
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[h][e] = sub_bf16x2(((q.q[h][w] >> (4 * e)) & 0x000f000fu) | 0x43004300u, q.z[h][i]);
      const uint32_t a0[4] = {f[0][0], f[1][0], f[0][1], f[1][1]};
      const uint32_t a1[4] = {f[0][2], f[1][2], f[0][3], f[1][3]};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 b = *reinterpret_cast<const uint4*>(xs + t * xstride + (w * 32 + lane) * 16);
        mma_bf16(d[t], a0, b.x, b.y);
        mma_bf16(d[t], a1, b.z, b.w);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      acc[t][0] = fmaf(q.s[0][i], d[t][0], acc[t][0]);
      acc[t][1] = fmaf(q.s[0][i], d[t][1], acc[t][1]);
      acc[t][2] = fmaf(q.s[1][i], d[t][2], acc[t][2]);
      acc[t][3] = fmaf(q.s[1][i], d[t][3], acc[t][3]);
    }
  }
}

// The values of chunks [c0, c0 + n) of tokens m0 .. m0 + 8 NT, in fragment order:
// [token tile][chunk][word][lane] of 16 bytes, inputs (0, 4, 1, 5, 2, 6, 3, 7).
template <int G, int NT>
__device__ __forceinline__ void stage_tokens(const W4Args& a, uint8_t* xs, int64_t m0, int64_t c0,
                                             int n) {
  for (int i = threadIdx.x; i < NT * n * 128; i += kThreads) {
    const int lane = i & 31, w = (i >> 5) & 3;
    const int ch = (i >> 7) % n, t = (i >> 7) / n;
    const int64_t m = m0 + t * 8 + (lane >> 2);
    const int64_t k = (c0 + ch) * kChunk + input_of<G>(w, lane & 3);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (m < a.M && k < a.K)
      v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.A) + m * a.K + k));
    uint4 o;  // v holds inputs 01 23 45 67
    o.x = __byte_perm(v.x, v.z, 0x5410);  // 0 4
    o.y = __byte_perm(v.x, v.z, 0x7632);  // 1 5
    o.z = __byte_perm(v.y, v.w, 0x5410);  // 2 6
    o.w = __byte_perm(v.y, v.w, 0x7632);  // 3 7
    *reinterpret_cast<uint4*>(xs + (size_t)t * n * kXChunk + (size_t)ch * kXChunk +
                              (w * 32 + lane) * 16) = o;
  }
}

struct W4Plan {
  int slice;    // chunks of the inputs held in shared memory at a time
  int slices;
  int ks;       // warps that share 16 outputs, each with a part of a slice
};

template <int G, bool ZEROS, int NT>
__global__ void __launch_bounds__(kThreads, 2) w4_kernel(const W4Args a, const W4Plan p) {
  extern __shared__ __align__(16) uint8_t sm[];
  uint8_t* xs = sm;
  float* red = reinterpret_cast<float*>(sm + (size_t)NT * p.slice * kXChunk);  // [warp][16][8 NT]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t m0 = (int64_t)blockIdx.y * 8 * NT;
  const int sets = kWarps / p.ks;  // 16-output blocks a block works on at a time
  const int set = warp / p.ks, part = warp % p.ks;
  const int64_t blocks = (a.N + 15) / 16;
  bool staged = false;
  for (int64_t b0 = (int64_t)blockIdx.x * sets; b0 < blocks; b0 += (int64_t)gridDim.x * sets) {
    const int64_t row0 = (b0 + set) * 16;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
    for (int sl = 0; sl < p.slices; ++sl) {
      const int64_t c0 = (int64_t)sl * p.slice;
      const int n = (int)(chunks - c0 < p.slice ? chunks - c0 : p.slice);
      if (!staged || p.slices > 1) {
        __syncthreads();
        stage_tokens<G, NT>(a, xs, m0, c0, n);
        __syncthreads();
        staged = true;
      }
      const int per = (n + p.ks - 1) / p.ks;
      const int e0 = part * per < n ? part * per : n, e1 = e0 + per < n ? e0 + per : n;
      if (row0 < a.N && e0 < e1) {
        Chunk<G> cur, nxt;
        load_chunk<G, ZEROS>(a, row0, (c0 + e0) * kChunk, lane, cur);
        for (int e = e0; e < e1; ++e) {
          if (e + 1 < e1) load_chunk<G, ZEROS>(a, row0, (c0 + e + 1) * kChunk, lane, nxt);
          chunk_products<G, NT>(cur, xs + (size_t)e * kXChunk, n * kXChunk, lane, acc);
          cur = nxt;
        }
      }
    }
    // the parts of a set, added in order
    float* mine = red + warp * 128 * NT;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mine[((lane >> 2) + (i >> 1) * 8) + 16 * (t * 8 + (lane & 3) * 2 + (i & 1))] = acc[t][i];
    __syncthreads();
    for (int i = threadIdx.x; i < sets * 128 * NT; i += kThreads) {
      const int st = i / (128 * NT), at = i % (128 * NT);
      const int64_t n = (b0 + st) * 16 + (at & 15), m = m0 + (at >> 4);
      if (n >= a.N || m >= a.M) continue;
      float v = red[st * p.ks * 128 * NT + at];
      for (int k = 1; k < p.ks; ++k) v += red[(st * p.ks + k) * 128 * NT + at];
      if (a.bias) v += __ldg(a.bias + n);
      if (M3_IN(m * a.N + n, a.M * a.N, a.status)) io_store(a.out, m * a.N + n, v, !a.out_f32);
    }
    __syncthreads();
  }
}

template <int G, bool ZEROS, int NT>
cudaError_t launch_nt(const W4Args& a, cudaStream_t s) {
  W4Plan p;
  const int64_t chunks = (a.K + kChunk - 1) / kChunk;
  const int red = kWarps * 128 * NT * 4;
  const int most = (kSmemMost - red) / (NT * kXChunk);
  p.slice = (int)(chunks < most ? chunks : most);
  p.slices = (int)((chunks + p.slice - 1) / p.slice);
  p.ks = kWarps;
  while (p.ks > 1 && p.ks > p.slice) p.ks >>= 1;
  const int smem = NT * p.slice * kXChunk + red;
  auto kern = w4_kernel<G, ZEROS, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0, per = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kThreads, smem);
  if (e != cudaSuccess) return e;
  const int64_t work = ((a.N + 15) / 16 + kWarps / p.ks - 1) / (kWarps / p.ks);
  const int64_t most_blocks = (int64_t)sms * (per < 1 ? 1 : per);
  const dim3 grid((unsigned)(work < most_blocks ? work : most_blocks),
                  (unsigned)((a.M + 8 * NT - 1) / (8 * NT)));
  kern<<<grid, kThreads, smem, s>>>(a, p);
  return cudaGetLastError();
}

template <int G, bool ZEROS>
cudaError_t launch_z(const W4Args& a, cudaStream_t s) {
  if (a.M <= 8) return launch_nt<G, ZEROS, 1>(a, s);
  if (a.M <= 16) return launch_nt<G, ZEROS, 2>(a, s);
  return launch_nt<G, ZEROS, 4>(a, s);
}

template <int G>
cudaError_t launch_g(const W4Args& a, cudaStream_t s) {
  return a.zeros ? launch_z<G, true>(a, s) : launch_z<G, false>(a, s);
}

// One warp per group: round to nearest, scale and zero point of the group's
// range.  The scale is rounded to bf16 first and the codes use the rounded one.
template <bool BF16>
__global__ void __launch_bounds__(256)
w4_quantize_kernel(int64_t N, int64_t K, int G, const void* W, uint8_t* codes,
                   __nv_bfloat16* scales, uint8_t* zeros) {
  const int lane = threadIdx.x & 31;
  const int64_t kg = K / G, groups = N * kg;
  for (int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); g < groups;
       g += (int64_t)gridDim.x * 8) {
    const int64_t base = g * G;  // a row is a whole number of groups
    float lo = 0.f, hi = 0.f;
    for (int i = lane; i < G; i += 32) {
      const float v = io_load(W, base + i, BF16);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float range = zeros ? __fdiv_rn(hi, 15.f) - __fdiv_rn(lo, 15.f)
                              : __fdiv_rn(fmaxf(hi, -lo), 7.f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(range);
    const float s = __bfloat162float(sb);
    const float inv_ok = s > 0.f;
    int z = 8;
    if (zeros) {
      z = inv_ok ? (int)rintf(fminf(__fdiv_rn(-lo, s), 15.f)) : 0;
      z = z < 0 ? 0 : z > 15 ? 15 : z;
    }
    for (int i = 2 * lane; i < G; i += 64) {
      uint32_t byte = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = io_load(W, base + i + e, BF16);
        const float q = inv_ok ? rintf(fminf(fmaxf(__fdiv_rn(v, s), -16.f), 16.f)) + (float)z : (float)z;
        const int c = q < 0.f ? 0 : q > 15.f ? 15 : (int)q;
        byte |= (uint32_t)c << (4 * e);
      }
      codes[(base + i) >> 1] = (uint8_t)byte;
    }
    if (lane == 0) {
      scales[g] = sb;
      if (zeros) zeros[g] = (uint8_t)z;
    }
  }
}

}  // namespace

cudaError_t w4_launch(const W4Args& a, cudaStream_t s) {
  switch (a.group) {
    case 32: return launch_g<32>(a, s);
    case 64: return launch_g<64>(a, s);
    default: return launch_g<128>(a, s);
  }
}

cudaError_t w4_quantize_launch(int64_t N, int64_t K, int group, bool bf16, const void* W,
                               uint8_t* codes, void* scales, uint8_t* zeros, cudaStream_t s) {
  const int64_t blocks = (N * (K / group) + 7) / 8;
  const unsigned grid = (unsigned)(blocks < kPlanSms * 16 ? blocks : kPlanSms * 16);
  __nv_bfloat16* sc = static_cast<__nv_bfloat16*>(scales);
  if (bf16)
    w4_quantize_kernel<true><<<grid, 256, 0, s>>>(N, K, group, W, codes, sc, zeros);
  else
    w4_quantize_kernel<false><<<grid, 256, 0, s>>>(N, K, group, W, codes, sc, zeros);
  return cudaGetLastError();
}

}  // namespace m3
