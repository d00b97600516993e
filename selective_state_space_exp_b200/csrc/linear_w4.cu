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
// A producer thread streams the codes by TMA, in boxes of 256 inputs (128
// bytes, swizzled) x 16 MT outputs, one box for each of eight warps in a stage.
// A warp turns its box into the product's A operand in registers: which input a
// fragment's slot stands for is free as long as both operands agree, so each
// lane takes the consecutive inputs of one wide shared-memory load, and the
// tokens' values are laid out once per block in that order.  A word of eight
// codes becomes four bf16 pairs: the codes of a pair (e, e + 4) are masked into
// the low mantissa bits of 128 (0x4300), which makes the number 128 + q, and
// 128 + z is taken off, both exactly.  The warps' parts of the inputs are added
// in shared memory in a fixed order.
#include <cuda.h>  // CUtensorMap

#include <cstring>

#include "lm_ops.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

using namespace tc;

constexpr int kWarps = 8;               // consumers; one more warp produces
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kBox = 256;               // inputs of a box: 128 bytes of codes
constexpr int kXChunk = 4 * 32 * 16;    // bytes of eight tokens' values of 128 inputs
constexpr int kMostStages = 8;
constexpr unsigned long long kWaitNs = 2000000000ull;

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

__device__ bool w4_wait(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  while (!mbar_try_wait(bar, parity)) {
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 > kWaitNs) {
      if (status) atomicCAS(status, 0, (int)M3_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Input of word w (0..3) of lane column c (0..3) in a chunk of 128: per group a
// lane has group / 4 consecutive inputs, eight a word.
template <int G>
__device__ __forceinline__ int input_of(int w, int c) {
  constexpr int words = G / 32;  // words of one group in a lane
  return (w / words) * G + c * (G / 4) + (w % words) * 8;
}

// Output (0..7) that fragment row r stands for: the rows of one shared-memory
// phase (2 for 16-byte loads, 4 for 8-byte ones) then differ in the swizzle bits
// that keep their pieces in different banks.
template <int G>
__device__ __forceinline__ int output_of(int r) {
  return G == 128 ? ((r & 1) << 2) | (r >> 1) : G == 64 ? ((r & 3) << 1) | (r >> 2) : r;
}

// Scales and zero points of a lane's two rows of one row tile over a box.
template <int G>
struct Params {
  static constexpr int NG = kBox / G;
  uint32_t s[2][(NG + 1) / 2];  // bf16 pairs
  uint32_t z[2][(NG + 3) / 4];  // bytes
};

template <int G, bool ZEROS>
__device__ __forceinline__ void load_params(const W4Args& a, bool vec, int64_t row0, int64_t k0,
                                            int lane, Params<G>& o) {
  constexpr int NG = Params<G>::NG;
  const int64_t kg = a.K / G;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = row0 + output_of<G>(lane >> 2) + 8 * h;
    const int64_t at = row * kg + k0 / G;
#pragma unroll
    for (int i = 0; i < (NG + 1) / 2; ++i) o.s[h][i] = 0;
#pragma unroll
    for (int i = 0; i < (NG + 3) / 4; ++i) o.z[h][i] = 0x08080808u;
    if (row >= a.N || k0 >= a.K) continue;
    const uint16_t* s = static_cast<const uint16_t*>(a.scales) + at;
    const uint8_t* z = a.zeros + at;
    if (vec) {  // K is a multiple of 256: a row's box is whole and aligned
      if constexpr (NG == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
        o.s[h][0] = v.x; o.s[h][1] = v.y; o.s[h][2] = v.z; o.s[h][3] = v.w;
      } else if constexpr (NG == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
        o.s[h][0] = v.x; o.s[h][1] = v.y;
      } else {
        o.s[h][0] = __ldg(reinterpret_cast<const uint32_t*>(s));
      }
      if constexpr (ZEROS) {
        if constexpr (NG == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
          o.z[h][0] = v.x; o.z[h][1] = v.y;
        } else if constexpr (NG == 4) {
          o.z[h][0] = __ldg(reinterpret_cast<const uint32_t*>(z));
        } else {
          o.z[h][0] = __ldg(reinterpret_cast<const uint16_t*>(z));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (k0 + i * G >= a.K) continue;
        o.s[h][i / 2] |= (uint32_t)__ldg(s + i) << (16 * (i & 1));
        if constexpr (ZEROS) {
          const int sh = 8 * (i & 3);
          o.z[h][i / 4] = (o.z[h][i / 4] & ~(0xffu << sh)) | ((uint32_t)__ldg(z + i) << sh);
        }
      }
    }
  }
}

// One box's products of a row tile, group by group, added to acc with the
// groups' scales.  codes: the tile's 16 rows of 128 swizzled bytes; xs: the
// tokens' values of the box's two chunks.
template <int G, bool ZEROS, int MT, int NT>
__device__ __forceinline__ void box_products(const uint8_t* codes, const uint8_t* xs, int xstride,
                                             const Params<G> (&pr)[MT], int lane,
                                             float (&acc)[MT][NT][4]) {
  constexpr int words = G / 32, NG = kBox / G;
  const int r = output_of<G>(lane >> 2), c = lane & 3;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int ch = i * G / 128, in = (i * G % 128) / 32;  // chunk, first word of the group in it
    uint32_t q[MT][2][words], zz[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* row = codes + (t * 16 + r + 8 * h) * 128;
        const int byte = i * (G / 2) + c * (G / 8);
        const uint8_t* p = row + ((((byte >> 4) ^ r) << 4) | (byte & 15));  // r + 8 swizzles as r
        if constexpr (G == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          q[t][h][0] = v.x; q[t][h][1] = v.y; q[t][h][2] = v.z; q[t][h][3] = v.w;
        } else if constexpr (G == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          q[t][h][0] = v.x; q[t][h][1] = v.y;
        } else {
          q[t][h][0] = *reinterpret_cast<const uint32_t*>(p);
        }
        zz[t][h] = ZEROS ? 0x43004300u + ((pr[t].z[h][i / 4] >> (8 * (i & 3))) & 15u) * 0x00010001u
                         : 0x43084308u;
      }
    }
    float d[MT][NT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) d[t][n][0] = d[t][n][1] = d[t][n][2] = d[t][n][3] = 0.f;
#pragma unroll
    for (int w = 0; w < words; ++w) {
      uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t f[4];  // pairs (e, e + 4), e = 0..3
#pragma unroll
          for (int e = 0; e < 4; ++e)
            f[e] = sub_bf16x2(((q[t][h][w] >> (4 * e)) & 0x000f000fu) | 0x43004300u, zz[t][h]);
          a0[t][h] = f[0]; a0[t][2 + h] = f[1];
          a1[t][h] = f[2]; a1[t][2 + h] = f[3];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = *reinterpret_cast<const uint4*>(xs + n * xstride + ch * kXChunk +
                                                        ((in + w) * 32 + lane) * 16);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma_bf16(d[t][n], a0[t], b.x, b.y);
          mma_bf16(d[t][n], a1[t], b.z, b.w);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float s0 = __uint_as_float((i & 1) ? pr[t].s[0][i / 2] & 0xffff0000u : pr[t].s[0][i / 2] << 16);
      const float s1 = __uint_as_float((i & 1) ? pr[t].s[1][i / 2] & 0xffff0000u : pr[t].s[1][i / 2] << 16);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[t][n][0] = fmaf(s0, d[t][n][0], acc[t][n][0]);
        acc[t][n][1] = fmaf(s0, d[t][n][1], acc[t][n][1]);
        acc[t][n][2] = fmaf(s1, d[t][n][2], acc[t][n][2]);
        acc[t][n][3] = fmaf(s1, d[t][n][3], acc[t][n][3]);
      }
    }
  }
}

// The values of `boxes` boxes from `box0` of tokens m0 .. m0 + 8 NT, in fragment
// order: [token tile][chunk][word][lane] of 16 bytes, inputs (0, 4, 1, 5, 2, 6, 3, 7).
template <int G, int NT>
__device__ __forceinline__ void stage_tokens(const W4Args& a, uint8_t* xs, int64_t m0,
                                             int64_t box0, int boxes) {
  const int n = 2 * boxes;
  for (int i = threadIdx.x; i < NT * n * 128; i += 32 * kWarps) {
    const int lane = i & 31, w = (i >> 5) & 3;
    const int ch = (i >> 7) % n, t = (i >> 7) / n;
    const int64_t m = m0 + t * 8 + (lane >> 2);
    const int64_t k = box0 * kBox + ch * 128 + input_of<G>(w, lane & 3);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (m < a.M && k < a.K)
      v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.A) + m * a.K + k));
    uint4 o;  // v holds inputs 01 23 45 67
    o.x = __byte_perm(v.x, v.z, 0x5410);  // 0 4
    o.y = __byte_perm(v.x, v.z, 0x7632);  // 1 5
    o.z = __byte_perm(v.y, v.w, 0x5410);  // 2 6
    o.w = __byte_perm(v.y, v.w, 0x7632);  // 3 7
    *reinterpret_cast<uint4*>(xs + ((size_t)t * n + ch) * kXChunk + (w * 32 + lane) * 16) = o;
  }
}

struct W4Plan {
  int boxes;    // boxes of a row in one stage (at most a warp each)
  int slices;   // stages of a row's inputs
  int rb;       // row blocks of 16 MT outputs in a stage
  int stages;
  int xboxes;   // boxes whose token values are held: all of a row's, or one slice's
  int64_t items;  // groups of rb row blocks
};

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

template <int G, bool ZEROS, int MT, int NT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 2 : 1)
w4_kernel(const W4Args a, const W4Plan p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t sm[];
  constexpr int kBoxBytes = 16 * MT * 128;
  constexpr int kRed = 16 * MT * 8 * NT;  // a warp's partial sums
  constexpr int kRedBufs = NT == 1 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nbox = p.boxes * p.rb;
  const int stage_bytes = nbox * kBoxBytes;
  uint8_t* xs = sm + p.stages * stage_bytes;
  float* red = reinterpret_cast<float*>(xs + (size_t)NT * p.xboxes * 2 * kXChunk);  // [bufs][warp][kRed]
  uint64_t* full = reinterpret_cast<uint64_t*>(red + kRedBufs * kWarps * kRed);
  uint64_t* empty = full + kMostStages;
  if ((smem_u32(sm) & 1023u) != 0) {  // the swizzled boxes need 1 KB alignment
    if (threadIdx.x == 0 && a.status) atomicCAS(a.status, 0, (int)M3_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    if (lane != 0) return;
    uint32_t it = 0;
    bool ok = true;
    for (int64_t item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
      for (int sl = 0; sl < p.slices; ++sl, ++it) {
        const int s = (int)(it % (uint32_t)p.stages);
        ok = w4_wait(&empty[s], ((it / (uint32_t)p.stages) & 1u) ^ 1u, a.status);
        if (!ok) break;
        mbar_expect_tx(&full[s], (uint32_t)stage_bytes);
        for (int b = 0; b < nbox; ++b) {
          const int64_t row = (item * p.rb + b / p.boxes) * 16 * MT;
          const int64_t box = (int64_t)sl * p.boxes + b % p.boxes;
          asm volatile(
              "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(sm + s * stage_bytes + b * kBoxBytes)),
              "l"(reinterpret_cast<uint64_t>(&map)), "r"((int)(box * (kBox / 2))), "r"((int)row),
              "r"(smem_u32(&full[s]))
              : "memory");
        }
      }
    }
    // let the last stages' copies land (bounded) before the block can exit
    const uint32_t st = (uint32_t)p.stages;
    for (uint32_t j = it > st ? it - st : 0; j < it; ++j)
      w4_wait(&full[j % st], (j / st) & 1u, a.status);
    return;
  }

  const int64_t m0 = (int64_t)blockIdx.y * 8 * NT;
  const bool vec = a.K % kBox == 0;
  const int mybox = warp % p.boxes, myrb = warp / p.boxes;
  const bool busy = warp < nbox;
  const bool whole = p.slices == 1 || p.xboxes > p.boxes;  // all token values are held
  if (whole) {
    stage_tokens<G, NT>(a, xs, m0, 0, p.xboxes);
    consumers_sync();
  }
  uint32_t it = 0, buf = 0;
  bool ok = true;
  Params<G> pr[MT];
  if (busy && blockIdx.x < p.items) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
      load_params<G, ZEROS>(a, vec, (((int64_t)blockIdx.x * p.rb + myrb) * MT + t) * 16,
                            (int64_t)mybox * kBox, lane, pr[t]);
  }
  for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x, buf ^= 1u) {
    float acc[MT][NT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.f;
    for (int sl = 0; sl < p.slices; ++sl, ++it) {
      if (!whole) {
        consumers_sync();
        stage_tokens<G, NT>(a, xs, m0, (int64_t)sl * p.boxes, p.xboxes);
        consumers_sync();
      }
      const int s = (int)(it % (uint32_t)p.stages);
      if (ok) ok = w4_wait(&full[s], (it / (uint32_t)p.stages) & 1u, a.status);
      // the next stage's scales are on their way while this one is multiplied
      Params<G> nx[MT];
      const bool more = sl + 1 < p.slices;
      const int64_t nitem = more ? item : item + gridDim.x;
      if (busy && nitem < p.items) {
        const int64_t nbx = (int64_t)(more ? sl + 1 : 0) * p.boxes + mybox;
#pragma unroll
        for (int t = 0; t < MT; ++t)
          load_params<G, ZEROS>(a, vec, ((nitem * p.rb + myrb) * MT + t) * 16, nbx * kBox, lane,
                                nx[t]);
      }
      if (busy && ok) {
        const int64_t xb = whole ? (int64_t)sl * p.boxes + mybox : mybox;
        if (xb < p.xboxes)
          box_products<G, ZEROS, MT, NT>(sm + s * stage_bytes + warp * kBoxBytes,
                                         xs + (size_t)xb * 2 * kXChunk, p.xboxes * 2 * kXChunk, pr,
                                         lane, acc);
      }
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[s])) : "memory");
#pragma unroll
      for (int t = 0; t < MT; ++t) pr[t] = nx[t];
    }
    // the warps' parts of the inputs, added in order; with two buffers one
    // barrier an item is enough
    if (kRedBufs == 1) consumers_sync();
    float* r = red + (kRedBufs == 1 ? 0 : buf * kWarps * kRed);
    if (busy) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            r[warp * kRed + t * 16 + output_of<G>(lane >> 2) + (i >> 1) * 8 +
              16 * MT * (n * 8 + (lane & 3) * 2 + (i & 1))] = acc[t][n][i];
    }
    consumers_sync();
    for (int i = threadIdx.x; i < p.rb * kRed; i += 32 * kWarps) {
      const int st = i / kRed, at = i % kRed;
      const int64_t n = (item * p.rb + st) * 16 * MT + at % (16 * MT), m = m0 + at / (16 * MT);
      if (n >= a.N || m >= a.M) continue;
      float v = r[st * p.boxes * kRed + at];
      for (int k = 1; k < p.boxes; ++k) v += r[(st * p.boxes + k) * kRed + at];
      if (a.bias) v += __ldg(a.bias + n);
      if (M3_IN(m * a.N + n, a.M * a.N, a.status)) io_store(a.out, m * a.N + n, v, !a.out_f32);
    }
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// The codes as [N][K / 2] bytes, boxes of 128 bytes x `rows`, rows past N and
// bytes past K / 2 read as zero.
bool encode_codes(CUtensorMap* m, const W4Args& a, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(a.K / 2), (cuuint64_t)a.N};
  const cuuint64_t strides[1] = {(cuuint64_t)(a.K / 2)};
  const cuuint32_t box[2] = {kBox / 2, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, bool ZEROS, int MT, int NT>
cudaError_t launch_nt(const W4Args& a, cudaStream_t s) {
  constexpr int kBoxBytes = 16 * MT * 128, kRed = 16 * MT * 8 * NT;
  constexpr int fixed = (NT == 1 ? 2 : 1) * kWarps * kRed * 4 + 2 * kMostStages * 8;
  constexpr int xbox = NT * 2 * kXChunk;
  constexpr int kHalf = 113 * 1024, kWhole = 226 * 1024;
  W4Plan p;
  const int64_t all = (a.K + kBox - 1) / kBox;
  p.slices = (int)((all + kWarps - 1) / kWarps);
  p.boxes = (int)((all + p.slices - 1) / p.slices);
  p.rb = kWarps / p.boxes;
  const int stage = p.boxes * p.rb * kBoxBytes;
  // the token values of a whole row where three stages still fit beside them
  p.xboxes = fixed + all * xbox + 3 * (int64_t)stage <= kWhole ? (int)all : p.boxes;
  const int need = fixed + p.xboxes * xbox;
  const int room = MT == 1 && need + 3 * stage <= kHalf ? kHalf : kWhole;
  p.stages = (room - need) / stage;
  if (p.stages > kMostStages) p.stages = kMostStages;
  if (p.stages < 1) return cudaErrorInvalidValue;
  const int smem = need + p.stages * stage;
  p.items = ((a.N + 16 * MT - 1) / (16 * MT) + p.rb - 1) / p.rb;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  if (!encode_codes(&map, a, 16 * MT)) return cudaErrorInvalidValue;
  auto kern = w4_kernel<G, ZEROS, MT, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sms * (room == kHalf ? 2 : 1);
  const dim3 grid((unsigned)(p.items < most ? p.items : most),
                  (unsigned)((a.M + 8 * NT - 1) / (8 * NT)));
  kern<<<grid, kThreads, smem, s>>>(a, p, map);
  return cudaGetLastError();
}

// Tokens are taken 8 NT at a time.  From two token tiles on a warp takes 32
// outputs, so that a token value read from shared memory serves two products.
template <int G, bool ZEROS>
cudaError_t launch_z(const W4Args& a, cudaStream_t s) {
  if (a.M <= 8) return launch_nt<G, ZEROS, 1, 1>(a, s);
  if (a.M <= 16) return launch_nt<G, ZEROS, 2, 2>(a, s);
  return launch_nt<G, ZEROS, 2, 4>(a, s);
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
