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
// Each of sixteen warps streams its own codes by TMA, in boxes of 256 inputs (128
// bytes, swizzled) x 16 MT outputs through a ring of its own, and refills a slot
// when it has read it: the warps meet only where their parts of the inputs are
// added.  A warp turns its box into the product's A operand in registers: which input a
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

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBox = 256;               // inputs of a box: 128 bytes of codes
constexpr int kXChunk = 4 * 32 * 16;    // bytes of eight tokens' values of 128 inputs
constexpr int kMostStages = 8;         // of a warp's ring
constexpr int kSmemMost = 226 * 1024;
constexpr unsigned long long kWaitNs = 2000000000ull;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a group: no accumulator to clear.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// (v & mask) | magic as one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(magic));
  return r;
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

// s, z: the lane's place in the first of its rows, at the box's first group;
// kg8: eight rows on.  rows, cols: how many rows and groups there are from here.
template <int G, bool ZEROS, int MT>
__device__ __forceinline__ void load_params(const uint16_t* s, const uint8_t* z, int64_t kg8,
                                            bool vec, int rows, int cols,
                                            Params<G> (&o)[MT]) {
  constexpr int NG = Params<G>::NG;
  if (vec && rows > 16 * MT - 8 && cols > 0) {  // whole rows, aligned pieces
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h, s += kg8, z += kg8) {
        Params<G>& p = o[t];
        if constexpr (NG == 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
          p.s[h][0] = v.x; p.s[h][1] = v.y; p.s[h][2] = v.z; p.s[h][3] = v.w;
        } else if constexpr (NG == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
          p.s[h][0] = v.x; p.s[h][1] = v.y;
        } else {
          p.s[h][0] = __ldg(reinterpret_cast<const uint32_t*>(s));
        }
        if constexpr (ZEROS) {
          if constexpr (NG == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
            p.z[h][0] = v.x; p.z[h][1] = v.y;
          } else if constexpr (NG == 4) {
            p.z[h][0] = __ldg(reinterpret_cast<const uint32_t*>(z));
          } else {
            p.z[h][0] = __ldg(reinterpret_cast<const uint16_t*>(z));
          }
        }
      }
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h, s += kg8, z += kg8) {
      Params<G>& p = o[t];
#pragma unroll
      for (int i = 0; i < (NG + 1) / 2; ++i) p.s[h][i] = 0;
#pragma unroll
      for (int i = 0; i < (NG + 3) / 4; ++i) p.z[h][i] = 0;
      if (t * 16 + h * 8 >= rows) continue;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (i >= cols) continue;
        p.s[h][i / 2] |= (uint32_t)__ldg(s + i) << (16 * (i & 1));
        if constexpr (ZEROS) p.z[h][i / 4] |= (uint32_t)__ldg(z + i) << (8 * (i & 3));
      }
    }
  }
}

// One box's products of a row tile, group by group, added to acc with the
// groups' scales.  codes: the tile's 16 rows of 128 swizzled bytes; xs: the
// tokens' values of the box's two chunks.
template <int G, bool ZEROS, int MT, int NT>
__device__ __forceinline__ void box_products(const uint8_t* codes, const uint8_t* xs, int xstride,
                                             const Params<G> (&pr)[MT], int lane, uint32_t mask,
                                             uint32_t magic, float (&acc)[MT][NT][4]) {
  constexpr int words = G / 32, NG = kBox / G;
  const int r = output_of<G>(lane >> 2), c = lane & 3;
  // a lane's piece of group i: byte i * G / 2 + c * G / 8 of its row, the 16-byte
  // pieces swizzled by the row (r + 8 swizzles as r)
  const uint8_t* row = codes + r * 128 + ((c * (G / 8)) & 15);
  const uint32_t piece = (uint32_t)(((c * (G / 8)) & ~15) ^ (r << 4));
  uint32_t zb[MT][2][(NG + 3) / 4];
  if constexpr (ZEROS) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < (NG + 3) / 4; ++i) zb[t][h][i] = pr[t].z[h][i] & 0x0f0f0f0fu;
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int ch = i * G / 128, in = (i * G % 128) / 32;  // chunk, first word of the group in it
    uint32_t q[MT][2][words], zz[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* p = row + (t * 16 + 8 * h) * 128 + (piece ^ (uint32_t)(i * (G / 2)));
        if constexpr (G == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          q[t][h][0] = v.x; q[t][h][1] = v.y; q[t][h][2] = v.z; q[t][h][3] = v.w;
        } else if constexpr (G == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          q[t][h][0] = v.x; q[t][h][1] = v.y;
        } else {
          q[t][h][0] = *reinterpret_cast<const uint32_t*>(p);
        }
        // 128 + z, twice: the zero point's byte below 0x43
        zz[t][h] = ZEROS ? __byte_perm(zb[t][h][i / 4], 0x43434343u, 0x4040u | ((i & 3) * 0x0101u))
                         : 0x43084308u;
      }
    }
    float d[MT][NT][4];
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
            f[e] = sub_bf16x2(and_or(q[t][h][w] >> (4 * e), mask, magic), zz[t][h]);
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
          if (w == 0)
            mma_bf16_first(d[t][n], a0[t], b.x, b.y);
          else
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
  for (int i = threadIdx.x; i < NT * n * 128; i += kThreads) {
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
  int ks;       // warps that share a row block's inputs, box by box in turn
  int slices;   // boxes of each of them
  int rb;       // row blocks of 16 MT outputs in an item
  int stages;   // boxes of a warp's ring
  int xboxes;   // boxes whose token values are held: all of a row's, or ks
  int items;    // groups of rb row blocks
  int all;      // boxes of a row
  // 0x000f000f and 0x43004300: as kernel arguments they are operands from the
  // constant bank; as literals each use first moved one into a register
  uint32_t mask, magic;
};

template <int G, bool ZEROS, int MT, int NT>
__global__ void __launch_bounds__(kThreads, 1)
w4_kernel(const W4Args a, const W4Plan p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t sm[];
  constexpr int kBoxBytes = 16 * MT * 128;
  constexpr int kRed = 16 * MT * 8 * NT;  // a warp's partial sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = sm + warp * p.stages * kBoxBytes;
  uint8_t* xs = sm + kWarps * p.stages * kBoxBytes;
  float* red = reinterpret_cast<float*>(xs + (size_t)NT * p.xboxes * 2 * kXChunk);  // [warp][kRed]
  uint64_t* full = reinterpret_cast<uint64_t*>(red + kWarps * kRed) + warp * kMostStages;
  if ((smem_u32(sm) & 1023u) != 0) {  // the swizzled boxes need 1 KB alignment
    if (threadIdx.x == 0 && a.status) atomicCAS(a.status, 0, (int)M3_ERR_CUDA);
    return;
  }
  const int64_t m0 = (int64_t)blockIdx.y * 8 * NT;
  const bool vec = a.K % kBox == 0;
  const int part = warp % p.ks, myrb = warp / p.ks;
  const bool busy = myrb < p.rb;
  const int row_step = (int)gridDim.x * p.rb * 16 * MT;  // from an item to the block's next

  // lane 0 keeps the ring full: the next box's row, slice and slot
  int pitem = (int)blockIdx.x, prow = ((int)blockIdx.x * p.rb + myrb) * 16 * MT, psl = 0, pslot = 0;
  auto ask = [&] {
    if (pitem >= p.items) return;
    mbar_expect_tx(&full[pslot], (uint32_t)kBoxBytes);
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(ring + pslot * kBoxBytes)),
        "l"(reinterpret_cast<uint64_t>(&map)), "r"((psl * p.ks + part) * (kBox / 2)), "r"(prow),
        "r"(smem_u32(&full[pslot]))
        : "memory");
    if (++pslot == p.stages) pslot = 0;
    if (++psl == p.slices) {
      psl = 0;
      prow += row_step;
      pitem += (int)gridDim.x;
    }
  };
  if (busy && lane == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    for (int s = 0; s < p.stages; ++s) ask();
  }
  __syncwarp();
  const uint32_t magic = p.magic;
  const bool whole = p.xboxes >= p.ks * p.slices;  // all token values are held
  if (whole) {
    stage_tokens<G, NT>(a, xs, m0, 0, p.xboxes);
    __syncthreads();
  }

  // the lane's place in scales and zeros: its first row of the item, its box
  const int kg = (int)(a.K / G);
  int left = (int)a.N - (((int)blockIdx.x * p.rb + myrb) * 16 * MT + output_of<G>(lane >> 2));
  int64_t at = ((int64_t)a.N - left) * kg + part * (kBox / G);
  const int64_t to_item = (int64_t)row_step * kg - (int64_t)(p.slices - 1) * p.ks * (kBox / G);
  const int to_slice = p.ks * (kBox / G);
  auto params = [&](int box, Params<G>(&o)[MT]) {
    load_params<G, ZEROS, MT>(static_cast<const uint16_t*>(a.scales) + at, a.zeros + at,
                              8 * (int64_t)kg, vec, left, box < p.all ? kg - box * (kBox / G) : 0, o);
  };
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  Params<G> pr[MT];
  if (busy) params(part, pr);
  for (int item = (int)blockIdx.x; item < p.items; item += (int)gridDim.x) {
    float acc[MT][NT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.f;
    for (int sl = 0; sl < p.slices; ++sl) {
      if (!whole) {
        __syncthreads();
        stage_tokens<G, NT>(a, xs, m0, (int64_t)sl * p.ks, p.xboxes);
        __syncthreads();
      }
      if (!busy) continue;
      if (ok) ok = __all_sync(0xffffffffu, w4_wait(&full[slot], phase, a.status));
      // the next box's scales are on their way while this one is multiplied
      Params<G> nx[MT];
      const bool more = sl + 1 < p.slices;
      at += more ? (int64_t)to_slice : to_item;
      if (!more) left -= row_step;
      params(more ? (sl + 1) * p.ks + part : part, nx);
      if (ok) {
        const int xb = whole ? sl * p.ks + part : part;
        box_products<G, ZEROS, MT, NT>(ring + slot * kBoxBytes, xs + (size_t)xb * 2 * kXChunk,
                                       p.xboxes * 2 * kXChunk, pr, lane, p.mask, magic, acc);
      }
      __syncwarp();  // every lane has read the slot
      if (ok && lane == 0) ask();
      if (ok && ++slot == p.stages) {
        slot = 0;
        phase ^= 1u;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) pr[t] = nx[t];
    }
    // the warps' parts of the inputs, added in order
    if (busy) {
      float* r = red + warp * kRed + output_of<G>(lane >> 2) + 16 * MT * 2 * (lane & 3);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            r[t * 16 + (i >> 1) * 8 + 16 * MT * (n * 8 + (i & 1))] = acc[t][n][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.rb * kRed; i += kThreads) {
      const int st = i / kRed, o = i % kRed;
      const int64_t n = (item * p.rb + st) * 16 * MT + o % (16 * MT), m = m0 + o / (16 * MT);
      if (n >= a.N || m >= a.M) continue;
      const float* r = red + st * p.ks * kRed + o;
      float v = r[0];
      for (int k = 1; k < p.ks; ++k) v += r[k * kRed];
      if (a.bias) v += __ldg(a.bias + n);
      if (M3_IN(m * a.N + n, a.M * a.N, a.status)) io_store(a.out, m * a.N + n, v, !a.out_f32);
    }
    if (item + (int)gridDim.x < p.items) __syncthreads();  // before the sums are overwritten
  }
  // after a wait that gave up: the copies asked for land (bounded) before the
  // block can exit; of a slot's copies only the last can still be out
  if (busy && !ok && lane == 0)
    for (int k = 0; k < p.stages; ++k) {
      if (slot == k) continue;
      w4_wait(&full[k], phase ^ (k < slot ? 1u : 0u), a.status);
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

// How the work is cut for `MT` row tiles a warp and `NT` token tiles; false
// where a ring of two boxes does not fit beside all of a row's token values.
bool make_plan(const W4Args& a, int MT, int NT, bool whole, W4Plan* p) {
  const int box = 16 * MT * 128, red = kWarps * 16 * MT * 8 * NT * 4;
  const int64_t all = (a.K + kBox - 1) / kBox;  // boxes of a row
  const int64_t rows = (a.N + 16 * MT - 1) / (16 * MT);
  // warps that share a row block: few, so that what an item costs besides its
  // boxes (about 0.7 boxes) comes seldom, but enough to keep every SM busy
  double best = 0;
  for (int ks = 1; ks <= kWarps; ks *= 2) {
    const int64_t slices = (all + ks - 1) / ks, rb = kWarps / ks;
    const int64_t rounds = ((rows + rb - 1) / rb + kPlanSms - 1) / kPlanSms;
    const double cost = (double)rounds * ((double)slices + 0.7);
    if (ks == 1 || cost < best) {
      best = cost;
      p->ks = ks;
      p->slices = (int)slices;
      p->rb = (int)rb;
    }
    if (ks >= all) break;
  }
  p->all = (int)all;
  p->mask = 0x000f000fu;
  p->magic = 0x43004300u;
  p->items = (int)((rows + p->rb - 1) / p->rb);
  p->xboxes = whole ? p->ks * p->slices : p->ks;
  const int64_t left = kSmemMost - red - kWarps * kMostStages * 8 - (int64_t)p->xboxes * NT * 2 * kXChunk;
  p->stages = left < 0 ? 0 : (int)(left / (kWarps * box));
  if (p->stages > kMostStages) p->stages = kMostStages;
  return p->stages >= 2;
}

template <int G, bool ZEROS, int MT, int NT>
cudaError_t launch_plan(const W4Args& a, const W4Plan& p, cudaStream_t s) {
  const int smem = kWarps * p.stages * 16 * MT * 128 + p.xboxes * NT * 2 * kXChunk +
                   kWarps * 16 * MT * 8 * NT * 4 + kWarps * kMostStages * 8;
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
  const dim3 grid((unsigned)(p.items < sms ? p.items : sms),
                  (unsigned)((a.M + 8 * NT - 1) / (8 * NT)));
  kern<<<grid, kThreads, smem, s>>>(a, p, map);
  return cudaGetLastError();
}

// A warp takes 32 outputs, so that a token value read from shared memory serves
// two products; 16 where a ring of two such boxes does not fit beside the token
// values of a whole row; and where neither fits, the token values are read
// again for each slice.
template <int G, bool ZEROS, int NT>
cudaError_t launch_nt(const W4Args& a, cudaStream_t s) {
  W4Plan p;
  if (make_plan(a, 2, NT, true, &p)) return launch_plan<G, ZEROS, 2, NT>(a, p, s);
  if (make_plan(a, 1, NT, true, &p)) return launch_plan<G, ZEROS, 1, NT>(a, p, s);
  if (make_plan(a, 1, NT, false, &p)) return launch_plan<G, ZEROS, 1, NT>(a, p, s);
  return cudaErrorInvalidValue;
}

template <int G, bool ZEROS>
cudaError_t launch_z(const W4Args& a, cudaStream_t s) {
  return a.M <= 8 ? launch_nt<G, ZEROS, 1>(a, s) : launch_nt<G, ZEROS, 2>(a, s);
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
