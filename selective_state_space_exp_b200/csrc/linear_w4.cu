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
//
// From 17 tokens on the products are tcgen05's: eight warps write the decoded
// weights to TMEM as the A operand, the tokens' values come by TMA as B, eight more
// warps add the groups' sums with their scales out of TMEM.
//
// Rounding: sums, scales' products and bias in fp32, out rounded once.
//
// Measured: one token, 50257 x 2048: 17.3 us (groups of 128), 20.4 us (of 32, zero
// points): 3.0 TB/s of codes and scales.  230 instructions for 16 x 128 codes, 88 of them
// a word's shifts, masks and subtractions, the others loads, scales, zero points and
// additions; issue slots are 53 % used, no unit is at its limit.  11 tokens 24.9 us, 32
// tokens 25.7, 64 tokens 31.8, 128 tokens x 8192 x 4096 19.8 us: there the decoding, the
// products and the sums of a step wait on one another.  One token, 4096 x 2048: 5.5 us,
// most of it the start of a kernel and the way to memory and back.
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

// A constant that stays in a register: as a plain one it is moved into a new
// register at each use.
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (v & mask) | magic as one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(magic));
  return r;
}

// Waits for a phase: the timer is read only every so many tries (each try may
// itself suspend for a while).
__device__ __forceinline__ bool w4_wait(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitNs) {
      if (status) atomicCAS(status, 0, (int)M3_ERR_TIMEOUT);
      return false;
    }
  }
}

// By a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool w4_wait_all(uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, w4_wait(bar, parity, status));
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
                                             uint32_t magic, uint32_t bytes,
                                             float (&acc)[MT][NT][4]) {
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
        zz[t][h] = ZEROS ? __byte_perm(zb[t][h][i / 4], bytes, 0x4040u | ((i & 3) * 0x0101u)) : bytes;
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
  const int n = 2 * boxes, all = NT * n * 128;
  constexpr int U = 4;  // loads in flight together
  for (int i0 = threadIdx.x; i0 < all; i0 += U * kThreads) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      const int lane = i & 31, w = (i >> 5) & 3, ch = (i >> 7) % n, t = (i >> 7) / n;
      const int64_t m = m0 + t * 8 + (lane >> 2);
      const int64_t k = box0 * kBox + ch * 128 + input_of<G>(w, lane & 3);
      v[u] = make_uint4(0, 0, 0, 0);
      if (i < all && m < a.M && k < a.K)
        v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.A) + m * a.K + k));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= all) break;
      uint4 o;  // v holds inputs 01 23 45 67
      o.x = __byte_perm(v[u].x, v[u].z, 0x5410);  // 0 4
      o.y = __byte_perm(v[u].x, v[u].z, 0x7632);  // 1 5
      o.z = __byte_perm(v[u].y, v[u].w, 0x5410);  // 2 6
      o.w = __byte_perm(v[u].y, v[u].w, 0x7632);  // 3 7
      *reinterpret_cast<uint4*>(xs + (size_t)i * 16) = o;  // [tile][chunk][word][lane]
    }
  }
}

// Outputs n .. n + 3 of token m, those there are.
__device__ __forceinline__ void store_outputs(const W4Args& a, int64_t m, int64_t n, float4 f) {
  float v[4] = {f.x, f.y, f.z, f.w};
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) v[j] += __ldg(a.bias + n + j);
  }
  const int64_t at = m * a.N + n;
  if (!M3_IN(at + (a.N % 4 == 0 ? 3 : 0), a.M * a.N, a.status)) return;
  if (a.N % 4 == 0) {  // whole and aligned
    if (a.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) io_store(a.out, at + j, v[j], !a.out_f32);
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
  // 0x000f000f (as an argument an operand from the constant bank), 0x43004300, and
  // 0x43434343 with zero points or 128 + 8 twice without
  uint32_t mask, magic, bytes;
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
  const int tokens = (int)(a.M - m0 < 8 * NT ? a.M - m0 : 8 * NT);
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
  const uint32_t magic = in_register(p.magic), bytes = in_register(p.bytes);
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
                                       p.xboxes * 2 * kXChunk, pr, lane, p.mask, magic, bytes, acc);
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
    // the warps' parts of the inputs, added in order, four outputs a thread
    if (busy) {
      float* r = red + warp * kRed + output_of<G>(lane >> 2);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int tok = n * 8 + (lane & 3) * 2 + j;
          if (tok >= tokens) continue;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            r[16 * MT * tok + t * 16] = acc[t][n][j];
            r[16 * MT * tok + t * 16 + 8] = acc[t][n][2 + j];
          }
        }
    }
    __syncthreads();
    constexpr int kQuads = 4 * MT;  // of a row block's outputs
    for (int i = threadIdx.x; i < p.rb * tokens * kQuads; i += kThreads) {
      const int qd = i % kQuads, rest = i / kQuads, tok = rest % tokens, st = rest / tokens;
      const int64_t n = (int64_t)(item * p.rb + st) * 16 * MT + qd * 4, m = m0 + tok;
      if (n >= a.N) continue;
      const float* r = red + st * p.ks * kRed + 16 * MT * tok + qd * 4;
      float4 v = *reinterpret_cast<const float4*>(r);
#pragma unroll 4
      for (int k = 1; k < p.ks; ++k) {
        const float4 f = *reinterpret_cast<const float4*>(r + k * kRed);
        v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
      }
      store_outputs(a, m, n, v);
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
  p->bytes = a.zeros ? 0x43434343u : 0x43084308u;
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
  // the same limit whatever the plan: another host thread may set it between this and the launch
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
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

// ---- tcgen05 form ---------------------------------------------------------------

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 16) {
    tmem_ld16(taddr, v);
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
  }
}

// 16 consecutive 32-bit columns of this thread's TMEM lane (warp-wide).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}

// D (TMEM) [+]= A (TMEM) * B (smem), issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int c0, int c1,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// A place in a ring of n slots and the parity of its current use.
struct Turn {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

constexpr int kTileRows = 128;               // outputs of a tile
constexpr int kStep = 256;                   // inputs of a step
constexpr int kCodeBox = kTileRows * 128;    // bytes: a step's codes
constexpr int kABufs = 2, kACols = kStep / 2;  // TMEM: a step's weights, bf16 pairs
constexpr int kDCols = 512 - kABufs * kACols;  // TMEM left for sums
constexpr int kBlock = 8;                    // groups whose scales are staged at a time
constexpr int kWG = 2;                       // warpgroups of each of the two roles below
constexpr int kWorkers = 4 * kWG;            // warps that decode, and as many that add up
constexpr int kTcThreads = 32 * (2 * kWorkers + 4);

template <int G, int NTOK>
struct TcCfg {
  // Sums of SUB inputs each, CI of them accumulated in turn: MMAs into one
  // accumulator wait on each other, so few tokens want several chains.
  static constexpr int CI = NTOK >= 128 ? 1 : NTOK == 64 ? 2 : 4;
  static constexpr int SUB = CI == 1 ? G : G < 64 ? G : 64;
  static constexpr int SETS = kStep / SUB / CI;         // of a step
  static constexpr int DBUFS = kDCols / (CI * NTOK);    // sets in TMEM
  static constexpr int COLS = NTOK / kWG;               // tokens of an adding thread
  static constexpr int XBYTES = NTOK * kStep * 2;       // a step's token values
  static constexpr int XBUFS = NTOK >= 128 ? 2 : 4;
  static constexpr int CBUFS = NTOK >= 128 ? 4 : NTOK == 64 ? 4 : 8;
  static constexpr int X_OFF = CBUFS * kCodeBox;
  static constexpr int P_OFF = X_OFF + XBUFS * XBYTES;  // scales, then zero points
  static constexpr int PBYTES = kBlock * kTileRows * 4;
  static constexpr int BAR_OFF = P_OFF + 4 * PBYTES;
  static constexpr int BARS = 2 * CBUFS + 2 * XBUFS + kABufs + 2 * DBUFS + 4 + 1;
  static constexpr int SMEM = BAR_OFF + BARS * 8 + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(NTOK * kTileRows * 4 <= P_OFF, "the split sums reuse the rings");
};

struct TcPlan {
  int tiles;     // of 128 outputs
  int split;     // CTAs of a cluster that share a tile's inputs
  int steps;     // of a row
  int per;       // steps of one split, a multiple of what a block of scales covers
  uint32_t mask, magic;
};

template <int G, bool ZEROS, int NTOK>
__global__ void __launch_bounds__(kTcThreads, 1)
w4_tc_kernel(const W4Args a, const TcPlan p, const __grid_constant__ CUtensorMap cmap,
             const __grid_constant__ CUtensorMap xmap) {
  using Cf = TcCfg<G, NTOK>;
  constexpr int NG = kStep / G;             // groups of a step
  constexpr int CB = kBlock / NG;           // steps of a block of scales
  extern __shared__ __align__(1024) uint8_t sm[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if ((smem_u32(sm) & 1023u) != 0) {
    if (threadIdx.x == 0 && a.status) atomicCAS(a.status, 0, (int)M3_ERR_CUDA);
    return;
  }
  float* s_scale = reinterpret_cast<float*>(sm + Cf::P_OFF);                         // [2][8][128]
  uint32_t* s_zero = reinterpret_cast<uint32_t*>(sm + Cf::P_OFF + 2 * Cf::PBYTES);  // [2][8][128]
  uint64_t* c_full = reinterpret_cast<uint64_t*>(sm + Cf::BAR_OFF);
  uint64_t* c_empty = c_full + Cf::CBUFS;
  uint64_t* x_full = c_empty + Cf::CBUFS;
  uint64_t* a_full = x_full + Cf::XBUFS;
  uint64_t* s_done = a_full + kABufs;       // a step's MMAs: its weights and token values are free
  uint64_t* d_full = s_done + Cf::XBUFS;
  uint64_t* d_empty = d_full + Cf::DBUFS;
  uint64_t* p_full = d_empty + Cf::DBUFS;   // blocks of scales
  uint64_t* p_empty = p_full + 2;
  uint64_t* s_fin = p_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_fin + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cf::CBUFS; ++i) { mbar_init(&c_full[i], 1); mbar_init(&c_empty[i], kWorkers); }
    for (int i = 0; i < Cf::XBUFS; ++i) { mbar_init(&x_full[i], 1); mbar_init(&s_done[i], 1); }
    for (int i = 0; i < kABufs; ++i) mbar_init(&a_full[i], 32 * kWorkers);
    for (int i = 0; i < Cf::DBUFS; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 32 * kWorkers); }
    for (int i = 0; i < 2; ++i) { mbar_init(&p_full[i], 64); mbar_init(&p_empty[i], ZEROS ? 2 * kWorkers : kWorkers); }
    mbar_init(s_fin, 1);
    fence_mbar_init();
  }
  if (warp == 2 * kWorkers + 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *s_tmem;                        // A buffers, then the groups' sums
  const uint32_t td = tm + kABufs * kACols;

  const int m0 = (int)blockIdx.y * NTOK;
  const int rank = (int)blockIdx.x % p.split;         // of the cluster: its part of the inputs
  const int tile0 = (int)blockIdx.x / p.split, tstep = (int)gridDim.x / p.split;
  const int c0 = rank * p.per;
  const int c1 = c0 + p.per < p.steps ? c0 + p.per : p.steps;
  const int nc = c1 - c0;                             // steps of this CTA, in every tile
  bool ok = true;

  float* red = reinterpret_cast<float*>(sm);          // [NTOK][128], over the idle rings
  if (warp < kWorkers) {
    // ---- decoders: codes to bf16 weights in TMEM ------------------------------------
    const int q = warp & 3, wg = warp >> 2;
    const int r = 32 * q + lane;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const uint32_t magic = in_register(p.magic);
    constexpr int WORDS = 32 / kWG;                   // of a row's step, a thread's part
    Turn code, at, done;                              // done: two steps behind
    uint32_t it = 0, blk = 0;                                 // blocks of scales so far
    for (int tile = tile0; tile < p.tiles && ok; tile += tstep) {
      for (int c = 0; c < nc; ++c) {
        if (ZEROS && c % CB == 0) ok = w4_wait(&p_full[blk & 1u], (blk >> 1) & 1u, a.status);
        ok = ok && w4_wait(&c_full[code.slot], code.phase, a.status);
        if (it >= kABufs) {
          ok = ok && w4_wait(&s_done[done.slot], done.phase, a.status);
          done.next(Cf::XBUFS);
        }
        ++it;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint8_t* row = sm + code.slot * kCodeBox + r * 128;
        uint32_t w[WORDS];
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
          const int piece = wg * (WORDS / 4) + i;
          const uint4 v = *reinterpret_cast<const uint4*>(row + ((piece ^ (r & 7)) << 4));
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        const uint32_t* zs = s_zero + ((blk & 1u) * kBlock + (c % CB) * NG) * kTileRows + r;
        const uint32_t acol = tm + lane_base + at.slot * kACols + wg * (4 * WORDS);
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
          const uint32_t z = ZEROS ? zs[((wg * WORDS + i) * 8 / G) * kTileRows] : 0x43084308u;
          uint32_t f[16];  // four words' codes in order: the pairs of one byte's halves
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t odd = w[i + j] >> 4;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[4 * j + e] = sub_bf16x2(
                  and_or(__byte_perm(w[i + j], odd, 0x4400u + 0x1111u * e), p.mask, magic), z);
          }
          tmem_st16(acol + i * 4, f);
        }
        tmem_st_wait();
        tc_fence_before();
        bar_arrive(&a_full[at.slot]);
        at.next(kABufs);
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&c_empty[code.slot]);
          if (ZEROS && (c % CB == CB - 1 || c + 1 == nc)) bar_arrive(&p_empty[blk & 1u]);
        }
        if (c % CB == CB - 1 || c + 1 == nc) ++blk;
        code.next(Cf::CBUFS);
      }
    }
  } else if (warp < 2 * kWorkers) {
    // ---- adders: the groups' sums out of TMEM, times their scales -------------------
    const int q = warp & 3, wg = (warp - kWorkers) >> 2;
    const int r = 32 * q + lane;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    Turn dt;
    uint32_t blk = 0;
    float acc[Cf::COLS];
#pragma unroll
    for (int i = 0; i < Cf::COLS; ++i) acc[i] = 0.f;
    for (int tile = tile0; tile < p.tiles && ok; tile += tstep) {
      for (int c = 0; c < nc; ++c) {
        if (c % CB == 0) ok = w4_wait(&p_full[blk & 1u], (blk >> 1) & 1u, a.status);
        const float* sc = s_scale + ((blk & 1u) * kBlock + (c % CB) * NG) * kTileRows + r;
#pragma unroll
        for (int g = 0; g < Cf::SETS; ++g) {
          float sv[Cf::CI];
#pragma unroll
          for (int h = 0; h < Cf::CI; ++h) sv[h] = sc[((g * Cf::CI + h) * Cf::SUB / G) * kTileRows];
          ok = __all_sync(0xffffffffu, ok && w4_wait(&d_full[dt.slot], dt.phase, a.status));
          if (!ok) break;
          tc_fence_after();
          const uint32_t dcol = td + lane_base + dt.slot * (Cf::CI * NTOK) + wg * Cf::COLS;
          constexpr int LD = Cf::COLS == 16 ? 16 : 8;  // few registers beside 64 sums
#pragma unroll
          for (int i = 0; i < Cf::COLS; i += LD) {
#pragma unroll
            for (int h = 0; h < Cf::CI; h += 2) {
              uint32_t v[2][LD];
              tmem_ld<LD>(dcol + h * NTOK + i, v[0]);
              if (h + 1 < Cf::CI) tmem_ld<LD>(dcol + (h + 1) * NTOK + i, v[1]);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < LD; ++j) acc[i + j] = fmaf(sv[h], __uint_as_float(v[0][j]), acc[i + j]);
              if (h + 1 < Cf::CI) {
#pragma unroll
                for (int j = 0; j < LD; ++j)
                  acc[i + j] = fmaf(sv[h + 1 < Cf::CI ? h + 1 : h], __uint_as_float(v[1][j]), acc[i + j]);
              }
            }
          }
          tc_fence_before();
          bar_arrive(&d_empty[dt.slot]);
          dt.next(Cf::DBUFS);
        }
        if (!ok) break;
        if (c % CB == CB - 1 || c + 1 == nc) {
          __syncwarp();
          if (lane == 0) bar_arrive(&p_empty[blk & 1u]);
          ++blk;
        }
      }
      if (ok && p.split == 1) {
        const int64_t n = (int64_t)tile * kTileRows + r;
        if (n < a.N) {
          const float b = a.bias ? __ldg(a.bias + n) : 0.f;
          const int left = (int)(a.M - m0) - wg * Cf::COLS;  // tokens from here
          const int64_t at = (int64_t)(m0 + wg * Cf::COLS) * a.N + n;
          if (a.out_f32) {
            float* o = static_cast<float*>(a.out) + at;
#pragma unroll
            for (int i = 0; i < Cf::COLS; ++i, o += a.N)
              if (i < left && M3_IN(at + i * a.N, a.M * a.N, a.status)) *o = acc[i] + b;
          } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
            for (int i = 0; i < Cf::COLS; ++i, o += a.N)
              if (i < left && M3_IN(at + i * a.N, a.M * a.N, a.status)) *o = __float2bfloat16_rn(acc[i] + b);
          }
        }
#pragma unroll
        for (int i = 0; i < Cf::COLS; ++i) acc[i] = 0.f;
      }
    }
    if (p.split > 1) {  // one tile: its last sum is in, so the rings are idle
#pragma unroll
      for (int i = 0; i < Cf::COLS; ++i) red[(wg * Cf::COLS + i) * kTileRows + r] = acc[i];
    }
  } else if (warp >= 2 * kWorkers + 2) {
    // ---- stagers: scales and zero points, a block of groups at a time ----------------
    const int i0 = threadIdx.x - 32 * (2 * kWorkers + 2);  // 0..63: rows i0 and i0 + 64 of a tile
    const int kg = (int)(a.K / G);
    uint32_t blk = 0;
    for (int tile = tile0; tile < p.tiles && ok; tile += tstep) {
      for (int c = 0; c < nc; c += CB, ++blk) {
        const uint32_t slot = blk & 1u;
        const int g0 = (c0 + c) * NG;  // first group
        uint32_t sw[2][kBlock / 2] = {}, zw[2][2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t row = (int64_t)tile * kTileRows + i0 + 64 * h;
          const int left = row < a.N ? kg - g0 : 0;
          const uint16_t* sp = static_cast<const uint16_t*>(a.scales) + row * kg + g0;
          const uint8_t* zp = a.zeros + row * kg + g0;
          if (left >= kBlock && kg % kBlock == 0) {  // g0 is a multiple of a block
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp));
            sw[h][0] = v.x; sw[h][1] = v.y; sw[h][2] = v.z; sw[h][3] = v.w;
            if constexpr (ZEROS) {
              const uint2 z = __ldg(reinterpret_cast<const uint2*>(zp));
              zw[h][0] = z.x; zw[h][1] = z.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
              if (j >= left) continue;
              sw[h][j / 2] |= (uint32_t)__ldg(sp + j) << (16 * (j & 1));
              if constexpr (ZEROS) zw[h][j / 4] |= (uint32_t)__ldg(zp + j) << (8 * (j & 3));
            }
          }
        }
        ok = w4_wait(&p_empty[slot], ((blk >> 1) & 1u) ^ 1u, a.status);
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < kBlock; ++j) {
            const int at = (slot * kBlock + j) * kTileRows + i0 + 64 * h;
            s_scale[at] = __uint_as_float((j & 1) ? sw[h][j / 2] & 0xffff0000u : sw[h][j / 2] << 16);
            if constexpr (ZEROS)
              s_zero[at] = 0x43004300u + ((zw[h][j / 4] >> (8 * (j & 3))) & 15u) * 0x00010001u;
          }
        }
        bar_arrive(&p_full[slot]);
      }
    }
  } else if (warp == 2 * kWorkers) {
    // ---- TMA ------------------------------------------------------------------------
    Turn code, xt;
    uint32_t nx = 0, ncode = 0;
    for (int tile = tile0; tile < p.tiles && ok; tile += tstep) {
      for (int c = 0; c < nc && ok; ++c) {
        ok = w4_wait_all(&c_empty[code.slot], code.phase ^ 1u, a.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_expect_tx(&c_full[code.slot], kCodeBox);
          tma_box(sm + code.slot * kCodeBox, &cmap, (c0 + c) * (kStep / 2), tile * kTileRows,
                  &c_full[code.slot]);
        }
        __syncwarp();
        code.next(Cf::CBUFS);
        ++ncode;
        ok = w4_wait_all(&s_done[xt.slot], xt.phase ^ 1u, a.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_expect_tx(&x_full[xt.slot], Cf::XBYTES);
          uint8_t* xs = sm + Cf::X_OFF + xt.slot * Cf::XBYTES;
#pragma unroll
          for (int i = 0; i < kStep / 64; ++i)
            tma_box(xs + i * NTOK * 128, &xmap, (c0 + c) * kStep + i * 64, m0, &x_full[xt.slot]);
        }
        __syncwarp();
        xt.next(Cf::XBUFS);
        ++nx;
      }
    }
    // the last copies have landed (bounded) before the block can exit
    for (uint32_t k = ncode > Cf::CBUFS ? ncode - Cf::CBUFS : 0; k < ncode; ++k)
      w4_wait(&c_full[k % Cf::CBUFS], (k / Cf::CBUFS) & 1u, a.status);
    for (uint32_t k = nx > Cf::XBUFS ? nx - Cf::XBUFS : 0; k < nx; ++k)
      w4_wait(&x_full[k % Cf::XBUFS], (k / Cf::XBUFS) & 1u, a.status);
  } else if (warp == 2 * kWorkers + 1) {
    // ---- MMA issue: the sums of a set in turn, so that none waits on the last; the
    // whole warp keeps step and one lane issues (descriptors in uniform registers) -------
    constexpr uint32_t idesc = idesc_bf16(kTileRows, NTOK, 0, 0);
    const uint64_t x0 = sw128_desc(smem_u32(sm) + Cf::X_OFF, 16, 1024);
    Turn at, xt, dt;
    for (int tile = tile0; tile < p.tiles && ok; tile += tstep) {
      for (int c = 0; c < nc && ok; ++c) {
        // three lanes wait at once
        uint64_t* bar = lane == 0 ? &x_full[xt.slot] : lane == 1 ? &a_full[at.slot] : &d_empty[dt.slot];
        const uint32_t ph = lane == 0 ? xt.phase : lane == 1 ? at.phase : dt.phase ^ 1u;
        if (lane < 3) ok = w4_wait(bar, ph, a.status);
        ok = __all_sync(0xffffffffu, ok);
        const uint64_t xd = x0 + xt.slot * (Cf::XBYTES >> 4);
        const uint32_t acol = tm + at.slot * kACols;
#pragma unroll
        for (int g = 0; g < Cf::SETS; ++g) {
          if (g > 0) ok = w4_wait_all(&d_empty[dt.slot], dt.phase ^ 1u, a.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < Cf::SUB / 16; ++k) {
#pragma unroll
              for (int h = 0; h < Cf::CI; ++h) {
                const int ks = (g * Cf::CI + h) * (Cf::SUB / 16) + k;  // of the step's sixteen
                mma_bf16_ts(td + (dt.slot * Cf::CI + h) * NTOK, acol + ks * 8,
                            xd + (uint64_t)((ks / 4) * NTOK * 8 + (ks % 4) * 2), idesc, k > 0);
              }
            }
            mma_commit(&d_full[dt.slot]);
            if (g == Cf::SETS - 1) mma_commit(&s_done[xt.slot]);
          }
          __syncwarp();
          dt.next(Cf::DBUFS);
        }
        at.next(kABufs);
        xt.next(Cf::XBUFS);
      }
    }
  }

  // every MMA issued has completed before TMEM is released (bounded)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2 * kWorkers + 1) {
    if (elect_one()) mma_commit(s_fin);
    __syncwarp();
    w4_wait(s_fin, 0, a.status);
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
  if (p.split == 1) return;

  // ---- split inputs: the cluster's sums, added in rank order -------------------------
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
  {
    const int mine = NTOK / p.split;  // tokens this CTA adds, four outputs at a time
    for (int i = threadIdx.x; i < mine * (kTileRows / 4); i += kTcThreads) {
      const int t = rank * mine + i / (kTileRows / 4), r = i % (kTileRows / 4) * 4;
      const int64_t m = m0 + t, n = (int64_t)tile0 * kTileRows + r;
      if (m >= a.M || n >= a.N) continue;
      const uint32_t local = smem_u32(red + t * kTileRows + r);
      float f[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= p.split) break;
        uint32_t remote;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(k));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f[k][0]), "=f"(f[k][1]), "=f"(f[k][2]), "=f"(f[k][3])
                     : "r"(remote));
      }
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = f[0][j];
#pragma unroll
        for (int k = 1; k < 8; ++k)
          if (k < p.split) v[j] += f[k][j];
      }
      store_outputs(a, m, n, make_float4(v[0], v[1], v[2], v[3]));
    }
  }
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

bool encode_tokens(CUtensorMap* m, const W4Args& a, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.M};
  const cuuint64_t strides[1] = {(cuuint64_t)a.K * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.A), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, bool ZEROS, int NTOK>
cudaError_t launch_tc(const W4Args& a, cudaStream_t s) {
  using Cf = TcCfg<G, NTOK>;
  TcPlan p;
  p.tiles = (int)((a.N + kTileRows - 1) / kTileRows);
  p.steps = (int)((a.K + kStep - 1) / kStep);
  p.mask = 0x000f000fu;
  p.magic = 0x43004300u;
  // splits of the inputs, of whole blocks of scales each
  constexpr int unit = kBlock * G / kStep;  // steps of a block: 1, 2 or 4
  const int64_t token_tiles = (a.M + NTOK - 1) / NTOK;
  p.split = 1;
  while (p.split < 8 && (int64_t)p.tiles * token_tiles * p.split * 2 <= kPlanSms &&
         p.steps > unit * p.split)
    p.split *= 2;
  p.per = (p.steps + p.split - 1) / p.split;
  p.per = (p.per + unit - 1) / unit * unit;
  CUtensorMap cmap, xmap;
  memset(&cmap, 0, sizeof(cmap));
  memset(&xmap, 0, sizeof(xmap));
  if (!encode_codes(&cmap, a, kTileRows) || !encode_tokens(&xmap, a, NTOK))
    return cudaErrorInvalidValue;
  auto kern = w4_tc_kernel<G, ZEROS, NTOK>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  // with a split every cluster has one tile: its sums meet once, at the end
  const int64_t ctas = p.split > 1 ? (int64_t)p.tiles * p.split : p.tiles < sms ? p.tiles : sms;
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)token_tiles);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = Cf::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, p, cmap, xmap);
}

// Up to 16 tokens the mma.sync form: the tcgen05 one pays the same for any few
// tokens (50257 x 2048, groups of 128, one token: 22 us against 17.3; 16 tokens:
// 25.6 against 25.0; 32 tokens: 25.7 against 47).
//
// Above 64 tokens, tiles of 128 or several of 64, which decode the weights again.
// Tiles of 64 where groups are of 32 (their sums wait for TMEM columns, of which 128
// tokens leave two sets: 128 x 8192 x 4096 28.3 us against 34.9), or where even with
// them the SMs are not filled twice (300 x 500 x 1024 8.9 us against 13.5).  Else
// tiles of 128 (512 x 8192 x 4096, groups of 128, 55 us against 79; of 64, 67
// against 83).
template <int G, bool ZEROS>
cudaError_t launch_m(const W4Args& a, cudaStream_t s) {
  if (a.M <= 16) return launch_z<G, ZEROS>(a, s);
  if (a.M <= 32) return launch_tc<G, ZEROS, 32>(a, s);
  if (a.M <= 64) return launch_tc<G, ZEROS, 64>(a, s);
  if constexpr (G > 32) {
    const int64_t tiles = ((a.N + kTileRows - 1) / kTileRows) * ((a.M + 63) / 64);
    if (2 * tiles > kPlanSms) return launch_tc<G, ZEROS, 128>(a, s);
  }
  return launch_tc<G, ZEROS, 64>(a, s);
}

template <int G>
cudaError_t launch_g(const W4Args& a, cudaStream_t s) {
  return a.zeros ? launch_m<G, true>(a, s) : launch_m<G, false>(a, s);
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

cudaError_t w4_launch(const W4Args& all, cudaStream_t s) {
  // tiles of tokens are a grid's second dimension, which ends at 65535
  constexpr int64_t most = (int64_t)1 << 20;
  cudaError_t e = cudaSuccess;
  for (int64_t m = 0; m < all.M && e == cudaSuccess; m += most) {
    W4Args a = all;
    a.M = all.M - m < most ? all.M - m : most;
    a.A = static_cast<const char*>(all.A) + m * all.K * 2;
    a.out = static_cast<char*>(all.out) + m * all.N * (all.out_f32 ? 4 : 2);
    e = a.group == 32 ? launch_g<32>(a, s) : a.group == 64 ? launch_g<64>(a, s) : launch_g<128>(a, s);
  }
  return e;
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
