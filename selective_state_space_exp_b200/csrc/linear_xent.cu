// linear_xent.cu -- softmax cross entropy of a head over a large vocabulary, from
// the hidden states and the head's weights; the logits are never kept.
//
//   l_tv = sum_k h_tk W_vk,   lse_t = log sum_v exp l_tv,
//   loss_t = lse_t - l_{t,y_t}   (0 where y_t is the ignored target)
//   d_tv = (exp(l_tv - lse_t) - [v = y_t]) dloss_t
//   dh_tk = sum_v d_tv W_vk,   dW_vk = sum_t d_tv h_tk
//
// Everything is a matrix product on the tensor cores with an epilogue:
//   stats    l tiles of 128 tokens x 256 classes; each tile leaves a running
//            maximum and sum of exponentials per token (one pass over the
//            accumulator) and the target's logit; a small kernel joins them.
//   dlogits  the same tiles again for one piece of the vocabulary, the
//            epilogue turning them into d / c, rounded to bf16 (the operand type
//            of the next two products; sums stay fp32).  c is the largest
//            |dloss|: with the usual equal dloss the targets' entries, which
//            carry most of the gradient, are then p - 1, whose roundings differ
//            from token to token, and not all the one rounding of dloss.
//   grads    dW of the piece (reduction over tokens: both operands are read
//            with the reduction as their outer dimension, MN-major) and the
//            piece's share of dh (W MN-major), accumulated over the pieces in
//            fp32 and rounded once.
// The piece is chosen so that its d fits a fixed workspace.  Bound by the tensor
// cores at training sizes: 2 M V K forward, 6 M V K backward (2 of them the
// recomputed logits).  Where there are too few output tiles to fill the SMs the
// reduction is split, the partial sums being added in a fixed order.
//
// Measured at 2048 tokens, 32000 classes, width 2048 (268 GFLOP a product), each alone:
// stats 167 us, dlogits 170, dW 174, dh 182 (1.47 to 1.61 PFLOP/s, the tensor pipe 92 to
// 96 % active; a GPU at a higher clock took 148 for stats); back to back the power limit
// makes it 845 us in all.  16384 tokens, 50257 classes: 10.6 to 10.9 ms, 1.24 to 1.27
// PFLOP/s.  4096 tokens, 32768 classes, width 1024, forward alone: 214 to 219 us, where a
// tile's exponentials outlast half its products.
//
// The tensor cores truncate addends as they align them to an fp32 accumulator: loss and
// lse are good to about 2.5e-6 of their value at widths of 2700 and more.
//
// Kernel: persistent, one CTA per SM, warp-specialised: warp 0 streams operand
// tiles by TMA (128-byte swizzle) through a ring of stages, one lane of warp 1
// issues tcgen05.mma into two TMEM accumulators in turn, warps 2-9 run the
// epilogue of the other one.  Every wait is bounded (M3_ERR_TIMEOUT).
#include <cuda.h>  // CUtensorMap

#include <cstring>

#include "lm_ops.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

using namespace tc;

constexpr int kBM = 128, kBK = 64;       // a CTA's rows of a tile, reduction step
constexpr int kWide = 256, kMiddle = 128, kNarrow = 64;  // columns of a tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBlk = 64 * kBK * 2;  // an MN-major block: 64 columns x 64 reduction rows

// CG: CTAs that share a tile of CG * 128 rows (a pair's tensor cores work on one
// tile, each CTA holding its own rows of A and half the columns of B, which
// halves what the pair reads of B).
template <int CG, int BN>
struct Cfg {
  static constexpr int A_BYTES = kBM * kBK * 2;
  static constexpr int B_COLS = BN / CG;
  static constexpr int TMEM = 2 * BN;  // columns of two accumulators
  static constexpr int STAGE = A_BYTES + B_COLS * kBK * 2;
  static constexpr int STAGES = BN == kNarrow ? 8 : BN == kMiddle || CG == 2 ? 6 : 4;
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int SMEM = BAR_OFF + (2 * STAGES + 5) * 8 + 16;
  static_assert(SMEM + 1024 <= 232448, "shared memory");
};

constexpr int kGroupRows = 2048;  // rows that share a column tile while it is in L2
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kStats = 0, kDlogits = 1, kGrad = 2 };

struct GemmArgs {
  int64_t M, N;           // extent of the output
  int kb, kb_per;         // reduction blocks in all, and of one split
  int cg, bn;             // CTAs of a tile, its columns
  int mt, nt, splits;     // tiles
  int a_rows;             // of A that a stage loads: fewer than kBM where M is smaller
  bool dependent;         // not the call's first kernel
  int* status;
  // stats, dlogits: rows are tokens, columns classes v0 + n
  const int64_t* targets;
  int64_t ignore, V, v0;
  float2* stat;           // [2 nt][M]: maximum (base 2) and sum, per half tile
  float* tlogit;          // [M]
  const float* lse;
  const float* dloss;
  __nv_bfloat16* d;       // [M][ldd]
  int64_t ldd;
  const __nv_bfloat16* h; // [M][K], copied by the first piece's dlogits
  __nv_bfloat16* scored;  // to here with zeros for the tokens that are not scored, or nullptr
  int64_t K;
  float* unit;            // c: written by the first piece's dlogits, a factor of out in grads
  // grads
  float* acc;             // [splits][M][N] partial sums or running sum
  __nv_bfloat16* out;     // [M][N], written when set
  bool add;               // acc holds an earlier sum
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Maps {
  CUtensorMap a, b;
};

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// The clock is read now and then only: its value takes longer than most waits.
__device__ bool wait(uint64_t* bar, uint32_t parity, int* status) {
  unsigned long long t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if (i % 64 != 0) continue;
    const unsigned long long t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitNs) {
      if (status) atomicCAS(status, 0, (int)M3_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// By a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, wait(bar, parity, status));
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tma_2d(void* dst, const void* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Pair forms (CTA group 2): both CTAs' loads complete on the first one's barrier,
// whose thread issues the MMAs of both; a commit reaches the barriers of both.
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void tma_2d_pair(void* dst, const void* map, int c0, int c1,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1) {
    mma_bf16_ss(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
  }
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG, int COLS>
__device__ __forceinline__ void alloc(uint32_t* holder) {
  if constexpr (CG == 1) {
    tmem_alloc(holder, COLS);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(holder)),
                 "r"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG, int COLS>
__device__ __forceinline__ void dealloc(uint32_t taddr) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, COLS);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(COLS)
                 : "memory");
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

struct Tile {
  int m, n, split;
};

// Tiles of one split first; inside it bands of kGroupRows rows, down each column
// of a band before the next column: the CTAs running at one time share a few row
// and column tiles, which stay in L2.
template <int CG>
__device__ __forceinline__ Tile tile_of(const GemmArgs& g, int64_t t) {
  constexpr int kGroupM = kGroupRows / (CG * kBM);
  const int64_t per = (int64_t)g.mt * g.nt;
  Tile o;
  o.split = (int)(t / per);
  const int64_t r = t % per;
  const int64_t band = r / ((int64_t)kGroupM * g.nt);
  const int64_t q = r % ((int64_t)kGroupM * g.nt);
  const int rows = g.mt - (int)band * kGroupM < kGroupM ? g.mt - (int)band * kGroupM : kGroupM;
  o.n = (int)(q / rows);
  o.m = (int)band * kGroupM + (int)(q % rows);
  return o;
}

// Operand tiles of one stage: K-major [rows][64] as one box; MN-major as blocks
// of 64 columns, each 64 reduction rows of 128 bytes.  bar: a shared::cluster
// address.
template <int CG, bool MN, int ROWS>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, int row0, int k0,
                                             uint64_t* own, uint32_t bar) {
  auto load = [&](uint8_t* d, int c0, int c1) {
    if constexpr (CG == 1) tma_2d(d, map, c0, c1, own);
    else tma_2d_pair(d, map, c0, c1, bar);
  };
  if constexpr (MN) {
#pragma unroll
    for (int i = 0; i < ROWS / 64; ++i) load(dst + i * kBlk, row0 + i * 64, k0);
  } else {
    load(dst, k0, row0);
  }
}

// The largest |dloss| of a scored token, or 1 where that is no positive finite
// number; every epilogue thread takes part and gets it.
__device__ __forceinline__ float largest_dloss(const GemmArgs& g, float* s_max) {
  const int i = threadIdx.x - 64;
  float c = 0.f;
#pragma unroll 4
  for (int64_t m = i; m < g.M; m += 32 * kEpiWarps) {
    const int64_t t = g.targets[m];
    if (t != g.ignore && t >= 0 && t < g.V) c = fmaxf(c, fabsf(g.dloss[m]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
  if ((i & 31) == 0) s_max[i >> 5] = c;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
  c = s_max[0];
#pragma unroll
  for (int w = 1; w < kEpiWarps; ++w) c = fmaxf(c, s_max[w]);
  return c > 0.f && c < INFINITY ? c : 1.f;
}

// Lane j of four gets the others' w[j]: w[i] becomes lane i's w[j].  A lane has a
// row of an accumulator; with its pieces stored as they are, a store touches 32 rows
// by 16 bytes each, after the exchange 8 rows by 64: the backward of 4096 x 32768 x
// 1024 took 685 us before and 580 us after, of 300 x 50257 x 1024 197 and 148 us.
__device__ __forceinline__ void turn4(uint4 (&w)[4], int lane) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & o) continue;
      uint4 &a = w[i], &b = w[i | o];
      const uint4 give = up ? a : b;
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, o), __shfl_xor_sync(0xffffffffu, give.y, o),
                                   __shfl_xor_sync(0xffffffffu, give.z, o), __shfl_xor_sync(0xffffffffu, give.w, o));
      if (up) a = got;
      else b = got;
    }
  }
}

// The hidden states that dW = d^T h is taken from: d is 0 in a token that is not
// scored, but 0 times a NaN or an infinity that stands there (padding) is not.
// Done by the warps that wait for the first tile: 2 M K bytes read and written.
__device__ __forceinline__ void copy_scored(const GemmArgs& g) {
  const int warp = (threadIdx.x - 64) >> 5, lane = threadIdx.x & 31;
  const int nvec = (int)(g.K / 8);
  for (int64_t m = (int64_t)blockIdx.x * kEpiWarps + warp; m < g.M; m += (int64_t)gridDim.x * kEpiWarps) {
    const int64_t t = g.targets[m];
    const bool live = t != g.ignore && t >= 0 && t < g.V;
    const uint4* from = reinterpret_cast<const uint4*>(g.h + m * g.K);
    uint4* to = reinterpret_cast<uint4*>(g.scored + m * g.K);
#pragma unroll 4
    for (int v = lane; v < nvec; v += 32) {
      const uint4 x = from[v];  // does not wait for the target
      if (M3_IN(m * g.K + 8 * v + 7, g.M * g.K, g.status)) to[v] = live ? x : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int MODE, int BN>
__device__ __forceinline__ void epilogue(const GemmArgs& g, const Tile& t, int64_t row0,
                                         uint32_t tcol, int q, int half, int lane, float unit) {
  const int64_t m = row0 + 32 * q + lane;
  const int64_t n0 = (int64_t)t.n * BN + half * (BN / 2);
  const bool on = m < g.M;
  if constexpr (MODE == kStats) {
    int64_t tgt = -1;
    if (on) tgt = g.targets[m];
    const int64_t rel = tgt - n0;  // the target's column in this half tile
    float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += 32) {
      uint32_t v[32];
      tmem_ld32(tcol + (uint32_t)c, v);
      tmem_ld_wait();
      float f[32];
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        f[e] = n0 + c + e < g.V ? __uint_as_float(v[e]) : -INFINITY;
        top = fmaxf(top, f[e]);
      }
      if (on && rel >= c && rel < c + 32 && tgt < g.V && tgt != g.ignore) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (rel == c + e) g.tlogit[m] = f[e];
      }
      const float nm = fmaxf(mx, top * kLog2e);
      if (nm > -INFINITY) {
        sum = sum * ex2(mx - nm);
#pragma unroll
        for (int e = 0; e < 32; ++e) sum += ex2(fmaf(f[e], kLog2e, -nm));
        mx = nm;
      } else {  // -infinity or NaN only
#pragma unroll
        for (int e = 0; e < 32; ++e) sum += f[e] > -INFINITY || f[e] != f[e] ? f[e] : 0.f;
      }
    }
    if (on && M3_IN((int64_t)(2 * t.n + half) * g.M + m, (int64_t)2 * g.nt * g.M, g.status))
      g.stat[(int64_t)(2 * t.n + half) * g.M + m] = make_float2(mx, sum);
  } else if constexpr (MODE == kDlogits) {
    int64_t tgt = -1;
    float scale = 0.f, off = 0.f;
    bool live = false;
    if (on) {
      tgt = g.targets[m];
      live = tgt != g.ignore && tgt >= 0 && tgt < g.V;
      if (live) {
        scale = __fdiv_rn(g.dloss[m], unit);
        off = g.lse[m] * kLog2e;
      }
    }
    const int64_t rel = tgt - g.v0 - n0;
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += 32) {
      uint32_t v[32];
      tmem_ld32(tcol + (uint32_t)c, v);
      tmem_ld_wait();
      float f[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float p = ex2(fmaf(__uint_as_float(v[e]), kLog2e, -off));
        if (rel == c + e) p -= 1.f;
        f[e] = live ? p * scale : 0.f;
      }
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = make_uint4(pack_bf16(f[8 * i], f[8 * i + 1]), pack_bf16(f[8 * i + 2], f[8 * i + 3]),
                          pack_bf16(f[8 * i + 4], f[8 * i + 5]), pack_bf16(f[8 * i + 6], f[8 * i + 7]));
      // four lanes turn their rows' pieces about, so that a store writes 64 bytes of a row
      turn4(w, lane);
      const int64_t n = n0 + c + 8 * (lane & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = m - (lane & 3) + i;
        if (row < g.M && n < g.ldd && M3_IN(row * g.ldd + n + 7, g.M * g.ldd, g.status))
          *reinterpret_cast<uint4*>(g.d + row * g.ldd + n) = w[i];
      }
    }
  } else {
    // as above: after the exchange a lane holds its piece of four rows
    const int64_t first = m - (lane & 3);
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += 32) {
      uint32_t v[32];
      tmem_ld32(tcol + (uint32_t)c, v);
      tmem_ld_wait();
      if (!g.acc) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * i + e]) * unit;
          w[i] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                            pack_bf16(f[6], f[7]));
        }
        turn4(w, lane);
        const int64_t n = n0 + c + 8 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // N is a multiple of 8
          if (first + i < g.M && n < g.N && M3_IN((first + i) * g.N + n + 7, g.M * g.N, g.status))
            *reinterpret_cast<uint4*>(g.out + (first + i) * g.N + n) = w[i];
        continue;
      }
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = make_uint4(v[h + 4 * i], v[h + 4 * i + 1], v[h + 4 * i + 2], v[h + 4 * i + 3]);
        turn4(w, lane);
        const int64_t n = n0 + c + h + 4 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (first + i >= g.M || n >= g.N || !M3_IN((first + i) * g.N + n + 3, g.M * g.N, g.status)) continue;
          float4* acc = reinterpret_cast<float4*>(g.acc + ((int64_t)t.split * g.M + first + i) * g.N + n);
          float4 f = make_float4(__uint_as_float(w[i].x), __uint_as_float(w[i].y), __uint_as_float(w[i].z),
                                 __uint_as_float(w[i].w));
          if (g.add) {
            const float4 x = *acc;
            f.x += x.x; f.y += x.y; f.z += x.z; f.w += x.w;
          }
          if (g.out)
            *reinterpret_cast<uint2*>(g.out + (first + i) * g.N + n) =
                make_uint2(pack_bf16(f.x * unit, f.y * unit), pack_bf16(f.z * unit, f.w * unit));
          else
            *acc = f;
        }
      }
    }
  }
}

template <int CG, int BN, int MODE, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
xent_gemm_kernel(const GemmArgs g, const __grid_constant__ Maps maps) {
  using C = Cfg<CG, BN>;
  constexpr int kStages = C::STAGES;
  let_next_start();
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if ((sbase & 1023u) != 0) {  // the swizzled layout needs 1 KB alignment
    if (tid == 0 && g.status) atomicCAS(g.status, 0, (int)M3_ERR_CUDA);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* s_fin = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_fin + 1);
  const int64_t tiles = (int64_t)g.mt * g.nt * g.splits;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;  // a pair is two neighbouring blocks
  const int64_t first = blockIdx.x / CG, step = gridDim.x / CG;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * kEpiWarps);
    }
    mbar_init(s_fin, 1);
    fence_mbar_init();
  }
  if (CG == 2) {
    __syncthreads();
    pair_sync();  // the other CTA's barriers are ready
  }
  if (warp == 1) alloc<CG, C::TMEM>(s_tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *s_tmem;
  wait_for_previous();

  if (warp == 0) {
    const uint32_t bytes = (uint32_t)(CG * (g.a_rows * kBK * 2 + C::B_COLS * kBK * 2));
    uint32_t s = 0, phase = 0;
    int64_t loads = 0;
    bool ok = true;
    for (int64_t t = first; t < tiles && ok; t += step) {
      const Tile tl = tile_of<CG>(g, t);
      const int k0 = tl.split * g.kb_per, k1 = k0 + g.kb_per < g.kb ? k0 + g.kb_per : g.kb;
      const int arow = (tl.m * CG + rank) * kBM, brow = tl.n * BN + rank * C::B_COLS;
      for (int kb = k0; kb < k1; ++kb, ++loads) {
        if (!wait_all(&empty[s], phase ^ 1u, g.status)) { ok = false; break; }
        if (elect_one()) {
          uint8_t* st = sm + s * C::STAGE;
          const uint32_t bar = CG == 2 ? in_first_cta(&full[s]) : 0;
          if (rank == 0) mbar_expect_tx(&full[s], bytes);
          load_operand<CG, AMN, kBM>(st, &maps.a, arow, kb * kBK, &full[s], bar);
          load_operand<CG, BMN, C::B_COLS>(st + C::A_BYTES, &maps.b, brow, kb * kBK, &full[s], bar);
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // let the last stages' copies land (bounded) before the CTA can exit: the
    // first CTA's barriers see both CTAs' copies, the other CTA waits for the
    // MMAs that have read its own
    for (int64_t j = loads > kStages ? loads - kStages : 0; j < loads; ++j)
      wait(rank == 0 ? &full[j % kStages] : &empty[j % kStages], (uint32_t)(j / kStages) & 1u, g.status);
  } else if (warp == 1 && rank == 0) {
    // the whole warp keeps step and one lane issues: descriptors then live in
    // uniform registers, where a single lane's branch would move each operand of
    // each instruction there (a step of four MMAs: about 120 cycles against 283)
    constexpr uint32_t idesc = idesc_bf16(CG * kBM, BN, AMN, BMN);
    // K-major: 16 reduction columns are 32 bytes on; MN-major: 16 rows of 128 bytes
    const uint64_t a0 = sw128_desc(sbase, AMN ? kBlk : 16, 1024);
    const uint64_t b0 = sw128_desc(sbase + C::A_BYTES, BMN ? kBlk : 16, 1024);
    uint32_t s = 0, phase = 0;
    int j = 0;
    bool ok = true;
    for (int64_t t = first; t < tiles && ok; t += step, ++j) {
      const Tile tl = tile_of<CG>(g, t);
      const int k0 = tl.split * g.kb_per, k1 = k0 + g.kb_per < g.kb ? k0 + g.kb_per : g.kb;
      const int b = j & 1;
      if (!wait_all(&acc_empty[b], ((j >> 1) & 1) ^ 1u, g.status)) break;
      tc_fence_after();
      const uint32_t dcol = tm + (uint32_t)(b * BN);
      for (int kb = k0; kb < k1; ++kb) {
        if (!wait_all(&full[s], phase, g.status)) { ok = false; break; }
        tc_fence_after();
        const uint64_t ad = a0 + s * (C::STAGE >> 4), bd = b0 + s * (C::STAGE >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k4 = 0; k4 < kBK / 16; ++k4)
            mma<CG>(dcol, ad + (uint64_t)(k4 * (AMN ? 128 : 2)),
                    bd + (uint64_t)(k4 * (BMN ? 128 : 2)), idesc, kb > k0 || k4 > 0);
          commit<CG>(&empty[s]);
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (ok && elect_one()) commit<CG>(&acc_full[b]);
      __syncwarp();
    }
  } else if (warp >= 2) {
    const int q = warp & 3;  // TMEM lane quadrant this warp may access
    const int half = (warp - 2) >> 2;
    float unit = 1.f;
    if constexpr (MODE == kDlogits) {
      __shared__ float s_max[kEpiWarps];
      if (g.dependent) {  // a later piece
        unit = *g.unit;
      } else {
        unit = largest_dloss(g, s_max);
        if (blockIdx.x == 0 && tid == 64) *g.unit = unit;
        if (g.scored) copy_scored(g);
      }
    }
    if constexpr (MODE == kGrad) unit = *g.unit;
    int j = 0;
    for (int64_t t = first; t < tiles; t += step, ++j) {
      const int b = j & 1;
      if (!wait_all(&acc_full[b], (j >> 1) & 1u, g.status)) break;
      tc_fence_after();
      const Tile tl = tile_of<CG>(g, t);
      epilogue<MODE, BN>(g, tl, (int64_t)(tl.m * CG + rank) * kBM,
                     tm + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * BN + half * (BN / 2)), q,
                     half, lane, unit);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // the MMA thread's CTA learns it from both
        if constexpr (CG == 1) arrive(&acc_empty[b]);
        else arrive_at(in_first_cta(&acc_empty[b]));
      }
    }
  }

  // every MMA issued has completed before TMEM is released (bounded); of a pair each CTA
  // waits on its own barrier, so that the other's arrival does not reach a CTA that is gone
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (rank == 0 && elect_one()) commit<CG>(s_fin);
    __syncwarp();
    wait(s_fin, 0, g.status);
  }
  __syncwarp();
  if (CG == 2) pair_sync();
  if (warp == 1) dealloc<CG, C::TMEM>(tm);
}

// (maximum, sum) of the exponentials of two sets.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float nm = fmaxf(a.x, b.x);
  // both sets -infinity only: their sums hold 0 or NaN
  return nm > -INFINITY ? make_float2(nm, a.y * ex2(a.x - nm) + b.y * ex2(b.x - nm))
                        : make_float2(nm, a.y + b.y);
}

// Joins the tiles' maxima and sums of a token: kJoinTokens tokens a block, the
// other threads over the tiles.
constexpr int kJoinTokens = 8, kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
xent_join_kernel(const float2* stat, int parts, int64_t M, int64_t V, const int64_t* targets,
                 int64_t ignore, const float* tlogit, float* loss, float* lse, int* status) {
  constexpr int kRows = kJoinThreads / kJoinTokens;
  let_next_start();
  wait_for_previous();
  __shared__ float2 s[kRows][kJoinTokens];
  const int t = threadIdx.x % kJoinTokens, w = threadIdx.x / kJoinTokens;
  const int64_t m = (int64_t)blockIdx.x * kJoinTokens + t;
  float2 v = make_float2(-INFINITY, 0.f);
  if (m < M) {
#pragma unroll 4
    for (int p = w; p < parts; p += kRows) v = join(v, stat[(int64_t)p * M + m]);
  }
  s[w][t] = v;
  __syncthreads();
#pragma unroll
  for (int h = kRows / 2; h > 0; h >>= 1) {  // a tree of fixed order
    if (w < h) s[w][t] = join(s[w][t], s[w + h][t]);
    __syncthreads();
  }
  if (w != 0 || m >= M) return;
  v = s[0][t];
  const float z = (v.x + log2f(v.y)) * kLn2;
  if (lse) lse[m] = z;
  if (!loss) return;
  const int64_t y = targets[m];
  if (y == ignore) {
    loss[m] = 0.f;
  } else if (y < 0 || y >= V) {
    if (status) atomicCAS(status, 0, (int)M3_ERR_INVALID_ARGUMENT);
    loss[m] = __int_as_float(0x7fffffff);  // NaN
  } else {
    loss[m] = z - tlogit[m];
  }
}

// out = c times the sum over splits of part[s], rounded to bf16; n is a multiple of
// 8.  LANES threads share the splits of four neighbouring sums.
template <int LANES>
__global__ void __launch_bounds__(256)
xent_sum_kernel(const float* part, int splits, int64_t n, const float* unit, __nv_bfloat16* out) {
  constexpr int kCols = 256 / LANES;
  let_next_start();
  wait_for_previous();
  __shared__ float4 s_part[LANES][kCols];
  const int x = threadIdx.x % kCols, y = threadIdx.x / kCols;
  const float c = *unit;
  for (int64_t i0 = (int64_t)blockIdx.x * kCols * 4; i0 < n; i0 += (int64_t)gridDim.x * kCols * 4) {
    const int64_t i = i0 + x * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
#pragma unroll 4
      for (int s = y; s < splits; s += LANES) {
        const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)s * n + i);
        f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
      }
    }
    if constexpr (LANES > 1) {
      s_part[y][x] = f;
      __syncthreads();
      if (y == 0) {
#pragma unroll
        for (int l = 1; l < LANES; ++l) {
          const float4 v = s_part[l][x];
          f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
        }
      }
      __syncthreads();
    }
    if (y == 0 && i < n)
      *reinterpret_cast<uint2*>(out + i) =
          make_uint2(pack_bf16(f.x * c, f.y * c), pack_bf16(f.z * c, f.w * c));
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

// [rows][cols] bf16 with `ld` elements a row, boxes of 64 columns x box_rows.
bool encode(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld,
            int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One operand: [rows][cols] of memory; mn: the columns are the output's extent
// and the rows the reduction.
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
};

template <int CG, int BN, int MODE, bool AMN, bool BMN>
cudaError_t gemm_cg(const GemmArgs& g0, const Operand& a, const Operand& b, cudaStream_t s) {
  using C = Cfg<CG, BN>;
  // the rows of a stage behind A's last keep what shared memory held: they give
  // rows of the output that are not stored
  GemmArgs g = g0;
  g.a_rows = !AMN && g.M < kBM ? (int)ceil_div(g.M, 8) * 8 : kBM;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  if (!encode(&maps.a, a.p, a.rows, a.cols, a.ld, AMN ? kBK : g.a_rows) ||
      !encode(&maps.b, b.p, b.rows, b.cols, b.ld, BMN ? kBK : C::B_COLS))
    return cudaErrorInvalidValue;
  auto kern = xent_gemm_kernel<CG, BN, MODE, AMN, BMN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int64_t ctas = (int64_t)g.mt * g.nt * g.splits;
  // tokens are copied a warp each: CTAs without a tile help
  if (MODE == kDlogits && g.scored && !g.dependent && ctas < ceil_div(g.M, CG * kEpiWarps))
    ctas = ceil_div(g.M, CG * kEpiWarps);
  if (ctas > sms / CG) ctas = sms / CG;
  return launch_kernel(kern, dim3((unsigned)(CG * ctas)), kThreads, C::SMEM, s, g.dependent, CG, g, maps);
}

template <int MODE, bool AMN, bool BMN>
cudaError_t gemm(const GemmArgs& g, const Operand& a, const Operand& b, cudaStream_t s) {
  if (g.cg == 2) return gemm_cg<2, kWide, MODE, AMN, BMN>(g, a, b, s);
  if (g.bn == kNarrow) return gemm_cg<1, kNarrow, MODE, AMN, BMN>(g, a, b, s);
  if (g.bn == kMiddle) return gemm_cg<1, kMiddle, MODE, AMN, BMN>(g, a, b, s);
  return gemm_cg<1, kWide, MODE, AMN, BMN>(g, a, b, s);
}

// How a product's output is cut.
struct Cut {
  int cg, bn, splits;
};

// A product with M x N outputs, reduced over K in steps of 64.  Pairs of CTAs on
// 256 x 256 tiles where these fill three quarters of the SMs or more and have rows for
// both CTAs (the loss forward of 64 tokens x 20000 classes x 256 16.3 us with pairs, 10.6
// without; 128 x 32000 x 1024 22.1 and 15.7; 128 x 50257 x 2048 47.1 and 46.1); else single
// ones, with the columns and the splits of the reduction for which the longest
// CTA loads least (24, 32 or 48 KB a step; a step's time goes with that: 0.16 to
// 0.42 us).  Splits are at least eight steps long, and the launch that adds them
// counts as sixteen narrow steps.  Measured: 77 x 1003 classes x 256, the four
// products of a loss with gradients, 21 us with narrow tiles against 32 us with
// wide ones; logits of 28 x 10776 x 1744 15.4 us (middle) against 19.2 (wide); but
// dh of 391 x 56104 x 3296 181 us (wide, two splits) against 280 (middle).
Cut cut_of(int64_t M, int64_t N, int64_t K, bool split) {
  if (M > kBM && ceil_div(M, 2 * kBM) * ceil_div(N, kWide) >= kPlanSms / 2 * 3 / 4) return Cut{2, kWide, 1};
  const int64_t mt = ceil_div(M, kBM), kb = ceil_div(K, kBK);
  Cut best{1, kWide, 1};
  int64_t least = INT64_MAX;
  for (int bn : {kWide, kMiddle, kNarrow}) {
    const int64_t tiles = mt * ceil_div(N, bn);
    int64_t s = split ? kPlanSms / tiles : 1;
    if (s > kb / 8) s = kb / 8;
    if (s < 1) s = 1;
    s = ceil_div(kb, ceil_div(kb, s));
    const int64_t loads = ceil_div(tiles * s, kPlanSms) * ceil_div(kb, s) * (kBM + bn) / 8 + (s > 1 ? 16 * 24 : 0);
    if (loads < least) {
      least = loads;
      best = Cut{1, bn, (int)s};
    }
  }
  return best;
}

void set_tiles(GemmArgs* g, int64_t M, int64_t N, int64_t K, const Cut& c) {
  g->M = M;
  g->N = N;
  g->cg = c.cg;
  g->bn = c.bn;
  g->mt = (int)ceil_div(M, c.cg * kBM);
  g->nt = (int)ceil_div(N, c.bn);
  g->kb = (int)ceil_div(K, kBK);
  g->kb_per = (int)ceil_div(g->kb, c.splits);
  g->splits = (int)ceil_div(g->kb, g->kb_per);
}

// Bytes that the workspace may hold of d at a time: large enough that the
// products over a piece fill the SMs many times, small beside the memory.
constexpr int64_t kPieceBytes = (int64_t)256 << 20;

struct BwdPlan {
  int64_t piece, ldd;  // classes of one piece, and its row length (a multiple of 64)
  int pieces;
  Cut dh, dw;
  size_t d_bytes, dh_bytes, dw_bytes, h_bytes;
};

BwdPlan bwd_plan(const XentArgs& a) {
  BwdPlan p;
  int64_t most = kPieceBytes / 2 / a.M / kWide * kWide;
  if (most < kWide) most = kWide;
  p.pieces = (int)ceil_div(a.V, most);
  p.piece = ceil_div(ceil_div(a.V, p.pieces), kWide) * kWide;
  p.pieces = (int)ceil_div(a.V, p.piece);
  if (p.pieces == 1) p.piece = a.V;
  p.ldd = ceil_div(p.piece, 64) * 64;
  p.dh = cut_of(a.M, a.K, p.piece, true);
  p.dw = cut_of(p.piece, a.K, a.M, true);
  p.d_bytes = align_up((size_t)a.M * p.ldd * 2, 256);
  // sums of a gradient, and the copy of the hidden states for dW, only where it is wanted
  p.dh_bytes = a.dh && (p.pieces > 1 || p.dh.splits > 1)
                   ? align_up((size_t)p.dh.splits * a.M * a.K * 4, 256) : 0;
  p.dw_bytes = a.dW && p.dw.splits > 1 ? align_up((size_t)p.dw.splits * p.piece * a.K * 4, 256) : 0;
  p.h_bytes = a.dW ? align_up((size_t)a.M * a.K * 2, 256) : 0;
  return p;
}

size_t fwd_stat_bytes(const XentArgs& a) {
  return align_up((size_t)2 * ceil_div(a.V, cut_of(a.M, a.V, a.K, false).bn) * a.M * sizeof(float2), 256);
}

cudaError_t sum_splits(const float* part, int splits, int64_t n, const float* unit, void* out,
                       cudaStream_t s) {
  // few sums: eight threads each
  const bool few = n < (int64_t)kPlanSms * 1024 && splits >= 8;
  const int64_t blocks = ceil_div(n, few ? 128 : 1024);
  return launch_kernel(few ? xent_sum_kernel<8> : xent_sum_kernel<1>,
                       dim3((unsigned)(blocks < kPlanSms * 8 ? blocks : kPlanSms * 8)), 256, 0, s, true, 1,
                       part, splits, n, unit, static_cast<__nv_bfloat16*>(out));
}

}  // namespace

size_t xent_workspace(const XentArgs& a, bool backward) {
  if (a.M == 0) return 0;
  if (!backward) return fwd_stat_bytes(a) + align_up((size_t)a.M * 4, 256);
  if (!a.dh && !a.dW) return 0;
  const BwdPlan p = bwd_plan(a);
  return p.d_bytes + p.dh_bytes + p.dw_bytes + p.h_bytes + 256;
}

cudaError_t xent_fwd_launch(const XentArgs& a, cudaStream_t s) {
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  set_tiles(&g, a.M, a.V, a.K, cut_of(a.M, a.V, a.K, false));
  g.status = a.status;
  g.targets = a.targets;
  g.ignore = a.ignore;
  g.V = a.V;
  g.stat = reinterpret_cast<float2*>(a.ws);
  g.tlogit = reinterpret_cast<float*>(a.ws + fwd_stat_bytes(a));
  cudaError_t e = gemm<kStats, false, false>(g, Operand{a.h, a.M, a.K, a.K},
                                             Operand{a.W, a.V, a.K, a.K}, s);
  if (e != cudaSuccess) return e;
  return launch_kernel(xent_join_kernel, dim3((unsigned)ceil_div(a.M, kJoinTokens)), kJoinThreads, 0, s,
                       true, 1, (const float2*)g.stat, 2 * g.nt, a.M, a.V, a.targets, a.ignore,
                       (const float*)g.tlogit, a.loss, a.lse, a.status);
}

cudaError_t xent_bwd_launch(const XentArgs& a, cudaStream_t s) {
  const BwdPlan p = bwd_plan(a);
  __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(a.ws);
  float* dh32 = reinterpret_cast<float*>(a.ws + p.d_bytes);
  float* dw32 = reinterpret_cast<float*>(a.ws + p.d_bytes + p.dh_bytes);
  __nv_bfloat16* scored = reinterpret_cast<__nv_bfloat16*>(a.ws + p.d_bytes + p.dh_bytes + p.dw_bytes);
  float* unit = reinterpret_cast<float*>(a.ws + p.d_bytes + p.dh_bytes + p.dw_bytes + p.h_bytes);
  for (int i = 0; i < p.pieces; ++i) {
    const int64_t v0 = (int64_t)i * p.piece, n = a.V - v0 < p.piece ? a.V - v0 : p.piece;
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.W) + v0 * a.K;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    set_tiles(&g, a.M, n, a.K, cut_of(a.M, n, a.K, false));
    g.dependent = i > 0;
    g.status = a.status;
    g.targets = a.targets;
    g.ignore = a.ignore;
    g.V = a.V;
    g.v0 = v0;
    g.lse = a.lse;
    g.dloss = a.dloss;
    g.d = d;
    g.ldd = p.ldd;
    g.unit = unit;
    g.h = static_cast<const __nv_bfloat16*>(a.h);
    g.scored = a.dW ? scored : nullptr;
    g.K = a.K;
    cudaError_t e = gemm<kDlogits, false, false>(g, Operand{a.h, a.M, a.K, a.K},
                                                 Operand{W, n, a.K, a.K}, s);
    if (e != cudaSuccess) return e;
    if (a.dW) {  // [n][K] = d^T h
      GemmArgs w;
      memset(&w, 0, sizeof(w));
      set_tiles(&w, n, a.K, a.M, p.dw);
      w.dependent = true;
      w.status = a.status;
      w.unit = unit;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dW) + v0 * a.K;
      if (w.splits > 1) w.acc = dw32; else w.out = out;
      e = gemm<kGrad, true, true>(w, Operand{d, a.M, n, p.ldd}, Operand{scored, a.M, a.K, a.K}, s);
      if (e == cudaSuccess && w.splits > 1) e = sum_splits(dw32, w.splits, n * a.K, unit, out, s);
      if (e != cudaSuccess) return e;
    }
    if (a.dh) {  // [M][K] += d W
      GemmArgs h;
      memset(&h, 0, sizeof(h));
      set_tiles(&h, a.M, a.K, n, p.dh);
      h.dependent = true;
      h.status = a.status;
      h.unit = unit;
      const bool last = i + 1 == p.pieces;
      h.add = i > 0;
      if (p.dh_bytes) h.acc = dh32;
      if (last && p.dh.splits == 1) h.out = static_cast<__nv_bfloat16*>(a.dh);
      e = gemm<kGrad, false, true>(h, Operand{d, a.M, n, p.ldd}, Operand{W, n, a.K, a.K}, s);
      if (e == cudaSuccess && last && p.dh.splits > 1)
        e = sum_splits(dh32, p.dh.splits, a.M * a.K, unit, a.dh, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace m3
