// The linear layer around the attention, with its epilogue, and its gradient,
// on the tensor cores (TMA + tcgen05/TMEM).
//
//   forward   z = x W^T + bias,  y = residual + gate[sample] * act(z)
//   backward  dz = gate * dy * act'(z);  dx = dz W;  dW = dz^T x;
//             dbias = sum dz;  dgate[sample] = sum dy act(z)
//
// x [rows, n_in] and W [n_out, n_in] are bf16, products accumulate in fp32, and
// bias, activation, gate and residual are applied to the fp32 accumulator, so
// y is rounded once. The backward's dz is rounded to bf16 for its two products
// (the tensor cores take 16-bit operands); dbias and dgate are summed from the
// unrounded values.
//
// One kernel runs the three products: D[M, N] = A[M, K] B[N, K]^T with each
// operand either K-major (rows of K) or MN-major (stored transposed, read
// through MN-major shared-memory descriptors), so no operand is transposed in
// memory: forward x, W K-major; dx = dz (K-major) and W (MN-major over n_in);
// dW = dz and x, both MN-major with K = rows.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tc_sm100.h"
#include "tile_map.h"
#include "vsa_internal.h"

namespace vsa {
namespace {

using namespace tc;

// ------------------------------------------------------------ activation ----

// sigmoid(x) = 1 / (1 + e^-x); e^-x overflows to infinity for x << 0, which gives 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// gelu_tanh(z) = z (1 + tanh(u)) / 2 = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGeluB = 1.5957691216057308f;   // 2 sqrt(2/pi)
__device__ __forceinline__ float act_fwd(float z, int act) {
  if (act == VSA_ACT_GELU_TANH) return z * sigmoid(kGeluB * z * fmaf(0.044715f * z, z, 1.f));
  if (act == VSA_ACT_SILU) return z * sigmoid(z);
  return z;
}
// act(z) and act'(z), with the accurate exponential: they go into fp32 sums.
__device__ __forceinline__ void act_both(float z, int act, float& f, float& df) {
  if (act == VSA_ACT_NONE) {
    f = z;
    df = 1.f;
    return;
  }
  const bool gelu = act == VSA_ACT_GELU_TANH;
  const float u = gelu ? kGeluB * z * fmaf(0.044715f * z, z, 1.f) : z;
  const float du = gelu ? kGeluB * fmaf(3.f * 0.044715f * z, z, 1.f) : 1.f;
  const float s = 1.f / (1.f + expf(-u));
  f = z * s;
  df = fmaf(f * (1.f - s), du, s);
}

// -------------------------------------------------------------- epilogue ----

struct Epilogue {
  __nv_bfloat16* out;              // [M, N], row stride ld_out
  const float* bias;               // [N] or null
  const float* gate;               // [samples, N] or null
  const __nv_bfloat16* residual;   // row stride ld_res, or null
  __nv_bfloat16* pre;              // row stride ld_pre, or null
  int64_t ld_out, ld_res, ld_pre, ld_gate;
  int32_t rows_per_gate, act;
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ uint4 to_bf16x8(const float (&v)[8]) {
  return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// Eight columns of one row: v holds the accumulator, b the columns' bias.
__device__ __forceinline__ void store8(const Epilogue& e, int64_t row, int col, float (&v)[8], const float (&b)[8]) {
  // the loads first: they do not wait for the arithmetic
  uint4 res = make_uint4(0, 0, 0, 0);
  float g[8];
  if (e.residual) res = __ldcs(reinterpret_cast<const uint4*>(e.residual + row * e.ld_res + col));
  if (e.gate) load8(e.gate + (row / e.rows_per_gate) * e.ld_gate + col, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
  if (e.pre) *reinterpret_cast<uint4*>(e.pre + row * e.ld_pre + col) = to_bf16x8(v);
  if (e.act != VSA_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_fwd(v[i], e.act);
  }
  if (e.gate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i];
  }
  if (e.residual) {
    float r[8];
    bf16x8_to_f32(res, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  *reinterpret_cast<uint4*>(e.out + row * e.ld_out + col) = to_bf16x8(v);
}
__device__ __forceinline__ void load_bias(const Epilogue& e, int col, float (&b)[8]) {
  if (e.bias) {
    load8(e.bias + col, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
  }
}

// 32 rows by 32 columns of an accumulator, from one warp's TMEM lanes (lane =
// row; r: this lane's 32 columns) to the output: through 4 KB of shared memory,
// so that four lanes share a row and every global access moves 64 bytes of a row
// instead of 16. The 16-byte chunks of a staged row are swizzled by the row, which
// keeps both sides free of bank conflicts. partial: fp32 results instead.
__device__ __forceinline__ void store_chunk(const Epilogue& e, float* partial, int64_t M, int N, int64_t row0, int col0,
                                            const uint32_t (&r)[32], uint8_t* stage, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) * 16)) =
        make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
  __syncwarp();
  const int c8 = lane & 3;                       // my eight columns
  const int col = col0 + 8 * c8;
  if (col < N) {                                 // N is a multiple of eight
    float b[8];
    if (!partial) load_bias(e, col, b);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int rr = it * 8 + (lane >> 2);
      const int64_t row = row0 + rr;
      if (row >= M) continue;
      const float4 lo = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * c8) ^ (rr & 7)) * 16));
      const float4 hi = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * c8 + 1) ^ (rr & 7)) * 16));
      if (partial) {
        float4* dst = reinterpret_cast<float4*>(partial + row * N + col);
        dst[0] = lo;
        dst[1] = hi;
      } else {
        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store8(e, row, col, v, b);
      }
    }
  }
  __syncwarp();                                  // the stage is rewritten for the next chunk
}

// --------------------------------------------------------------- product ----

constexpr int kGThreads = 320;   // warp 0 producer, warp 1 MMA, warps 2-9 epilogue
constexpr int kEWarps = 8;       // two per TMEM lane quarter, half of the columns each: a GELU's chain of
                                 // dependent steps leaves one warp per scheduler idle most of the time

struct GemmParams {
  Epilogue ep;
  float* partial;          // splits > 1: fp32 [splits][M][N]
  uint32_t* state;         // [0] error word
  uint64_t wait_ns;
  int32_t M, N, kblocks;   // K in blocks of 64
  int32_t tiles_m, tiles_n, splits;
};

template <int BN>
struct GSmem {
  static constexpr uint32_t kA = 128 * 128;        // 128 x 64 bf16
  static constexpr uint32_t kB = BN * 128;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr uint32_t oOut = kStages * kStage;           // the epilogue warps' 4 KB each
  static constexpr uint32_t oBar = oOut + kEWarps * 4096;
  static constexpr uint32_t oMisc = oBar + 24 * 8;
  static constexpr uint32_t oEnd = oMisc + 16;
};
enum { G_FULL = 0, G_EMPTY = 8, G_AFULL = 16, G_AEMPTY = 18, G_DRAIN = 20 };

// The tile and k range of work unit u: the splits of a tile are neighbours, and
// tiles run down groups of eight row tiles before the next column tile, so that
// the CTAs at work share operand tiles in L2.
struct Unit {
  int m, n, k0, k1, split;
};
__device__ __forceinline__ Unit unit_of(const GemmParams& p, int u) {
  Unit r;
  r.split = u % p.splits;
  const int t = u / p.splits;
  const int per_group = 8 * p.tiles_n;
  const int grp = t / per_group, in = t - grp * per_group;
  const int rows = min(8, p.tiles_m - grp * 8);
  r.m = grp * 8 + in % rows;
  r.n = in / rows;
  r.k0 = int(int64_t(p.kblocks) * r.split / p.splits);
  r.k1 = int(int64_t(p.kblocks) * (r.split + 1) / p.splits);
  return r;
}

template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kGThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const __grid_constant__ GemmParams prm) {
  using L = GSmem<BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::oBar + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile uint32_t* abort_flag = misc + 1;
  uint32_t* gerr = prm.state;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = prm.tiles_m * prm.tiles_n * prm.splits;
  constexpr uint32_t kCols = 2 * BN;             // two accumulators

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(G_FULL + i), 1);
      mbar_init(bar(G_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(G_AFULL + i), 1);
      mbar_init(bar(G_AEMPTY + i), kEWarps);     // one arrival per epilogue warp
    }
    mbar_init(bar(G_DRAIN), 1);
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + L::oMisc),
                 "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;                           // k blocks issued
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Unit t = unit_of(prm, u);
        for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
          const int st = int(it % L::kStages);
          const uint32_t ph = (it / L::kStages) & 1;
          if (!(ok = wait_bar(bar(G_EMPTY + st), ph ^ 1, abort_flag, gerr, prm.wait_ns))) break;
          const uint32_t fb = bar(G_FULL + st);
          const uint32_t sa = sbase + st * L::kStage, sb = sa + L::kA;
          mbar_expect_tx(fb, L::kStage);
          if constexpr (A_MN) {                  // 64 columns of M by 64 rows of K per box
            tma_load_2d(sa, &ta, t.m * 128, kb * 64, fb);
            tma_load_2d(sa + 8192, &ta, t.m * 128 + 64, kb * 64, fb);
          } else {                               // 64 columns of K by 128 rows of M
            tma_load_2d(sa, &ta, kb * 64, t.m * 128, fb);
          }
          if constexpr (B_MN) {
            for (int i = 0; i < BN / 64; ++i) tma_load_2d(sb + 8192 * i, &tb, t.n * BN + 64 * i, kb * 64, fb);
          } else {
            tma_load_2d(sb, &tb, kb * 64, t.n * BN, fb);
          }
        }
      }
      if (*abort_flag)                           // let the copies land before shared memory is released
        for (uint32_t j = it >= uint32_t(L::kStages) ? it - L::kStages : 0; j < it; ++j)
          drain_wait(bar(G_FULL + int(j % L::kStages)), (j / L::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(128, BN, A_MN, B_MN);
      uint32_t it = 0, n = 0;                    // k blocks, tiles
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++n) {
        const Unit t = unit_of(prm, u);
        const int ab = n & 1;
        if (!(ok = wait_bar(bar(G_AEMPTY + ab), ((n >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
        for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
          const int st = int(it % L::kStages);
          if (!(ok = wait_bar(bar(G_FULL + st), (it / L::kStages) & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint32_t sa = sbase + st * L::kStage;
          const uint64_t da = A_MN ? sw128_desc(sa, 8192, 1024) : sw128_desc(sa, 16, 1024);
          const uint64_t db = B_MN ? sw128_desc(sa + L::kA, 8192, 1024) : sw128_desc(sa + L::kA, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)         // 16 of K per instruction
            tc_mma(tmem + ab * BN, da + ((kk * (A_MN ? 2048 : 32)) >> 4), db + ((kk * (B_MN ? 2048 : 32)) >> 4), idesc,
                   (kb > t.k0 || kk > 0) ? 1u : 0u);
          tc_commit(bar(G_EMPTY + st));
        }
        if (ok) tc_commit(bar(G_AFULL + ab));
      }
      tc_commit(bar(G_DRAIN));                   // nothing of ours may run when TMEM is freed
      drain_wait(bar(G_DRAIN), 0);
    }
    __syncwarp();
  } else {
    const int q4 = warp & 3, c0 = ((warp - 2) >> 2) * (BN / 2);   // my lanes and columns
    uint8_t* stage = smem + L::oOut + (warp - 2) * 4096;
    uint32_t n = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++n) {
      const Unit t = unit_of(prm, u);
      const int ab = n & 1;
      const bool ok = wait_bar(bar(G_AFULL + ab), (n >> 1) & 1, abort_flag, gerr, prm.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int64_t row0 = int64_t(t.m) * 128 + q4 * 32;
      float* partial = prm.splits > 1 ? prm.partial + int64_t(t.split) * prm.M * prm.N : nullptr;
#pragma unroll 1
      for (int c = c0; c < c0 + BN / 2; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + ab * BN + (uint32_t(q4 * 32) << 16) + c, r);
        tmem_wait_ld(r);
        if (c + 32 >= c0 + BN / 2) {             // the accumulator is read: the next tile may use it
          tc_fence_before();
          warp_arrive(bar(G_AEMPTY + ab));
        }
        store_chunk(prm.ep, partial, prm.M, prm.N, row0, t.n * BN + c, r, stage, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
}

// The same product on CTA pairs: a cluster of two CTAs computes a 256 x 256 tile
// with cta_group::2 products, each CTA holding its 128 rows of A and its half of
// the 256 columns of B, so that a k block moves 32 KB into each SM where two
// single CTAs would move 48 KB for the same work, and one 256 x 256 instruction
// (128 cycles) is long enough for one issuing thread. The leader (rank 0) issues;
// loads of both CTAs count on the leader's full barrier, the products' completion
// arrives in both CTAs. Two 256-column accumulators fill TMEM: a tile's epilogue
// runs under the next tile's products.
constexpr int kPStages = 6;
struct PSmem {
  static constexpr uint32_t kA = 128 * 128, kB = 128 * 128, kStage = kA + kB;
  static constexpr uint32_t oOut = kPStages * kStage;
  static constexpr uint32_t oBar = oOut + kEWarps * 4096;
  static constexpr uint32_t oMisc = oBar + 24 * 8;
  static constexpr uint32_t oEnd = oMisc + 16;
};

template <bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                     const __grid_constant__ GemmParams prm) {
  using L = PSmem;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::oBar + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile uint32_t* abort_flag = misc + 1;
  uint32_t* gerr = prm.state;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);
  const int units = prm.tiles_m * prm.tiles_n;   // 256 x 256 tiles

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(bar(G_FULL + i), 1);
      mbar_init(bar(G_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(G_AFULL + i), 1);
      mbar_init(bar(G_AEMPTY + i), 2 * kEWarps); // the epilogue warps of both CTAs
    }
    mbar_init(bar(G_DRAIN), 1);
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sbase + L::oMisc));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                // the pair's barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit t = unit_of(prm, u);
        const int m0 = t.m * 256 + int(rank) * 128, n0 = t.n * 256 + int(rank) * 128;
        for (int kb = 0; kb < prm.kblocks; ++kb, ++it) {
          const int st = int(it % kPStages);
          if (!(ok = wait_bar(bar(G_EMPTY + st), ((it / kPStages) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
          const uint32_t fb = map_to_rank(bar(G_FULL + st), 0);
          const uint32_t sa = sbase + st * L::kStage, sb = sa + L::kA;
          if (rank == 0) mbar_expect_tx(bar(G_FULL + st), 2 * L::kStage);
          if constexpr (A_MN) {
            tma_load_2d_pair(sa, &ta, m0, kb * 64, fb);
            tma_load_2d_pair(sa + 8192, &ta, m0 + 64, kb * 64, fb);
          } else {
            tma_load_2d_pair(sa, &ta, kb * 64, m0, fb);
          }
          if constexpr (B_MN) {
            tma_load_2d_pair(sb, &tb, n0, kb * 64, fb);
            tma_load_2d_pair(sb + 8192, &tb, n0 + 64, kb * 64, fb);
          } else {
            tma_load_2d_pair(sb, &tb, kb * 64, n0, fb);
          }
        }
      }
      // every stage is consumed (in both CTAs) before the CTA may end; after an abort the
      // copies in flight are given time to land
      if (ok) {
        for (uint32_t j = it >= uint32_t(kPStages) ? it - kPStages : 0; j < it && ok; ++j)
          ok = wait_bar(bar(G_EMPTY + int(j % kPStages)), (j / kPStages) & 1, abort_flag, gerr, prm.wait_ns);
      }
      if (!ok) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(256, 256, A_MN, B_MN);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs, ++n) {
        const int ab = n & 1;
        if (!(ok = wait_bar(bar(G_AEMPTY + ab), ((n >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
        for (int kb = 0; kb < prm.kblocks; ++kb, ++it) {
          const int st = int(it % kPStages);
          if (!(ok = wait_bar(bar(G_FULL + st), (it / kPStages) & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint32_t sa = sbase + st * L::kStage;
          const uint64_t da = A_MN ? sw128_desc(sa, 8192, 1024) : sw128_desc(sa, 16, 1024);
          const uint64_t db = B_MN ? sw128_desc(sa + L::kA, 8192, 1024) : sw128_desc(sa + L::kA, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_pair(tmem + ab * 256, da + ((kk * (A_MN ? 2048 : 32)) >> 4), db + ((kk * (B_MN ? 2048 : 32)) >> 4),
                        idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          tc_commit_pair(bar(G_EMPTY + st));
        }
        if (ok) tc_commit_pair(bar(G_AFULL + ab));
      }
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar(G_DRAIN))
                   : "memory");
      drain_wait(bar(G_DRAIN), 0);
    }
    __syncwarp();
  } else {
    const int q4 = warp & 3, c0 = ((warp - 2) >> 2) * 128;
    uint8_t* stage = smem + L::oOut + (warp - 2) * 4096;
    uint32_t n = 0;
    for (int u = pair; u < units; u += pairs, ++n) {
      const Unit t = unit_of(prm, u);
      const int ab = n & 1;
      const bool ok = wait_bar(bar(G_AFULL + ab), (n >> 1) & 1, abort_flag, gerr, prm.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int64_t row0 = int64_t(t.m) * 256 + rank * 128 + q4 * 32;
#pragma unroll 1
      for (int c = c0; c < c0 + 128; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + ab * 256 + (uint32_t(q4 * 32) << 16) + c, r);
        tmem_wait_ld(r);
        if (c == c0 + 96) {                      // the accumulator is read: the leader may use it again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(bar(G_AEMPTY + ab), 0));
        }
        store_chunk(prm.ep, nullptr, prm.M, prm.N, row0, t.n * 256 + c, r, stage, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                // neither CTA's shared memory or TMEM is in use any more
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The splits of K joined in order, then the epilogue: eight columns per thread.
__global__ void __launch_bounds__(256) split_join_kernel(const __grid_constant__ GemmParams prm) {
  const int64_t per_row = prm.N / 8, total = int64_t(prm.M) * per_row;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / per_row;
    const int col = int(i - row * per_row) * 8;
    float v[8] = {};
    for (int s = 0; s < prm.splits; ++s) {
      float t[8];
      load8(prm.partial + (int64_t(s) * prm.M + row) * prm.N + col, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += t[j];
    }
    float b[8];
    load_bias(prm.ep, col, b);
    store8(prm.ep, row, col, v, b);
  }
}

// ----------------------------------------------------- gradient of the rest ----

struct GradParams {
  const __nv_bfloat16 *dy, *pre;   // row strides ld_dy, ld_pre; pre may be null
  __nv_bfloat16* dz;               // [rows][N] contiguous, or null (dz = dy)
  const float* gate;               // [samples][N] or null
  float *part_z, *part_g;          // column sums of dz and of dy act(z): [chunks][N], or null
  int64_t ld_dy, ld_pre, rows, rows_per_sample;
  int32_t N, act, chunk, chunks_per_sample;
};

// dz and the column sums in one pass. A block takes 256 columns (32 lanes of
// eight) of one chunk of rows, which lies in one sample; its eight warps take
// every eighth row and meet in shared memory.
__global__ void __launch_bounds__(256) linear_dz_kernel(const __grid_constant__ GradParams p) {
  __shared__ float red[2][8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = int(blockIdx.y) * 256 + lane * 8;
  const int64_t sample = blockIdx.x / p.chunks_per_sample;
  const int64_t r0 = sample * p.rows_per_sample + int64_t(blockIdx.x % p.chunks_per_sample) * p.chunk;
  const int64_t end = (sample + 1) * p.rows_per_sample;
  int64_t r1 = r0 + p.chunk;
  if (r1 > end) r1 = end;
  if (r1 > p.rows) r1 = p.rows;
  float sz[8] = {}, sg[8] = {}, gt[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gt[i] = 1.f;
  const bool on = col < p.N;
  if (on && p.gate) load8(p.gate + sample * p.N + col, gt);
  if (on) {
    for (int64_t r = r0 + warp; r < r1; r += 8) {
      float dy[8], z[8];
      bf16x8_to_f32(__ldcs(reinterpret_cast<const uint4*>(p.dy + r * p.ld_dy + col)), dy);
      if (p.pre) {
        bf16x8_to_f32(__ldcs(reinterpret_cast<const uint4*>(p.pre + r * p.ld_pre + col)), z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, df;
          act_both(z[i], p.act, f, df);
          sg[i] = fmaf(dy[i], f, sg[i]);
          dy[i] *= gt[i] * df;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] *= gt[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sz[i] += dy[i];
      if (p.dz) *reinterpret_cast<uint4*>(p.dz + r * p.N + col) = to_bf16x8(dy);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[0][warp][lane * 8 + i] = sz[i];
    red[1][warp][lane * 8 + i] = sg[i];
  }
  __syncthreads();
  const int c = int(blockIdx.y) * 256 + threadIdx.x;
  if (c < p.N) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      a += red[0][w][threadIdx.x];
      b += red[1][w][threadIdx.x];
    }
    if (p.part_z) p.part_z[int64_t(blockIdx.x) * p.N + c] = a;
    if (p.part_g) p.part_g[int64_t(blockIdx.x) * p.N + c] = b;
  }
}

// The chunks' column sums joined in order, in fp64: block s < samples the gate
// gradient of sample s, block `samples` the bias gradient over every chunk.
__global__ void __launch_bounds__(256) linear_colsum_kernel(const float* __restrict__ part_z,
                                                            const float* __restrict__ part_g, int samples,
                                                            int chunks_per_sample, int N, float* dbias, float* dgate) {
  __shared__ double red[8][32];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int col = int(blockIdx.y) * 32 + lane;
  const bool is_bias = int(blockIdx.x) == samples;
  const float* src = is_bias ? part_z : part_g;
  float* dst = is_bias ? dbias : dgate;
  if (!dst) return;                              // uniform over the block
  const int64_t c0 = is_bias ? 0 : int64_t(blockIdx.x) * chunks_per_sample;
  const int64_t c1 = is_bias ? int64_t(samples) * chunks_per_sample : c0 + chunks_per_sample;
  double s = 0.0;
  if (col < N)
    for (int64_t i = c0 + sl; i < c1; i += 8) s += double(src[i * N + col]);
  red[sl][lane] = s;
  __syncthreads();
  if (sl == 0 && col < N) {
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    dst[(is_bias ? 0 : int64_t(blockIdx.x) * N) + col] = float(s);
  }
}

// ------------------------------------------------------------------ host ----

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

constexpr int kBN = 128;

// Pairs of CTAs on 256 x 256 tiles, or single CTAs on 128 x 128 tiles and splits of
// K: pairs from the point where their tiles fill most of the SMs.
bool use_pairs(const vsa_plan* p, int64_t M, int64_t N) {
  return cdiv64(M, 256) * cdiv64(N, 256) * 2 >= p->num_sms * 3 / 4;
}

// Splits of K: one tile per CTA leaves SMs idle when there are fewer tiles than
// half the SMs; each split keeps at least four k blocks of work.
int choose_splits(const vsa_plan* p, int64_t M, int64_t N, int64_t K) {
  if (use_pairs(p, M, N)) return 1;
  const int64_t tiles = cdiv64(M, 128) * cdiv64(N, kBN), kb = cdiv64(K, 64);
  if (tiles * 2 > p->num_sms) return 1;
  int64_t s = p->num_sms / tiles;
  if (s > kb / 4) s = kb / 4;
  if (s > 32) s = 32;
  return int(s < 1 ? 1 : s);
}
int64_t split_bytes(const vsa_plan* p, int64_t M, int64_t N, int64_t K) {
  const int s = choose_splits(p, M, N, K);
  return s > 1 ? round256(int64_t(s) * M * N * 4) : 0;
}

// A 2-D bf16 tensor map, columns innermost, `ld` elements per row.
bool make_map2(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows) {
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
  return make_map_nd(m, base, 2, dims, strides, box);
}

// D[M, N] = A B^T over K. A: [M, K] (K-major) or [K, M] (a_mn), B likewise.
template <bool A_MN, bool B_MN>
cudaError_t run_gemm(const vsa_plan* p, const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t M, int64_t N,
                     int64_t K, const Epilogue& ep, void* partial, cudaStream_t s) {
  using L = GSmem<kBN>;
  const bool pairs = use_pairs(p, M, N);
  const int bn = pairs ? 128 : kBN;              // rows of B one CTA loads
  CUtensorMap ta, tb;
  const bool ma = A_MN ? make_map2(&ta, a, K, M, ld_a, 64, 64) : make_map2(&ta, a, M, K, ld_a, 64, 128);
  const bool mb = B_MN ? make_map2(&tb, b, K, N, ld_b, 64, 64) : make_map2(&tb, b, N, K, ld_b, 64, bn);
  if (!ma || !mb) return cudaErrorInvalidValue;
  GemmParams prm;
  prm.ep = ep;
  prm.partial = static_cast<float*>(partial);
  prm.state = p->d_state;
  prm.wait_ns = p->wait_ns;
  prm.M = int32_t(M);
  prm.N = int32_t(N);
  prm.kblocks = int32_t(cdiv64(K, 64));
  prm.tiles_m = int32_t(cdiv64(M, pairs ? 256 : 128));
  prm.tiles_n = int32_t(cdiv64(N, pairs ? 256 : kBN));
  prm.splits = choose_splits(p, M, N, K);
  const int64_t units = int64_t(prm.tiles_m) * prm.tiles_n * prm.splits;
  if (pairs) {
    const int smem = 1024 + int(PSmem::oEnd);
    const cudaError_t e =
        cudaFuncSetAttribute(gemm_pair_kernel<A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t most = p->num_sms / 2;
    gemm_pair_kernel<A_MN, B_MN><<<2 * unsigned(units < most ? units : most), kGThreads, smem, s>>>(ta, tb, prm);
    return cudaGetLastError();
  }
  const int grid = int(units < p->num_sms ? units : p->num_sms);
  const int smem = 1024 + int(L::oEnd);
  cudaError_t e = cudaFuncSetAttribute(gemm_kernel<kBN, A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  gemm_kernel<kBN, A_MN, B_MN><<<grid, kGThreads, smem, s>>>(ta, tb, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess || prm.splits == 1) return e;
  const int64_t want = cdiv64(M * (N / 8), 256), cap = int64_t(p->num_sms) * 8;
  split_join_kernel<<<unsigned(want < cap ? want : cap), 256, 0, s>>>(prm);
  return cudaGetLastError();
}

struct GradPlan {
  int32_t samples, chunk, chunks_per_sample;
  int64_t rows_per_sample;
  bool needs_dz;
  int64_t dz_bytes, part_bytes;    // part_bytes: one of the two column-sum tables
};

GradPlan grad_plan(const vsa_plan* p, int64_t rows, int64_t N, int act, bool gate, int64_t rows_per_gate) {
  GradPlan g;
  g.needs_dz = act != VSA_ACT_NONE || gate;
  g.rows_per_sample = gate ? rows_per_gate : rows;
  g.samples = int32_t(cdiv64(rows, g.rows_per_sample));
  const int64_t blocks_y = cdiv64(N, 256);
  int64_t want = cdiv64(int64_t(p->num_sms) * 4, blocks_y);
  int64_t chunk = cdiv64(rows, want);
  if (chunk < 32) chunk = 32;
  if (chunk > g.rows_per_sample) chunk = g.rows_per_sample;
  g.chunk = int32_t(chunk);
  g.chunks_per_sample = int32_t(cdiv64(g.rows_per_sample, chunk));
  g.dz_bytes = g.needs_dz ? round256(rows * N * 2) : 0;
  g.part_bytes = round256(int64_t(g.samples) * g.chunks_per_sample * N * 4);
  return g;
}

}  // namespace

int64_t linear_workspace_bytes(const vsa_plan* p, int64_t rows, int64_t n_in, int64_t n_out, bool backward,
                               int64_t rows_per_gate) {
  if (rows == 0) return 0;
  if (!backward) return split_bytes(p, rows, n_out, n_in);
  // whatever the activation: the largest need
  const GradPlan g = grad_plan(p, rows, n_out, VSA_ACT_SILU, rows_per_gate > 0, rows_per_gate);
  const int64_t a = split_bytes(p, rows, n_in, n_out), b = split_bytes(p, n_out, n_in, rows);
  return g.dz_bytes + 2 * g.part_bytes + (a > b ? a : b);
}

cudaError_t launch_linear(const vsa_plan* p, const vsa_linear_args& a, void* workspace, cudaStream_t s) {
  Epilogue ep = {};
  ep.out = static_cast<__nv_bfloat16*>(a.y);
  ep.ld_out = a.ld_y;
  ep.bias = a.bias;
  ep.gate = a.gate;
  ep.ld_gate = a.n_out;
  ep.rows_per_gate = a.gate ? int32_t(a.rows_per_gate) : 1;
  ep.residual = static_cast<const __nv_bfloat16*>(a.residual);
  ep.ld_res = a.ld_residual;
  ep.pre = static_cast<__nv_bfloat16*>(a.pre);
  ep.ld_pre = a.ld_pre;
  ep.act = a.act;
  return run_gemm<false, false>(p, a.x, a.ld_x, a.w, a.n_in, a.rows, a.n_out, a.n_in, ep, workspace, s);
}

cudaError_t launch_linear_bwd(const vsa_plan* p, const vsa_linear_grad_args& a, void* workspace, cudaStream_t s) {
  const GradPlan g = grad_plan(p, a.rows, a.n_out, a.act, a.gate != nullptr, a.rows_per_gate);
  char* ws = static_cast<char*>(workspace);
  auto* dz = reinterpret_cast<__nv_bfloat16*>(ws);
  float* part_z = reinterpret_cast<float*>(ws + g.dz_bytes);
  float* part_g = reinterpret_cast<float*>(ws + g.dz_bytes + g.part_bytes);
  void* split = ws + g.dz_bytes + 2 * g.part_bytes;
  const bool products = a.dx || a.dw;
  if ((g.needs_dz && products) || a.dbias || a.dgate) {
    GradParams gp;
    gp.dy = static_cast<const __nv_bfloat16*>(a.dy);
    gp.pre = a.act != VSA_ACT_NONE || a.dgate ? static_cast<const __nv_bfloat16*>(a.pre) : nullptr;
    gp.dz = g.needs_dz && products ? dz : nullptr;
    gp.gate = a.gate;
    gp.part_z = a.dbias ? part_z : nullptr;
    gp.part_g = a.dgate ? part_g : nullptr;
    gp.ld_dy = a.ld_dy;
    gp.ld_pre = a.ld_pre;
    gp.rows = a.rows;
    gp.rows_per_sample = g.rows_per_sample;
    gp.N = a.n_out;
    gp.act = a.act;
    gp.chunk = g.chunk;
    gp.chunks_per_sample = g.chunks_per_sample;
    const dim3 grid(unsigned(g.samples) * unsigned(g.chunks_per_sample), unsigned(cdiv64(a.n_out, 256)));
    linear_dz_kernel<<<grid, 256, 0, s>>>(gp);
    if (a.dbias || a.dgate)
      linear_colsum_kernel<<<dim3(unsigned(g.samples) + 1, unsigned(cdiv64(a.n_out, 32))), 256, 0, s>>>(
          part_z, part_g, g.samples, g.chunks_per_sample, a.n_out, a.dbias, a.dgate);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const void* zsrc = g.needs_dz ? static_cast<const void*>(dz) : a.dy;
  const int64_t ld_z = g.needs_dz ? a.n_out : a.ld_dy;
  Epilogue ep = {};
  ep.rows_per_gate = 1;
  if (a.dx) {
    ep.out = static_cast<__nv_bfloat16*>(a.dx);
    ep.ld_out = a.ld_dx;
    const cudaError_t e =
        run_gemm<false, true>(p, zsrc, ld_z, a.w, a.n_in, a.rows, a.n_in, a.n_out, ep, split, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    ep.out = static_cast<__nv_bfloat16*>(a.dw);
    ep.ld_out = a.n_in;
    return run_gemm<true, true>(p, zsrc, ld_z, a.x, a.ld_x, a.n_out, a.n_in, a.rows, ep, split, s);
  }
  return cudaSuccess;
}

}  // namespace vsa
