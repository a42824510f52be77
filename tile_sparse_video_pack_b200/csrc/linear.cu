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
#include <string.h>

#include <type_traits>

#include "tc_sm100.h"
#include "tile_map.h"
#include "vsa_internal.h"

namespace vsa {
namespace {

using namespace tc;

// ------------------------------------------------------------ activation ----

// gelu_tanh(z) = z (1 + tanh(u)) / 2 = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3);
// sigmoid(x) = 1 / (1 + 2^(-x log2 e)): 2^x overflows to infinity for x << 0, which gives 0.
// The approximate exponential and reciprocal are within 2^-21 for the arguments that
// matter, far below the output's rounding to bf16. Two elements at a time in packed fp32.
constexpr float kGeluB = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// SiLU has no cubic term: as GELU's with a coefficient of 0 it would be 0 times infinity from |z| = 2^64 on.
__device__ __forceinline__ void act_fwd(float (&v)[8], int act) {
  if (act == VSA_ACT_NONE) return;
  const uint64_t one = f2pack(1.f, 1.f);
  auto apply = [&](auto exponent) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t z = f2pack(v[i], v[i + 1]);
      float x0, x1;
      f2unpack(exponent(z), x0, x1);
      f2unpack(fadd2(f2pack(ex2(x0), ex2(x1)), one), x0, x1);
      f2unpack(fmul2(z, f2pack(rcp(x0), rcp(x1))), v[i], v[i + 1]);
    }
  };
  if (act == VSA_ACT_GELU_TANH) {
    constexpr float c1 = -kGeluB * kLog2e, c3 = -0.044715f * kGeluB * kLog2e;
    const uint64_t c1p = f2pack(c1, c1), c3p = f2pack(c3, c3);
    apply([&](uint64_t z) { return fmul2(z, ffma2(fmul2(z, z), c3p, c1p)); });   // -2u log2 e
  } else {
    const uint64_t c1p = f2pack(-kLog2e, -kLog2e);
    apply([&](uint64_t z) { return fmul2(z, c1p); });                            // -z log2 e
  }
}
// act(z) and act'(z) of two elements: with s = sigmoid(u), f = z s and
// f' = s + f (1 - s) u' (SiLU: u = z; GELU: u the 2u above), one polynomial for both.
// Far out s is 0 or 1 exactly and so is f', but with |z| past 2^64 the polynomial (SiLU: 0
// times infinity) and f' (0 times an infinite f or u') are NaN: FAR has their values.
template <bool FAR>
__device__ __forceinline__ void act_both(uint64_t z, int act, uint64_t& f, uint64_t& df) {
  const uint64_t one = f2pack(1.f, 1.f);
  if (act == VSA_ACT_NONE) {
    f = z;
    df = one;
    return;
  }
  const bool gelu = act == VSA_ACT_GELU_TANH;
  const float c1 = gelu ? kGeluB : 1.f, c3 = gelu ? 0.044715f * kGeluB : 0.f;
  const uint64_t z2 = fmul2(z, z);
  uint64_t x = fmul2(z, f2pack(-kLog2e, -kLog2e));
  if (!FAR || gelu) x = fmul2(x, ffma2(z2, f2pack(c3, c3), f2pack(c1, c1)));
  float x0, x1;
  f2unpack(x, x0, x1);
  f2unpack(fadd2(f2pack(ex2(x0), ex2(x1)), one), x0, x1);
  const uint64_t s = f2pack(rcp(x0), rcp(x1));
  f = fmul2(z, s);
  const uint64_t du = ffma2(z2, f2pack(3.f * c3, 3.f * c3), f2pack(c1, c1));
  df = ffma2(fmul2(f, ffma2(s, f2pack(-1.f, -1.f), one)), du, s);
  if constexpr (FAR) {
    constexpr float kFar = 1e4f;
    float z0, z1, s0, s1, d0, d1;
    f2unpack(z, z0, z1);
    f2unpack(s, s0, s1);
    f2unpack(df, d0, d1);
    df = f2pack(fabsf(z0) > kFar ? s0 : d0, fabsf(z1) > kFar ? s1 : d1);
  }
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

__device__ __forceinline__ uint4 load_residual(const Epilogue& e, int64_t row, int col) {
  return e.residual ? __ldcs(reinterpret_cast<const uint4*>(e.residual + row * e.ld_res + col)) : make_uint4(0, 0, 0, 0);
}
// The gate row of an output row (rows fit 32 bits).
__device__ __forceinline__ const float* gate_row(const Epilogue& e, int64_t row) {
  return e.gate ? e.gate + int64_t(uint32_t(row) / uint32_t(e.rows_per_gate)) * e.ld_gate : nullptr;
}

// Eight columns of one row: v holds the accumulator, b the columns' bias, res the
// residual's eight values, loaded before (y may overwrite the residual).
__device__ __forceinline__ void store8(const Epilogue& e, int64_t row, int col, float (&v)[8], const float (&b)[8],
                                       uint4 res, const float* gate) {
  float g[8];
  if (gate) load8(gate + col, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
  if (e.pre) __stcs(reinterpret_cast<uint4*>(e.pre + row * e.ld_pre + col), to_bf16x8(v));
  act_fwd(v, e.act);
  if (gate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i];
  }
  if (e.residual) {
    float r[8];
    bf16x8_to_f32(res, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  __stcs(reinterpret_cast<uint4*>(e.out + row * e.ld_out + col), to_bf16x8(v));
}
__device__ __forceinline__ void load_bias(const Epilogue& e, int col, float (&b)[8]) {
  if (e.bias) {
    load8(e.bias + col, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
  }
}

// The rows of a warp's 32-row strip that this lane stores (four lanes share a row,
// four rows each) and their gate rows: fixed for a tile.
struct StripRows {
  int64_t row0;
  int n;                           // how many of the four are inside the matrix
  const float* gate[4];
};
__device__ __forceinline__ StripRows strip_rows(const Epilogue& e, int64_t M, int64_t row0, int lane) {
  StripRows r;
  r.row0 = row0 + (lane >> 2);
  r.n = 0;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int64_t row = r.row0 + it * 8;
    r.gate[it] = row < M ? gate_row(e, row) : nullptr;
    r.n += row < M;
  }
  return r;
}
// The residual of a 32-column chunk of the strip: requested ahead of the chunk (one at a
// time before its store, each load held up the next: 164 us for the output projection).
struct Chunk {
  uint4 res[4];
};
__device__ __forceinline__ Chunk load_chunk(const Epilogue& e, const StripRows& rows, int N, int col0, int lane) {
  Chunk c;
  const int col = col0 + 8 * (lane & 3);
#pragma unroll
  for (int it = 0; it < 4; ++it)
    c.res[it] = it < rows.n && col < N ? load_residual(e, rows.row0 + it * 8, col) : make_uint4(0, 0, 0, 0);
  return c;
}

// 32 rows by 32 columns of an accumulator, from one warp's TMEM lanes (lane =
// row; r: this lane's 32 columns) to the output: through 4 KB of shared memory,
// so that four lanes share a row and every global access moves 64 bytes of a row
// instead of 16. The 16-byte chunks of a staged row are swizzled by the row, which
// keeps both sides free of bank conflicts.
__device__ __forceinline__ void store_chunk(const Epilogue& e, const StripRows& rows, const Chunk& in, int N, int col0,
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
    load_bias(e, col, b);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int rr = it * 8 + (lane >> 2);
      if (it >= rows.n) continue;
      const float4 lo = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * c8) ^ (rr & 7)) * 16));
      const float4 hi = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * c8 + 1) ^ (rr & 7)) * 16));
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      store8(e, rows.row0 + it * 8, col, v, b, in.res[it], rows.gate[it]);
    }
  }
  __syncwarp();                                  // the stage is rewritten for the next chunk
}

// --------------------------------------------------------------- product ----

constexpr int kGThreads = 320;   // warp 0 producer, warp 1 MMA, warps 2-9 epilogue
constexpr int kEWarps = 8;       // two per TMEM lane quarter, half of the columns each: a GELU's chain of
                                 // dependent steps leaves one warp per scheduler idle most of the time

// One product. a_mn / b_mn: that operand is stored [K][M] / [K][N].
struct Product {
  Epilogue ep;
  int32_t M, N, kblocks;   // K in blocks of 64
  int32_t tiles_m, tiles_n;
  int32_t a_mn, b_mn;
};
struct GemmParams {
  Product prod[2];
  uint32_t* state;         // [0] error word
  uint64_t wait_ns;
  int32_t n_prod, units;   // products and the tiles of all of them
  int32_t splits;          // CTAs of a cluster that share a tile's K
  int32_t group;           // row tiles per group of the tile order
  int32_t hold;            // test hook: the epilogue waits for a second arrival, which nothing makes
};
struct GemmMaps {
  CUtensorMap a[2], b[2];
};

constexpr int kBM = 128;
template <bool SPLIT, int BN>
struct GSmem {
  static constexpr uint32_t kA = kBM * 128, kB = BN * 128, kStage = kA + kB;   // 64 of K
  static constexpr int kStages = BN == 64 && !SPLIT ? 8 : 6;
  static constexpr uint32_t oOut = kStages * kStage;           // the epilogue warps' 4 KB each, or the shares of my rows
  static constexpr uint32_t oBar = oOut + (SPLIT ? kBM * BN * 4 : kEWarps * 4096);
  static constexpr uint32_t oMisc = oBar + 24 * 8;
  static constexpr uint32_t oEnd = oMisc + 16;
};
// The bound of the epilogue's wait for a tile's products: the plan's limit and, because a sum over rows may have millions
// of k blocks, 10 us for each (one takes 0.1 to 0.8, the latter with all SMs at HBM). A stall is found within the
// limit all the same: producer and issuer wait for one k block at a time.
__device__ __forceinline__ uint64_t tile_limit(uint64_t wait_ns, int kblocks) { return wait_ns + uint64_t(kblocks) * 10000u; }

enum { G_FULL = 0, G_EMPTY = 8, G_AFULL = 16, G_AEMPTY = 18, G_DRAIN = 20 };

// Tile u: tiles run down groups of `group` row tiles before the next column tile,
// so that the CTAs at work share operand tiles in L2.
struct Tile {
  int prod, m, n;
};
__device__ __forceinline__ Tile tile_of(const GemmParams& p, int u) {
  Tile r;
  const int first = p.prod[0].tiles_m * p.prod[0].tiles_n;
  r.prod = u >= first ? 1 : 0;
  if (r.prod) u -= first;
  const Product& q = p.prod[r.prod];
  const int per_group = p.group * q.tiles_n;
  const int grp = u / per_group, in = u - grp * per_group;
  const int rows = min(p.group, q.tiles_m - grp * p.group);
  r.m = grp * p.group + in % rows;
  r.n = in / rows;
  return r;
}

// Loads of one k block: 128 (64) rows of a K-major operand are one box of 64 of K by
// that many rows, of an MN-major one two boxes (one) of 64 columns by 64 of K.
template <bool PAIR, int ROWS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, bool mn, int row0, int kb, uint32_t fb) {
  auto load = [&](uint32_t d, int x, int y) {
    if (PAIR) tma_load_2d_pair(d, map, x, y, fb);
    else tma_load_2d(d, map, x, y, fb);
  };
  if (mn) {
    load(dst, row0, kb * 64);
    if (ROWS == 128) load(dst + 8192, row0 + 64, kb * 64);
  } else {
    load(dst, kb * 64, row0);
  }
}
// Shared-memory descriptor of an operand's stage and the advance per 16 of K.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
  return mn ? sw128_desc(addr, 8192, 1024) : sw128_desc(addr, 16, 1024);
}
__device__ __forceinline__ uint32_t operand_step(bool mn) { return (mn ? 2048u : 32u) >> 4; }

__device__ __forceinline__ void st_cluster(uint32_t addr, const uint32_t* v) {   // addr: mapped into a CTA of the cluster
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// SPLIT = false: every CTA works through tiles on its own, the epilogue of one tile
// under the products of the next. SPLIT = true, for problems with few tiles: the
// `splits` CTAs of a cluster (2, 4 or 8) take a share of a tile's K each and write
// their fp32 accumulators, 128 / splits rows to each CTA, into that CTA's shared
// memory; each joins its rows' shares in rank order -- one launch, no partial sums
// in global memory, the same result every time. Writing to the joining CTA takes
// the remote latency once, before the barrier; reading from the others took it
// again for every row. The exchange runs at some 13 bytes a cycle and CTA, so a split
// tile has 64 columns, and rows past the matrix are not sent.
template <bool SPLIT, int BN>
__global__ void __launch_bounds__(kGThreads, 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams prm) {
  using L = GSmem<SPLIT, BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::oBar + 8u * uint32_t(i); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile uint32_t* abort_flag = misc + 1;
  uint32_t* gerr = prm.state;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = SPLIT ? prm.splits : 1;
  const int rank = SPLIT ? int(cluster_rank()) : 0;
  const int u0 = int(blockIdx.x) / splits, du = int(gridDim.x) / splits;
  constexpr uint32_t kCols = 2 * BN;            // two accumulators

  if (threadIdx.x == 0) {
    for (int i = 0; i < prm.n_prod; ++i) {
      prefetch_map(&maps.a[i]);
      prefetch_map(&maps.b[i]);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(G_FULL + i), 1);
      mbar_init(bar(G_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(G_AFULL + i), prm.hold ? 2 : 1);
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
  if constexpr (SPLIT) cluster_sync();           // the others' shared memory exists from here on
  allow_successor();
  wait_predecessor();

  uint32_t it = 0, n = 0;                        // k blocks and tiles so far, counted alike by every role
  bool ok = true;
  for (int u = u0; u < prm.units; u += du, ++n) {
    const Tile t = tile_of(prm, u);
    const Product& pr = prm.prod[t.prod];
    const int k0 = int(int64_t(pr.kblocks) * rank / splits), k1 = int(int64_t(pr.kblocks) * (rank + 1) / splits);
    const int ab = n & 1;
    if (warp == 0) {
      if (lane == 0) {
        const CUtensorMap* ta = &maps.a[t.prod];
        const CUtensorMap* tb = &maps.b[t.prod];
        for (int kb = k0; kb < k1 && ok; ++kb, ++it) {
          const int st = int(it % L::kStages);
          if (!(ok = wait_bar(bar(G_EMPTY + st), ((it / L::kStages) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
          const uint32_t sa = sbase + st * L::kStage;
          mbar_expect_tx(bar(G_FULL + st), L::kStage);
          load_operand<false, 128>(sa, ta, pr.a_mn, t.m * kBM, kb, bar(G_FULL + st));
          load_operand<false, BN>(sa + L::kA, tb, pr.b_mn, t.n * BN, kb, bar(G_FULL + st));
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0 && ok) {
        const uint32_t idesc = idesc_bf16(kBM, BN, pr.a_mn, pr.b_mn);
        const uint32_t as = operand_step(pr.a_mn), bs = operand_step(pr.b_mn);
        ok = wait_bar(bar(G_AEMPTY + ab), ((n >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns);
        for (int kb = k0; kb < k1 && ok; ++kb, ++it) {
          const int st = int(it % L::kStages);
          if (!(ok = wait_bar(bar(G_FULL + st), (it / L::kStages) & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint32_t sa = sbase + st * L::kStage;
          const uint64_t da = operand_desc(sa, pr.a_mn), db = operand_desc(sa + L::kA, pr.b_mn);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)         // 16 of K per instruction
            tc_mma(tmem + ab * BN, da + kk * as, db + kk * bs, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
          tc_commit(bar(G_EMPTY + st));
        }
        if (ok) tc_commit(bar(G_AFULL + ab));
      }
      __syncwarp();
    } else if (ok) {
      const int ew = warp - 2, q4 = warp & 3, c0 = (ew >> 2) * (BN / 2);   // my lanes and columns
      StripRows rows;
      Chunk next;
      if constexpr (!SPLIT) {                    // while the products run
        rows = strip_rows(pr.ep, pr.M, int64_t(t.m) * kBM + q4 * 32, lane);
        next = load_chunk(pr.ep, rows, pr.N, t.n * BN + c0, lane);
      }
      ok = wait_bar(bar(G_AFULL + ab), (n >> 1) & 1, abort_flag, gerr, tile_limit(prm.wait_ns, k1 - k0));
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int c = c0; c < c0 + BN / 2; c += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + ab * BN + (uint32_t(q4 * 32) << 16) + c, r);
          tmem_wait_ld(r);
          if (c + 32 >= c0 + BN / 2) {          // the accumulator is read: the next tile may use it
            tc_fence_before();
            warp_arrive(bar(G_AEMPTY + ab));
          }
          if constexpr (SPLIT) {
            // share `rank` at the CTA that joins this row: rows of BN floats, 16-byte chunks swizzled by the row
            const int row = q4 * 32 + lane, per = kBM / splits, owner = row / per;
            const uint32_t to = map_to_rank(sbase + L::oOut + uint32_t(rank * per + row % per) * (BN * 4), owner);
            if (int64_t(t.m) * kBM + row < pr.M) {
#pragma unroll
              for (int i = 0; i < 8; ++i) st_cluster(to + (((c >> 2) + i) ^ (row & 7)) * 16, r + 4 * i);
            }
          } else {
            const Chunk in = next;
            if (c + 32 < c0 + BN / 2) next = load_chunk(pr.ep, rows, pr.N, t.n * BN + c + 32, lane);
            store_chunk(pr.ep, rows, in, pr.N, t.n * BN + c, r, smem + L::oOut + ew * 4096, lane);
          }
        }
      }
    }
    if constexpr (SPLIT) {
      // what the join needs besides the shares, before the barrier
      constexpr int LPR = BN / 8, RPW = 32 / LPR;     // lanes to a row (eight columns each), rows per warp and step
      const int per = kBM / splits, cg = lane % LPR;  // rows this CTA joins
      const int col = t.n * BN + 8 * cg;
      float bias[8] = {};
      if (warp >= 2 && ok && col < pr.N) load_bias(pr.ep, col, bias);
      cluster_sync();                            // every share is where it is joined
      if (warp >= 2 && ok) {
        for (int rr = (warp - 2) * RPW + lane / LPR; rr < per; rr += RPW * kEWarps) {
          const int in_tile = rank * per + rr;
          const int64_t row = int64_t(t.m) * kBM + in_tile;
          if (row >= pr.M || col >= pr.N) continue;
          const uint4 res = load_residual(pr.ep, row, col);
          float v[8] = {};
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < splits) {
              const uint8_t* at = smem + L::oOut + (s * per + rr) * (BN * 4);
              const float4 x = *reinterpret_cast<const float4*>(at + ((2 * cg) ^ (in_tile & 7)) * 16);
              const float4 y = *reinterpret_cast<const float4*>(at + ((2 * cg + 1) ^ (in_tile & 7)) * 16);
              v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
              v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
            }
          store8(pr.ep, row, col, v, bias, res, gate_row(pr.ep, row));
        }
      }
      // every CTA has read its shares before any is written again; a CTA whose shares are all
      // in may end
      if (u + du < prm.units) cluster_sync();
    }
  }
  // Every copy lands before shared memory is released, whatever the abort flag says by now: a role that is
  // still at work may give up after this one has left (at the usual end the last stages are on their way)
  if (warp == 0 && lane == 0)
    for (uint32_t j = it >= uint32_t(L::kStages) ? it - L::kStages : 0; j < it; ++j)
      drain_wait(bar(G_FULL + int(j % L::kStages)), (j / L::kStages) & 1);
  if (warp == 1 && lane == 0) {                  // nothing of ours may run when TMEM is freed
    tc_commit(bar(G_DRAIN));
    drain_wait(bar(G_DRAIN), 0);
  }
  __syncwarp();
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
// 18,944 x 2,048 with K 8,192: 468 us, 1,360 TFLOP/s at 1,965 MHz, 554 us once the power cap holds (1,400 MHz), 380 on
// zeros; K 2,048 with gate and residual (18,560 rows) 126 to 131 us, 147 to 153 with the cap. The tensor pipe is
// active 66 to 71 % of the time (K 2,048).
constexpr int kPStages = 6;
struct PSmem {
  static constexpr uint32_t kA = 128 * 128, kB = 128 * 128, kStage = kA + kB;
  static constexpr uint32_t oOut = kPStages * kStage;
  static constexpr uint32_t oBar = oOut + kEWarps * 4096;
  static constexpr uint32_t oMisc = oBar + 24 * 8;
  static constexpr uint32_t oEnd = oMisc + 16;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    gemm_pair_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams prm) {
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
  const int units = prm.units;                   // 256 x 256 tiles of one product
  const Product& pr = prm.prod[0];
  const bool a_mn = pr.a_mn, b_mn = pr.b_mn;

  if (threadIdx.x == 0) {
    prefetch_map(&maps.a[0]);
    prefetch_map(&maps.b[0]);
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(bar(G_FULL + i), 1);
      mbar_init(bar(G_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(G_AFULL + i), prm.hold ? 2 : 1);
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
  allow_successor();
  wait_predecessor();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Tile t = tile_of(prm, u);
        const int m0 = t.m * 256 + int(rank) * 128, n0 = t.n * 256 + int(rank) * 128;
        for (int kb = 0; kb < pr.kblocks; ++kb, ++it) {
          const int st = int(it % kPStages);
          if (!(ok = wait_bar(bar(G_EMPTY + st), ((it / kPStages) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
          const uint32_t fb = map_to_rank(bar(G_FULL + st), 0);
          const uint32_t sa = sbase + st * L::kStage, sb = sa + L::kA;
          if (rank == 0) mbar_expect_tx(bar(G_FULL + st), 2 * L::kStage);
          load_operand<true, 128>(sa, &maps.a[0], a_mn, m0, kb, fb);
          load_operand<true, 128>(sb, &maps.b[0], b_mn, n0, kb, fb);
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
      const uint32_t idesc = idesc_bf16(256, 256, a_mn, b_mn);
      const uint32_t as = operand_step(a_mn), bs = operand_step(b_mn);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs, ++n) {
        const int ab = n & 1;
        if (!(ok = wait_bar(bar(G_AEMPTY + ab), ((n >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
        for (int kb = 0; kb < pr.kblocks; ++kb, ++it) {
          const int st = int(it % kPStages);
          if (!(ok = wait_bar(bar(G_FULL + st), (it / kPStages) & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint32_t sa = sbase + st * L::kStage;
          const uint64_t da = operand_desc(sa, a_mn), db = operand_desc(sa + L::kA, b_mn);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_pair(tmem + ab * 256, da + kk * as, db + kk * bs, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
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
      const Tile t = tile_of(prm, u);
      const int ab = n & 1;
      // while the products run
      const StripRows rows = strip_rows(pr.ep, pr.M, int64_t(t.m) * 256 + rank * 128 + q4 * 32, lane);
      Chunk next = load_chunk(pr.ep, rows, pr.N, t.n * 256 + c0, lane);
      bool ok = wait_bar(bar(G_AFULL + ab), (n >> 1) & 1, abort_flag, gerr, tile_limit(prm.wait_ns, pr.kblocks));
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
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
        const Chunk in = next;
        if (c + 32 < c0 + 128) next = load_chunk(pr.ep, rows, pr.N, t.n * 256 + c + 32, lane);
        store_chunk(pr.ep, rows, in, pr.N, t.n * 256 + c, r, stage, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                // neither CTA's shared memory or TMEM is in use any more
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Up to sixteen rows (a timestep's conditioning, single tokens): bound by reading W once,
// so no tile is staged. A block takes 8 T columns, its W warps every W-th chunk of 64 of
// K; their sums are joined in shared memory in the warps' order and stored by the common
// epilogue. T: eights of rows. A lane's 16-byte load holds eight k of one column of W, or
// of one row of x, which is two steps of m16n8k16 fragments when the k within a chunk are
// taken in the lanes' order, the same for both operands: nothing is shuffled, and 16 rows
// cost no more arithmetic than one (the warp-level instruction takes its operands from
// registers; its rate does not matter here). Each warp keeps U chunks of loads in flight.
// Rows past the last are zeros in registers. fp32 products on the plain cores took 20.8 us
// for 8 rows at 1,536 x 9,216, this takes 6.5 (4.3 at the copy rate) and 6.4 for one row;
// the tiles of 128 rows take 15.
template <int T, int W, int U>
__global__ void __launch_bounds__(W * 32) few_rows_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld_x,
                                                          const __nv_bfloat16* __restrict__ w, int rows, int K, int N,
                                                          const __grid_constant__ Epilogue ep) {
  __shared__ float4 part[W][T * 8][T * 2];
  allow_successor();
  wait_predecessor();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int n0 = int(blockIdx.x) * 8 * T;
  const __nv_bfloat16 *wp[T], *xp[T];
  bool w_in[T], x_in[T];
#pragma unroll
  for (int j = 0; j < T; ++j) {
    w_in[j] = n0 + j * 8 < N;                      // N is a multiple of eight, and so is K
    wp[j] = w + int64_t(w_in[j] ? n0 + j * 8 + g : 0) * K;
    x_in[j] = g + j * 8 < rows;
    xp[j] = x + int64_t(x_in[j] ? g + j * 8 : 0) * ld_x;
  }
  uint4 wv[U][2][T], xv[U][2][T];
  auto load = [&](int d, int k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = k0 + i * 32 + t * 8;
#pragma unroll
      for (int j = 0; j < T; ++j) {
        wv[d][i][j] = k < K && w_in[j] ? __ldcs(reinterpret_cast<const uint4*>(wp[j] + k)) : make_uint4(0, 0, 0, 0);
        xv[d][i][j] = k < K && x_in[j] ? __ldg(reinterpret_cast<const uint4*>(xp[j] + k)) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  float acc[T][4] = {};
#pragma unroll
  for (int d = 0; d < U; ++d) load(d, (d * W + warp) * 64);
  for (int k0 = warp * 64; k0 < K; k0 += 64 * W * U) {     // the same steps for all lanes: a product is the whole warp's
#pragma unroll
    for (int d = 0; d < U; ++d) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 lo = xv[d][i][0], hi = T > 1 ? xv[d][i][T - 1] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < T; ++j) {
          mma_16x8x16(acc[j], lo.x, hi.x, lo.y, hi.y, wv[d][i][j].x, wv[d][i][j].y);
          mma_16x8x16(acc[j], lo.z, hi.z, lo.w, hi.w, wv[d][i][j].z, wv[d][i][j].w);
        }
      }
      load(d, k0 + 64 * W * (U + d));
    }
  }
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int r = 0; r < T; ++r)
      reinterpret_cast<float2*>(&part[warp][r * 8 + g][j * 2])[t] = make_float2(acc[j][2 * r], acc[j][2 * r + 1]);
  __syncthreads();
  const int row = int(threadIdx.x) / T, j = int(threadIdx.x) % T, col = n0 + j * 8;
  if (row >= rows || col >= N) return;             // rows <= 8 T
  float v[8] = {}, b[8];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float4 lo = part[i][row][j * 2], hi = part[i][row][j * 2 + 1];
    v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
    v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
  }
  load_bias(ep, col, b);
  store8(ep, row, col, v, b, load_residual(ep, row, col), gate_row(ep, row));
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
// every eighth row, four at a time so that enough loads are in flight (one row at a time
// and the library's exponential and division: 238 us at 9,280 x 8,192, where the bytes take 70;
// now 89), and meet in shared memory.
__global__ void __launch_bounds__(256) linear_dz_kernel(const __grid_constant__ GradParams p) {
  __shared__ float red[2][8][256];
  allow_successor();
  wait_predecessor();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = int(blockIdx.y) * 256 + lane * 8;
  const int64_t sample = blockIdx.x / p.chunks_per_sample;
  const int64_t r0 = sample * p.rows_per_sample + int64_t(blockIdx.x % p.chunks_per_sample) * p.chunk;
  const int64_t end = (sample + 1) * p.rows_per_sample;
  int64_t r1 = r0 + p.chunk;
  if (r1 > end) r1 = end;
  if (r1 > p.rows) r1 = p.rows;
  uint64_t sz[4], sg[4], gt[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) gt[i] = f2pack(1.f, 1.f);
  const bool on = col < p.N;
  if (on && p.gate) {
    float g[8];
    load8(p.gate + sample * p.N + col, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) gt[i] = f2pack(g[2 * i], g[2 * i + 1]);
  }
  // this thread's columns of its rows
  auto walk = [&](auto far) {
    constexpr int U = 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) sz[i] = sg[i] = 0ull;
    if (!on) return;
    for (int64_t r = r0 + warp; r < r1; r += 8 * U) {
      uint4 vy[U], vz[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t rr = r + 8 * u;
        if (rr < r1) {
          vy[u] = __ldcs(reinterpret_cast<const uint4*>(p.dy + rr * p.ld_dy + col));
          if (p.pre) vz[u] = __ldcs(reinterpret_cast<const uint4*>(p.pre + rr * p.ld_pre + col));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t rr = r + 8 * u;
        if (rr >= r1) break;
        float dy[8], z[8];
        bf16x8_to_f32(vy[u], dy);
        if (p.pre) bf16x8_to_f32(vz[u], z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint64_t d = f2pack(dy[2 * i], dy[2 * i + 1]), f, df;
          if (p.pre) {
            act_both<decltype(far)::value>(f2pack(z[2 * i], z[2 * i + 1]), p.act, f, df);
            sg[i] = ffma2(d, f, sg[i]);
            d = fmul2(fmul2(d, gt[i]), df);
          } else {
            d = fmul2(d, gt[i]);
          }
          sz[i] = fadd2(sz[i], d);
          f2unpack(d, dy[2 * i], dy[2 * i + 1]);
        }
        if (p.dz) *reinterpret_cast<uint4*>(p.dz + rr * p.N + col) = to_bf16x8(dy);
      }
    }
  };
  walk(std::false_type{});
  // A pre-activation too far out for the common polynomial has made its column's sum NaN: once more, with care. (The
  // two comparisons that this takes cost 8 % when every element makes them.)
  uint64_t all = fadd2(fadd2(sz[0], sz[1]), fadd2(sz[2], sz[3]));
  float all0, all1;
  f2unpack(all, all0, all1);
  if (p.pre && isnan(all0 + all1)) walk(std::true_type{});
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2unpack(sz[i], red[0][warp][lane * 8 + 2 * i], red[0][warp][lane * 8 + 2 * i + 1]);
    f2unpack(sg[i], red[1][warp][lane * 8 + 2 * i], red[1][warp][lane * 8 + 2 * i + 1]);
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
  allow_successor();
  wait_predecessor();
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

// Row tiles per group of the tile order. At 18,944 x 2048 -> 8192 groups of 8 read
// 392 MB from DRAM and groups of 16 234 MB (operands: 111 MB), in the same time.
constexpr int kGroup = 16;

// A 2-D bf16 tensor map, columns innermost, `ld` elements per row.
bool make_map2(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows) {
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
  return make_map_nd(m, base, 2, dims, strides, box);
}

// D[M, N] = A B^T over K. a: [M, K], or [K, M] with a_mn; b: [N, K], or [K, N] with b_mn.
struct Problem {
  const void *a, *b;
  int64_t ld_a, ld_b, M, N, K;
  bool a_mn, b_mn;
  Epilogue ep;
};

// Rounds of tiles over the SMs decide between pairs of CTAs on 256 x 256 tiles and single
// CTAs on 128 x 128 ones: a round of pairs, four times a tile's work on two SMs, takes about 1.1
// times as long (K 2,048, us, singles / pairs: 1,024 x 2,048 17.7 / 18.6, one round each; 512 x 5,120
// 30.2 / 19.6, two and one; 3,584 x 2,048 56 / 31, four and two).
bool use_pairs(const vsa_plan* p, int64_t M, int64_t N) {
  const int64_t pairs = cdiv64(cdiv64(M, 256) * cdiv64(N, 256), p->num_sms / 2);
  return 11 * pairs < 10 * cdiv64(cdiv64(M, 128) * cdiv64(N, 128), p->num_sms);
}

// tile_m x tile_n per unit; a CTA loads 128 rows of A and b_rows of B.
bool add_product(GemmMaps& maps, GemmParams& prm, const Problem& q, int tile_m, int tile_n, int b_rows) {
  const int i = prm.n_prod++;
  const bool ma = q.a_mn ? make_map2(&maps.a[i], q.a, q.K, q.M, q.ld_a, 64, 64)
                         : make_map2(&maps.a[i], q.a, q.M, q.K, q.ld_a, 64, 128);
  const bool mb = q.b_mn ? make_map2(&maps.b[i], q.b, q.K, q.N, q.ld_b, 64, 64)
                         : make_map2(&maps.b[i], q.b, q.N, q.K, q.ld_b, 64, b_rows);
  Product& r = prm.prod[i];
  r.ep = q.ep;
  r.M = int32_t(q.M);
  r.N = int32_t(q.N);
  r.kblocks = int32_t(cdiv64(q.K, 64));
  r.tiles_m = int32_t(cdiv64(q.M, tile_m));
  r.tiles_n = int32_t(cdiv64(q.N, tile_n));
  r.a_mn = q.a_mn;
  r.b_mn = q.b_mn;
  prm.units += r.tiles_m * r.tiles_n;
  return ma && mb;
}

// One or two products: in one launch where both go to single CTAs.
cudaError_t run_products(const vsa_plan* p, const Problem* q, int n, cudaStream_t s) {
  GemmMaps maps;
  GemmParams prm;
  auto start = [&] {
    memset(&prm, 0, sizeof(prm));
    prm.state = p->d_state;
    prm.wait_ns = p->wait_ns;
    prm.hold = p->test_hold;
    prm.group = kGroup;
    prm.splits = 1;
  };
  const unsigned sms = unsigned(p->num_sms);
  int64_t units128 = 0, units64 = 0, kb = 1 << 30;   // tiles of the single CTAs' products; k blocks of the shortest
  for (int i = 0; i < n; ++i) {
    if (!use_pairs(p, q[i].M, q[i].N)) {
      units128 += cdiv64(q[i].M, 128) * cdiv64(q[i].N, 128);
      units64 += cdiv64(q[i].M, 128) * cdiv64(q[i].N, 64);
      kb = cdiv64(q[i].K, 64) < kb ? cdiv64(q[i].K, 64) : kb;
      continue;
    }
    start();
    if (!add_product(maps, prm, q[i], 256, 256, 128)) return cudaErrorInvalidValue;
    const unsigned pairs = unsigned(prm.units) < sms / 2 ? unsigned(prm.units) : sms / 2;
    const cudaError_t r = launch_after(gemm_pair_kernel, dim3(2 * pairs), unsigned(kGThreads),
                                       size_t(1024 + PSmem::oEnd), s, 1, maps, prm);
    if (r != cudaSuccess) return r;
  }
  if (units128 == 0) return cudaSuccess;
  // Tiles of 128 x 64 while one round of them covers the products (K 2,048, us: 128 tiles of 64
  // columns 14.9, the 64 of 128 columns 17.2; 160 tiles of 64 columns 26.1, 80 of 128 17.6), and K
  // shared by clusters of 2, 4 or 8 while the clusters fit the SMs at once and every CTA keeps two k
  // blocks (32 tiles, shared by 1, 2, 4: 14.7, 10.7, 8.7). Clusters of 8 leave more SMs out (16 tiles of
  // K 1,024, shared by 4 and 8: 7.4 and 12.0; 14 tiles: 6.4 and 6.3; 4 tiles of K 2,048: 6.6 and 5.9).
  const bool narrow = units64 <= sms;
  int splits = 1;
  while (splits < 8 && units64 * splits * 2 <= sms * (splits == 4 ? 8 : 9) / 10 && kb >= splits * 4) splits *= 2;
  start();
  prm.splits = splits;
  for (int i = 0; i < n; ++i)
    if (!use_pairs(p, q[i].M, q[i].N) &&
        !add_product(maps, prm, q[i], 128, narrow ? 64 : 128, narrow ? 64 : 128))
      return cudaErrorInvalidValue;
  if (splits > 1)
    return launch_after(gemm_kernel<true, 64>, dim3(unsigned(prm.units * splits)), unsigned(kGThreads),
                        size_t(1024 + GSmem<true, 64>::oEnd), s, unsigned(splits), maps, prm);
  const dim3 grid(unsigned(prm.units) < sms ? unsigned(prm.units) : sms);
  if (narrow)
    return launch_after(gemm_kernel<false, 64>, grid, unsigned(kGThreads), size_t(1024 + GSmem<false, 64>::oEnd), s, 1,
                        maps, prm);
  return launch_after(gemm_kernel<false, 128>, grid, unsigned(kGThreads), size_t(1024 + GSmem<false, 128>::oEnd), s, 1,
                      maps, prm);
}

// Sixteen warps share a block's K where the blocks are few, four where they fill the SMs
// several times over or K is short (one row, us, sixteen / four warps: K 2,048 by 512 columns
// 2.3 / 2.5, by 2,048 3.3 / 4.3, by 8,192 9.8 / 7.0; K 512 by 1,536 2.1 / 1.8).
cudaError_t run_few_rows(const vsa_plan* p, const Problem& q, cudaStream_t s) {
  auto* x = static_cast<const __nv_bfloat16*>(q.a);
  auto* w = static_cast<const __nv_bfloat16*>(q.b);
  const int t = q.M <= 8 ? 1 : 2;
  const int64_t blocks = cdiv64(q.N, 8 * t);
  const bool few = blocks * t <= int64_t(p->num_sms) * 2 && q.K >= 1024;
#define VSA_FEW(T, W, U)                                                                                             \
  launch_after(few_rows_kernel<T, W, U>, dim3(unsigned(blocks)), unsigned(W * 32), 0, s, 1, x, q.ld_a, w, int(q.M), \
               int(q.K), int(q.N), q.ep)
  if (t == 1) return few ? VSA_FEW(1, 16, 2) : VSA_FEW(1, 4, 2);
  return few ? VSA_FEW(2, 16, 2) : VSA_FEW(2, 4, 3);
#undef VSA_FEW
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
  int64_t want = cdiv64(int64_t(p->num_sms) * 16, blocks_y);   // many small blocks: no long last round
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

// Shared-memory limits of the products, once per device (plan creation).
cudaError_t prepare_linear() {
  const auto at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(gemm_pair_kernel, at, 1024 + int(PSmem::oEnd));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_kernel<false, 128>, at, 1024 + int(GSmem<false, 128>::oEnd));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_kernel<false, 64>, at, 1024 + int(GSmem<false, 64>::oEnd));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_kernel<true, 64>, at, 1024 + int(GSmem<true, 64>::oEnd));
  return e;
}

int64_t linear_bwd_workspace_bytes(const vsa_plan* p, int64_t rows, int64_t n_out, int64_t rows_per_gate) {
  if (rows == 0) return 0;
  // whatever the activation: the largest need
  const GradPlan g = grad_plan(p, rows, n_out, VSA_ACT_SILU, rows_per_gate > 0, rows_per_gate);
  return g.dz_bytes + 2 * g.part_bytes;
}

cudaError_t launch_linear(const vsa_plan* p, const vsa_linear_args& a, cudaStream_t s) {
  Problem q = {};
  q.a = a.x;
  q.ld_a = a.ld_x;
  q.b = a.w;
  q.ld_b = a.n_in;
  q.M = a.rows;
  q.N = a.n_out;
  q.K = a.n_in;
  q.ep.out = static_cast<__nv_bfloat16*>(a.y);
  q.ep.ld_out = a.ld_y;
  q.ep.bias = a.bias;
  q.ep.gate = a.gate;
  q.ep.ld_gate = a.n_out;
  q.ep.rows_per_gate = a.gate ? int32_t(a.rows_per_gate) : 1;
  q.ep.residual = static_cast<const __nv_bfloat16*>(a.residual);
  q.ep.ld_res = a.ld_residual;
  q.ep.pre = static_cast<__nv_bfloat16*>(a.pre);
  q.ep.ld_pre = a.ld_pre;
  q.ep.act = a.act;
  return q.M <= 16 ? run_few_rows(p, q, s) : run_products(p, &q, 1, s);
}

cudaError_t launch_linear_bwd(const vsa_plan* p, const vsa_linear_grad_args& a, void* workspace, cudaStream_t s) {
  const GradPlan g = grad_plan(p, a.rows, a.n_out, a.act, a.gate != nullptr, a.rows_per_gate);
  char* ws = static_cast<char*>(workspace);
  auto* dz = reinterpret_cast<__nv_bfloat16*>(ws);
  float* part_z = reinterpret_cast<float*>(ws + g.dz_bytes);
  float* part_g = reinterpret_cast<float*>(ws + g.dz_bytes + g.part_bytes);
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
    cudaError_t e = launch_after(linear_dz_kernel, grid, 256u, 0, s, 1, gp);
    if (e == cudaSuccess && (a.dbias || a.dgate))
      e = launch_after(linear_colsum_kernel, dim3(unsigned(g.samples) + 1, unsigned(cdiv64(a.n_out, 32))), 256u, 0, s, 1,
                       part_z, part_g, g.samples, g.chunks_per_sample, a.n_out, a.dbias, a.dgate);
    if (e != cudaSuccess) return e;
  }
  const void* zsrc = g.needs_dz ? static_cast<const void*>(dz) : a.dy;
  const int64_t ld_z = g.needs_dz ? a.n_out : a.ld_dy;
  Problem q[2] = {};
  int n = 0;
  if (a.dx) {                                    // dx = dz W: W is stored with n_out, the K of this product, as its rows
    Problem& d = q[n++];
    d.a = zsrc;
    d.ld_a = ld_z;
    d.b = a.w;
    d.ld_b = a.n_in;
    d.b_mn = true;
    d.M = a.rows;
    d.N = a.n_in;
    d.K = a.n_out;
    d.ep.out = static_cast<__nv_bfloat16*>(a.dx);
    d.ep.ld_out = a.ld_dx;
    d.ep.rows_per_gate = 1;
  }
  if (a.dw) {                                    // dW = dz^T x: K = rows, both stored with K as their rows
    Problem& d = q[n++];
    d.a = zsrc;
    d.ld_a = ld_z;
    d.a_mn = true;
    d.b = a.x;
    d.ld_b = a.ld_x;
    d.b_mn = true;
    d.M = a.n_out;
    d.N = a.n_in;
    d.K = a.rows;
    d.ep.out = static_cast<__nv_bfloat16*>(a.dw);
    d.ep.ld_out = a.n_in;
    d.ep.rows_per_gate = 1;
  }
  return n ? run_products(p, q, n, s) : cudaSuccess;
}

}  // namespace vsa
