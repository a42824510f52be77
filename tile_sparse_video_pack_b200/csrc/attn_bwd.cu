// Gradient of the tile-sparse attention (TMA + tcgen05/TMEM).
//
// With P = exp(scale q k^T - lse) over the key tiles each query tile keeps,
// o = P v and delta = rowsum(do o):
//   dV = P^T dO,   dS = P (dO V^T - delta),   dQ = scale dS K,   dK = scale dS^T Q.
// P is rebuilt from the forward's log-sum-exp, so nothing of size rows x keys
// is stored.
//
// Two passes of one kernel, each with its own stationary 64-row tile whose
// gradient stays in tensor memory from its first to its last partner, so that
// no sum is spread over CTAs and no atomics decide its order:
//   key pass    stationary key tile (K, V), streamed query tiles (Q, dO): dK, dV
//   query pass  stationary query tile (Q, dO), streamed key tiles (K, V): dQ
// Write X, Y for the streamed pair (Q, dO or K, V) and Xs, Ys for the
// stationary one (K, V or Q, dO). Two streamed tiles make 128 rows, so every
// product has M = 128 without merging two tiles' lists:
//   S = X Xs^T, dP = Y Ys^T           128 x 64, rows = streamed tokens (TMEM lanes)
//   acc1^T += X^T dS (dK or dQ)       d x 64, and in the key pass acc0^T += Y^T P (dV)
// The accumulators are transposed (lanes = channels) so that M is 128 for them
// too; the streamed tile serves its first product K-major and its second
// MN-major from the same shared-memory image. P and dS go through shared
// memory as bf16, the operand type of the forward's P (half a step, 2^-9,
// of each term).
// The two passes cost 14 d operations per (query, key) pair where one pass
// with a summed dQ would cost 10 d, but that sum would go through global
// atomics, 32 KB per tile pair.
//
// Which tiles meet is a bit matrix per (batch, head), [query tile][key tile]:
// built from the index lists (validated on the way), its transpose by 32 x 32
// ballots. The producer walks the stationary tile's row of it.
//
// Warp roles (416 threads): warp 0 producer (item, bit row, TMA); warps 1-3 and
// 12 one MMA issuer for each of S, dP, acc1 and acc0, because an issuing thread
// spends about 88 cycles on each instruction and its barriers where these N = 64
// products take 32 to 48 (one thread for all four: 4,030 cycles per streamed pair
// in the key pass); warps 4-11 two warpgroups that turn S and dP into P and dS,
// half of the columns each, and write the finished gradients. Both work on the
// same pair: with alternate pairs the step from S to P took twice as long, and it
// is on the path of a stage's release. P and dS stay in registers until the
// previous pair's products have read theirs, so that one buffer does; at d = 64, where
// two fit, two take 3 % off (32 heads of 38 tiles: 115 -> 112 us). Every wait is bounded as in the
// forward.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tc_sm100.h"
#include "tile_map.h"
#include "vsa_internal.h"

namespace vsa {
namespace {

using namespace tc;

constexpr int kBThreads = 416;
constexpr int kWarpS = 1, kWarpDp = 2, kWarpAcc1 = 3, kWarpAcc0 = 12;   // MMA issuers
constexpr uint32_t kBox = 64 * 64 * 2;           // one 64 x 64 bf16 TMA box

// ------------------------------------------------------------ preparation ----

struct BitParams {
  const int32_t *idx, *idx_ref, *ref_tiles, *prefix_ref;
  uint32_t *bits, *bits_t;   // [B * heads][words * 32][words]: query-major and its transpose
  uint32_t* state;
  int32_t heads, nt_max, ntv_max, k_max, n_pre, n_ref, k_ref_max, words;
  int32_t ntv[VSA_MAX_HEADS], k[VSA_MAX_HEADS], k_ref[VSA_MAX_HEADS];
};

// Per packed row: log-sum-exp in log2 units, and delta = sum of do * o. Rows of
// unused slots (and of tiles past a head's own) get +inf, so that P is 0.
template <int CPR>
__device__ __forceinline__ void prepare_rows(const Geometry& g, int block, int blocks, const uint4* o, const uint4* dO,
                                             const float* lse, const int32_t* counts, float* lse2, float* delta) {
  const int64_t rows = int64_t(g.B) * g.Hh * g.nt_max * VSA_TILE;
  const int c = threadIdx.x % CPR;
  constexpr int R = 256 / CPR;
  for (int64_t r0 = int64_t(block) * R; r0 < rows; r0 += int64_t(blocks) * R) {
    const int64_t row = r0 + threadIdx.x / CPR;  // rows is a multiple of R: every lane has one
    const int64_t tile = row / VSA_TILE;
    const int h = int((tile / g.nt_max) % g.Hh);
    const bool valid = int(row % VSA_TILE) < counts[int64_t(h) * g.nt_max + tile % g.nt_max];
    float s = 0.f;
    if (valid) {
      float a[8], b[8];
      bf16x8_to_f32(__ldcs(o + row * CPR + c), a);
      bf16x8_to_f32(__ldcs(dO + row * CPR + c), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
    }
#pragma unroll
    for (int x = CPR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (c == 0) {
      lse2[row] = valid ? lse[row] * 1.4426950408889634f : INFINITY;
      delta[row] = s;
    }
  }
}

// One warp per (batch, head, query tile): its row of the bit matrix. A list out
// of range or not ascending latches the error and leaves the row empty.
__device__ __forceinline__ void prepare_bits(const BitParams& p, int64_t index, uint32_t* row) {
  const int lane = threadIdx.x & 31;
  const int rows = p.words * 32;
  const int bh = int(index / rows), i = int(index - int64_t(bh) * rows), h = bh % p.heads;
  const int nt = p.n_pre + p.ntv[h];
  for (int w = lane; w < p.words; w += 32) row[w] = 0u;
  __syncwarp();
  bool bad = false;
  if (i < p.n_pre) {
    for (int t = lane; t < nt; t += 32) atomicOr(row + (t >> 5), 1u << (t & 31));
  } else if (i < nt) {
    for (int t = lane; t < p.n_pre; t += 32)
      if (!p.idx_ref || p.prefix_ref[t] < 0) atomicOr(row + (t >> 5), 1u << (t & 31));
    const int64_t vrow = int64_t(bh) * p.ntv_max + (i - p.n_pre);
    auto add = [&](const int32_t* list, int n, int limit, bool ref) {
      for (int e = lane; e < n; e += 32) {
        const int j = list[e], before = e > 0 ? list[e - 1] : -1;
        if (j < 0 || j >= limit || j <= before) {
          bad = true;
        } else {
          const int t = ref ? p.ref_tiles[j] : p.n_pre + j;
          atomicOr(row + (t >> 5), 1u << (t & 31));
        }
      }
    };
    if (p.idx_ref) add(p.idx_ref + vrow * p.k_ref_max, p.k_ref[h], p.n_ref, true);
    add(p.idx + vrow * p.k_max, p.k[h], p.ntv[h], false);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) atomicOr(p.state, kErrBadIndex);
  __syncwarp();
  uint32_t* out = p.bits + index * p.words;
  for (int w = lane; w < p.words; w += 32) out[w] = bad ? 0u : row[w];
}

// Both in one launch: the first `row_blocks` blocks the rows, the others eight rows of
// the bit matrix each; block 0 also clears the two work counters.
template <int CPR>
__global__ void __launch_bounds__(256)
    bwd_prepare_kernel(const __grid_constant__ Geometry g, int row_blocks, const uint4* __restrict__ o,
                       const uint4* __restrict__ dO, const float* __restrict__ lse,
                       const int32_t* __restrict__ counts, float* __restrict__ lse2, float* __restrict__ delta,
                       uint32_t* __restrict__ counters, const __grid_constant__ BitParams p, int64_t bit_rows) {
  extern __shared__ uint32_t sm[];               // [8][words]
  allow_successor();
  wait_predecessor();
  if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0u;
  if (int(blockIdx.x) < row_blocks) {
    prepare_rows<CPR>(g, blockIdx.x, row_blocks, o, dO, lse, counts, lse2, delta);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int64_t index = (int64_t(blockIdx.x) - row_blocks) * 8 + warp;
  if (index < bit_rows) prepare_bits(p, index, sm + warp * p.words);
}

// Transpose by 32 x 32 blocks: one warp per block.
__global__ void __launch_bounds__(256) bwd_transpose_kernel(const uint32_t* __restrict__ bits,
                                                            uint32_t* __restrict__ bits_t, int words, int64_t blocks) {
  allow_successor();
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const int64_t blk = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (blk >= blocks) return;
  const int64_t bh = blk / (int64_t(words) * words);
  const int in = int(blk - bh * words * words);
  const int wi = in / words, wj = in % words;
  const int64_t base = bh * words * 32;
  const uint32_t x = bits[(base + wi * 32 + lane) * words + wj];
  uint32_t mine = 0u;
#pragma unroll
  for (int b = 0; b < 32; ++b) {
    const uint32_t v = __ballot_sync(0xffffffffu, (x >> b) & 1u);
    if (lane == b) mine = v;
  }
  bits_t[(base + wj * 32 + lane) * words + wi] = mine;
}

// ------------------------------------------------------------------ kernel ----

struct BwdItem {
  int32_t bh, tile, pairs, count;   // pairs: streamed pairs; count: valid rows of the stationary tile
  int32_t end, pad[3];
};
struct BwdPair {
  int32_t ta, tb;                   // streamed tiles (tb < 0: none)
};

template <int D, bool KEY>
struct BSmem {
  static constexpr uint32_t kHalf = 128 * 128;                 // 128 rows x 64 channels
  static constexpr uint32_t kTensor = (D / 64) * kHalf;        // one slot: one streamed tensor's pair of tiles
  static constexpr int kSlots = D == 128 ? 5 : 8;              // what fits beside the rest (D = 64: ample)
  static constexpr uint32_t kStat = (D / 64) * kBox;           // one stationary tile
  static constexpr uint32_t kPd = 128 * 128;                   // P or dS of a pair: 128 rows x 64 bf16
  static constexpr uint32_t oStat = kSlots * kTensor;          // Xs, Ys
  static constexpr int kPdBufs = D == 128 ? 1 : 2;             // one is what fits at D = 128
  static constexpr uint32_t oDs = oStat + 2 * kStat;
  static constexpr uint32_t oP = oDs + kPdBufs * kPd;          // key pass
  static constexpr uint32_t oBar = oP + (KEY ? kPdBufs : 0) * kPd;
  static constexpr uint32_t oItem = oBar + 40 * 8;
  static constexpr uint32_t oPair = oItem + 2 * sizeof(BwdItem);
  static constexpr uint32_t oCol = oPair + 4 * sizeof(BwdPair);              // query pass: lse2, delta of the tile
  static constexpr uint32_t oEnd = oCol + (KEY ? 0 : 2 * 2 * 64 * 4);        // two items' worth
};

// Slot and use count of streamed pair g's X or Y. d = 128, key pass: both live
// from their load to the end of acc0 / acc1, so one ring of five alternates them
// (2.5 pairs). Query pass: Y is done after dP, X after acc1: rings of two and
// three. d = 64: slots in pairs, [Y; X] one operand of 128 channels, four pairs.
struct SlotUse {
  uint32_t slot, use;
};
template <int D, bool KEY>
__device__ __forceinline__ SlotUse slot_of(uint32_t g, bool is_x) {
  if (D == 64) return {2 * (g % 4) + (is_x ? 1u : 0u), g / 4};
  if (KEY) {
    const uint32_t n = 2 * g + (is_x ? 0 : 1);
    return {n % 5, n / 5};
  }
  return is_x ? SlotUse{g % 3, g / 3} : SlotUse{3 + g % 2, g / 2};
}
// Whether pair g's X or Y is the last load into its slot, after gx loads of X and gy of Y.
template <int D, bool KEY>
__device__ __forceinline__ bool last_use(uint32_t g, bool is_x, uint32_t gx, uint32_t gy) {
  if (D == 64) return g + 4 >= (is_x ? gx : gy);
  if (KEY) return is_x ? g + 2 >= gy : g + 3 >= gx;   // five slots on: Y of pair g + 2, X of pair g + 3
  return is_x ? g + 3 >= gx : g + 2 >= gy;
}

enum {
  Q_FULL = 0, Q_EMPTY = 8, Q_SFULL = 16, Q_SFREE = 18, Q_IFULL = 20, Q_IEMPTY = 22, Q_PREADY = 24, Q_PFREE = 26,
  Q_STATFULL = 28, Q_STATEMPTY, Q_ACCFULL, Q_ACCFREE, Q_COLS, Q_DRAIN, Q_COUNT
};
static_assert(Q_COUNT <= 40, "barrier slots");

struct BwdParams {
  const uint32_t* bits;             // this pass's bit matrix (rows = stationary tiles)
  __nv_bfloat16 *out0, *out1;       // key pass: dV, dK; query pass: out1 = dQ
  uint32_t* counter;                // work counter of this pass
};
struct BwdCommon {
  uint32_t* state;                  // [0] error word
  uint64_t wait_ns;
  int64_t n_items;
  const float *lse2, *delta;        // [B * heads][nt_max][64]
  const int32_t* counts;            // [heads][nt_max]
  int32_t heads, bh_total, nt_max, words, key_ctas, by_head;
  float scale_log2, scale;
  int32_t hold;                     // test hook: the step to P waits for a third arrival, which nothing makes
};
struct BwdMaps {
  CUtensorMap q, k, v, dO;
};

// One pass, from this CTA's first item to the end of the pass's queue. Returns with every
// role done and its copies and products finished.
template <int D, bool KEY>
__device__ __forceinline__ void bwd_pass(const CUtensorMap& tx, const CUtensorMap& ty, const CUtensorMap& txs,
                                         const CUtensorMap& tys, const BwdCommon& prm, const BwdParams& pass,
                                         uint8_t* smem, uint32_t tmem, volatile uint32_t* abort_flag) {
  using L = BSmem<D, KEY>;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::oBar + 8u * uint32_t(i); };
  BwdItem* items = reinterpret_cast<BwdItem*>(smem + L::oItem);
  BwdPair* pairs = reinterpret_cast<BwdPair*>(smem + L::oPair);
  uint32_t* gerr = prm.state;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kH = D / 64;                     // 64-channel halves
  constexpr int kIssuers = KEY ? 4 : 3;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(bar(Q_FULL + i), 1);
      mbar_init(bar(Q_EMPTY + i), D == 64 && KEY ? 2 : 1);   // d = 64: acc0 and acc1 read both of [Y; X]
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Q_SFULL + i), prm.hold ? 3 : 2);   // S and dP
      mbar_init(bar(Q_SFREE + i), 8);            // one arrival per warp of the warpgroups
      mbar_init(bar(Q_IFULL + i), 1);
      mbar_init(bar(Q_IEMPTY + i), kIssuers + 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Q_PREADY + i), 8);
      mbar_init(bar(Q_PFREE + i), kIssuers - 2);
    }
    mbar_init(bar(Q_STATFULL), 1);
    mbar_init(bar(Q_STATEMPTY), 2);              // S and dP
    mbar_init(bar(Q_ACCFULL), kIssuers - 2);
    mbar_init(bar(Q_ACCFREE), 8);
    mbar_init(bar(Q_COLS), 8);
    mbar_init(bar(Q_DRAIN), kIssuers);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  // TMEM: buffer b at columns 128 b: S [0, 64), dP [64, 128); acc0 (dV^T) at 256, acc1 (dK^T / dQ^T) at 320

  if (warp == 0) {
    // ---------------------------------------------------------- producer ---
    uint32_t g = 0;                              // streamed pairs issued by this lane (0: X, 1: Y)
    int stat_it = -1;                            // last item whose stationary phase is under way or over
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      if (lane == 0) ok = wait_bar(bar(Q_IEMPTY + slot), ((it >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      uint32_t item = 0;
      if (lane == 0) item = atomicAdd(pass.counter, 1u);
      item = __shfl_sync(0xffffffffu, item, 0);
      if (int64_t(item) >= prm.n_items) {
        if (lane == 0) {
          items[slot].end = 1;
          mbar_arrive(bar(Q_IFULL + slot));
        }
        break;
      }
      // prefix tiles, which meet every tile, first: of all heads, or head by head
      const uint32_t per = prm.by_head ? prm.nt_max : prm.bh_total;
      const int hi = int(item / per), lo = int(item % per);
      const int bh = prm.by_head ? hi : lo, tile = prm.by_head ? lo : hi;
      const int h = bh % prm.heads;
      const uint32_t* row = pass.bits + (int64_t(bh) * prm.words * 32 + tile) * prm.words;
      int n = 0;
      for (int w = lane; w < prm.words; w += 32) n += __popc(row[w]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      const int npairs = (n + 1) >> 1;
      if (lane == 0) {
        BwdItem& b = items[slot];
        b.bh = bh;
        b.tile = tile;
        b.pairs = npairs;
        b.count = prm.counts[int64_t(h) * prm.nt_max + tile];
        b.end = 0;
        mbar_arrive(bar(Q_IFULL + slot));
        ok = wait_bar(bar(Q_STATEMPTY), (it & 1) ^ 1, abort_flag, gerr, prm.wait_ns);
        if (ok && npairs > 0) {
          mbar_expect_tx(bar(Q_STATFULL), 2 * L::kStat);
          const int y = (bh * prm.nt_max + tile) * 64;
          for (int c = 0; c < kH; ++c) {
            tma_load_2d(sbase + L::oStat + c * kBox, &txs, 64 * c, y, bar(Q_STATFULL));
            tma_load_2d(sbase + L::oStat + L::kStat + c * kBox, &tys, 64 * c, y, bar(Q_STATFULL));
          }
        } else if (ok) {
          mbar_arrive(bar(Q_STATFULL));          // nothing to load: keep the phases in step with the items
        }
        if (ok) stat_it = int(it);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      // the streamed tiles, two at a time, in ascending order: lane 0 loads X, lane 1 Y, each
      // at its own pace (diverged lanes make independent progress)
      if (lane < 2) {
        const bool is_x = lane == 0;
        const CUtensorMap* map = is_x ? &tx : &ty;
        int first = -1;
        uint32_t next = row[0];
        for (int w = 0; w < prm.words && ok; ++w) {
          uint32_t bitsw = next;
          const bool last = w + 1 == prm.words;
          if (!last) next = row[w + 1];
          while (ok && (bitsw || (last && first >= 0))) {
            int t = -1;                          // a tile left over at the end streams alone
            if (bitsw) {
              t = w * 32 + __ffs(bitsw) - 1;
              bitsw &= bitsw - 1;
              if (first < 0) {
                first = t;
                continue;
              }
            }
            const SlotUse u = slot_of<D, KEY>(g, is_x);
            ok = wait_bar(bar(Q_EMPTY + int(u.slot)), (u.use & 1) ^ 1, abort_flag, gerr, prm.wait_ns);
            if (!ok) break;
            if (is_x) pairs[g & 3] = BwdPair{first, t};   // read before this pair's stage is free again
            const uint32_t fb = bar(Q_FULL + int(u.slot));
            mbar_expect_tx(fb, L::kTensor);
            const int ya = (bh * prm.nt_max + first) * 64, yb = t >= 0 ? (bh * prm.nt_max + t) * 64 : ya;
            const uint32_t dst = sbase + u.slot * L::kTensor;
            for (int c = 0; c < kH; ++c) {
              tma_load_2d(dst + c * L::kHalf, map, 64 * c, ya, fb);
              tma_load_2d(dst + c * L::kHalf + kBox, map, 64 * c, yb, fb);
            }
            ++g;
            first = -1;
          }
        }
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, ok);
    }
    // Every copy lands before shared memory serves anything else, whatever the abort flag says by now: a role
    // that is still at work may give up after this one has left. Each lane waits for the last use of its slots;
    // a slot that has been used again since was empty before that.
    const uint32_t gx = __shfl_sync(0xffffffffu, g, 0), gy = __shfl_sync(0xffffffffu, g, 1);
    if (lane < 2) {
      if (lane == 0 && stat_it >= 0) drain_wait(bar(Q_STATFULL), uint32_t(stat_it) & 1);
      for (uint32_t j = g >= 4 ? g - 4 : 0; j < g; ++j) {
        const SlotUse u = slot_of<D, KEY>(j, lane == 0);
        if (last_use<D, KEY>(j, lane == 0, gx, gy)) drain_wait(bar(Q_FULL + int(u.slot)), u.use & 1);
      }
    }
    __syncwarp();
  } else if (warp == kWarpS || warp == kWarpDp) {
    // -------------------------------------------- S = X Xs^T, dP = Y Ys^T ---
    if (lane == 0) {
      const bool is_s = warp == kWarpS;
      constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0);
      const uint64_t db = sw128_desc(sbase + L::oStat + (is_s ? 0 : L::kStat), 16, 1024);
      const uint64_t da0 = sw128_desc(sbase, 16, 1024);
      const uint32_t td = tmem + (is_s ? 0 : 64);
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t it = 0; ok; ++it) {
        const int slot = it & 1;
        if (!(ok = wait_bar(bar(Q_IFULL + slot), (it >> 1) & 1, abort_flag, gerr, prm.wait_ns))) break;
        const int npairs = items[slot].pairs;
        const bool end = items[slot].end != 0;
        mbar_arrive(bar(Q_IEMPTY + slot));
        if (end) break;
        if (!(ok = wait_bar(bar(Q_STATFULL), it & 1, abort_flag, gerr, prm.wait_ns))) break;
        for (int j = 0; j < npairs; ++j, ++g) {
          const uint32_t b = g & 1;
          const SlotUse u = slot_of<D, KEY>(g, is_s);
          // The buffer's previous pair has been read: first, because it also says that the slot's previous load has
          // landed. In the ring that X and Y share, Y of pair g follows X of pair g - 2, which this issuer has not
          // waited for: with that load still on its way, the parity of Y's phase reads as if it had passed.
          if (!(ok = wait_bar(bar(Q_SFREE + int(b)), ((g >> 1) & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
          if (!(ok = wait_bar(bar(Q_FULL + int(u.slot)), u.use & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint64_t da = da0 + u.slot * (L::kTensor >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma(td + b * 128, da + (((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4),
                   db + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
          tc_commit(bar(Q_SFULL + int(b)));
          if constexpr (!KEY && D == 128) {
            if (!is_s) tc_commit(bar(Q_EMPTY + int(u.slot)));   // dP is the query pass's only use of Y
          }
        }
        if (ok) tc_commit(bar(Q_STATEMPTY));
      }
      tc_commit(bar(Q_DRAIN));
      drain_wait(bar(Q_DRAIN), 0);
    }
    __syncwarp();
  } else if (warp == kWarpAcc1 || warp == kWarpAcc0) {
    // ---------------------------------- acc1^T += X^T dS, acc0^T += Y^T P ---
    if (lane == 0 && (KEY || warp == kWarpAcc1)) {
      const bool is1 = warp == kWarpAcc1;
      constexpr uint32_t idA = idesc_bf16(128, 64, 1, 1);
      // A = X^T or Y^T, MN-major: 64-channel chunks kHalf apart. For d = 64 both are one
      // operand of 128 channels, [Y; X]: dV^T is in lanes 0-63 of acc0, dK^T / dQ^T in
      // lanes 64-127 of acc1, and the other halves are not used (Y's stage is then read
      // here too, so its release counts this product).
      const bool a_is_x = is1 && D == 128;
      const uint64_t da0 = sw128_desc(sbase, L::kHalf, 1024);
      const uint64_t db0 = sw128_desc(sbase + (is1 ? L::oDs : L::oP), 8192, 1024);
      const uint32_t td = tmem + (is1 ? 320 : 256);
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t it = 0; ok; ++it) {
        const int slot = it & 1;
        if (!(ok = wait_bar(bar(Q_IFULL + slot), (it >> 1) & 1, abort_flag, gerr, prm.wait_ns))) break;
        const int npairs = items[slot].pairs;
        const bool end = items[slot].end != 0;
        mbar_arrive(bar(Q_IEMPTY + slot));
        if (end) break;
        // the accumulators are free once the previous item's gradients are read
        if (!(ok = wait_bar(bar(Q_ACCFREE), (it & 1) ^ 1, abort_flag, gerr, prm.wait_ns))) break;
        for (int j = 0; j < npairs; ++j, ++g) {
          const SlotUse u = slot_of<D, KEY>(g, a_is_x);
          if (!(ok = wait_bar(bar(Q_FULL + int(u.slot)), u.use & 1, abort_flag, gerr, prm.wait_ns))) break;
          const uint32_t pb = g % L::kPdBufs;
          if (!(ok = wait_bar(bar(Q_PREADY + int(pb)), (g / L::kPdBufs) & 1, abort_flag, gerr, prm.wait_ns))) break;
          tc_fence_after();
          const uint64_t da = da0 + u.slot * (L::kTensor >> 4), db = db0 + pb * (L::kPd >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)         // 16 streamed rows per step
            tc_mma(td, da + ((kk * 2048) >> 4), db + ((kk * 2048) >> 4), idA, (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit(bar(Q_PFREE + int(pb)));
          tc_commit(bar(Q_EMPTY + int(u.slot)));
          if (D == 64) tc_commit(bar(Q_EMPTY + int(u.slot) + 1));   // X of [Y; X]
        }
        if (ok) tc_commit(bar(Q_ACCFULL));
      }
      tc_commit(bar(Q_DRAIN));
      drain_wait(bar(Q_DRAIN), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- P, dS, output ---
    const int wg = (warp - 4) >> 2;
    const int q4 = warp & 3;                     // TMEM lane quarter this warp may read
    const int r = q4 * 32 + lane;                // streamed row, TMEM lane
    const uint32_t lane_off = uint32_t(q4 * 32) << 16;
    const int c0 = 32 * wg;                      // my warpgroup's 32 of the stationary tile's 64 rows
    float* cols = reinterpret_cast<float*>(smem + L::oCol);   // query pass: -lse2 [64], -delta [64] of two items
    const uint64_t c2 = f2pack(prm.scale_log2, prm.scale_log2);
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      ok = wait_bar(bar(Q_IFULL + slot), (it >> 1) & 1, abort_flag, gerr, prm.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      const BwdItem inf = items[slot];
      warp_arrive(bar(Q_IEMPTY + slot));
      if (inf.end) break;
      const int h = inf.bh % prm.heads;
      const int64_t base = int64_t(inf.bh) * prm.nt_max;
      if constexpr (!KEY) {
        // the stationary queries' lse2 and delta, negated, in this item's buffer: every warp has
        // read what it held two items ago before it arrived for the last item
        float* col = cols + slot * 128;
        if (warp < 8) {
          const int x = (warp - 4) * 32 + lane;
          col[x] = -(x < 64 ? prm.lse2[(base + inf.tile) * 64 + x] : prm.delta[(base + inf.tile) * 64 + x - 64]);
        }
        warp_arrive(bar(Q_COLS));
        ok = wait_bar(bar(Q_COLS), it & 1, abort_flag, gerr, prm.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      for (int j = 0; j < inf.pairs; ++j, ++g) {
        const SlotUse u = slot_of<D, KEY>(g, true);
        ok = wait_bar(bar(Q_FULL + int(u.slot)), u.use & 1, abort_flag, gerr, prm.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const BwdPair pr = pairs[g & 3];
        const int tile = r < 64 ? pr.ta : pr.tb;
        // key pass: minus lse2 and minus delta of my query row (an unused slot's lse2 is +inf,
        // which makes its P and dS 0); query pass: whether my key row is one
        float rl = -INFINITY, rd = 0.f;
        bool live = true;
        if constexpr (KEY) {
          if (tile >= 0) {
            rl = -prm.lse2[(base + tile) * 64 + (r & 63)];
            rd = -prm.delta[(base + tile) * 64 + (r & 63)];
          }
        } else {
          live = tile >= 0 && (r & 63) < prm.counts[int64_t(h) * prm.nt_max + tile];
        }
        const int b = int(g & 1);
        ok = wait_bar(bar(Q_SFULL + b), (g >> 1) & 1, abort_flag, gerr, prm.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[32], dp[32];
        tmem_ld32(tmem + b * 128 + lane_off + c0, s);
        tmem_ld32(tmem + b * 128 + 64 + lane_off + c0, dp);
        tmem_wait_ld(s);
        reg_fence(dp);
        tc_fence_before();
        warp_arrive(bar(Q_SFREE + b));
        const uint64_t rl2 = f2pack(rl, rl), rd2 = f2pack(rd, rd);
        uint32_t pk[KEY ? 16 : 1], dk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint64_t l2 = rl2, dl = rd2;
          if constexpr (!KEY) {
            l2 = *reinterpret_cast<const uint64_t*>(cols + slot * 128 + c0 + 2 * e);
            dl = *reinterpret_cast<const uint64_t*>(cols + slot * 128 + 64 + c0 + 2 * e);
          }
          float x0, x1, d0, d1;
          f2unpack(ffma2(f2pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, l2), x0, x1);
          x0 = ex2(x0);
          x1 = ex2(x1);
          if constexpr (!KEY) {
            x0 = live ? x0 : 0.f;
            x1 = live ? x1 : 0.f;
          }
          f2unpack(fmul2(f2pack(x0, x1),
                         fadd2(f2pack(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1])), dl)),
                   d0, d1);
          if constexpr (KEY) pk[e] = bf16x2(x0, x1);
          dk[e] = bf16x2(d0, d1);
        }
        // the P and dS last in this buffer have been consumed by their products
        const uint32_t pb = g % L::kPdBufs;
        ok = wait_bar(bar(Q_PFREE + int(pb)), ((g / L::kPdBufs) & 1) ^ 1, abort_flag, gerr, prm.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        // row r: 128 bytes, 16-byte chunks swizzled by the row; my warpgroup's four
        uint8_t* drow = smem + L::oDs + pb * L::kPd + r * 128;
        uint8_t* prow = smem + L::oP + pb * L::kPd + r * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = ((4 * wg + i) ^ (r & 7)) * 16;
          *reinterpret_cast<uint4*>(drow + at) = make_uint4(dk[4 * i], dk[4 * i + 1], dk[4 * i + 2], dk[4 * i + 3]);
          if constexpr (KEY)
            *reinterpret_cast<uint4*>(prow + at) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        warp_arrive(bar(Q_PREADY + int(pb)));
      }
      if (!ok) break;
      // the finished gradients: lanes = channels, columns = the tile's rows. Key pass:
      // warpgroup 0 writes dV, 1 writes dK; query pass: 32 rows of dQ each.
      ok = wait_bar(bar(Q_ACCFULL), it & 1, abort_flag, gerr, prm.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const bool is_v = KEY && wg == 0;
      const int ch = D == 128 ? r : (is_v ? r : r - 64);
      const bool mine = ch >= 0 && ch < D;
      __nv_bfloat16* out = (is_v ? pass.out0 : pass.out1) + (base + inf.tile) * 64 * D + (mine ? ch : 0);
      const float f = is_v ? 1.f : prm.scale;
#pragma unroll 1
      for (int c = KEY ? 0 : c0; c < (KEY ? 64 : c0 + 32); c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + (is_v ? 256 : 320) + lane_off + c, v);
        tmem_wait_ld(v);
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int row = c + i;
            const float x = (row < inf.count && inf.pairs > 0) ? __uint_as_float(v[i]) * f : 0.f;
            out[int64_t(row) * D] = __float2bfloat16_rn(x);
          }
        }
      }
      tc_fence_before();
      warp_arrive(bar(Q_ACCFREE));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0)                          // the other pass lays out shared memory anew
    for (int i = 0; i < Q_COUNT; ++i) mbar_inval(bar(i));
}

// The two passes in one launch: the first key_ctas CTAs begin with the key pass, the others
// with the query pass, and each goes on to the other pass's queue when its own is empty.
template <int D>
__global__ void __launch_bounds__(kBThreads, 1)
    attn_bwd_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdCommon prm,
                    const __grid_constant__ BwdParams key, const __grid_constant__ BwdParams qry) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint32_t misc[2];                   // TMEM base, abort flag
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    misc[1] = 0u;
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
    prefetch_map(&maps.dO);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(misc)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  volatile uint32_t* abort_flag = misc + 1;
  wait_predecessor();
  const bool key_first = int(blockIdx.x) < prm.key_ctas;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if ((i == 0) == key_first)
      bwd_pass<D, true>(maps.q, maps.dO, maps.k, maps.v, prm, key, smem, tmem, abort_flag);
    else
      bwd_pass<D, false>(maps.k, maps.v, maps.q, maps.dO, prm, qry, smem, tmem, abort_flag);
    if (*abort_flag) break;                      // uniform: every role has passed the barrier at the pass's end
  }
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// -------------------------------------------------------------------- host ----

inline int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

struct BwdLayout {
  int words;
  int64_t rows_bytes, bits_bytes;
  int64_t oLse, oDelta, oBits, oBitsT, total;
};
BwdLayout bwd_layout(const Geometry& g) {
  BwdLayout l;
  l.words = (g.nt_max + 31) / 32;
  l.rows_bytes = round256(int64_t(g.B) * g.Hh * g.nt_max * VSA_TILE * 4);
  l.bits_bytes = round256(int64_t(g.B) * g.Hh * l.words * 32 * l.words * 4);
  l.oLse = 256;                                  // the two work counters first
  l.oDelta = l.oLse + l.rows_bytes;
  l.oBits = l.oDelta + l.rows_bytes;
  l.oBitsT = l.oBits + l.bits_bytes;
  l.total = l.oBitsT + l.bits_bytes;
  return l;
}

template <int D>
constexpr int kBwdSmem =
    1024 + int(BSmem<D, true>::oEnd > BSmem<D, false>::oEnd ? BSmem<D, true>::oEnd : BSmem<D, false>::oEnd);
static_assert(kBwdSmem<64> <= kBwdSmem<128> && kBwdSmem<128> + 1024 <= 227 * 1024, "shared memory of one CTA");
constexpr int kMaxBitSmem = 8 * (65536 / 32) * 4;   // eight rows of the largest bit matrix

template <int D>
cudaError_t run_passes(const vsa_plan* p, const BwdMaps& maps, const BwdCommon& prm, const BwdParams& key,
                       const BwdParams& qry, cudaStream_t s) {
  const int64_t items = 2 * prm.n_items;
  return launch_after(attn_bwd_kernel<D>, dim3(unsigned(items < p->num_sms ? items : p->num_sms)), unsigned(kBThreads),
                      size_t(kBwdSmem<D>), s, 1, maps, prm, key, qry);
}

template <int CPR>
cudaError_t run_prepare(const vsa_plan* p, const void* op, const void* dop, const float* lse, float* lse2, float* delta,
                        uint32_t* counters, const BitParams& bp, int64_t bit_rows, cudaStream_t s) {
  const Geometry& g = p->geo;
  const int64_t rows = int64_t(g.B) * g.Hh * g.nt_max * VSA_TILE, per = 256 / CPR;
  const int64_t want = (rows + per - 1) / per, cap = int64_t(p->num_sms) * 8;
  const int row_blocks = int(want < cap ? want : cap);
  const int smem = 8 * bp.words * 4;
  return launch_after(bwd_prepare_kernel<CPR>, dim3(unsigned(row_blocks + (bit_rows + 7) / 8)), 256u, size_t(smem), s, 1,
                      g, row_blocks, static_cast<const uint4*>(op), static_cast<const uint4*>(dop), lse,
                      p->d_tile_count, lse2, delta, counters, bp, bit_rows);
}

}  // namespace

// Shared-memory limits of the kernels, once per device (plan creation).
cudaError_t prepare_attn_bwd() {
  const auto at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_kernel<128>, at, kBwdSmem<128>);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_bwd_kernel<64>, at, kBwdSmem<64>);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(bwd_prepare_kernel<16>, at, kMaxBitSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(bwd_prepare_kernel<8>, at, kMaxBitSmem);
  return e;
}

int64_t attn_bwd_workspace_bytes(const vsa_plan* p) { return bwd_layout(p->geo).total; }

cudaError_t launch_attn_bwd(const vsa_plan* p, const void* qp, const void* kp, const void* vp, const void* op,
                            const float* lse, const void* dop, const int32_t* idx, const int32_t* idx_ref,
                            const int32_t* k, void* dqp, void* dkp, void* dvp, void* workspace, cudaStream_t s) {
  const Geometry& g = p->geo;
  const BwdLayout l = bwd_layout(g);
  char* ws = static_cast<char*>(workspace);
  const int64_t rows = int64_t(g.B) * g.Hh * g.nt_max * VSA_TILE;
  BwdMaps maps;
  if (!make_map(&maps.q, qp, rows, g.d) || !make_map(&maps.k, kp, rows, g.d) || !make_map(&maps.v, vp, rows, g.d) ||
      !make_map(&maps.dO, dop, rows, g.d))
    return cudaErrorInvalidValue;
  float* lse2 = reinterpret_cast<float*>(ws + l.oLse);
  float* delta = reinterpret_cast<float*>(ws + l.oDelta);
  uint32_t* counters = reinterpret_cast<uint32_t*>(ws);

  BitParams bp;
  bp.idx = idx;
  bp.idx_ref = idx_ref;
  bp.ref_tiles = p->d_ref_tiles;
  bp.prefix_ref = p->d_prefix_ref;
  bp.bits = reinterpret_cast<uint32_t*>(ws + l.oBits);
  bp.bits_t = reinterpret_cast<uint32_t*>(ws + l.oBitsT);
  bp.state = p->d_state;
  bp.heads = g.Hh;
  bp.nt_max = g.nt_max;
  bp.ntv_max = g.ntv_max;
  bp.k_max = g.k_max;
  bp.n_pre = g.n_pre_tiles;
  bp.n_ref = g.n_ref;
  bp.k_ref_max = g.k_ref_max;
  bp.words = l.words;
  for (int h = 0; h < VSA_MAX_HEADS; ++h) {
    bp.ntv[h] = h < g.Hh ? g.ntv[h] : 0;
    bp.k[h] = h < g.Hh ? k[h] : 0;
    bp.k_ref[h] = h < g.Hh ? g.k_ref[h] : 0;
  }
  const int bh = g.B * g.Hh;
  const int64_t bit_rows = int64_t(bh) * l.words * 32;
  cudaError_t e = g.d == 128 ? run_prepare<16>(p, op, dop, lse, lse2, delta, counters, bp, bit_rows, s)
                             : run_prepare<8>(p, op, dop, lse, lse2, delta, counters, bp, bit_rows, s);
  if (e != cudaSuccess) return e;
  const int64_t blocks = int64_t(bh) * l.words * l.words;
  e = launch_after(bwd_transpose_kernel, dim3(unsigned((blocks + 7) / 8)), 256u, 0, s, 1, bp.bits, bp.bits_t, l.words,
                   blocks);
  if (e != cudaSuccess) return e;

  BwdCommon prm;
  prm.state = p->d_state;
  prm.wait_ns = p->wait_ns;
  prm.hold = p->test_hold;
  prm.n_items = int64_t(bh) * g.nt_max;
  prm.lse2 = lse2;
  prm.delta = delta;
  prm.counts = p->d_tile_count;
  prm.heads = g.Hh;
  prm.nt_max = g.nt_max;
  prm.words = l.words;
  prm.scale = p->desc.softmax_scale;
  prm.scale_log2 = p->desc.softmax_scale * 1.4426950408889634f;
  // Few items: both passes at once, three fifths of the CTAs on the key pass, which takes about
  // 1.45 times the query pass's time, and the heavy items of all heads first (ragged case: 66 -> 42 us;
  // 48 head by head). Many: head by head and the key pass first, so that one head's pair of streams
  // stays in L2 (clip, three heads: 32.8 ms the first way, 29.1 head by head, 26.8 one pass
  // after the other as well; 24 medium heads: no difference).
  prm.bh_total = bh;
  const int64_t ctas = 2 * prm.n_items < p->num_sms ? 2 * prm.n_items : p->num_sms;
  prm.by_head = prm.n_items >= 4 * ctas;
  prm.key_ctas = int32_t(prm.by_head ? ctas : (ctas * 3 + 4) / 5);
  BwdParams key, qry;
  key.bits = bp.bits_t;
  key.counter = counters;
  key.out0 = static_cast<__nv_bfloat16*>(dvp);
  key.out1 = static_cast<__nv_bfloat16*>(dkp);
  qry.bits = bp.bits;
  qry.counter = counters + 1;
  qry.out0 = nullptr;
  qry.out1 = static_cast<__nv_bfloat16*>(dqp);
  return g.d == 128 ? run_passes<128>(p, maps, prm, key, qry, s) : run_passes<64>(p, maps, prm, key, qry, s);
}

}  // namespace vsa
