// RMS norm of every head's query and key row and the rotary position embedding
// in one pass, before the layer: token-major to token-major, or fused with the
// tile pack and the score stage's pooling; and the gradient of both.
//
// Forward, for a row x of head_dim d with weights w:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,
//   every channel pair (a, b) of n turns by the token's angle of that pair:
//   (a, b) -> (a cos - b sin, a sin + b cos).
// Backward, for the gradient dy of the result: dn turns back,
//   dn = (da cos + db sin, -da sin + db cos),  xr = x r,  g = dn w,
//   dx = r (g - xr mean(g xr)),  dw = sum over the rows of dn xr.
// Statistics, rotation and sums are fp32; each output is rounded to bf16 once.
//
// A row is held by d / 8 lanes, eight channels each, as four rotation pairs:
// lane c owns pairs 4c .. 4c + 3, which are channels 8c .. 8c + 7 of the
// interleaved layout (one 16-byte load) and channels 4c .. 4c + 3 and
// d/2 + 4c .. + 3 of the halves layout (two 8-byte loads that fill their
// sectors across the lanes). So both members of a pair are in one lane, the
// table rows are one float4 of cosines and one of sines per lane in either
// layout, and the only shuffles are those of the mean.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tc_sm100.h"
#include "tile_map.h"
#include "vsa_internal.h"

namespace vsa {
namespace {

using tc::f2pack;
using tc::f2unpack;
using tc::fadd2;
using tc::ffma2;
using tc::fmul2;

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// One lane's eight channels of a row in shared memory: four words of two channels.
// Interleaved: word j is pair j. Halves: words 0, 1 hold the first members of
// pairs 0 .. 3, words 2, 3 the second.
template <bool HALVES>
__device__ __forceinline__ uint4 row_of(const __nv_bfloat16* row, int d, int c) {
  if (HALVES) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * c);
    const uint2 b = *reinterpret_cast<const uint2*>(row + d / 2 + 4 * c);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  return reinterpret_cast<const uint4*>(row)[c];
}
template <bool HALVES>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int d, int c, uint4 v) {
  if (HALVES) {
    *reinterpret_cast<uint2*>(row + 4 * c) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + d / 2 + 4 * c) = make_uint2(v.z, v.w);
  } else {
    reinterpret_cast<uint4*>(row)[c] = v;
  }
}
template <bool HALVES>
__device__ __forceinline__ void to_pairs(uint4 v, float (&a)[4], float (&b)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (HALVES) {
      a[j] = (j & 1) ? hi_f32(w[j >> 1]) : lo_f32(w[j >> 1]);
      b[j] = (j & 1) ? hi_f32(w[2 + (j >> 1)]) : lo_f32(w[2 + (j >> 1)]);
    } else {
      a[j] = lo_f32(w[j]);
      b[j] = hi_f32(w[j]);
    }
  }
}
template <bool HALVES>
__device__ __forceinline__ uint4 from_pairs(const float (&a)[4], const float (&b)[4]) {
  if (HALVES)
    return make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]));
  return make_uint4(pack_bf16(a[0], b[0]), pack_bf16(a[1], b[1]), pack_bf16(a[2], b[2]), pack_bf16(a[3], b[3]));
}
// The channel of member m (0: a, 1: b) of the lane's pair j.
template <bool HALVES>
__device__ __forceinline__ int channel_of(int d, int c, int j, int m) {
  return HALVES ? m * (d / 2) + 4 * c + j : 8 * c + 2 * j + m;
}

struct Weights {
  float a[4], b[4];
};
// The lane's weights of one head (ones for a null table; rows are 16-byte aligned).
template <bool HALVES>
__device__ __forceinline__ Weights load_weights(const float* w, int d, int c) {
  Weights r;
  if (!w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.a[j] = r.b[j] = 1.f;
    return r;
  }
  const float4 x = __ldg(reinterpret_cast<const float4*>(w) + (HALVES ? c : 2 * c));
  const float4 y = __ldg(reinterpret_cast<const float4*>(w) + (HALVES ? d / 8 + c : 2 * c + 1));
  if (HALVES) {
    r.a[0] = x.x; r.a[1] = x.y; r.a[2] = x.z; r.a[3] = x.w;
    r.b[0] = y.x; r.b[1] = y.y; r.b[2] = y.z; r.b[3] = y.w;
  } else {
    r.a[0] = x.x; r.b[0] = x.y; r.a[1] = x.z; r.b[1] = x.w;
    r.a[2] = y.x; r.b[2] = y.y; r.a[3] = y.z; r.b[3] = y.w;
  }
  return r;
}

struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn load_turn(const NormRopeArgs& n, int tok, int d, int c) {
  Turn t;
  if (n.cos) {
    const float4 cs = __ldg(reinterpret_cast<const float4*>(n.cos + int64_t(tok) * (d / 2)) + c);
    const float4 sn = __ldg(reinterpret_cast<const float4*>(n.sin + int64_t(tok) * (d / 2)) + c);
    t.c[0] = cs.x; t.c[1] = cs.y; t.c[2] = cs.z; t.c[3] = cs.w;
    t.s[0] = sn.x; t.s[1] = sn.y; t.s[2] = sn.z; t.s[3] = sn.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t.c[j] = 1.f;
      t.s[j] = 0.f;
    }
  }
  return t;
}

// Sum over the CPR lanes of a row (aligned groups of the warp).
template <int CPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = CPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One level of a summing tree over lanes, of 2 n values per lane: the lane gives the
// half of them that its partner keeps and keeps the sums of the other half, so
// that the level costs n exchanges and leaves n values, different ones in the
// two lanes.
template <int N>
__device__ __forceinline__ void halve(float (&v)[2 * N], float (&out)[N], int lane_bit) {
  const bool upper = threadIdx.x & lane_bit;
#pragma unroll
  for (int i = 0; i < N; ++i)
    out[i] = (upper ? v[N + i] : v[i]) + __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[N + i], lane_bit);
}

// Sum of squares of a row by halving: channels d / 2, d / 4, .. apart are added, the
// same tree in either layout, so that every term passes through few roundings. At
// d = 128 four neighbouring channels are first added in a chain (one value per lane of
// a full warp). Squares of bf16 values are exact in fp32. Between levels in one lane
// and levels across lanes, halve() keeps the exchanges at 4 to 10 per row.
template <int CPR, bool HALVES>
__device__ __forceinline__ float square_sum(const float (&a)[4], const float (&b)[4]) {
  float s;
  if constexpr (CPR == 16) {
    float q[2];                                  // two quads: halves c and c + 16, interleaved 2c and 2c + 1
    if constexpr (HALVES) {
      q[0] = fmaf(a[3], a[3], fmaf(a[2], a[2], fmaf(a[1], a[1], a[0] * a[0])));
      q[1] = fmaf(b[3], b[3], fmaf(b[2], b[2], fmaf(b[1], b[1], b[0] * b[0])));
      s = q[0] + q[1];                           // quads 16 apart
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    } else {
      q[0] = fmaf(b[1], b[1], fmaf(a[1], a[1], fmaf(b[0], b[0], a[0] * a[0])));
      q[1] = fmaf(b[3], b[3], fmaf(a[3], a[3], fmaf(b[2], b[2], a[2] * a[2])));
      float one[1];
      halve<1>(q, one, 8);                       // quads 16 apart; the lane keeps one of its two
      s = one[0];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s += __shfl_xor_sync(0xffffffffu, s, 8);   // neighbouring quads
    }
  } else {
    float two[2], one[1];
    if constexpr (HALVES) {                      // channels 4c + j and 32 + 4c + j
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fmaf(a[j], a[j], b[j] * b[j]);   // 32 apart
      halve<2>(v, two, 4);                       // 16
      halve<1>(two, one, 2);                     // 8
      s = one[0] + __shfl_xor_sync(0xffffffffu, one[0], 1);               // 4
      s += __shfl_xor_sync(0xffffffffu, s, 4);   // 2
      s += __shfl_xor_sync(0xffffffffu, s, 2);   // 1
    } else {                                     // channels 8c .. 8c + 7
      float v[8], four[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = a[j] * a[j];
        v[2 * j + 1] = b[j] * b[j];
      }
      halve<4>(v, four, 4);                      // 32
      halve<2>(four, two, 2);                    // 16
      halve<1>(two, one, 1);                     // 8
      s = one[0] + __shfl_xor_sync(0xffffffffu, one[0], 4);               // 4
      s += __shfl_xor_sync(0xffffffffu, s, 2);   // 2
      s += __shfl_xor_sync(0xffffffffu, s, 1);   // 1
    }
  }
  return s;
}

// The normed and turned row as stored (bf16 words). Each product of the rotation
// is rounded by itself, as the formula is written: with a fused multiply-add one
// of a pair's two products would be exact and the other not (packed multiplies
// and adds get fused, so the rotation is in scalars).
template <int CPR, bool HALVES>
__device__ __forceinline__ uint4 norm_rope_row(uint4 v, const Weights& w, const Turn& t, float eps) {
  float a[4], b[4];
  to_pairs<HALVES>(v, a, b);
  const float r = rsqrtf(square_sum<CPR, HALVES>(a, b) * (1.f / (CPR * 8)) + eps);
  const uint64_t r2 = f2pack(r, r);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    f2unpack(fmul2(fmul2(f2pack(a[j], a[j + 1]), r2), f2pack(w.a[j], w.a[j + 1])), a[j], a[j + 1]);
    f2unpack(fmul2(fmul2(f2pack(b[j], b[j + 1]), r2), f2pack(w.b[j], w.b[j + 1])), b[j], b[j + 1]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float na = a[j], nb = b[j];
    a[j] = __fsub_rn(__fmul_rn(na, t.c[j]), __fmul_rn(nb, t.s[j]));
    b[j] = __fadd_rn(__fmul_rn(na, t.s[j]), __fmul_rn(nb, t.c[j]));
  }
  return from_pairs<HALVES>(a, b);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {   // off: sixteen zero bytes
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Token-major to token-major. One warp per token; its 32 / CPR lane groups
// walk the heads, so the token's table row is loaded once for all heads.
// Bound by HBM: a warp's next steps (32 / CPR rows of q and of k each) are
// requested into shared memory ahead of the one at work, across tokens too, and
// the next token's angles into registers. Sixteen rounds of blocks at most: the
// SMs do not get the same share of HBM, and with one round, every warp's tokens
// fixed, the last is 20 % behind (24 heads of 128, 112,512 tokens: 530 us; 2 rounds
// 485, 4 455, 16 434 = 6.5 TB/s; direct loads, two in flight, 500 to 590). Results may
// overwrite their inputs: a row is requested once, by the warp that writes it, and
// written after it is read.
constexpr int kFwdStages = 5, kFwdBlocks = 3;    // blocks per SM
template <int CPR, bool HALVES>
__global__ void __launch_bounds__(256, kFwdBlocks) norm_rope_kernel(NormRopeArgs n, int B, int n_tok, int heads,
                                                                    const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                                    __nv_bfloat16* qo, __nv_bfloat16* ko) {
  constexpr int D = CPR * 8, G = 32 / CPR;
  __shared__ __align__(16) uint8_t sm[8][kFwdStages][2][512];
  tc::allow_successor();
  tc::wait_predecessor();
  const int lane = threadIdx.x & 31, c = lane % CPR, grp = lane / CPR, warp = threadIdx.x >> 5;
  const int steps = (heads + G - 1) / G, dt = int(gridDim.x) * 8;
  const int64_t first = int64_t(blockIdx.x) * 8 + warp, total = int64_t(B) * n_tok;
  struct At {                                    // a place in the walk: alike in all lanes
    int b, tok, step;
    int64_t left;                                // tokens of the walk from here
  };
  auto next_token = [&](At& a) {                 // without a division
    a.left -= dt;
    a.tok += dt;
    while (a.tok >= n_tok) {
      a.tok -= n_tok;
      ++a.b;
    }
  };
  At now;
  now.b = int(first / n_tok);
  now.tok = int(first - int64_t(now.b) * n_tok);
  now.step = 0;
  now.left = total - first;
  At ahead = now;                                // the step to request next
  uint32_t issued = 0, done = 0;                 // steps, which take the stages in turn
  auto request_next = [&] {                      // one group of copies for every step, past the end an empty one
    if (ahead.left > 0) {
      const int h = ahead.step * G + grp;
      const bool on = h < heads;
      const int64_t off = (on ? h : 0) * D + 8 * c;
      const uint32_t dst = tc::smem_u32(sm[warp][issued % kFwdStages][0]) + lane * 16;
      cp_async16(dst, q + ahead.b * n.st[0].batch + ahead.tok * n.st[0].token + off, on);
      cp_async16(dst + 512, k + ahead.b * n.st[1].batch + ahead.tok * n.st[1].token + off, on);
      if (++ahead.step == steps) {
        ahead.step = 0;
        next_token(ahead);
      }
    }
    cp_commit();
    ++issued;
  };
#pragma unroll
  for (int i = 0; i < kFwdStages - 1; ++i) request_next();
  Weights wq = load_weights<HALVES>(n.w_q, D, c), wk = load_weights<HALVES>(n.w_k, D, c);
  Turn next = load_turn(n, now.left > 0 ? now.tok : 0, D, c);
  while (now.left > 0) {
    const Turn t = next;
    __nv_bfloat16* qw = qo + now.b * n.st[2].batch + now.tok * n.st[2].token;
    __nv_bfloat16* kw = ko + now.b * n.st[3].batch + now.tok * n.st[3].token;
    next_token(now);
    if (now.left > 0) next = load_turn(n, now.tok, D, c);
    for (int step = 0; step < steps; ++step, ++done) {
      request_next();
      cp_wait<kFwdStages - 1>();
      __syncwarp();                              // a row's chunks were requested by the lanes that share it
      const int h = step * G + grp;
      const uint8_t* in = sm[warp][done % kFwdStages][0] + grp * CPR * 16;
      if (n.per_head && h < heads) {
        wq = load_weights<HALVES>(n.w_q ? n.w_q + h * D : nullptr, D, c);
        wk = load_weights<HALVES>(n.w_k ? n.w_k + h * D : nullptr, D, c);
      }
      const uint4 yq = norm_rope_row<CPR, HALVES>(row_of<HALVES>(reinterpret_cast<const __nv_bfloat16*>(in), D, c), wq, t, n.eps);
      const uint4 yk =
          norm_rope_row<CPR, HALVES>(row_of<HALVES>(reinterpret_cast<const __nv_bfloat16*>(in + 512), D, c), wk, t, n.eps);
      if (h < heads) {
        store_row<HALVES>(qw + h * D, D, c, yq);
        store_row<HALVES>(kw + h * D, D, c, yk);
      }
      __syncwarp();                              // the stage may be filled again
    }
  }
}

// Fused with the pack and the pooling: one CTA of 256 threads per (batch, tile, a
// run of `run` heads). Bound by HBM, and next to it by L2: the table rows of a
// tile are two thirds of its q, k and v rows' bytes, so a thread keeps its rows'
// angles in registers for all heads of the run that share a tile shape. The rows
// of a head (48 KB at d = 128) are requested at once into one of two buffers, the
// next head's while this one is worked on, so that the bytes in flight do not
// depend on registers. Unused slots arrive as zeros. Full clip (24 heads of 128, 112,512
// tokens): 0.66 ms, 6.4 TB/s; 0.78 with a table read per head, 1.20 with one pass of
// loads per thread into registers. Lanes and rows as in the pack kernel; the
// descriptors are pooled from the rounded rows in the same order as there, so packed
// tiles and descriptors equal, bit for bit, those of the token-major pass followed by
// the pack. Tiles past a head's own are zero, their descriptors too.
template <int CPR, bool TRIP>
struct PackSmem {
  static constexpr int D = CPR * 8, NS = TRIP ? 3 : 1;
  static constexpr uint32_t kTensor = VSA_TILE * D * 2;
  static constexpr uint32_t kPart = NS * 2 * 8 * D * 4;        // pooling partials, over the rows once they are read
  static constexpr uint32_t kBuf = 3 * kTensor > kPart ? 3 * kTensor : kPart;
  static constexpr uint32_t kBytes = 2 * kBuf;
};
template <int CPR, bool HALVES, bool TRIP>
__global__ void __launch_bounds__(256, 2)
    norm_rope_pack_kernel(NormRopeArgs n, Geometry g, int run, const __nv_bfloat16* q, const __nv_bfloat16* k,
                          const __nv_bfloat16* v, __nv_bfloat16* qp, __nv_bfloat16* kp, __nv_bfloat16* vp,
                          const int32_t* __restrict__ counts, float* pq, float* pk) {
  constexpr int D = CPR * 8;
  constexpr int KD = TRIP ? 3 * D : D;
  constexpr int RG = 256 / CPR, RPT = 64 / RG;
  constexpr int NS = TRIP ? 3 : 1;
  extern __shared__ __align__(16) uint8_t rows[];              // two of [q, k, v][64][D] bf16
  __shared__ int32_t toks[2][VSA_TILE];
  using L = PackSmem<CPR, TRIP>;
  const int runs = (g.Hh + run - 1) / run;
  const int h0 = int(blockIdx.x % runs) * run, h1 = min(g.Hh, h0 + run);
  const int64_t bn = blockIdx.x / runs;
  const int tile_n = int(bn % g.nt_max), b = int(bn / g.nt_max);
  const int c = threadIdx.x % CPR, rg = threadIdx.x / CPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vt = tile_n - g.n_pre_tiles;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint32_t base = tc::smem_u32(rows);
  tc::allow_successor();
  tc::wait_predecessor();

  // Which token list head h uses: a head of another tile shape than the one before it
  // fills the other list (the divisions cost more than a row's arithmetic: once per slot).
  int list_next = 0;
  auto same_tiles = [&](int a, int h) { return g.pt[a] == g.pt[h] && g.ph[a] == g.ph[h] && g.pw[a] == g.pw[h]; };
  auto make_list = [&](int h) {                  // uniform over the CTA
    if (h > h0) {
      if (same_tiles(h - 1, h)) return;
      list_next ^= 1;
    }
    if (threadIdx.x < VSA_TILE) toks[list_next][threadIdx.x] = src_token(g, h, tile_n, threadIdx.x);
    __syncthreads();
  };
  auto request = [&](int h, int buf) {
    const __nv_bfloat16* src[3] = {q, k, v};
#pragma unroll
    for (int z = 0; z < 3; ++z) {
      const __nv_bfloat16* at = src[z] + b * n.st[z].batch + h * D + 8 * c;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int s = rg + RG * i, tok = toks[list_next][s];
        cp_async16(base + buf * L::kBuf + z * L::kTensor + (s * D + 8 * c) * 2, at + (tok >= 0 ? tok : 0) * n.st[z].token,
                   tok >= 0);
      }
    }
  };
  make_list(h0);
  request(h0, 0);
  cp_commit();
  int list = 0;                                  // the list of the head at work
  Turn turn[RPT];
  Weights wq = load_weights<HALVES>(n.w_q, D, c), wk = load_weights<HALVES>(n.w_k, D, c);
  for (int h = h0; h < h1; ++h) {
    const int buf = (h - h0) & 1;
    if (h == h0 || !same_tiles(h - 1, h)) {
      list = list_next;                          // made when this head's rows were requested
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int tok = toks[list][rg + RG * i];
        turn[i] = load_turn(n, tok >= 0 ? tok : 0, D, c);
      }
    }
    if (n.per_head) {
      wq = load_weights<HALVES>(n.w_q ? n.w_q + h * D : nullptr, D, c);
      wk = load_weights<HALVES>(n.w_k ? n.w_k + h * D : nullptr, D, c);
    }
    if (h + 1 < h1) {
      make_list(h + 1);
      request(h + 1, buf ^ 1);
    }
    cp_commit();
    cp_wait<1>();                                // this head's rows
    __syncwarp();                                // a row's chunks were requested by the lanes that share it
    const int bh = b * g.Hh + h;
    const int64_t tile = int64_t(bh) * g.nt_max + tile_n;
    const bool pool = vt >= 0 && vt < g.ntv[h];  // uniform over the CTA
    float st[NS][2][8];                          // [statistic][q, k][pair j: a, then b]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        st[0][t][e] = 0.f;
        if (TRIP) {
          st[NS - 2][t][e] = -INFINITY;
          st[NS - 1][t][e] = INFINITY;
        }
      }
    const __nv_bfloat16* sm = reinterpret_cast<const __nv_bfloat16*>(rows + buf * L::kBuf);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int s = rg + RG * i;
      const bool on = toks[list][s] >= 0;
      const int64_t row = (tile * VSA_TILE + s) * D;
      uint4 y[2];
      y[0] = norm_rope_row<CPR, HALVES>(row_of<HALVES>(sm + s * D, D, c), wq, turn[i], n.eps);
      y[1] = norm_rope_row<CPR, HALVES>(row_of<HALVES>(sm + (VSA_TILE + s) * D, D, c), wk, turn[i], n.eps);
      if (!on) y[0] = y[1] = zero;
      store_row<HALVES>(qp + row, D, c, y[0]);
      store_row<HALVES>(kp + row, D, c, y[1]);
      reinterpret_cast<uint4*>(vp + row)[c] = *reinterpret_cast<const uint4*>(sm + (2 * VSA_TILE + s) * D + 8 * c);
      if (pool && on) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float a[4], bb[4];
          to_pairs<HALVES>(y[z], a, bb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            st[0][z][j] += a[j];
            st[0][z][4 + j] += bb[j];
            if (TRIP) {
              st[NS - 2][z][j] = fmaxf(st[NS - 2][z][j], a[j]);
              st[NS - 2][z][4 + j] = fmaxf(st[NS - 2][z][4 + j], bb[j]);
              st[NS - 1][z][j] = fminf(st[NS - 1][z][j], a[j]);
              st[NS - 1][z][4 + j] = fminf(st[NS - 1][z][4 + j], bb[j]);
            }
          }
        }
      }
    }
    if (pool) {
#pragma unroll
      for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            st[0][t][e] += __shfl_xor_sync(0xffffffffu, st[0][t][e], o);
            if (TRIP) {
              st[NS - 2][t][e] = fmaxf(st[NS - 2][t][e], __shfl_xor_sync(0xffffffffu, st[NS - 2][t][e], o));
              st[NS - 1][t][e] = fminf(st[NS - 1][t][e], __shfl_xor_sync(0xffffffffu, st[NS - 1][t][e], o));
            }
          }
      __syncthreads();                           // every row is read: the partials take their place
      float* part = reinterpret_cast<float*>(rows + buf * L::kBuf);   // [statistic][q, k][warp][D]
      if (lane < CPR) {
#pragma unroll
        for (int z = 0; z < NS; ++z)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              part[((z * 2 + t) * 8 + warp) * D + channel_of<HALVES>(D, c, e & 3, e >> 2)] = st[z][t][e];
      }
      __syncthreads();
      if (threadIdx.x < 2 * D) {
        const int t = threadIdx.x / D, ch = threadIdx.x % D;
        float sum = 0.f, mx = -INFINITY, mn = INFINITY;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          sum += part[(t * 8 + w) * D + ch];
          if (TRIP) {
            mx = fmaxf(mx, part[(((NS - 2) * 2 + t) * 8 + w) * D + ch]);
            mn = fminf(mn, part[(((NS - 1) * 2 + t) * 8 + w) * D + ch]);
          }
        }
        const float cnt = float(counts[h * g.nt_max + tile_n]);
        float* out = (t ? pk : pq) + (int64_t(bh) * g.ntv_max + vt) * KD;
        out[ch] = sum / cnt;
        if (TRIP) {
          out[D + ch] = mx;
          out[2 * D + ch] = mn;
        }
      }
    } else if (vt >= 0 && threadIdx.x < 2 * D) { // no such tile in this head
      for (int z = 0; z < NS; ++z)
        (threadIdx.x / D ? pk : pq)[(int64_t(bh) * g.ntv_max + vt) * KD + z * D + threadIdx.x % D] = 0.f;
    }
    __syncthreads();                             // the buffer (and the other token list) may be filled again
  }
}

// Gradient rows: dx from dy and x, and the row's share of dw, two pairs at a time in packed fp32.
template <int CPR, bool HALVES>
__device__ __forceinline__ uint4 norm_rope_grad_row(uint4 vy, uint4 vx, const Weights& w, const Turn& t, float eps,
                                                    uint64_t (&dwa)[2], uint64_t (&dwb)[2]) {
  float xa[4], xb[4], ya[4], yb[4];
  to_pairs<HALVES>(vx, xa, xb);
  to_pairs<HALVES>(vy, ya, yb);
  const float r = rsqrtf(square_sum<CPR, HALVES>(xa, xb) * (1.f / (CPR * 8)) + eps);
  const uint64_t r2 = f2pack(r, r);
  uint64_t ra[2], rb[2], ga[2], gb[2], dot = 0ull;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint64_t c = f2pack(t.c[2 * j], t.c[2 * j + 1]), s = f2pack(t.s[2 * j], t.s[2 * j + 1]);
    const uint64_t y0 = f2pack(ya[2 * j], ya[2 * j + 1]), y1 = f2pack(yb[2 * j], yb[2 * j + 1]);
    const uint64_t da = ffma2(y0, c, fmul2(y1, s));
    const uint64_t db = ffma2(y1, c, fmul2(y0, s) ^ 0x8000000080000000ull);
    ra[j] = fmul2(f2pack(xa[2 * j], xa[2 * j + 1]), r2);
    rb[j] = fmul2(f2pack(xb[2 * j], xb[2 * j + 1]), r2);
    dwa[j] = ffma2(da, ra[j], dwa[j]);
    dwb[j] = ffma2(db, rb[j], dwb[j]);
    ga[j] = fmul2(da, f2pack(w.a[2 * j], w.a[2 * j + 1]));
    gb[j] = fmul2(db, f2pack(w.b[2 * j], w.b[2 * j + 1]));
    dot = ffma2(ga[j], ra[j], ffma2(gb[j], rb[j], dot));
  }
  float d0, d1;
  f2unpack(dot, d0, d1);
  const float m = -row_sum<CPR>(d0 + d1) * (1.f / (CPR * 8));
  const uint64_t m2 = f2pack(m, m);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f2unpack(fmul2(r2, ffma2(ra[j], m2, ga[j])), ya[2 * j], ya[2 * j + 1]);
    f2unpack(fmul2(r2, ffma2(rb[j], m2, gb[j])), yb[2 * j], yb[2 * j + 1]);
  }
  return from_pairs<HALVES>(ya, yb);
}

// One warp per token and all heads (weights shared by the heads), or with
// PER_HEAD one lane group per token of the block's own head (blockIdx.y), so
// that the lanes' weight-gradient sums belong to one weight row in both.
// PACKED: dy (and dv, which is only moved) come from packed tiles. The blocks'
// partial sums of dw go to `part` [blockIdx.y][blockIdx.x][q, k][d], summed in
// block order by the kernel below: no atomics, the same result every time.
// Bound by HBM: a warp's next steps (32 / CPR rows of every input each) are
// requested into shared memory ahead of the one at work, across tokens too; the
// clip takes 0.86 ms, 6.5 TB/s (weights per head 0.95), with one step's loads in
// registers 1.08. With PER_HEAD a step is a
// token, so its table rows are requested along with it.
template <int CPR, bool PACKED, bool PER_HEAD>
struct GradSmem {
  static constexpr int kStages = PER_HEAD ? 3 : 2;
  static constexpr int kRows = PACKED ? 5 : 4;                 // dy_q, dy_k, q, k (, dv)
  static constexpr int kIn = kRows + (PER_HEAD ? 2 : 0);       // (, cos, sin)
  static constexpr uint32_t kStep = kIn * 512;                 // one warp's step: 32 chunks of each input
  static constexpr uint32_t oRed = 8 * kStages * kStep;
  static constexpr uint32_t oRow = oRed + 8 * 2 * CPR * 8 * 4;
  static constexpr uint32_t kBytes = oRow + 8 * VSA_MAX_HEADS * 4;
};
template <int CPR, bool HALVES, bool PACKED, bool PER_HEAD>
__global__ void __launch_bounds__(256, 2) norm_rope_bwd_kernel(NormRopeArgs n, Geometry g, const __nv_bfloat16* dyq,
                                                               const __nv_bfloat16* dyk, const __nv_bfloat16* dyv,
                                                               const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                               __nv_bfloat16* dq, __nv_bfloat16* dk,
                                                               __nv_bfloat16* dv, float* part) {
  constexpr int D = CPR * 8, G = 32 / CPR;
  using L = GradSmem<CPR, PACKED, PER_HEAD>;
  extern __shared__ __align__(16) uint8_t sm[];
  tc::allow_successor();
  tc::wait_predecessor();
  const int lane = threadIdx.x & 31, c = lane % CPR, grp = lane / CPR, warp = threadIdx.x >> 5;
  uint8_t* stage = sm + warp * L::kStages * L::kStep;
  int32_t* prow = reinterpret_cast<int32_t*>(sm + L::oRow) + warp * VSA_MAX_HEADS;   // the requested token's, by head
  const int64_t woff = PER_HEAD && n.per_head ? int64_t(blockIdx.y) * D : 0;
  const Weights wq = load_weights<HALVES>(n.w_q ? n.w_q + woff : nullptr, D, c);
  const Weights wk = load_weights<HALVES>(n.w_k ? n.w_k + woff : nullptr, D, c);
  uint64_t acc[2][2][2] = {}, tok_acc[2][2][2] = {};   // [q, k][a, b][two pairs]; a token's own sum first: shorter chains
  const int64_t total = int64_t(g.B) * g.n_tokens;
  constexpr int TPW = PER_HEAD ? G : 1;          // tokens per warp and step
  const int64_t first = (int64_t(blockIdx.x) * 8 + warp) * TPW + (PER_HEAD ? grp : 0);
  const int dt = int(gridDim.x) * 8 * TPW;
  const int steps = PER_HEAD ? 1 : (g.Hh + G - 1) / G;         // per token

  // A place in the walk: this lane's token (a lane group's own with PER_HEAD) and, among
  // its steps, the head. left: tokens of the whole walk from here, which decides
  // alike for all lanes; on: this lane has a row.
  struct At {
    int b, tok, step;
    int64_t left;
  };
  auto advance = [&](At& a) {                    // the next step, or the next token without a division
    if (++a.step < steps) return;
    a.step = 0;
    a.left -= dt;
    a.tok += dt;
    while (a.tok >= g.n_tokens) {
      a.tok -= g.n_tokens;
      ++a.b;
    }
  };
  auto head_of = [&](const At& a) { return PER_HEAD ? int(blockIdx.y) : a.step * G + grp; };
  auto on = [&](const At& a) { return a.b < g.B && head_of(a) < g.Hh; };
  auto more = [&](const At& a) { return a.left > 0; };
  auto request = [&](const At& a, uint32_t buf) {   // warp-wide
    const bool is_on = on(a);
    const int h = is_on ? head_of(a) : 0, bb = is_on ? a.b : 0, tok = is_on ? a.tok : 0;
    if constexpr (PACKED && !PER_HEAD) {
      if (a.step == 0) {                         // a new token: every head's packed row
        __syncwarp();                            // the previous token's rows are read
        for (int i = lane; i < g.Hh; i += 32) prow[i] = packed_row(g, i, a.tok);
        __syncwarp();
      }
    }
    const __nv_bfloat16* src[5];
    if constexpr (PACKED) {
      const int pr = PER_HEAD ? packed_row(g, h, tok) : prow[h];
      const int64_t row = (int64_t(bb * g.Hh + h) * g.nt_max * VSA_TILE + pr) * D;
      src[0] = dyq + row;
      src[1] = dyk + row;
      src[4] = dyv + row;
    } else {
      src[0] = dyq + bb * n.st[5].batch + tok * n.st[5].token + h * D;
      src[1] = dyk + bb * n.st[6].batch + tok * n.st[6].token + h * D;
    }
    src[2] = q + bb * n.st[0].batch + tok * n.st[0].token + h * D;
    src[3] = k + bb * n.st[1].batch + tok * n.st[1].token + h * D;
    const uint32_t dst = tc::smem_u32(stage + buf * L::kStep) + lane * 16;
#pragma unroll
    for (int z = 0; z < L::kRows; ++z) cp_async16(dst + z * 512, src[z] + 8 * c, is_on);
    if constexpr (PER_HEAD) {
      if (n.cos) {
        cp_async16(dst + L::kRows * 512, n.cos + int64_t(tok) * (D / 2) + 4 * c, is_on);
        cp_async16(dst + (L::kRows + 1) * 512, n.sin + int64_t(tok) * (D / 2) + 4 * c, is_on);
      }
    }
  };

  At now;
  now.b = int(first / g.n_tokens);
  now.tok = int(first - int64_t(now.b) * g.n_tokens);
  now.step = 0;
  now.left = total - (first - (PER_HEAD ? grp : 0));
  At next = now;                                 // the step to request next
  uint32_t issued = 0, done = 0;                 // steps, which take the stages in turn
  auto request_next = [&] {                      // one group of copies for every step, past the end an empty one
    if (more(next)) {
      request(next, issued % L::kStages);
      advance(next);
    }
    cp_commit();
    ++issued;
  };
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) request_next();
  while (more(now)) {
    Turn turn = {};
    if (!PER_HEAD || !n.cos) turn = load_turn(n, now.b < g.B ? now.tok : 0, D, c);
    for (int step = 0; step < steps; ++step, ++done) {
      request_next();
      cp_wait<L::kStages - 1>();
      __syncwarp();
      const uint32_t buf = done % L::kStages;
      // lane group grp's row of input z: 16 * CPR bytes
      const uint8_t* in = stage + buf * L::kStep + grp * CPR * 16;
      auto row = [&](int z) { return row_of<HALVES>(reinterpret_cast<const __nv_bfloat16*>(in + z * 512), D, c); };
      if constexpr (PER_HEAD) {
        if (n.cos) {                             // this lane's own chunks
          const float4 cs = *reinterpret_cast<const float4*>(in + L::kRows * 512 + 16 * c);
          const float4 sn = *reinterpret_cast<const float4*>(in + (L::kRows + 1) * 512 + 16 * c);
          turn = Turn{{cs.x, cs.y, cs.z, cs.w}, {sn.x, sn.y, sn.z, sn.w}};
        }
      }
      const float eps = on(now) ? n.eps : 1.f;   // a lane without a row has zeros: with eps 0 they would be 0 * inf
      const uint4 yq = norm_rope_grad_row<CPR, HALVES>(row(0), row(2), wq, turn, eps, tok_acc[0][0], tok_acc[0][1]);
      const uint4 yk = norm_rope_grad_row<CPR, HALVES>(row(1), row(3), wk, turn, eps, tok_acc[1][0], tok_acc[1][1]);
      if (on(now)) {
        const int off = head_of(now) * D;
        store_row<HALVES>(dq + now.b * n.st[2].batch + now.tok * n.st[2].token + off, D, c, yq);
        store_row<HALVES>(dk + now.b * n.st[3].batch + now.tok * n.st[3].token + off, D, c, yk);
        if constexpr (PACKED)
          reinterpret_cast<uint4*>(dv + now.b * n.st[4].batch + now.tok * n.st[4].token + off)[c] =
              *reinterpret_cast<const uint4*>(in + 4 * 512 + 16 * c);
      }
      __syncwarp();                              // the buffer may be filled again
      advance(now);
    }
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[z][m][j] = fadd2(acc[z][m][j], tok_acc[z][m][j]);
          tok_acc[z][m][j] = 0ull;
        }
  }
  float(*red)[2][D] = reinterpret_cast<float(*)[2][D]>(sm + L::oRed);
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[2];
        f2unpack(acc[z][m][j >> 1], v[0], v[1]);
        float x = v[j & 1];
#pragma unroll
        for (int o = CPR; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane < CPR) red[warp][z][channel_of<HALVES>(D, c, j, m)] = x;
      }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int z = threadIdx.x / D, ch = threadIdx.x % D;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[w][z][ch];
    part[((int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 2 + z) * D + ch] = s;
  }
}

// dw[row][z][ch] = sum over the nb partials of that row: 32 interleaved chains per
// channel in fp64, joined in a fixed order. Grid (rows, 2, d / 32).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int nb, int D, float* dw_q,
                                                       float* dw_k) {
  __shared__ double red[32][32];
  tc::wait_predecessor();
  const int lane = threadIdx.x & 31, ch = int(blockIdx.z) * 32 + lane, sl = threadIdx.x >> 5, z = blockIdx.y;
  double s = 0.0;
#pragma unroll 4
  for (int i = sl; i < nb; i += 32) s += double(part[((int64_t(blockIdx.x) * nb + i) * 2 + z) * D + ch]);
  red[sl][lane] = s;
  __syncthreads();
  if (sl == 0) {
    for (int i = 1; i < 32; ++i) s += red[i][lane];
    float* out = z ? dw_k : dw_q;
    if (out) out[int64_t(blockIdx.x) * D + ch] = float(s);
  }
}

// Blocks along x of the gradient kernel: one token for each of eight warps (or their
// lane groups) at least, what is resident at once, two blocks per SM, at most
// (weights per head: shared among the heads). From packed tiles and with shared
// weights up to eight rounds of that, one for every 64 steps of a warp, so that SMs
// with a smaller share of HBM get fewer blocks: 937 us with one round, 869 with eight
// at 24 heads of 128 and 112,512 tokens (570 steps); 59 and 75 at 45 steps. From
// token-major rows 677 and 682, with weights per head 952 and 1,053.
int bwd_blocks(const vsa_plan* p, bool per_head, bool packed) {
  const Geometry& g = p->geo;
  const int64_t tokens = int64_t(g.B) * g.n_tokens;
  const int tpb = per_head ? 8 * (32 / (g.d / 8)) : 8;
  const int64_t want = (tokens + tpb - 1) / tpb;
  const int64_t resident = int64_t(p->num_sms) * 2, per_token = (g.Hh + 32 / (g.d / 8) - 1) / (32 / (g.d / 8));
  int64_t rounds = per_head || !packed ? 1 : tokens * per_token / (resident * 8 * 64);
  rounds = rounds < 1 ? 1 : rounds > 8 ? 8 : rounds;
  const int64_t cap = resident * rounds / (per_head ? g.Hh : 1);
  return int(want < cap ? want : cap < 1 ? 1 : cap);
}

}  // namespace

// Shared-memory limits of the kernels above, once per device (plan creation).
cudaError_t prepare_norm_rope() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* kernel, uint32_t bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  };
#define VSA_SET(CPR, HV)                                                                 \
  set(norm_rope_pack_kernel<CPR, HV, false>, PackSmem<CPR, false>::kBytes);              \
  set(norm_rope_pack_kernel<CPR, HV, true>, PackSmem<CPR, true>::kBytes);                \
  set(norm_rope_bwd_kernel<CPR, HV, false, false>, GradSmem<CPR, false, false>::kBytes);        \
  set(norm_rope_bwd_kernel<CPR, HV, false, true>, GradSmem<CPR, false, true>::kBytes);         \
  set(norm_rope_bwd_kernel<CPR, HV, true, false>, GradSmem<CPR, true, false>::kBytes);          \
  set(norm_rope_bwd_kernel<CPR, HV, true, true>, GradSmem<CPR, true, true>::kBytes)
  VSA_SET(16, true);
  VSA_SET(16, false);
  VSA_SET(8, true);
  VSA_SET(8, false);
#undef VSA_SET
  return e;
}

cudaError_t launch_norm_rope(const vsa_plan* p, const NormRopeArgs& n, const void* q, const void* k, void* qo, void* ko,
                             cudaStream_t s) {
  const Geometry& g = p->geo;
  const int64_t want = (int64_t(g.B) * g.n_tokens + 7) / 8, cap = int64_t(p->num_sms) * kFwdBlocks * 16;
  const unsigned grid = unsigned(want < cap ? want : cap);
  auto* q2 = static_cast<const __nv_bfloat16*>(q);
  auto* k2 = static_cast<const __nv_bfloat16*>(k);
  auto* qo2 = static_cast<__nv_bfloat16*>(qo);
  auto* ko2 = static_cast<__nv_bfloat16*>(ko);
#define VSA_RUN(CPR, HV) \
  return tc::launch_after(norm_rope_kernel<CPR, HV>, dim3(grid), 256u, 0, s, 1, n, g.B, g.n_tokens, g.Hh, q2, k2, qo2, ko2)
  if (g.d == 128) {
    if (n.halves) VSA_RUN(16, true);
    else VSA_RUN(16, false);
  } else {
    if (n.halves) VSA_RUN(8, true);
    else VSA_RUN(8, false);
  }
#undef VSA_RUN
}

cudaError_t launch_norm_rope_pack(const vsa_plan* p, const NormRopeArgs& n, const void* q, const void* k, const void* v,
                                  void* qp, void* kp, void* vp, float* pooled_q, float* pooled_k, cudaStream_t s) {
  const Geometry& g = p->geo;
  // Heads per CTA: up to eight, while two CTAs per SM still get four rounds of work.
  int64_t run = int64_t(g.B) * g.Hh * g.nt_max / (int64_t(p->num_sms) * 8);
  run = run < 1 ? 1 : run > 8 ? 8 : run;
  const unsigned grid = unsigned(int64_t(g.B) * g.nt_max * ((g.Hh + run - 1) / run));
  const bool trip = p->desc.score_mode == VSA_SCORE_TRIPPOOL;
#define VSA_RUN(CPR, HV, TR)                                                                                       \
  return tc::launch_after(norm_rope_pack_kernel<CPR, HV, TR>, dim3(grid), 256u, size_t(PackSmem<CPR, TR>::kBytes), s, \
                          1, n, g, int(run), static_cast<const __nv_bfloat16*>(q),                                 \
                          static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),              \
                          static_cast<__nv_bfloat16*>(qp), static_cast<__nv_bfloat16*>(kp),                        \
                          static_cast<__nv_bfloat16*>(vp), p->d_tile_count, pooled_q, pooled_k)
  if (g.d == 128) {
    if (n.halves) {
      if (trip) VSA_RUN(16, true, true);
      else VSA_RUN(16, true, false);
    } else {
      if (trip) VSA_RUN(16, false, true);
      else VSA_RUN(16, false, false);
    }
  } else {
    if (n.halves) {
      if (trip) VSA_RUN(8, true, true);
      else VSA_RUN(8, true, false);
    } else {
      if (trip) VSA_RUN(8, false, true);
      else VSA_RUN(8, false, false);
    }
  }
#undef VSA_RUN
}

int64_t norm_bwd_workspace_bytes(const vsa_plan* p) {
  const int64_t shared = bwd_blocks(p, false, true), per_head = int64_t(bwd_blocks(p, true, true)) * p->geo.Hh;
  return (shared > per_head ? shared : per_head) * 2 * p->geo.d * int64_t(sizeof(float));
}

cudaError_t launch_norm_rope_bwd(const vsa_plan* p, const NormRopeArgs& n, bool packed, const void* dyq, const void* dyk,
                                 const void* dyv, const void* q, const void* k, void* dq, void* dk, void* dv, float* dw_q,
                                 float* dw_k, void* workspace, cudaStream_t s) {
  const Geometry& g = p->geo;
  const int nb = bwd_blocks(p, n.per_head, packed);
  const dim3 grid(nb, n.per_head ? g.Hh : 1);
  float* part = static_cast<float*>(workspace);
  cudaError_t e = cudaSuccess;
#define VSA_RUN(CPR, HV, PK, PH)                                                                                   \
  e = tc::launch_after(norm_rope_bwd_kernel<CPR, HV, PK, PH>, grid, 256u, size_t(GradSmem<CPR, PK, PH>::kBytes), s, 1, n, \
                       g, static_cast<const __nv_bfloat16*>(dyq), static_cast<const __nv_bfloat16*>(dyk),          \
                       static_cast<const __nv_bfloat16*>(dyv), static_cast<const __nv_bfloat16*>(q),               \
                       static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(dq),                      \
                       static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv), part)
#define VSA_RUN2(CPR, HV)                  \
  do {                                     \
    if (packed) {                          \
      if (n.per_head) VSA_RUN(CPR, HV, true, true);  \
      else VSA_RUN(CPR, HV, true, false);  \
    } else {                               \
      if (n.per_head) VSA_RUN(CPR, HV, false, true); \
      else VSA_RUN(CPR, HV, false, false); \
    }                                      \
  } while (0)
  if (g.d == 128) {
    if (n.halves) VSA_RUN2(16, true);
    else VSA_RUN2(16, false);
  } else {
    if (n.halves) VSA_RUN2(8, true);
    else VSA_RUN2(8, false);
  }
#undef VSA_RUN2
#undef VSA_RUN
  if (e != cudaSuccess || (!dw_q && !dw_k)) return e;
  return tc::launch_after(norm_dw_kernel, dim3(grid.y, 2, unsigned(g.d / 32)), 1024u, 0, s, 1, part, nb, g.d, dw_q, dw_k);
}

}  // namespace vsa
