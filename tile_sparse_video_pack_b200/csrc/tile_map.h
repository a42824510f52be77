// The tile permutation on the device -- packed slot -> token, token -> packed
// row -- and the row loads shared by the kernels that move tiles (pack.cu,
// norm_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "vsa_internal.h"

namespace vsa {

// Token held by slot s of packed tile n of head h, or -1 for an unused slot.
// Prefix tiles: 64 consecutive tokens of one segment. Video tiles: the tile's
// tokens in (t, h, w) raster order over its actual extent (tiles cut by the
// grid's far edge hold fewer tokens, packed into the first slots).
__device__ __forceinline__ int src_token(const Geometry& g, int h, int n, int s) {
  if (n < g.n_pre_tiles) {
    int i = 0;
#pragma unroll 1
    while (i + 1 < g.n_seg && n >= g.seg_tile0[i + 1]) ++i;
    const int j = (n - g.seg_tile0[i]) * VSA_TILE + s;
    return j < g.seg_len[i] ? g.seg_tok0[i] + j : -1;
  }
  const int v = n - g.n_pre_tiles;
  if (v >= g.ntv[h]) return -1;
  const int nX = g.nX[h], nYX = g.nY[h] * nX;
  const int ti = v / nYX;
  const int r = v - ti * nYX;
  const int yi = r / nX;
  const int xi = r - yi * nX;
  const int t0 = ti * g.pt[h], y0 = yi * g.ph[h], x0 = xi * g.pw[h];
  const int et = min(g.pt[h], g.T - t0), eh = min(g.ph[h], g.H - y0), ew = min(g.pw[h], g.W - x0);
  if (s >= et * eh * ew) return -1;
  const int ehw = eh * ew;
  const int dt = s / ehw;
  const int r2 = s - dt * ehw;
  const int dy = r2 / ew;
  const int dx = r2 - dy * ew;
  return g.n_pre_tok + ((t0 + dt) * g.H + (y0 + dy)) * g.W + (x0 + dx);
}

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Packed row of token `tok` for head h: (tile, slot) -> tile * 64 + slot, the
// inverse of src_token. Prefix tokens: their segment's tiles of 64 consecutive
// tokens. Video tokens (t, y, x): the tile (t / pt, y / ph, x / pw) and the
// token's (t, h, w) raster position inside that tile's actual extent.
__device__ __forceinline__ int packed_row(const Geometry& g, int h, int tok) {
  if (tok < g.n_pre_tok) {
    int i = 0;
#pragma unroll 1
    while (i + 1 < g.n_seg && tok >= g.seg_tok0[i + 1]) ++i;
    const int off = tok - g.seg_tok0[i];
    return (g.seg_tile0[i] + off / VSA_TILE) * VSA_TILE + off % VSA_TILE;
  }
  const int v = tok - g.n_pre_tok;
  const int hw = g.H * g.W;
  const int t = v / hw;
  const int r = v - t * hw;
  const int y = r / g.W;
  const int x = r - y * g.W;
  const int pt = g.pt[h], ph = g.ph[h], pw = g.pw[h];
  const int ti = t / pt, yi = y / ph, xi = x / pw;
  const int eh = min(ph, g.H - yi * ph), ew = min(pw, g.W - xi * pw);
  const int slot = ((t - ti * pt) * eh + (y - yi * ph)) * ew + (x - xi * pw);
  const int n = g.n_pre_tiles + (ti * g.nY[h] + yi) * g.nX[h] + xi;
  return n * VSA_TILE + slot;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

}  // namespace vsa
