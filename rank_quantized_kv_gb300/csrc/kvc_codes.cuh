// How stored codes are read by the CUDA-core attention kernels: packed positions
// and chunks of a basis, bit fields of a row, sums over a warp.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kvc_internal.h"

namespace kvc {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Packed position j of basis beta: component (-1: padding) and width.
__device__ inline int position_component(const Params& p, int beta, int j, int* width) {
  int4 e[kMaxSeg];  // start byte, width, first order slot, count; all read at once
#pragma unroll
  for (int s = 0; s < kMaxSeg; ++s)
    e[s] = reinterpret_cast<const int4*>(p.seg)[(size_t)beta * kMaxSeg + s];
  int at = -1, nch = 0;
#pragma unroll
  for (int s = 0; s < kMaxSeg; ++s) {
    const int m = j - nch * 8;
    if (m >= 0 && m < e[s].w) {
      at = e[s].z + m;
      *width = e[s].y;
    }
    nch += (e[s].w + 7) / 8;
  }
  return at < 0 ? -1 : p.order[(size_t)beta * p.r + at];
}

// Chunk c (8 packed positions) of basis beta: first byte | width << 16 |
// valid << 31, 0 past the last one.
__device__ inline uint32_t chunk_entry(const Params& p, int beta, int c) {
  int nch = 0;
  for (int s = 0; s < kMaxSeg; ++s) {
    const int32_t* e = p.seg + ((size_t)beta * kMaxSeg + s) * 4;
    if (!e[3]) break;
    const int n = (e[3] + 7) / 8;
    if (c < nch + n) return (uint32_t)(e[0] + e[1] * (c - nch)) | ((uint32_t)e[1] << 16) | (1u << 31);
    nch += n;
  }
  return 0u;
}

__device__ __forceinline__ uint2 bits_at(const unsigned char* base, int a) {
  const uint32_t* wp = reinterpret_cast<const uint32_t*>(base) + (a >> 2);
  const uint32_t w0 = wp[0], w1 = wp[1], w2 = wp[2];
  const uint32_t sh = 8 * (a & 3);
  return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
}

__device__ __forceinline__ uint32_t chunk_code(uint2 b, int w, int e) {
  if (w == 8) return ((e < 4 ? b.x : b.y) >> (8 * (e & 3))) & 0xffu;
  return (b.x >> (w * e)) & ((1u << w) - 1u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

}  // namespace

}  // namespace kvc
