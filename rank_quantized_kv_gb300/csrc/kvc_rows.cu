// Stored rows moved between and inside layers: a row is its packed bytes and
// its fp16 side words, so the codes move as they are and no row is decoded.
//
//   gather  dst rows [len, len + n) of every (b, h) from a source layer: row
//           start + j, or index[b][j], of batch entry parent[b] (or b);
//   accept  of the last N rows keep rows index[b][0 .. n) in that order.
//
// Bound: HBM, each row read once and written once.  Payload and side words are
// two byte ranges per slot, cut into 16-byte chunks of the destination; a chunk
// is put together from pieces of V bytes, V the largest power of two (at most
// 16) that keeps every piece inside one row and aligned on both sides.
//
// Measured: 128 slots of 16384 int8 rows, 16 entries from about ten distinct parents
// (448 MB that have to move), in 82 us, 0.8 of the copy rate; 5461 chosen ones of
// 16384 rows of 48 bytes for 128 slots in 28 us, 2.5 TB/s of the rows' own bytes (a
// row at random draws one or two 64-byte pieces of DRAM, its norm another); accept
// of 17 of 64 rows for 128 slots 5 us, a launch.
#include <algorithm>

#include "kvc_internal.h"
#include "kvc_launch.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;              // chunks per thread: loads issued before stores
constexpr int kAcceptStage = 96 * 1024;    // shared memory of accept

// One byte range of a gather: `rows` rows of P bytes.  Contiguous source rows
// are one row of the whole range.
struct Part {
  int64_t P, rows;
  int64_t dst_byte;  // first byte written, from the start of the slot's region
  int64_t src_byte;  // contiguous rows: first byte read
  int V;             // piece size
};

template <int V> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };
template <> struct Piece<1> { using T = uint8_t; };

// Source address of byte x of the range, or null (and *bad) where the row's
// index lies outside the source.
__device__ __forceinline__ const uint8_t* src_of(const Part& q, const uint8_t* src,
                                                 const int32_t* idx, int64_t src_len, int64_t x,
                                                 bool* bad) {
  if (!idx) return src + q.src_byte + x;
  // 32-bit division where it suffices: the 64-bit one is a subroutine
  const int64_t row = x < ((int64_t)1 << 32) ? (int64_t)((uint32_t)x / (uint32_t)q.P) : x / q.P;
  const int64_t s = idx[row];
  if (s < 0 || s >= src_len) {
    *bad = true;
    return nullptr;
  }
  return src + s * q.P + (x - row * q.P);
}

template <int V>
__device__ void gather_part(const Part& q, uint8_t* dst, const uint8_t* src, const int32_t* idx,
                            int64_t src_len, bool* bad) {
  using T = typename Piece<V>::T;
  const int64_t total = q.P * q.rows;
  const int64_t a0 = q.dst_byte & ~int64_t(15), lead = q.dst_byte - a0;
  const int64_t chunks = (lead + total + 15) >> 4;
  const int64_t step = (int64_t)gridDim.y * kThreads;
  for (int64_t c0 = (int64_t)blockIdx.y * kThreads + threadIdx.x; c0 < chunks;
       c0 += step * kPerThread) {
    union { T t[16 / V]; uint4 w; } v[kPerThread];
    uint32_t have[kPerThread];  // bit per piece
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
      const int64_t c = c0 + u * step, x0 = c * 16 - lead;
      have[u] = 0;
      if (c >= chunks || x0 < 0 || x0 + 16 > total) continue;
#pragma unroll
      for (int e = 0; e < 16 / V; ++e) {
        const uint8_t* s = src_of(q, src, idx, src_len, x0 + e * V, bad);
        if (s) {
          v[u].t[e] = *reinterpret_cast<const T*>(s);
          have[u] |= 1u << e;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
      const int64_t c = c0 + u * step, x0 = c * 16 - lead;
      if (c >= chunks) continue;
      uint8_t* d = dst + a0 + c * 16;
      if (x0 < 0 || x0 + 16 > total) {  // an edge of the range: byte by byte
        const int64_t x1 = x0 + 16 < total ? x0 + 16 : total;
        for (int64_t x = x0 < 0 ? 0 : x0; x < x1; ++x) {
          const uint8_t* s = src_of(q, src, idx, src_len, x, bad);
          if (s) d[x - x0] = *s;
        }
      } else if (have[u] == (1u << (16 / V)) - 1u) {
        *reinterpret_cast<uint4*>(d) = v[u].w;
      } else {
#pragma unroll
        for (int e = 0; e < 16 / V; ++e)
          if (have[u] >> e & 1u) reinterpret_cast<T*>(d)[e] = v[u].t[e];
      }
    }
  }
}

// grid (destination slots, chunk blocks, payload | side words)
__global__ void __launch_bounds__(kThreads)
    gather_kernel(const Params dp, const Params sp, const GatherArgs a) {
  const int slot = blockIdx.x, side = blockIdx.z;
  const int b = slot / dp.Hg, h = slot - b * dp.Hg;
  const int sb = a.parent ? a.parent[b] : b;
  if (sb < 0 || sb >= sp.B) {
    if (threadIdx.x == 0) atomicCAS(dp.err, 0, kErrIndex);
    return;
  }
  const int ss = sb * sp.Hg + h;
  const int64_t P = side ? dp.side_bytes : dp.P[dp.basis_of[slot]];
  if (P == 0) return;
  const int32_t* idx = a.index ? a.index + (int64_t)b * a.n : nullptr;
  Part q;
  q.dst_byte = a.dst_row0 * P;
  if (idx) {
    q.P = P;
    q.rows = a.n;
    q.src_byte = 0;
    q.V = (int)min((int64_t)16, P & -P);  // rows start at multiples of P
  } else {
    q.P = P * a.n;
    q.rows = 1;
    q.src_byte = a.src_row0 * P;
    const int64_t off = (q.src_byte - q.dst_byte) & 15;
    q.V = off ? (int)(off & -off) : 16;
  }
  bool bad = false;
  uint8_t* dst = dp.store + (side ? dp.side_off[slot] : dp.pay_off[slot]);
  const uint8_t* src = sp.store + (side ? sp.side_off[ss] : sp.pay_off[ss]);
  switch (q.V) {
    case 16: gather_part<16>(q, dst, src, idx, a.src_len, &bad); break;
    case 8: gather_part<8>(q, dst, src, idx, a.src_len, &bad); break;
    case 4: gather_part<4>(q, dst, src, idx, a.src_len, &bad); break;
    case 2: gather_part<2>(q, dst, src, idx, a.src_len, &bad); break;
    default: gather_part<1>(q, dst, src, idx, a.src_len, &bad);
  }
  if (bad) atomicCAS(dp.err, 0, kErrIndex);
}

// The columns [c0, c0 + w) of the accepted rows, through shared memory: every
// row is read before any is written, so the index may have any order.
template <int V>
__device__ void accept_columns(uint8_t* region, int64_t P, int c0, int w, const AcceptArgs& a,
                               const int32_t* idx, uint8_t* stage, bool* bad) {
  using T = typename Piece<V>::T;
  const int ppr = w / V;  // pieces of a row
  const int64_t total = a.n * ppr;
  T* st = reinterpret_cast<T*>(stage);
  for (int64_t i = threadIdx.x; i < total; i += kThreads) {
    const int64_t j = i / ppr;
    const int32_t s = idx[j];
    if (s < 0 || s >= a.N) *bad = true;
    else st[i] = *reinterpret_cast<const T*>(region + (a.base + s) * P + c0 + (i - j * ppr) * V);
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < total; i += kThreads) {
    const int64_t j = i / ppr;
    const int32_t s = idx[j];
    if (s >= 0 && s < a.N)
      *reinterpret_cast<T*>(region + (a.base + j) * P + c0 + (i - j * ppr) * V) = st[i];
  }
}

// grid (slots, column chunks of the payload, then of the side words)
__global__ void __launch_bounds__(kThreads) accept_kernel(const Params p, const AcceptArgs a) {
  extern __shared__ __align__(16) uint8_t stage[];
  const int slot = blockIdx.x, y = blockIdx.y, side = y >= a.pay_chunks;
  const int64_t P = side ? p.side_bytes : p.P[p.basis_of[slot]];
  const int c0 = (side ? y - a.pay_chunks : y) * a.cw;
  if (c0 >= P) return;
  const int w = (int)min((int64_t)a.cw, P - c0);
  const int32_t* idx = a.index + (int64_t)(slot / p.Hg) * a.n;
  uint8_t* region = p.store + (side ? p.side_off[slot] : p.pay_off[slot]);
  const int64_t bits = P | a.cw | 16;  // V divides the row, the chunk and 16
  bool bad = false;
  switch ((int)(bits & -bits)) {
    case 16: accept_columns<16>(region, P, c0, w, a, idx, stage, &bad); break;
    case 8: accept_columns<8>(region, P, c0, w, a, idx, stage, &bad); break;
    case 4: accept_columns<4>(region, P, c0, w, a, idx, stage, &bad); break;
    case 2: accept_columns<2>(region, P, c0, w, a, idx, stage, &bad); break;
    default: accept_columns<1>(region, P, c0, w, a, idx, stage, &bad);
  }
  if (bad) atomicCAS(p.err, 0, kErrIndex);
}

}  // namespace

cudaError_t launch_gather(const Params& dp, const Params& sp, const GatherArgs& a, int pmax,
                          int sms, cudaStream_t s, int* nk) {
  if (std::max(pmax, dp.side_bytes) == 0) return cudaSuccess;  // rows of no bytes
  // blocks for one round of the longer range, at most about eight a SM in all
  const int64_t chunks = (a.n * std::max(pmax, dp.side_bytes) + 15) / 16 + 1;
  const int64_t need = (chunks + kThreads * kPerThread - 1) / (kThreads * kPerThread);
  const int64_t most = std::max<int64_t>(1, (8 * (int64_t)sms + dp.n_slots - 1) / dp.n_slots);
  const dim3 grid((unsigned)dp.n_slots, (unsigned)std::min(need, most), dp.side_bytes ? 2 : 1);
  gather_kernel<<<grid, kThreads, 0, s>>>(dp, sp, a);
  ++*nk;
  return cudaGetLastError();
}

int accept_columns_per_block(int64_t n, int widest) {
  const int64_t most = kAcceptStage / n;  // bytes of a row that a block can stage
  if (most >= 16) return (int)std::min<int64_t>((widest + 15) / 16 * 16, most / 16 * 16);
  for (int w = 8; w >= 1; w /= 2)
    if (most >= w) return w;
  return 0;
}

cudaError_t launch_accept(const Params& p, AcceptArgs a, int pmax, cudaStream_t s, int* nk) {
  const int widest = std::max(pmax, p.side_bytes);
  if (widest == 0) return cudaSuccess;  // every component dropped: rows of no bytes
  a.cw = accept_columns_per_block(a.n, widest);
  a.pay_chunks = (pmax + a.cw - 1) / a.cw;
  const int side_chunks = (p.side_bytes + a.cw - 1) / a.cw;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(accept_kernel), kAcceptStage);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.n_slots, (unsigned)(a.pay_chunks + side_chunks));
  accept_kernel<<<grid, kThreads, (size_t)a.n * a.cw, s>>>(p, a);
  ++*nk;
  return cudaGetLastError();
}

}  // namespace kvc
