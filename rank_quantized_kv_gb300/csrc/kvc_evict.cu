// Eviction: of the S rows of every slot (b, h) of a key and a value layer, n are
// kept, in their order, and the others dropped.  Ranked from the top:
//   the sinks, tokens [first, first + sinks), and the last `recent` tokens;
//   the others from first on by accumulated weight, larger first; NaN below all;
//   the padding before first;
// and among equals the lower token first.
//
// Select: a cluster per slot, its CTAs sharing the tokens out.  A weight becomes a
// 32-bit key of the same order; three passes over the keys (11, 11 and 10 bits)
// find the n-th largest by histograms that the cluster adds up through distributed
// shared memory; a last pass numbers the kept tokens by a scan and writes them.
// Move: kept rows, payload and side words of both layers, in 16-byte chunks of the
// destination put together from the largest pieces that stay inside a row.
//
// In place a kept row moves down or stays (the j-th kept row is at j or above), so
// a chunk's destination lies at or below its sources.  A cluster per range moves a
// stretch of chunks at a time, reads before a cluster barrier and writes after it:
// what it writes lies below the sources of all later stretches.
//
// Bound: HBM, the weights read once (and twice more from L2) and the kept rows read
// and written; for small caches two launches.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvc_codes.cuh"
#include "kvc_internal.h"
#include "kvc_launch.cuh"

namespace kvc {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512, kPer = 4, kSelStep = kSelThreads * kPer;
constexpr int kBins = 2048;
constexpr uint32_t kForced = 0xffffffffu, kNaNKey = 1u, kPadKey = 0u;

// The order of a token: forced ones above every weight, NaN and padding below.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return kNaNKey;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Slot {
  const float* w;
  int S, first, sink_end, recent0;
  __device__ uint32_t key(int t) const {
    if (t < first) return kPadKey;
    if (t < sink_end || t >= recent0) return kForced;
    return w ? order_key(w[t]) : 0x80000000u;
  }
};

// Inclusive scan over the block's threads; the block's total in *total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSelThreads / 32; ++i) {
    const uint32_t x = warp_sums[i];
    if (i < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

// grid: clusters of gridDim.x CTAs, one per slot (y)
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[3][kBins];
  __shared__ uint32_t sum[kBins];
  __shared__ uint32_t warp_sums[kSelThreads / 32];
  __shared__ uint32_t counts[2];  // keys above the threshold, equal to it
  __shared__ uint32_t digit_s, left_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)gridDim.x, me = (int)blockIdx.x, tid = threadIdx.x;
  const int slot = blockIdx.y, b = slot / a.H, h = slot - b * a.H;
  Slot s;
  s.w = a.weights ? a.weights + b * a.w_sb + h * a.w_sh : nullptr;
  s.S = a.S;
  s.first = a.first ? min(max(a.first[b], 0), a.S) : 0;
  s.sink_end = (int)min((int64_t)s.first + a.sinks, (int64_t)a.S);
  s.recent0 = a.S - a.recent;
  if (h == 0 && me == 0 && tid == 0 && a.first_out) a.first_out[b] = max(0, a.n - (a.S - s.first));
  // this CTA's tokens
  const int seg = ((a.S + ctas - 1) / ctas + kPer - 1) / kPer * kPer;
  const int t0 = (int)min((int64_t)a.S, (int64_t)me * seg), t1 = (int)min((int64_t)a.S, (int64_t)t0 + seg);
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0u;
  __syncthreads();
  // the key of the n-th largest, digit by digit: `known` bits fixed so far
  uint32_t thr = 0u, left = (uint32_t)a.n;  // (n >= 1)
  int known = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = 32 - known - bits;
    uint32_t* hp = hist[pass];
    for (int t = t0 + tid; t < t1; t += kSelThreads) {
      const uint32_t k = s.key(t);
      if (known == 0 || (k >> (32 - known)) == (thr >> (32 - known)))
        atomicAdd(&hp[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    cluster.sync();
    for (int i = tid; i < kBins; i += kSelThreads) {
      uint32_t v = 0;
      for (int c = 0; c < ctas; ++c) v += cluster.map_shared_rank(hp, c)[i];
      sum[i] = v;
    }
    __syncthreads();
    // from the top: the digit at which the running count reaches `left`
    uint32_t v = 0, mine[kBins / kSelThreads];
#pragma unroll
    for (int u = 0; u < kBins / kSelThreads; ++u) {
      mine[u] = sum[kBins - 1 - (tid * (kBins / kSelThreads) + u)];
      v += mine[u];
    }
    uint32_t total;
    const uint32_t end = block_scan(v, warp_sums, &total);
    uint32_t at = end - v;
#pragma unroll
    for (int u = 0; u < kBins / kSelThreads; ++u) {
      if (at < left && at + mine[u] >= left) {
        digit_s = kBins - 1 - (tid * (kBins / kSelThreads) + u);
        left_s = left - at;
      }
      at += mine[u];
    }
    __syncthreads();
    thr |= digit_s << shift;
    left = left_s;
    known += bits;
    __syncthreads();
  }
  // keys above thr, and the first `left` of those equal to it, are kept
  uint32_t gt = 0, eq = 0;
  for (int t = t0 + tid; t < t1; t += kSelThreads) {
    const uint32_t k = s.key(t);
    gt += k > thr;
    eq += k == thr;
  }
  uint32_t n_gt, n_eq;
  block_scan(gt, warp_sums, &n_gt);
  block_scan(eq, warp_sums, &n_eq);
  if (tid == 0) {
    counts[0] = n_gt;
    counts[1] = n_eq;
  }
  cluster.sync();
  uint32_t gt0 = 0, eq0 = 0;  // of the CTAs before this one
  for (int c = 0; c < me; ++c) {
    const uint32_t* p = cluster.map_shared_rank(counts, c);
    gt0 += p[0];
    eq0 += p[1];
  }
  grid_dependents_launch();
  int32_t* index = a.index + (int64_t)slot * a.n;
  float* dw = a.dst_weights && !a.in_place ? a.dst_weights + b * a.dw_sb + h * a.dw_sh + a.dst_row0 : nullptr;
#pragma unroll 1
  for (int tb = t0; tb < t1; tb += kSelStep) {
    const int t = tb + tid * kPer;
    uint32_t k[kPer], v = 0;  // counts of both in halves of a word: at most 2048 each
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      k[u] = t + u < t1 ? s.key(t + u) : 0u;
      if (t + u < t1) v += k[u] > thr ? 1u : k[u] == thr ? 0x10000u : 0u;
    }
    uint32_t total;
    uint32_t at = block_scan(v, warp_sums, &total) - v;
    uint32_t g = gt0 + (at & 0xffffu), e = eq0 + (at >> 16);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (t + u >= t1) break;
      const bool above = k[u] > thr, equal = k[u] == thr;
      if (above || (equal && e < left)) {
        const uint32_t to = g + min(e, left);
        index[to] = t + u;
        if (dw) dw[to] = s.w ? s.w[t + u] : 0.f;
      }
      g += above;
      e += equal;
    }
    gt0 += total & 0xffffu;
    eq0 += total >> 16;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- move

constexpr int kMoveThreads = 256, kChunks = 4;  // chunks of 16 bytes a thread has in flight

template <int V> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };
template <> struct Piece<1> { using T = uint8_t; };

// Rows idx[0 .. n) of src, P bytes each, to dst from byte dst0 on.
struct Move {
  const uint8_t* src;
  uint8_t* dst;
  const int32_t* idx;
  int64_t P, n, dst0;
};

__device__ __forceinline__ int64_t row_of(int64_t x, int64_t P) {
  // 32-bit division where it suffices: the 64-bit one is a subroutine
  return x < ((int64_t)1 << 32) ? (int64_t)((uint32_t)x / (uint32_t)P) : x / P;
}

// CTA `me` of `ctas`; `barrier` separates the reads of a stretch from its writes.
template <int V, class Barrier>
__device__ void move_rows(const Move& q, int me, int ctas, Barrier barrier) {
  using T = typename Piece<V>::T;
  const int64_t total = q.P * q.n, lead = q.dst0 & 15;
  uint8_t* out = q.dst + (q.dst0 - lead);  // 16-byte aligned
  const int64_t chunks = (lead + total + 15) >> 4;
  const int64_t step = (int64_t)ctas * kMoveThreads;
  for (int64_t c0 = 0; c0 < chunks; c0 += step * kChunks) {
    union { uint8_t b[16]; T t[16 / V]; uint4 w; } v[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int64_t c = c0 + u * step + (int64_t)me * kMoveThreads + threadIdx.x;
      const int64_t x = c * 16 - lead;
      if (c >= chunks) continue;
      if (x >= 0 && x + 16 <= total) {
        int64_t row = row_of(x, q.P);
        int at = (int)(x - row * q.P);
        const uint8_t* from = q.src + q.idx[row] * q.P;
#pragma unroll
        for (int e = 0; e < 16 / V; ++e) {
          if (at == q.P) {
            at = 0;
            from = q.src + q.idx[++row] * q.P;
          }
          v[u].t[e] = *reinterpret_cast<const T*>(from + at);
          at += V;
        }
      } else {  // an edge of the range: byte by byte
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (x + e >= 0 && x + e < total) {
            const int64_t row = row_of(x + e, q.P);
            v[u].b[e] = q.src[q.idx[row] * q.P + (x + e - row * q.P)];
          }
      }
    }
    barrier();
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int64_t c = c0 + u * step + (int64_t)me * kMoveThreads + threadIdx.x;
      const int64_t x = c * 16 - lead;
      if (c >= chunks) continue;
      if (x >= 0 && x + 16 <= total) {
        *reinterpret_cast<uint4*>(out + c * 16) = v[u].w;
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (x + e >= 0 && x + e < total) out[c * 16 + e] = v[u].b[e];
      }
    }
  }
}

template <class Barrier>
__device__ void move_any(const Move& q, int me, int ctas, Barrier barrier) {
  switch ((int)min((int64_t)16, q.P & -q.P)) {  // rows start at multiples of P
    case 16: move_rows<16>(q, me, ctas, barrier); break;
    case 8: move_rows<8>(q, me, ctas, barrier); break;
    case 4: move_rows<4>(q, me, ctas, barrier); break;
    case 2: move_rows<2>(q, me, ctas, barrier); break;
    default: move_rows<1>(q, me, ctas, barrier);
  }
}

// grid: (CTAs of a range, slots, ranges): key and value payload, key and value side
// words and, in place, the weights.  In place the CTAs of a range are a cluster.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const Params kp, const Params vp, const Params dkp, const Params dvp, const EvictArgs a) {
  const int slot = blockIdx.y, range = blockIdx.z;
  const bool weights = range == 4, values = range & 1, side = range >= 2;
  const Params& sp = values ? vp : kp;
  const Params& dp = values ? dvp : dkp;
  Move q;
  q.idx = a.index + (int64_t)slot * a.n;
  q.n = a.n;
  float* w = nullptr;
  if (weights) {
    const int b = slot / a.H, h = slot - b * a.H;
    w = a.weights + b * a.w_sb + h * a.w_sh;
    // (the weights may start at any multiple of 4; dst0 is their place in a 16-byte chunk)
    const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(w) & 15);
    q.P = 4;
    q.src = reinterpret_cast<const uint8_t*>(w);
    q.dst = reinterpret_cast<uint8_t*>(w) - lead;
    q.dst0 = lead;
  } else {
    q.P = side ? sp.side_bytes : sp.P[sp.basis_of[slot]];
    q.src = sp.store + (side ? sp.side_off[slot] : sp.pay_off[slot]);
    q.dst = dp.store + (side ? dp.side_off[slot] : dp.pay_off[slot]);
    q.dst0 = a.dst_row0 * q.P;
  }
  grid_dependency_wait();  // the index comes from the launch before
  if (q.P == 0) return;    // (every CTA of the cluster)
  if (IN_PLACE) {
    cg::cluster_group cluster = cg::this_cluster();
    move_any(q, (int)blockIdx.x, (int)gridDim.x, [&] { cluster.sync(); });
    if (!weights) return;
    // tokens to come start at zero; the dropped weights above n have been read
    cluster.sync();
    for (int64_t t = a.n + (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; t < a.S;
         t += (int64_t)gridDim.x * kMoveThreads)
      w[t] = 0.f;
  } else {
    move_any(q, (int)blockIdx.x, (int)gridDim.x, [] {});
  }
}

template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), dim3 grid, unsigned block, unsigned cluster, bool dependent,
                           cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_evict(const Params& kp, const Params& vp, const Params& dkp, const Params& dvp,
                         const EvictArgs& a, int pmax, int sms, cudaStream_t s, int* nk) {
  // CTAs of a slot's cluster: as many as there is a step of tokens for, at most
  // eight (the portable size), and not far more than the device holds at once
  auto pick = [&](int64_t work, int64_t clusters, int most) {
    int c = 1;
    while (c < 8 && c < work && 2 * c * clusters <= most) c *= 2;
    return c;
  };
  const int sel = pick((a.S + kSelStep - 1) / kSelStep, a.n_slots, 4 * sms);
  cudaError_t e = launch_cluster(evict_select_kernel, dim3(sel, a.n_slots), kSelThreads, sel, false, s, a);
  ++*nk;
  if (e != cudaSuccess) return e;
  const int widest = std::max(pmax, std::max(kp.side_bytes, vp.side_bytes));
  const int64_t steps = ((int64_t)a.n * std::max(widest, 4) + 16 * kMoveThreads * kChunks - 1) / (16 * kMoveThreads * kChunks);
  const int ranges = a.in_place && a.weights ? 5 : kp.side_bytes || vp.side_bytes ? 4 : 2;
  ++*nk;
  if (a.in_place) {
    const int c = pick(steps, (int64_t)a.n_slots * 2, 8 * sms);
    return launch_cluster(evict_move_kernel<true>, dim3(c, a.n_slots, ranges), kMoveThreads, c, true, s, kp, vp,
                          dkp, dvp, a);
  }
  const int64_t most = std::max<int64_t>(1, 4 * (int64_t)sms / a.n_slots);
  return launch_cluster(evict_move_kernel<false>, dim3((unsigned)std::min(steps, most), a.n_slots, ranges),
                        kMoveThreads, 1, true, s, kp, vp, dkp, dvp, a);
}

}  // namespace kvc
