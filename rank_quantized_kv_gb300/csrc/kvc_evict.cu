// Eviction: of the S rows of every slot (b, h) of a key and a value layer, n are
// kept, in their order, and the others dropped.  Ranked from the top:
//   the sinks, tokens [first, first + sinks), and the last `recent` tokens;
//   the others from first on by accumulated weight, larger first; NaN below all;
//   the padding before first;
// and among equals the lower token first.
//
// Select: a cluster per slot, its CTAs sharing the tokens out.  A weight becomes a
// 32-bit key of the same order, in registers (16 a thread; more tokens are read again
// in every pass); three passes over the keys (11, 11 and 10 bits) find the n-th
// largest by histograms that the cluster adds up through distributed shared memory; a
// last one numbers the kept tokens by a scan and writes them.
// Move: kept rows, payload and side words of both layers, in 16-byte chunks of the
// destination put together from the largest pieces that stay inside a row.
//
// In place a kept row moves down or stays (the j-th kept row is at j or above), so
// a chunk's destination lies at or below its sources.  A cluster per range moves a
// stretch of chunks at a time, reads before a cluster barrier and writes after it:
// what it writes lies below the sources of all later stretches.
//
// Bound: the move by HBM's sectors, kept rows that start and end inside them: 128
// slots, 4096 of 16384 rows of 48 + 128 bytes kept, 94 MB of rows each way in 50 us,
// with 138 MB read in sectors.  Select by the latency of its passes: 128 slots of 16384
// tokens 16 us; 8 slots of 130001 tokens, eight CTAs each, 24, of which the cluster's
// exchanges take a third.  Small caches are two launches (6 + 4 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "kvc_codes.cuh"
#include "kvc_internal.h"
#include "kvc_launch.cuh"

namespace kvc {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024, kPer = 16, kSelStep = kSelThreads * kPer;
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
  __device__ uint32_t key(int t, float weight) const {
    if (t < first) return kPadKey;
    if (t < sink_end || t >= recent0) return kForced;
    return order_key(weight);
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
  static_assert(kSelThreads == 1024, "a sum per lane");
  uint32_t x = warp_sums[lane];  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  *total = __shfl_sync(kFull, x, 31);
  const uint32_t before = __shfl_sync(kFull, x, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0u);
}

// The halves of a cluster barrier (all threads).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// grid: clusters of gridDim.x CTAs, one per slot (y).  A warp takes PER times 32
// consecutive tokens at a time, a lane every 32nd of them.  RESIDENT: the CTA's tokens
// are one step, whose keys stay in registers.
template <int PER, bool RESIDENT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ __align__(8) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_sums[kSelThreads / 32];
  __shared__ uint32_t digit_s, left_s, equal_s;
  constexpr int kStep = kSelThreads * PER;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)gridDim.x, me = (int)blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int slot = blockIdx.y, b = slot / a.H, h = slot - b * a.H;
  Slot s;
  s.w = a.weights ? a.weights + b * a.w_sb + h * a.w_sh : nullptr;
  s.S = a.S;
  s.first = a.first ? min(max(a.first[b], 0), a.S) : 0;
  s.sink_end = (int)min((int64_t)s.first + a.sinks, (int64_t)a.S);
  s.recent0 = a.S - a.recent;
  if (h == 0 && me == 0 && tid == 0 && a.first_out) a.first_out[b] = max(0, a.n - (a.S - s.first));
  // this CTA's tokens
  const int seg = (a.S + ctas - 1) / ctas;
  const int t0 = (int)min((int64_t)a.S, (int64_t)me * seg), t1 = (int)min((int64_t)a.S, (int64_t)t0 + seg);
  uint32_t key[PER];  // of tokens t + 32 u
  auto read = [&](int t) {
    float w[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) w[u] = s.w && t + 32 * u < t1 ? s.w[t + 32 * u] : 0.f;
#pragma unroll
    for (int u = 0; u < PER; ++u) key[u] = s.key(t + 32 * u, w[u]);
  };
  // f(first token of the thread) for every step of the CTA's tokens
  const int lead = (tid & ~31) * PER + lane;
  auto each = [&](auto f) {
    if (RESIDENT) {
      f(t0 + lead);
    } else {
      for (int tb = t0; tb < t1; tb += kStep) {
        read(tb + lead);
        f(tb + lead);
      }
    }
  };
  if (RESIDENT) read(t0 + lead);
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0u;
  __syncthreads();
  // the key of the n-th largest, digit by digit: `known` bits fixed so far
  uint32_t thr = 0u, left = (uint32_t)a.n;  // (n >= 1)
  uint32_t above = 0u;  // of the CTAs before this one, in this thread's bins: keys above the n-th largest
  int known = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = 32 - known - bits;
    uint32_t* hp = hist[pass];
    const uint32_t high = known ? ~0u << (32 - known) : 0u;  // the bits that must agree
    each([&](int t) {
#pragma unroll
      for (int u = 0; u < PER; ++u)
        if (t + 32 * u < t1 && ((key[u] ^ thr) & high) == 0u)
          atomicAdd(&hp[(key[u] >> shift) & ((1u << bits) - 1u)], 1u);
    });
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    constexpr int kMine = kBins / kSelThreads;
    static_assert(kMine == 2, "a thread's bins in one load");
    uint2 two = *reinterpret_cast<const uint2*>(hp + kBins - 2 - 2 * tid);  // bins of this thread
    uint2 pre = make_uint2(0u, 0u);                                         // in the CTAs before this one
    if (ctas > 1) {
      two = make_uint2(0u, 0u);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < ctas) {
          const uint2 x = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hp, c) + kBins - 2 - 2 * tid);
          two.x += x.x;
          two.y += x.y;
          if (c < me) {
            pre.x += x.x;
            pre.y += x.y;
          }
        }
    }
    const uint32_t mine[kMine] = {two.y, two.x}, v = two.x + two.y;  // from the top
    // the digit at which the running count reaches `left`
    uint32_t total;
    const uint32_t end = block_scan(v, warp_sums, &total);
    uint32_t at = end - v;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      if (at < left && at + mine[u] >= left) {
        digit_s = kBins - 1 - (tid * kMine + u);
        left_s = left - at;
      }
      at += mine[u];
    }
    __syncthreads();
    const int high_bin = kBins - 1 - 2 * tid, digit = (int)digit_s;
    above += (high_bin > digit ? pre.y : 0u) + (high_bin - 1 > digit ? pre.x : 0u);
    if (high_bin == digit) equal_s = pre.y;
    if (high_bin - 1 == digit) equal_s = pre.x;
    thr |= digit_s << shift;
    left = left_s;
    known += bits;
    __syncthreads();
  }
  // Keys above thr, and the first `left` of those equal to it, are kept.  Counts of both
  // of a step in halves of a word: at most 16384 each.
  auto count = [&](int t) {  // of the warp's tokens, in lane 0
    uint32_t v = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const bool in = t + 32 * u < t1;
      v += __popc(__ballot_sync(kFull, in && key[u] > thr)) + (__popc(__ballot_sync(kFull, in && key[u] == thr)) << 16);
    }
    return lane == 0 ? v : 0u;
  };
  uint32_t gt0 = 0, eq0 = 0;  // of the CTAs before this one
  if (ctas > 1) {
    cluster_arrive();  // this CTA has read the others' shared memory
    block_scan(above, warp_sums, &gt0);
    eq0 = equal_s;
  }
  grid_dependents_launch();
  int32_t* index = a.index + (int64_t)slot * a.n;
  float* dw = a.dst_weights && !a.in_place ? a.dst_weights + b * a.dw_sb + h * a.dw_sh + a.dst_row0 : nullptr;
  const uint32_t before = (1u << lane) - 1u;
  each([&](int t) {
    uint32_t total;
    const uint32_t v = count(t);
    const uint32_t at = __shfl_sync(kFull, block_scan(v, warp_sums, &total) - v, 0);
    uint32_t g = gt0 + (at & 0xffffu), e = eq0 + (at >> 16);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const bool in = t + 32 * u < t1, above = in && key[u] > thr, equal = in && key[u] == thr;
      const uint32_t ma = __ballot_sync(kFull, above), me2 = __ballot_sync(kFull, equal);
      const uint32_t mine = e + __popc(me2 & before);  // equal ones before this token
      if (above || (equal && mine < left)) {
        const uint32_t to = g + __popc(ma & before) + min(mine, left);
        index[to] = t + 32 * u;
        if (dw) dw[to] = s.w ? s.w[t + 32 * u] : 0.f;
      }
      g += __popc(ma);
      e += __popc(me2);
    }
    gt0 += total & 0xffffu;
    eq0 += total >> 16;
  });
  if (ctas > 1) cluster_wait();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- move

constexpr int kMoveThreads = 256, kChunks = 4;  // 16-byte chunks of a stretch that a thread has
constexpr int kStretch = kMoveThreads * kChunks * 16;

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

template <int V>
__device__ __forceinline__ void copy_piece(uint32_t dst, const uint8_t* src) {
  if constexpr (V == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(V) : "memory");
}

// CTA `me` of `ctas`; `barrier` separates the reads of a stretch from its writes.  A
// thread puts its chunks together in its own places of two stages, by asynchronous
// copies where the pieces are of 4 bytes or more; the next stretch's reads are on
// their way while this one is written.  BIG: byte numbers past 32 bits.
template <int V, bool BIG, class Barrier>
__device__ void move_rows(const Move& q, uint4* stage, int me, int ctas, Barrier barrier) {
  using T = typename Piece<V>::T;
  using Num = typename std::conditional<BIG, int64_t, uint32_t>::type;
  const int64_t total = q.P * q.n;
  const int lead = (int)(q.dst0 & 15);
  uint8_t* out = q.dst + (q.dst0 - lead);  // 16-byte aligned
  const int64_t chunks = (lead + total + 15) >> 4;
  const int64_t step = (int64_t)ctas * kMoveThreads;
  auto read = [&](int64_t c0, uint4* buf) {
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int64_t c = c0 + u * step, x = c * 16 - lead;
      if (c >= chunks) break;
      uint4* to = buf + u * kMoveThreads;
      if (x >= 0 && x + 16 <= total) {
        int64_t row = (Num)x / (Num)q.P;
        int at = (int)(x - row * q.P);
        const uint8_t* from = q.src + q.idx[row] * q.P;
#pragma unroll
        for (int e = 0; e < 16 / V; ++e) {
          if (at == q.P) {
            at = 0;
            from = q.src + q.idx[++row] * q.P;
          }
          if constexpr (V >= 4) copy_piece<V>((uint32_t)__cvta_generic_to_shared(to) + e * V, from + at);
          else reinterpret_cast<T*>(to)[e] = *reinterpret_cast<const T*>(from + at);
          at += V;
        }
      } else {  // an edge of the range: byte by byte
#pragma unroll 1
        for (int e = 0; e < 16; ++e)
          if (x + e >= 0 && x + e < total) {
            const int64_t row = (Num)(x + e) / (Num)q.P;
            reinterpret_cast<uint8_t*>(to)[e] = q.src[q.idx[row] * q.P + (x + e - row * q.P)];
          }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t first = (int64_t)me * kMoveThreads + threadIdx.x;
  uint4* mine = stage + threadIdx.x;
  constexpr int kStage = kChunks * kMoveThreads;
  read(first, mine);
  int at = 0;
  for (int64_t c0 = 0; c0 < chunks; c0 += step * kChunks, at ^= 1) {
    read(c0 + step * kChunks + first, mine + (at ^ 1) * kStage);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    barrier();
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int64_t c = c0 + first + u * step, x = c * 16 - lead;
      if (c >= chunks) break;
      const uint4* from = mine + at * kStage + u * kMoveThreads;
      if (x >= 0 && x + 16 <= total) {
        *reinterpret_cast<uint4*>(out + c * 16) = *from;
      } else {
#pragma unroll 1
        for (int e = 0; e < 16; ++e)
          if (x + e >= 0 && x + e < total) out[c * 16 + e] = reinterpret_cast<const uint8_t*>(from)[e];
      }
    }
  }
}

template <bool BIG, class Barrier>
__device__ void move_pieces(const Move& q, uint4* stage, int me, int ctas, Barrier barrier) {
  switch ((int)min((int64_t)16, q.P & -q.P)) {  // rows start at multiples of P
    case 16: move_rows<16, BIG>(q, stage, me, ctas, barrier); break;
    case 8: move_rows<8, BIG>(q, stage, me, ctas, barrier); break;
    case 4: move_rows<4, BIG>(q, stage, me, ctas, barrier); break;
    case 2: move_rows<2, BIG>(q, stage, me, ctas, barrier); break;
    default: move_rows<1, BIG>(q, stage, me, ctas, barrier);
  }
}
template <class Barrier>
__device__ void move_any(const Move& q, uint4* stage, int me, int ctas, Barrier barrier) {
  if (q.P * q.n < ((int64_t)1 << 32) - 64) move_pieces<false>(q, stage, me, ctas, barrier);
  else move_pieces<true>(q, stage, me, ctas, barrier);
}

// Ranges of a slot: key and value payload, key and value side words and, in place, the
// weights.  grid: (CTAs, slots); in place a range's CTAs are a cluster, blockIdx.z the
// range; else the CTAs of all ranges stand in a row, those of range r from start[r] on.
struct Ranges { int start[5]; };
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const Params kp, const Params vp, const Params dkp, const Params dvp, const EvictArgs a,
                      const Ranges ranges) {
  __shared__ uint4 stage[2 * kChunks * kMoveThreads];
  const int slot = blockIdx.y, x = blockIdx.x;
  const int range = IN_PLACE ? (int)blockIdx.z : x < ranges.start[1] ? 0 : x < ranges.start[2] ? 1 : x < ranges.start[3] ? 2 : 3;
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
    move_any(q, stage, (int)blockIdx.x, (int)gridDim.x, [&] { cluster.sync(); });
    if (!weights) return;
    // tokens to come start at zero; the dropped weights above n have been read
    cluster.sync();
    for (int64_t t = a.n + (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; t < a.S;
         t += (int64_t)gridDim.x * kMoveThreads)
      w[t] = 0.f;
  } else {
    move_any(q, stage, x - ranges.start[range], ranges.start[range + 1] - ranges.start[range], [] {});
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
                         const EvictArgs& a, int pk, int pv, int sms, cudaStream_t s, int* nk) {
  // CTAs of a cluster: as many as there is work for, at most eight (the portable size),
  // and not far more than the device holds at once
  auto pick = [&](int64_t work, int64_t clusters, int64_t most) {
    int c = 1;
    while (c < 8 && c < work && 2 * c * clusters <= most) c *= 2;
    return c;
  };
  // select: one CTA where the keys of all tokens fit its registers (a cluster costs
  // its barriers and remote reads: 128 slots of 16384 tokens 16 us, 30 with two CTAs each)
  const int sel = pick((a.S + kSelStep - 1) / kSelStep, 1, 8);
  const int64_t per = (a.S + (int64_t)sel * kSelThreads - 1) / ((int64_t)sel * kSelThreads);
  const auto kernel = per <= 4    ? evict_select_kernel<4, true>
                      : per <= 8  ? evict_select_kernel<8, true>
                      : per <= 16 ? evict_select_kernel<kPer, true>
                                  : evict_select_kernel<kPer, false>;
  cudaError_t e = launch_cluster(kernel, dim3(sel, a.n_slots), kSelThreads, sel, false, s, a);
  ++*nk;
  if (e != cudaSuccess) return e;
  // move: about six CTAs per SM, shared out among the slots' ranges by their bytes
  const int rows[4] = {pk, pv, kp.side_bytes, vp.side_bytes};
  const int64_t all = std::max(1, rows[0] + rows[1] + rows[2] + rows[3]);
  const int64_t ctas = std::max<int64_t>(1, 6 * (int64_t)sms / a.n_slots);
  Ranges r{};
  int widest = 4;
  for (int i = 0; i < 4; ++i) {
    const int64_t most = ((int64_t)a.n * rows[i] + 15 + kStretch) / kStretch;  // stretches of the range
    const int64_t share = std::max<int64_t>(1, (ctas * rows[i] + all / 2) / all);
    r.start[i + 1] = r.start[i] + (rows[i] ? (int)std::min(most, share) : 0);
    widest = std::max(widest, rows[i]);
  }
  ++*nk;
  if (a.in_place) {
    const int64_t n = ((int64_t)a.n * widest + kStretch - 1) / kStretch;
    const int c = pick(n, (int64_t)a.n_slots * 2, 8 * (int64_t)sms);
    return launch_cluster(evict_move_kernel<true>, dim3(c, a.n_slots, a.weights ? 5 : 4), kMoveThreads, c, true, s,
                          kp, vp, dkp, dvp, a, r);
  }
  if (r.start[4] == 0) return cudaSuccess;  // rows of no bytes
  return launch_cluster(evict_move_kernel<false>, dim3((unsigned)r.start[4], a.n_slots), kMoveThreads, 1, true, s,
                        kp, vp, dkp, dvp, a, r);
}

}  // namespace kvc
