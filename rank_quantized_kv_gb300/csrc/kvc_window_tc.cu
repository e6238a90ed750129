// The windowed attention's tcgen05 kernel for many rows (the mathematics:
// kvc_window.cu): prompt chunks, or many queries that observe a prompt.
//
// A job is 128 rows (the M side of both products, a TMEM lane each) and walks tiles of
// 128 tokens:
//   S[row][token]    = W[row][K] A[token][K]^T   W: key weights, two fp16 pieces
//   O[row][channel] += P[row][token] V[token][channel]
// S lies in TMEM; a softmax thread owns a row, so maxima, sums and rescaling need no
// other thread; P goes back to TMEM in S's place as the second product's A operand.
// Two softmax groups of four warps take alternate tiles, each with its own S, O,
// references and sums, which meet at the job's end.
//
// One CTA per SM walks a run of (job, tile) pairs.  Roles, handing tiles on through
// mbarriers:
//   producer (1 thread)   bulk-copies packed rows and side words into stages;
//   decoders (8 warps)    codes -> fp16 operands in shared memory: keys K-major,
//                         values as they lie (MN-major);
//   two MMA warps         S and O;
//   softmax (2 x 4 warps) S -> P;
//   watchdog (1 thread)   gives up, for all roles, when no tile gets done.
//
// Precision: that of kvc_attend_tree (include/kvc.h).  Codes are exact in fp16,
// centroids rounded to fp16 after a common scale (2^-14 for eight Gaussian levels); W
// keeps 22 bits; P times the value scale is rounded to fp16.  References move lazily and
// are a row's own: that of the scores is its first maximum less 4, and moves when a score
// exceeds it by 8; that of the value scales the power of two above the largest that the
// row sees, moved when one exceeds it four times.  Their sum is one exponent, so a scale
// costs the loop nothing.
//
// Bound: latency in the softmax groups; no unit is near its rate.  8 slots of 8192 rows,
// a window of 2048 tokens, 3-bit keys and int8 values of 128 channels: 212 us, 61 tiles
// a CTA at 6100 cycles each, of which the tensor pipe works 1535 (three products of
// 128^3), a scheduler issues 2660 instructions and the XU pipe is busy for a tenth.  With
// clocks read in every role (15 % slower): a group is in the loop over a tile's columns for
// 36 to 50 % of its time (5000 to 6700 cycles for each of its 31 tiles), at the ends of
// segments for 13 % (11000 each, five a CTA), with the tile's scales for 5 % (mostly cold
// code at a segment's first tiles) and waits for scores for 2 to 12 %, the rest lies
// between these; the score products' warp waits for the groups for 63 %, the decoders for
// a place for values for 45 %.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kvc_launch.cuh"
#include "kvc_sm100.cuh"
#include "kvc_window.cuh"
#include "kvc_window_mma.cuh"

namespace kvc {

using namespace sm100;

namespace {

constexpr int kTile = 128, kRows = 128;
constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kProd = kSoftWarps + kDecWarps, kScore = kProd + 1, kSum = kProd + 2;
constexpr int kThreads = (kProd + 4) * 32;
constexpr int kMaxNS = 4;          // row stages
// Side words of a tile stay until its softmax has read them: the stage of tile i + 8
// is loaded once tile i + 8 - kMaxNS >= i + 4 is decoded, whose key operand needed the
// scores of the tile before, hence the S of two tiles before that: tile i is done.
constexpr int kSideRing = 8;
constexpr int kGroupBar = 1, kSoftBar = 3, kDecBar = 4;  // named barriers: groups 1, 2; all softmax; decoders
constexpr uint64_t kDrainNs = 2000000000ull;  // limit of the drains; the watchdog's is the layer's
constexpr uint32_t kTryNs = 20000;            // a try sleeps so long at most
constexpr float kSet = 4.f, kMove = 8.f;      // log2
constexpr float kScaleLowest = -24.f;         // log2 of the smallest positive scale
constexpr uint32_t kTransposeB = 1u << 16;

struct TcShape {
  int K, KC, DV;                 // K of the scores, its chunks of 8; channels of O
  int ns;                        // row stages
  int krow, stage;               // bytes of a stage's key rows; of a stage
  int off_k, off_v, off_stage;   // shared-memory offsets (W lies first)
  int smem;
};

// True in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p;
}
// tcgen05.mma and commit by the lane that has `lead`, predicated and not in a branch:
// the operands are then computed where the warp is converged.
__device__ __forceinline__ void mma_tmem_a(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %0, 0;\n setp.ne.b32 p, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n}" ::"r"(lead),
      "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_smem(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %0, 0;\n setp.ne.b32 p, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n}" ::"r"(lead),
      "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}" ::"r"(lead),
      "r"(smem_u32(bar))
      : "memory");
}
// Wait for the loads into v: its values are used below this, not above.
__device__ __forceinline__ void wait_loaded(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29])
               :
               : "memory");
  asm volatile("" : "+r"(v[30]), "+r"(v[31])::"memory");
}
// Wait for a phase, or until the watchdog has given up.  From then on every wait
// returns after one failed try, so that all roles walk to their ends and the named
// barriers stay matched; the results are undefined and the error word says so.
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag) return;
}

// A stretch of a job in a CTA's run: tiles [i0, i1) of the job's.
struct Segment {
  int job, slot, r0, nr, i0, i1;
  bool whole;  // the job lies in this CTA alone
  Sight sight;
  Tiles<kTile> tiles;
  __device__ Segment(const Params& kp, const WindowArgs& t, int64_t at, int64_t end, int job_)
      : job(job_), slot(job_ / t.row_tiles), r0((job_ - slot * t.row_tiles) * kRows), nr(min(kRows, t.rows - r0)),
        sight(t, slot / kp.H),
        tiles(sight, t.ctx + r0 / t.rep, t.ctx + (r0 + nr - 1) / t.rep) {
    const int64_t a0 = at - job_ * t.tps, count = tiles.count();
    i0 = (int)(count * a0 / t.tps);
    i1 = (int)(count * (a0 + (end - at)) / t.tps);
    whole = a0 == 0 && end - at == t.tps;
  }
};
// A softmax group's segment and place in the run, in shared memory so that they take no
// registers in its loop; one thread of the group walks, a segment ahead.  Divisions are
// done for the run's first and last segments alone: the others are whole jobs.
struct Place {
  int more;  // 0: the run is at its end
  int job, slot, jt, r0, nr, n, p0, p1;
  int whole;
  int first, sink_end, window;
  int part;          // number of the partial, where it leaves one
  int a, na, b, i0;  // tiles, as in Tiles, from number i0 on
  int64_t at, run1;
  __device__ void begin(const Params& kp, const WindowArgs& t) {
    at = window_run(t, blockIdx.x);
    run1 = window_run(t, blockIdx.x + 1);
    job = (int)(at / t.tps);
    slot = job / t.row_tiles;
    jt = job - slot * t.row_tiles;
    fill(kp, t);
  }
  __device__ void fill(const Params& kp, const WindowArgs& t) {
    more = at < run1;
    if (!more) return;
    const int64_t start = job * t.tps, end = min(run1, start + t.tps);
    r0 = jt * kRows;
    nr = min(kRows, t.rows - r0);
    p0 = t.ctx + r0 / t.rep;
    p1 = t.ctx + (r0 + nr - 1) / t.rep;
    const Sight s(t, slot / kp.H);
    const Tiles<kTile> tiles(s, p0, p1);
    first = s.first;
    sink_end = s.sink_end;
    window = s.window;
    a = tiles.a;
    na = tiles.na;
    b = tiles.b;
    i0 = 0;
    n = tiles.count();
    whole = at == start && end == start + t.tps;
    part = job + (int)blockIdx.x;
    if (t.cuts && !whole) {
      const int64_t c0 = at == start ? blockIdx.x : window_cta(t, start);
      part = (int)(window_part(t, job, c0) + blockIdx.x - c0);
    }
    if (!whole) {
      i0 = (int)((int64_t)n * (at - start) / t.tps);
      n = (int)((int64_t)n * (end - start) / t.tps) - i0;
    }
    at = end;
  }
  // This place's successor, into `to`.
  __device__ void next(const Params& kp, const WindowArgs& t, Place& to) const {
    to.at = at;
    to.run1 = run1;
    to.job = job + 1;
    to.slot = slot;
    to.jt = jt + 1;
    if (to.jt == t.row_tiles) {
      to.jt = 0;
      ++to.slot;
    }
    to.fill(kp, t);
  }
  __device__ int token(int i) const {  // the first of tile i of the segment
    const int x = i0 + i;
    return (x < na ? a + x : b + x - na) * kTile;
  }
};
// f(segment) for every stretch of the CTA's run.
template <class F>
__device__ __forceinline__ void walk(const Params& kp, const WindowArgs& t, F f) {
  const int64_t run1 = window_run(t, blockIdx.x + 1);
  for (int64_t at = window_run(t, blockIdx.x); at < run1;) {
    const int job = (int)(at / t.tps);
    const int64_t end = min(run1, (job + 1) * t.tps);
    const Segment g(kp, t, at, end, job);
    at = end;
    f(g);
  }
}

// Eight W-bit codes from bit 8 W q of the words as fp16 centroids: pairs from a table
// that holds every pair once per lane, singles at four bits.
template <int W, int M>
__device__ __forceinline__ uint4 centroids(const uint32_t (&w)[M], int q, const unsigned char* tab, uint32_t lane4) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (W <= 3) {
      constexpr uint32_t mask = ((1u << (2 * W)) - 1u) << 7;
      const int bit = 8 * W * q + 2 * W * i - 7, at = bit >> 5, sh = bit & 31;
      uint32_t v;
      if (bit < 0) v = w[0] << -bit;
      else if (sh + 2 * W + 7 <= 32 || at + 1 >= M) v = w[at] >> sh;
      else v = __funnelshift_r(w[at], w[(at + 1) % M], sh);
      r[i] = *reinterpret_cast<const uint32_t*>(tab + ((v & mask) | lane4));
    } else {
      const uint32_t x = w[q] >> (8 * i);
      const uint32_t a = *reinterpret_cast<const uint32_t*>(tab + (((x & 15u) << 7) | lane4));
      const uint32_t b = *reinterpret_cast<const uint32_t*>(tab + (((x & 0xf0u) << 3) | lane4));
      r[i] = __byte_perm(a, b, 0x5410);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// 32 consecutive codes (W words) as four chunks of an operand, 128 bytes apart.
template <int W>
__device__ __forceinline__ void centroids32(const unsigned char* src, const unsigned char* tab, uint32_t lane4,
                                            unsigned char* dst) {
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t*>(src)[i];
#pragma unroll
  for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(dst + q * 128) = centroids<W>(w, q, tab, lane4);
}
// Eight int8 values as fp16.
__device__ __forceinline__ uint4 int8_values(uint2 b) {
  const uint32_t x = b.x ^ 0x80808080u, y = b.y ^ 0x80808080u, sub = kMagic | 0x00800080u;
  return make_uint4(sub_f16x2(__byte_perm(x, 0x64646464u, 0x5140), sub), sub_f16x2(__byte_perm(x, 0x64646464u, 0x5342), sub),
                    sub_f16x2(__byte_perm(y, 0x64646464u, 0x5140), sub), sub_f16x2(__byte_perm(y, 0x64646464u, 0x5342), sub));
}
// The int8 values of one token block (8 rows of NV chunks of 8 bytes) as fp16: lane
// (octet, t8) takes token t8 and NV / 2 chunks from first on, modulo NV; all loads first.
template <int NV>
__device__ __forceinline__ void int8_block(const unsigned char* row, unsigned char* dst, int first) {
  uint2 b[NV / 2];
#pragma unroll
  for (int j = 0; j < NV / 2; ++j) b[j] = *reinterpret_cast<const uint2*>(row + ((first + j) & (NV - 1)) * 8);
#pragma unroll
  for (int j = 0; j < NV / 2; ++j)
    *reinterpret_cast<uint4*>(dst + ((first + j) & (NV - 1)) * 128) = int8_values(b[j]);
}
// Bits [lo, hi] of a word, those of them that it has.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  if (hi < 0 || lo > 31 || lo > hi) return 0u;
  return (~0u << max(lo, 0)) & (~0u >> (31 - min(hi, 31)));
}
// Eight centred codes of a chunk as fp16.
__device__ __forceinline__ uint4 centred(uint2 bits, uint32_t entry) {
  Width w;
  w.set(entry);
  const uint2 b = w.split(bits);
  return make_uint4(w.pair(b, 0), w.pair(b, 1), w.pair(b, 2), w.pair(b, 3));
}

// The largest finite scale of the columns in [ca, ca1] and [cb, cb1], a row's own, of 32
// at a time: a lane holds one for the warp's rows.  (Kept short: it runs twice a segment,
// and its instructions come from L2.)
__device__ __forceinline__ float largest_seen(const float* scale, int ca, int ca1, int cb, int cb1) {
  float most = 0.f;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t see = bits_between(ca - 32 * q, ca1 - 32 * q) | bits_between(cb - 32 * q, cb1 - 32 * q);
    if (!__any_sync(kFull, see)) continue;
    const float x = scale[32 * q + lane];
    const float y = x > 0.f && x <= 65504.f ? x : 0.f;
    if (__all_sync(kFull, see == 0u || see == ~0u)) {
      const uint32_t u = __reduce_max_sync(kFull, __float_as_uint(y));
      if (see) most = fmaxf(most, __uint_as_float(u));
    } else {
#pragma unroll 4
      for (int e = 0; e < 32; ++e) {
        const float w = __shfl_sync(kFull, y, e);
        if (see >> e & 1u) most = fmaxf(most, w);
      }
    }
  }
  return most;
}

template <int KMODE, int VMODE>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const Params kp, const Params vp, const WindowArgs t, const TcShape z) {
  constexpr bool CB = KMODE == KVC_MODE_CODEBOOK, VU = VMODE == KVC_MODE_UNIFORM;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t row_full[kMaxNS], row_empty[kMaxNS], k_full, k_empty, v_full[2], v_empty[2], s_full[2], p_full[2],
      o_done[2], side_full[kSideRing], w_full, w_empty, done_bar;
  __shared__ uint32_t kch[32], vch[32];
  __shared__ __align__(16) unsigned short side_s[kSideRing][2][kTile];  // norms, scales
  __shared__ __align__(16) float cn[2][2][kTile], cs[2][2][kTile];  // per group and turn: norms, scales
  __shared__ __align__(16) float red[2][2][4];  // per group and turn: the warps' largest scales
  __shared__ float gm[2][kRows], gl[2][kRows], gx[2][kRows];  // the groups' references and sums; NaN: spoilt rows
  __shared__ __align__(256) unsigned char tab[CB ? 64 * 32 * 4 : 16];
  __shared__ __align__(8) unsigned char place_s[4 * sizeof(Place)];  // per group this one and the next
  Place* place = reinterpret_cast<Place*>(place_s);
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag, tiles_done;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* Ks = smem + z.off_k;
  unsigned char* Vs = smem + z.off_v;
  unsigned char* Rs = smem + z.off_stage;
  const int w_piece = kRows * z.K * 2, v_bytes = kTile * z.DV * 2;
  const uint32_t s_col = 0, o_col = 2 * kTile;

  if (warp == kScore) tmem_alloc(&tmem_base, 512);
  if (tid == 0) {
    for (int i = 0; i < z.ns; ++i) { mbar_init(&row_full[i], 1); mbar_init(&row_empty[i], kDecWarps); }
    mbar_init(&k_full, kDecWarps);
    mbar_init(&k_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], kDecWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < kSideRing; ++i) mbar_init(&side_full[i], 1);
    mbar_init(&w_full, 1);
    mbar_init(&w_empty, 1);
    mbar_init(&done_bar, 2);
    fence_mbar_init();
    abort_flag = tiles_done = 0;
  }
  if (tid < 2) place[2 * tid].begin(kp, t);
  if (CB) {
    const int wb = kp.cb_bits, lm = (1 << wb) - 1, n = (wb <= 3 ? 1 << (2 * wb) : 16) * 32;
    auto half_of = [&](int c) { return (uint32_t)__half_as_ushort(__float2half_rn(kp.codebook[c] * t.cb_mul)); };
    for (int j = tid; j < n; j += kThreads)
      reinterpret_cast<uint32_t*>(tab)[j] = half_of((j >> 5) & lm) | (wb <= 3 ? half_of(j >> (5 + wb)) << 16 : 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  grid_dependency_wait();  // the key weights come from the launch before

  if (warp >= kProd) {
    if (warp == kProd && lane == 0) {
      // ---------------------------------------------------------- producer
      int issued = 0, segs = 0;
      walk(kp, t, [&](const Segment& g) {
        if (g.i0 == g.i1 || abort_flag) return;
        // the job's key weights, once the last segment's scores are done
        if (segs) wait_or_abort(&w_empty, (segs - 1) & 1, &abort_flag);
        if (abort_flag) return;
        mbar_arrive_expect_tx(&w_full, 2 * w_piece);
        bulk_load(smem, t.w16 + (size_t)g.job * 2 * kRows * z.K, 2 * w_piece, &w_full);
        ++segs;
        const int Pk = kp.P[kp.basis_of[g.slot]], Pv = VU ? vp.P[vp.basis_of[g.slot]] : vp.D;
        const unsigned char* ks = kp.store + kp.pay_off[g.slot];
        const unsigned char* vs = vp.store + vp.pay_off[g.slot];
        const unsigned char* kn = kp.store + kp.side_off[g.slot];
        const unsigned char* vsc = vp.store + vp.side_off[g.slot];
        for (int i = g.i0; i < g.i1; ++i, ++issued) {
          const int st = issued % z.ns;
          if (issued >= z.ns) wait_or_abort(&row_empty[st], (issued / z.ns - 1) & 1, &abort_flag);
          if (abort_flag) return;
          const int64_t t0 = (int64_t)g.tiles.tile(i) * kTile;
          const int n = (int)min((int64_t)kTile, t.S - t0);
          const uint32_t kb = (uint32_t)((n * Pk + 15) & ~15), vb = (uint32_t)((n * Pv + 15) & ~15);
          unsigned char* to = Rs + st * z.stage;
          mbar_arrive_expect_tx(&row_full[st], kb + vb);
          if (kb) bulk_load(to, ks + t0 * Pk, kb, &row_full[st]);
          if (vb) bulk_load(to + z.krow, vs + t0 * Pv, vb, &row_full[st]);
          const int sd = issued % kSideRing;
          const uint32_t sb = (uint32_t)((2 * n + 15) & ~15);
          mbar_arrive_expect_tx(&side_full[sd], (CB ? sb : 0) + (VU ? 0 : sb));
          if (CB) bulk_load(side_s[sd][0], kn + t0 * 2, sb, &side_full[sd]);
          if (!VU) bulk_load(side_s[sd][1], vsc + t0 * 2, sb, &side_full[sd]);
        }
      });
      // copies still in flight (after a time-out) land before the CTA exits
      if (segs) mbar_wait_bounded(&w_full, (segs - 1) & 1, kDrainNs);
      for (int j = max(0, issued - z.ns); j < issued; ++j)
        mbar_wait_bounded(&row_full[j % z.ns], (j / z.ns) & 1, kDrainNs);
      for (int j = max(0, issued - kSideRing); j < issued; ++j)
        mbar_wait_bounded(&side_full[j % kSideRing], (j / kSideRing) & 1, kDrainNs);
    } else if (warp == kScore) {
      // ---------------------------------------------------------- S = W A^T
      const uint32_t lead = elect_one(), tmu = __shfl_sync(kFull, tm, 0);
      constexpr uint32_t id = idesc_f16(kRows, kTile, 0);
      const uint64_t wd = desc_kmajor_noswizzle(smem_u32(smem), 128, (uint32_t)z.KC * 128);
      const uint64_t kd = desc_kmajor_noswizzle(smem_u32(Ks), 128, (uint32_t)z.KC * 128);
      int it = 0, segs = 0;
      walk(kp, t, [&](const Segment& g) {
        const int n = __shfl_sync(kFull, g.i1 - g.i0, 0);
        if (n == 0) return;
        wait_or_abort(&w_full, segs & 1, &abort_flag);
        ++segs;
        for (int i = 0; i < n; ++i, ++it) {
          const int s = it & 1;
          if (it >= 2) wait_or_abort(&o_done[s], ((it >> 1) - 1) & 1, &abort_flag);  // P has been read
          wait_or_abort(&k_full, it & 1, &abort_flag);
          __syncwarp();
          tc_fence_after();
          for (int p = 0; p < 2; ++p)
#pragma unroll 4
            for (int k = 0; k < z.K / 16; ++k)
              mma_smem(lead, tmu + s_col + s * kTile, wd + ((p * w_piece) >> 4) + k * 16, kd + k * 16, id, p + k > 0);
          commit_if(lead, &s_full[s]);
          commit_if(lead, &k_empty);
          if (i + 1 == n) commit_if(lead, &w_empty);
        }
      });
      if (lead) {
        umma_commit(&done_bar);  // TMEM is released only after every MMA has finished
        mbar_wait_bounded(&done_bar, 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp == kSum) {
      // ---------------------------------------------------------- O += P V
      const uint32_t lead = elect_one(), tmu = __shfl_sync(kFull, tm, 0);
      const uint32_t id = idesc_f16(kRows, z.DV, 0) | kTransposeB;
      const uint32_t v_k = (uint32_t)z.DV * 16;  // bytes between V's cores along the tokens
      const uint64_t vd0 = desc_kmajor_noswizzle(smem_u32(Vs), v_k, 128);
      int it = 0;
      walk(kp, t, [&](const Segment& g) {
        const int n = __shfl_sync(kFull, g.i1 - g.i0, 0);
        for (int i = 0; i < n; ++i, ++it) {
          const int s = it & 1;
          wait_or_abort(&v_full[s], (it >> 1) & 1, &abort_flag);
          wait_or_abort(&p_full[s], (it >> 1) & 1, &abort_flag);
          __syncwarp();
          tc_fence_after();
          const uint64_t vd = vd0 + ((s * v_bytes) >> 4);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_tmem_a(lead, tmu + o_col + s * kTile, tmu + s_col + s * kTile + k * 8, vd + k * ((2 * v_k) >> 4), id,
                       k > 0 || i >= 2);  // the group's first tile of the segment overwrites its O
          commit_if(lead, &o_done[s]);
          commit_if(lead, &v_empty[s]);
          tiles_done = it + 1;  // (every lane the same)
        }
      });
      if (lead) {
        umma_commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp > kSum && lane == 0) {
      // ---------------------------------------------------------- watchdog
      // Gives up when no tile has been summed for the limit, as it finds each time
      // that the end has not come within a try.
      int seen_done = 0;
      uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait_sleep(&done_bar, 0, kTryNs)) {
        const uint64_t now = global_timer_ns();
        if (now - t0 > t.wait_ns) {
          abort_flag = 1;
          break;
        }
        if (tiles_done != seen_done) {
          seen_done = tiles_done;
          t0 = now;
        }
      }
    }
  } else if (warp >= kSoftWarps) {
    // ------------------------------------------------------------ decoders
    const int dtid = tid - kSoftWarps * 32, tt = dtid & (kTile - 1), half = dtid >> 7;
    // values: eight lanes take eight tokens of one block, each another chunk of the row,
    // so that neither the reads nor the writes (cores 128 bytes apart) meet in a bank
    const int octet = lane >> 3, t8 = lane & 7, vblk = (dtid >> 5) * 2 + (octet >> 1);
    int it = 0;
    walk(kp, t, [&](const Segment& g) {
      if (g.i0 == g.i1) return;
      named_bar_sync(kDecBar, kDecWarps * 32);  // the last segment's tables have been read
      const int kbeta = kp.basis_of[g.slot], vbeta = VU ? vp.basis_of[g.slot] : 0;
      if (dtid < 32) kch[dtid] = chunk_entry(kp, kbeta, dtid);
      else if (VU && dtid < 64) vch[dtid - 32] = chunk_entry(vp, vbeta, dtid - 32);
      named_bar_sync(kDecBar, kDecWarps * 32);
      const int Pk = kp.P[kbeta], Pv = VU ? vp.P[vbeta] : vp.D;
      for (int i = g.i0; i < g.i1; ++i, ++it) {
        const int rs = it % z.ns, vb = it & 1;
        wait_or_abort(&row_full[rs], (it / z.ns) & 1, &abort_flag);
        if (it >= 1) wait_or_abort(&k_empty, (it - 1) & 1, &abort_flag);
        __syncwarp();
        const unsigned char* st = Rs + rs * z.stage;
        unsigned char* kd = Ks + (tt >> 3) * (z.KC * 128) + (tt & 7) * 16;
        if (CB) {
          const int W = kp.cb_bits, per = kp.D / 64;  // stretches of 32 codes of a half
          for (int x = 0; x < per; ++x) {
            const int c0 = (half * per + x) * 4;  // first chunk
            const unsigned char* src = st + tt * Pk + c0 * W;
            unsigned char* dst = kd + c0 * 128;
            if (W == 3) centroids32<3>(src, tab, 4 * lane, dst);
            else if (W == 4) centroids32<4>(src, tab, 4 * lane, dst);
            else if (W == 2) centroids32<2>(src, tab, 4 * lane, dst);
            else centroids32<1>(src, tab, 4 * lane, dst);
          }
        } else {
          for (int c = half; c < z.KC; c += 2) {
            const uint32_t e = kch[c];
            *reinterpret_cast<uint4*>(kd + c * 128) =
                e ? centred(bits_at(st, tt * Pk + (int)(e & 0xffffu)), e) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();  // the operand is read by the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full);
        if (it >= 2) wait_or_abort(&v_empty[vb], ((it >> 1) - 1) & 1, &abort_flag);
        __syncwarp();
        {
          const unsigned char* raw = st + z.krow;
          const int tok = vblk * 8 + t8, nv = z.DV / 8;
          unsigned char* dst = Vs + vb * v_bytes + vblk * (z.DV * 16) + t8 * 16;
          const int c0 = (octet & 1) * (nv / 2) + t8;
          if (!VU && nv == 16) {
            int8_block<16>(raw + tok * 128, dst, c0);
          } else if (!VU && nv == 8) {
            int8_block<8>(raw + tok * 64, dst, c0);
          } else {
            for (int j = 0; j < nv / 2; ++j) {
              int c = c0 + j;
              while (c >= nv) c -= nv;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (VU) {
                const uint32_t e = vch[c];
                if (e) v = centred(bits_at(raw, tok * Pv + (int)(e & 0xffffu)), e);
              } else {
                v = int8_values(*reinterpret_cast<const uint2*>(raw + tok * Pv + c * 8));
              }
              *reinterpret_cast<uint4*>(dst + c * 128) = v;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[vb]);
          mbar_arrive(&row_empty[rs]);
        }
      }
    });
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane, bar = kGroupBar + wg;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tm + lane_off + s_col + wg * kTile, o_tm = tm + lane_off + o_col;
    int it0 = 0, turn = 0;  // tiles of the run before the segment; the group's tiles so far
    for (int turns = 0;; ++turns) {
      volatile Place& vg = place[2 * wg + (turns & 1)];
      if (!vg.more) break;
      const Place& g = place[2 * wg + (turns & 1)];
      const int n = vg.n, x = vg.r0 + min(r, vg.nr - 1), pos = t.ctx + x / t.rep;  // (rows past the last: its sight)
      const float rs = t.wscale[(size_t)vg.job * kRows + r];
      // The row's l and O are in units of 2^ref, ref = score reference + sref, where sref
      // (log2) is that of the value scales: nothing of it depends on what other rows see.
      float ref = -INFINITY, sref = VU ? 0.f : kScaleLowest;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      bool seen = false, spoilt = false;  // the row sees a token; one with a value scale of NaN
      int mine = 0;  // the group's tiles of the segment
      for (int i = (it0 ^ wg) & 1; i < n; i += 2, ++turn, ++mine) {
        const int it = it0 + i, t0 = g.token(i), buf = turn & 1;
        const uint32_t par = (it >> 1) & 1;
        const int t1 = t0 + kTile - 1;
        const bool all = t0 >= vg.first && t1 <= vg.p0 && (t0 > vg.p1 - vg.window || t1 < vg.sink_end);
        // visible columns, where not all are: [ca, ca1] and [cb, cb1]
        int ca = 0, ca1 = kTile - 1, cb = 0, cb1 = -1;
        if (!all) {
          const int first = vg.first;
          ca = max(first, pos - vg.window + 1) - t0;
          ca1 = pos - t0;
          cb = first - t0;
          cb1 = min(vg.sink_end, pos + 1) - 1 - t0;
          seen |= max(ca, 0) <= min(ca1, kTile - 1) || max(cb, 0) <= min(cb1, kTile - 1);
        } else {
          seen = true;
        }
        // this thread's column: its norm (codebook keys) and scale for all rows
        if (CB || !VU) {
          const int sd = it % kSideRing, tok = t0 + r;
          wait_or_abort(&side_full[sd], (it / kSideRing) & 1, &abort_flag);
          if (!VU) {
            float scale = __half2float(__ushort_as_half(side_s[sd][1][r]));
            // a token that no row sees may hold anything; a scale of NaN counts as 0 in the
            // product, and the rows that see it are marked below
            if (tok >= t.S || tok < vg.first) scale = 0.f;
            float level = scale > 0.f && scale <= 65504.f ? scale : 0.f;
            if (scale != scale) {
              level = INFINITY;
              scale = 0.f;
            }
            cs[wg][buf][r] = fmaxf(fminf(scale, 3e38f), -3e38f);
            const uint32_t big = __reduce_max_sync(kFull, __float_as_uint(level));
            if (lane == 0) red[wg][buf][quarter] = __uint_as_float(big);
          }
          if (CB) cn[wg][buf][r] = __half2float(__ushort_as_half(side_s[sd][0][r]));
        }
        if (CB || !VU) named_bar_sync(bar, 128);
        if (!VU) {
          // the row's reference of the scales: the power of two above the largest finite one
          // that it sees, once one exceeds it four times (before S is waited for: the first
          // tiles of a segment, which move it, wait for S in any case)
          const float4 warps = *reinterpret_cast<const float4*>(red[wg][buf]);
          float most = fmaxf(fmaxf(warps.x, warps.y), fmaxf(warps.z, warps.w));
          const float limit = __int_as_float(((int)sref + 2 + 127) << 23);
          if (__any_sync(kFull, most > limit)) {
            const bool odd = most == INFINITY;  // (for all rows) a column has a scale of NaN
            if (odd)
#pragma unroll 1
              for (int c = 0; c < kTile && !spoilt; ++c)
                spoilt = ((c >= ca && c <= ca1) || (c >= cb && c <= cb1)) &&
                         __hisnan(__ushort_as_half(side_s[it % kSideRing][1][c]));
            if (!all || odd) {  // the largest may be hidden from this row
              most = largest_seen(cs[wg][buf], ca, ca1, cb, cb1);
            }
            float f = 1.f;
            if (most > limit) {
              const float to = (float)((__float_as_int(most) >> 23) - 126), now = ref + (to - sref);
              if (ref != -INFINITY) f = ex2(ref - now);
              ref = now;
              sref = to;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) l2[e] = __fmul2_rn(l2[e], make_float2(f, f));
            if (mine && __any_sync(kFull, f != 1.f)) {  // O holds sums: the last product is done once S has been written
              wait_or_abort(&s_full[wg], par, &abort_flag);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < z.DV; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_tm + wg * kTile + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_tm + wg * kTile + c, o);
              }
              tmem_wait_st();
            }
          }
        }
        wait_or_abort(&s_full[wg], par, &abort_flag);
        __syncwarp();
        tc_fence_after();
        // 32 columns at a time: P's 16 columns go where columns of S that have been read
        // were.  (The loop is kept rolled: unrolled, its instructions came from L2.)
        uint32_t v[32];
        tmem_ld32(s_tm, v);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          wait_loaded(v);
          float2 y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          if (CB) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 f = *reinterpret_cast<const float4*>(&cn[wg][buf][32 * q + 4 * e]);
              y[2 * e] = __fmul2_rn(y[2 * e], make_float2(f.x, f.y));
              y[2 * e + 1] = __fmul2_rn(y[2 * e + 1], make_float2(f.z, f.w));
            }
          }
          if (q < 3) tmem_ld32(s_tm + 32 * (q + 1), v);
          if (!all) {
            const uint32_t see = bits_between(ca - 32 * q, ca1 - 32 * q) | bits_between(cb - 32 * q, cb1 - 32 * q);
            if (__any_sync(kFull, see != ~0u)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (!(see >> (2 * e) & 1u)) y[e].x = -INFINITY;
                if (!(see >> (2 * e + 1) & 1u)) y[e].y = -INFINITY;
              }
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 16; ++e) top[e & 3] = max_nan(top[e & 3], y[e].x, y[e].y);
          const float most = max_nan(max_nan(top[0], top[1]), max_nan(top[2], top[3])) * rs;
          const bool need = most > -INFINITY && !(most - ref <= kMove - sref);
          if (__any_sync(kFull, need)) {
            // the first reference, or a new one, whole steps of log2 away
            float now = ref, f = 1.f;
            if (need && most > kWindowLowest) {
              const float to = most - kSet + sref, up = to - ref;
              now = up < 1048576.f ? ref + ceilf(up) : to;
              if (most - now > kMove - sref) now = most;  // (past 2^27 fp32 has no such steps)
              f = ex2(ref - now);
            }
            ref = now;
#pragma unroll
            for (int e = 0; e < 2; ++e) l2[e] = __fmul2_rn(l2[e], make_float2(f, f));
            const __half2 fh = __float2half2_rn(f);
#pragma unroll 1
            for (int c = 0; c < q; ++c) {  // the tile's weights so far
              uint32_t h[16];
              tmem_ld16(s_tm + 16 * c, h);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), fh);
                h[e] = *reinterpret_cast<const uint32_t*>(&p);
              }
              tmem_st16(s_tm + 16 * c, h);
            }
            if (mine)
#pragma unroll 1
              for (int c = 0; c < z.DV; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_tm + wg * kTile + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_tm + wg * kTile + c, o);
              }
            tmem_wait_st();
          }
          const float neg = ref == -INFINITY ? 0.f : -ref;
          const float2 rs2 = make_float2(rs, rs), neg2 = make_float2(neg, neg);
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
            if (!VU) f = *reinterpret_cast<const float4*>(&cs[wg][buf][32 * q + 4 * e]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 xx = __ffma2_rn(y[2 * e + u], rs2, neg2);
              const float2 p = make_float2(ex2(xx.x), ex2(xx.y));
              l2[u] = __fadd2_rn(l2[u], p);
              const float2 w = VU ? p : __fmul2_rn(p, u ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
              h[2 * e + u] = pack_f16(w.x, w.y);
            }
          }
          tmem_st16(s_tm + 16 * q, h);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg]);
      }
      // ---- the groups' states into one
      if (r == 0) g.next(kp, t, place[2 * wg + (~turns & 1)]);  // (read after the barriers below)
      const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      if (mine) {
        wait_or_abort(&o_done[wg], ((it0 + n - 1 - ((it0 + n - 1 - wg) & 1)) >> 1) & 1, &abort_flag);
        __syncwarp();
        tc_fence_after();
      }
      gm[wg][r] = l != 0.f ? ref : seen ? kWindowLowest : -INFINITY;
      gl[wg][r] = l;
      gx[wg][r] = spoilt ? NAN : 0.f;
      // each group reads the other's sums below: the reads come after the products that
      // the other one has waited for
      tc_fence_before();
      named_bar_sync(kSoftBar, kSoftWarps * 32);
      tc_fence_after();
      const float ma = gm[0][r], mb = gm[1][r], la = gl[0][r], lb = gl[1][r];
      const float M = fmaxf(ma, mb), add = gx[0][r] + gx[1][r];
      const float fa = la != 0.f ? ex2(ma - M) : 0.f, fb = lb != 0.f ? ex2(mb - M) : 0.f;
      const float L = (la != 0.f ? fa * la : 0.f) + (lb != 0.f ? fb * lb : 0.f);
      // tiles of either group in the segment
      const bool has_a = n > 1 || (n == 1 && !(it0 & 1)), has_b = n > 1 || (n == 1 && (it0 & 1));
      const float inv = L > 0.f || L != L ? 1.f / L : M == -INFINITY ? 0.f : NAN;
      const bool direct = vg.whole && !VU;
      const size_t part = vg.part;
      if (direct) {
        if (wg == 0 && r < vg.nr && t.stats)
          t.stats[(size_t)vg.slot * t.rows + vg.r0 + r] = make_float2(M == -INFINITY ? 0.f : M, inv);
      } else if (wg == 0) {
        t.ml[part * kRows + r] = make_float2(M, L);
      }
      const int b = vg.slot / kp.H, h = vg.slot - b * kp.H, nq = x / t.rep;
      const int64_t o0 = b * t.o_sb + (int64_t)(h * t.rep + x - nq * t.rep) * t.o_sh + nq * t.o_st;
#pragma unroll 1
      for (int c0 = 0; c0 < z.DV / 2; c0 += 16) {
        const int c = wg * (z.DV / 2) + c0;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = add;
        if (has_a) {
          uint32_t o[16];
          tmem_ld16(o_tm + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = fmaf(__uint_as_float(o[e]), fa, v[e]);
        }
        if (has_b) {
          uint32_t o[16];
          tmem_ld16(o_tm + kTile + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = fmaf(__uint_as_float(o[e]), fb, v[e]);
        }
        if (!direct) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c + e < t.Dv) t.part[(part * t.Dvp + c + e) * kRows + r] = v[e];
        } else if (r < vg.nr) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (a row that sees nothing is zero)
            const float p = inv == 0.f ? 0.f : v[2 * e] * inv, q = inv == 0.f ? 0.f : v[2 * e + 1] * inv;
            if (t.out_bf16) {
              const __nv_bfloat162 y2 = __floats2bfloat162_rn(p, q);
              w[e] = *reinterpret_cast<const uint32_t*>(&y2);
            } else {
              w[e] = pack_f16(p, q);
            }
          }
          unsigned short* out = static_cast<unsigned short*>(t.out) + o0 + c;
          if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
            reinterpret_cast<uint4*>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              out[2 * e] = (unsigned short)w[e];
              out[2 * e + 1] = (unsigned short)(w[e] >> 16);
            }
          }
        }
      }
      tc_fence_before();
      named_bar_sync(kSoftBar, kSoftWarps * 32);  // the next segment overwrites O and the exchange
      tc_fence_after();
      it0 += n;
    }
  }
  __syncthreads();
  grid_dependents_launch();
  if (abort_flag && tid == 0) atomicCAS(kp.err, 0, kErrTimeout);
  if (warp == kScore) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

using TcKernel = void (*)(const Params, const Params, const WindowArgs, const TcShape);

TcKernel kernel_for(const Params& kp, const Params& vp) {
  if (kp.mode == KVC_MODE_UNIFORM)
    return vp.mode == KVC_MODE_UNIFORM ? window_tc_kernel<KVC_MODE_UNIFORM, KVC_MODE_UNIFORM>
                                       : window_tc_kernel<KVC_MODE_UNIFORM, KVC_MODE_INT8>;
  return vp.mode == KVC_MODE_UNIFORM ? window_tc_kernel<KVC_MODE_CODEBOOK, KVC_MODE_UNIFORM>
                                     : window_tc_kernel<KVC_MODE_CODEBOOK, KVC_MODE_INT8>;
}

// The layout, or false where shared memory does not hold it.
bool shape_for(const Params& vp, const WindowArgs& t, TcShape* z) {
  const bool vu = vp.mode == KVC_MODE_UNIFORM;
  auto up = [](int v, int to) { return (v + to - 1) / to * to; };
  z->K = up(t.NCk, 16);
  z->KC = z->K / 8;
  z->DV = up(t.Dv, 32);
  z->krow = up(kTile * t.Pk_max + 16, 128);
  z->stage = z->krow + up(kTile * t.Pv_max + (vu ? 16 : 0), 128);
  z->off_k = 2 * kRows * z->K * 2;
  z->off_v = z->off_k + kTile * z->K * 2;
  z->off_stage = z->off_v + 2 * kTile * z->DV * 2;
  const int most = 227 * 1024 - 22 * 1024;  // the static arrays take up to 22 KB
  for (z->ns = kMaxNS; z->ns >= 2; --z->ns) {
    z->smem = z->off_stage + z->ns * z->stage;
    if (z->smem <= most) return true;
  }
  return false;
}

}  // namespace

int window_tc_k(const Params& kp, const Params& vp, const WindowArgs& t) {
  if (t.prod || !window_projects(kp, t) || t.Dv > 128) return 0;
  if (kp.mode == KVC_MODE_CODEBOOK && kp.cb_bits > 4) return 0;
  if (vp.mode == KVC_MODE_INT8 && vp.D % 32) return 0;
  TcShape z;
  return shape_for(vp, t, &z) ? z.K : 0;
}

cudaError_t launch_window_tc(const Params& kp, const Params& vp, const WindowArgs& t, cudaStream_t s, int* nk) {
  TcShape z;
  if (!shape_for(vp, t, &z)) return cudaErrorInvalidValue;
  const TcKernel k = kernel_for(kp, vp);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), z.smem);
  if (e != cudaSuccess) return e;
  ++*nk;
  return launch_dependent(k, (unsigned)t.grid, kThreads, (size_t)z.smem, s, kp, vp, t, z);
}

}  // namespace kvc
