// Tree attention on the tensor cores (the mathematics: kvc_attend_tree.cu).
//
// Tokens lie on the M side of both products, query rows on the N side:
//   S[token][row]   = A[token][K] W[row][K]^T   A: codes as fp16, in TMEM
//   O[channel][row] += V[token][channel]^T P[token][row]
// so a job of 16 rows costs an eighth of one of 128 (with rows on M it would
// cost the same), and the codes are decoded once per job of up to 128 rows.
//
// One CTA per SM walks a run of (job, 128-token tile) pairs.  Roles, handing
// tiles on through mbarrier rings:
//   producer (1 thread)   bulk-copies packed key and value rows into row stages;
//   decoders (8 or 16 warps; the second eight take every other tile)
//                         key codes -> fp16 A in TMEM (lane = token); value
//                         codes -> fp16 V in shared memory;
//   two MMA warps         S = A W^T, and O += V^T P;
//   softmax (2 groups of 4 warps; lane = token)
//                         S -> P in fp16 in shared memory, sums of P in fp32;
//   watchdog (1 thread)   gives up, for all roles, when no tile gets done.
// Jobs of up to 64 rows: the softmax groups take alternate tiles, each with its
// own references, sums and O, which the combine joins.  Jobs of 128 rows: TMEM
// does not hold two O, so the groups take half of the columns each.
//
// Precision.  Codes are exact in fp16 (centred codes up to 128, int8 values).
// Centroids are rounded to fp16 after a common scale, chosen at init so that
// they fall nearest to fp16 values (relative 2^-11 at most; 2^-14 for the eight
// levels of a Gaussian).  The key weights W are two fp16 pieces of weights that
// a power of two per row brings into fp16's upper range: 22 bits of the large
// ones, an error of at most 2^-19 of the row's largest.  P is rounded to fp16:
// one rounding of relative 2^-11 per weight, independent between tokens, below
// the rounding of the 16-bit output.  S, O, the sums and the softmax's reference
// are fp32.
//
// Softmax.  A weight is 2^(s - m) with m a reference per row, not the running
// maximum itself: m is set to the tile's maximum less 6 when the row first sees
// a token, and moves only when a score exceeds m by 12, so that the sums and O
// are rescaled (in registers and TMEM) only then.  Weights reach 2^12 at most,
// fp16's range keeps 2^-14 at full precision, and the sums are 32-bit.  The
// value scales s_t, which multiply the weights, are divided by a power of two
// (sref) that likewise moves only when a scale exceeds it four times.
//
// Bound.  A tile's path S -> softmax -> P -> O is a chain of latencies (TMEM
// loads, 128 x N exponentials, shared stores, barriers), so a CTA keeps four
// tiles in flight; what is left is that chain and instruction fetch (three unrolled
// loops, 85 % of the requests hit), with half of the issue slots used, a quarter
// of DRAM and an eighth of the tensor core.  Measured (this kernel alone, us): 16
// sequences of 8 heads, 32 rows a head, 16384 tokens of 3-bit keys and int8 values
// 148, about 2250 cycles a tile (0.38 of the rate at which HBM delivers the rows);
// with 128 rows 266 (5100 cycles a tile of four times the scores); one sequence of
// 130001 tokens, 20 rows a head 77.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvc_launch.cuh"
#include "kvc_sm100.cuh"
#include "kvc_tc.h"

namespace kvc {

using namespace sm100;

namespace {

constexpr int kTile = kTreeTile;
constexpr int kSoftWarps = 8;      // two softmax groups of four warps
constexpr int kGroupWarps = 8;     // warps of a decoder group
constexpr int kMaxNS = 4;          // row stages
// Side words (norms and scales of a tile) stay until the softmax has read them:
// a tile's stage is loaded once the decoders are done with the tile kMaxNS
// before, whose keys they decoded after the scores of the tile two before that
// were done, which waited for the softmax to have read S four tiles earlier (and
// the side words of up to two tiles more); so entries are never overwritten too
// soon, nor read too early.
constexpr int kSideRing = 16;
static_assert(kSideRing >= kMaxNS + 2 + 4, "side words overwritten before they are read");
constexpr int kSoftBar = 1, kDecBar = 3;  // named barriers: softmax groups 1, 2; decoder groups 3, 4
constexpr uint64_t kWaitNs = 2000000000ull;  // limit of the drains; the watchdog's is the layer's
constexpr uint32_t kTryNs = 20000;             // a try sleeps so long at most
constexpr float kSet = 6.f;        // a reference is set this far below the maximum (log2)
constexpr float kMove = 12.f;      // and moves when a score lies this far above it

// Roles by warp: softmax 0..7, decoders 8.., then producer, S and O issuers and
// watchdog (setmaxnreg works on whole groups of four).  Two decoder groups
// take alternate tiles; jobs of 128 rows, which decode a tile for twice the rows,
// give the second group's registers to the softmax.  The registers of the launch
// (65536 / threads, rounded down to 8) are split among the roles; ptxas is held
// to them by the launch bounds and the host checks that it used them all.
template <int NC, bool HALVES>
struct Roles {
  static constexpr int dec_groups = HALVES ? 1 : 2;
  static constexpr int prod = kSoftWarps + dec_groups * kGroupWarps;
  static constexpr int score = prod + 1, sum = prod + 2;
  static constexpr int threads = (prod + 4) * 32;
  static constexpr int launch_regs = 65536 / threads / 8 * 8;
  static constexpr int ctl_regs = HALVES ? 64 : NC <= 32 ? 56 : 48;
  static constexpr int dec_regs = HALVES ? 72 : NC <= 32 ? 56 : 48;
  static constexpr int soft_regs = HALVES ? 136 : NC <= 32 ? 112 : 128;
  static_assert(128 * (ctl_regs + 2 * dec_groups * dec_regs + 2 * soft_regs) <= threads * launch_regs,
                "register split exceeds the launch's registers");
};

struct Shape {
  int nc, halves, n;     // columns of a softmax thread; 2: the groups split the columns, 1: the tiles
  int K, KC;             // K of the score product, its 8-value chunks
  int mt;                // 128-channel tiles of O
  int a_cols, s_col, o_col, cols;  // TMEM layout
  int nv, ns;            // V buffers, row stages
  int krow, stage;       // bytes of a stage's key rows; of a stage
  int off_p, off_v, off_stage;  // shared-memory offsets
  int smem;
};

__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 bits from byte a of a 4-byte aligned buffer.
__device__ __forceinline__ uint2 bits_at(const unsigned char* base, int a) {
  const uint32_t* wp = reinterpret_cast<const uint32_t*>(base) + (a >> 2);
  const uint32_t w0 = wp[0], w1 = wp[1], w2 = wp[2];
  const uint32_t sh = 8 * (a & 3);
  return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
}

// Eight centred codes of width w as fp16: 0x6400 | c is 1024 + c exactly.
__device__ __forceinline__ uint4 centred_codes(uint2 b, int w) {
  const uint32_t sub = 0x64006400u | ((1u << (w - 1)) * 0x10001u);
  uint32_t o[4];
  if (w == 8) {
    o[0] = hsub2_bits(__byte_perm(b.x, 0x64646464u, 0x5140), sub);
    o[1] = hsub2_bits(__byte_perm(b.x, 0x64646464u, 0x5342), sub);
    o[2] = hsub2_bits(__byte_perm(b.y, 0x64646464u, 0x5140), sub);
    o[3] = hsub2_bits(__byte_perm(b.y, 0x64646464u, 0x5342), sub);
  } else {
    const uint32_t mask = (1u << w) - 1u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t x = b.x >> (2 * q * w);
      o[q] = hsub2_bits((x & mask) | ((x << (16 - w)) & (mask << 16)) | 0x64006400u, sub);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight int8 values as fp16: b + 128 in the low bits of 1024, less 1152.
__device__ __forceinline__ uint4 int8_values(uint2 b) {
  const uint32_t x = b.x ^ 0x80808080u, y = b.y ^ 0x80808080u;
  const uint32_t sub = 0x64806480u;  // 1152, twice
  return make_uint4(hsub2_bits(__byte_perm(x, 0x64646464u, 0x5140), sub),
                    hsub2_bits(__byte_perm(x, 0x64646464u, 0x5342), sub),
                    hsub2_bits(__byte_perm(y, 0x64646464u, 0x5140), sub),
                    hsub2_bits(__byte_perm(y, 0x64646464u, 0x5342), sub));
}

// Centroids of at most 8 levels as bytes: low bytes, then high bytes, of the
// fp16 values of levels 0..3 and 4..7.
struct Levels { uint32_t lo0, lo1, hi0, hi1; };

// The fp16 centroids of the eight W-bit codes in the low bits of x (what lies
// above them is ignored): the codes are spread to one per nibble (three steps
// of halving, each a shift and a select), which is the selector that a byte
// permute of the levels takes.
template <int W>
__device__ __forceinline__ uint4 centroids8(uint32_t x, const Levels& t) {
  auto select = [](uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); };
  x = select(x, x << (16 - 4 * W), 0x0000ffffu);
  x = select(x, x << (8 - 2 * W), 0x00ff00ffu);
  x = select(x, x << (4 - W), 0x0f0f0f0fu) & (0x11111111u * ((1u << W) - 1u));
  const uint32_t y = x >> 16;
  const uint32_t l0 = __byte_perm(t.lo0, t.lo1, x), h0 = __byte_perm(t.hi0, t.hi1, x);
  const uint32_t l1 = __byte_perm(t.lo0, t.lo1, y), h1 = __byte_perm(t.hi0, t.hi1, y);
  return make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362),
                    __byte_perm(l1, h1, 0x5140), __byte_perm(l1, h1, 0x7362));
}

// The int8 values of one token block (8 rows of NV chunks of 8 bytes) as fp16 V.
// Lane (octet, t8) takes token t8 and chunks (c0 + t8) mod NV: of eight lanes
// no two meet in a bank, neither reading (rows 8 NV bytes apart) nor writing
// (cores 128 bytes apart).
template <int NV>
__device__ __forceinline__ void int8_block(const unsigned char* row, unsigned char* dst, int c0) {
  // chunk (c0 + j) mod NV: two ascending runs, so that the addresses are a base
  // each and constants
  const int k = NV - (c0 & (NV - 1));  // chunks before the wrap
  const unsigned char* src = row + (c0 & (NV - 1)) * 8;
  unsigned char* to = dst + (c0 & (NV - 1)) * 128;
#pragma unroll
  for (int j = 0; j < NV / 2; j += 4) {
    uint2 b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = *reinterpret_cast<const uint2*>(src + (j + u) * 8 - (j + u >= k ? NV * 8 : 0));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(to + (j + u) * 128 - (j + u >= k ? NV * 128 : 0)) = int8_values(b[u]);
  }
}

// The 2 W bits at bit `off` of the words w as a byte offset into the pair table
// below (a field f at bit 7: f * 128), other bits undefined.
template <int W, int M>
__device__ __forceinline__ uint32_t pair_offset(const uint32_t (&w)[M], int off) {
  const int at = off - 7, i = at >> 5, sh = at & 31;
  if (at < 0) return w[0] << -at;
  return sh + 2 * W + 7 <= 32 || i + 1 >= M ? w[i] >> sh : __funnelshift_r(w[i], w[i + 1], sh);
}

// 64 consecutive codes (2 W words, 8-byte aligned) of a row of W-bit indices
// into 32 TMEM columns, two codes per lookup in a table that holds every pair of
// centroids once per lane (no bank conflicts): a shift, a select that also adds
// the lane (lane4: its number times 4), and a load per two codes.
template <int W>
__device__ __forceinline__ void codebook64(const unsigned char* src, const uint32_t* tab, uint32_t lane4,
                                           uint32_t a_tm) {
  uint32_t w[2 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint2 v = reinterpret_cast<const uint2*>(src)[i];
    w[2 * i] = v.x;
    w[2 * i + 1] = v.y;
  }
  constexpr uint32_t mask = ((1u << (2 * W)) - 1u) << 7;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t at = (pair_offset<W>(w, 2 * W * (16 * h + i)) & mask) | lane4;
      r[i] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const unsigned char*>(tab) + at);
    }
    tmem_st16(a_tm + h * 16, r);
  }
}

// Chunk c (8 packed positions) of basis beta: first byte | width << 16, 0 past the last.
__device__ uint32_t chunk_entry(const Params& p, int beta, int c) {
  int nch = 0;
  for (int s = 0; s < kMaxSeg; ++s) {
    const int32_t* e = p.seg + ((size_t)beta * kMaxSeg + s) * 4;
    if (!e[3]) break;
    const int n = (e[3] + 7) / 8;
    if (c < nch + n) return (uint32_t)(e[0] + e[1] * (c - nch)) | ((uint32_t)e[1] << 16);
    nch += n;
  }
  return 0u;
}

// MN-major operand without swizzle: core matrices of 8 (K) x 8 (MN) 16-bit
// elements, 128 contiguous bytes with MN contiguous; `k_stride` bytes between
// cores adjacent along K, `mn_stride` along M/N.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr, uint32_t k_stride, uint32_t mn_stride) {
  return desc_kmajor_noswizzle(saddr, k_stride, mn_stride);
}
constexpr uint32_t kTransposeAB = (1u << 15) | (1u << 16);  // both operands MN-major

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// tcgen05.mma and commit by the lane that has `lead`, predicated and not in a
// branch: the operands are then computed where the warp is converged and stay
// in uniform registers.
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

// Entries of the pair table that holds every pair of centroids once per lane:
// for codebooks of at most 8 levels at D = 128, else none, and the centroids come
// from byte permutes (16 sequences of 8 heads, 32 rows a head, 16384 tokens of 3-bit
// keys, the whole call: with the table 174 us, without 198; D = 64 without 146).
__host__ __device__ constexpr int pair_entries(int cb_bits, int D) {
  return cb_bits <= 3 && D == 128 ? 1 << (2 * cb_bits) : 0;
}

template <int REGS> __device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS> __device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// The larger of two, NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The warp's maximum, NaN where a lane has NaN.
__device__ __forceinline__ float warp_max_redux(float v) {
  float y;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
// Sums over the warp's lanes of 2 W columns: in each step a lane hands half of
// its columns to the lane that differs in bit O and keeps the other half; past
// one column the lanes just add.
template <int W, int O, int M>
__device__ __forceinline__ void sum_lanes(float (&v)[M], int lane) {
  if constexpr (O >= 1) {
    if constexpr (W >= 1) {
      const bool hi = lane & O;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float keep = hi ? v[i + W] : v[i], give = hi ? v[i] : v[i + W];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
    }
    sum_lanes<W / 2, O / 2>(v, lane);
  }
}

// A CTA's run of tiles, cut at the jobs' ends.  Divisions by tiles and row tiles
// are done once, for the run's first tile; the next segment starts the next job.
struct Segment {
  int job, slot, r0, nr, b;
  int tile0, tile1;  // tiles of the job (hidden context skipped)
};
struct Walk {
  int64_t left;      // tiles of the run not yet walked
  int job, slot, jt; // next segment's job: its slot and row tile
  int a;             // and its first tile
  __device__ explicit Walk(const TreeArgs& t) {
    const int64_t at = t.total * blockIdx.x / t.grid;
    left = t.total * (blockIdx.x + 1) / t.grid - at;
    job = (int)(at / t.tps);
    a = (int)(at - job * t.tps);
    slot = job / t.row_tiles;
    jt = job - slot * t.row_tiles;
  }
  __device__ bool next(const TreeArgs& t, int H, Segment& g) {
    if (left <= 0) return false;
    const int z = (int)min(t.tps, a + left);
    left -= z - a;
    g.job = job;
    g.slot = slot;
    g.r0 = jt * t.rt;
    g.nr = min(t.rt, t.rows - g.r0);
    g.b = slot / H;
    g.tile0 = a;
    g.tile1 = z;
    if (t.first)  // tiles of hidden context only
      g.tile0 = min(z, max(a, (int)(min((int64_t)max(t.first[g.b], 0), t.ctx) / kTile)));
    ++job;
    a = 0;
    if (++jt == t.row_tiles) {
      jt = 0;
      ++slot;
    }
    return true;
  }
};

// A group's segment and place in the run, kept in shared memory so that they
// take no registers in its loop; one thread of the group walks.
struct Place {
  Walk w;
  Segment g;
  int more;            // 0: the run is at its end
  // softmax
  int plain0, plain1;  // tiles that hold visible context alone
  int first;
  const uint32_t* mask;  // per draft, which drafts see it
  float fold;          // codebook keys: their common factor, else 1
  int Pk, Pv;          // decoders: row bytes
  __device__ void next(const TreeArgs& t, int H) { more = w.next(t, H, g); }
};

// Position in a ring of n buffers; next() moves on one use.
struct Ring {
  int n, slot;
  uint32_t phase;
  __device__ explicit Ring(int n_) : n(n_), slot(0), phase(0u) {}
  __device__ void next() {
    if (++slot == n) { slot = 0; phase ^= 1u; }
  }
};

// Wait for a phase, or until the watchdog has given up.  From then on every wait
// returns after one failed try, so that all roles walk to their ends and the
// named barriers stay matched; the results are undefined and the error word says
// so.  (The waits stand in every role's code and on the tiles' path: with a clock
// in each the serving batch took 180 us to 190 in place of 176.)
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  while (!mbar_try_wait_sleep(bar, parity, kTryNs))
    if (*abort_flag) return;
}

template <int KMODE, int VMODE, int NC, bool HALVES>
__global__ void __launch_bounds__(Roles<NC, HALVES>::threads, 1)
    tree_tc_kernel(const Params kp, const Params vp, const TreeArgs t, const Shape z) {
  using R = Roles<NC, HALVES>;
  constexpr bool VU = VMODE == KVC_MODE_UNIFORM;
  constexpr int N = HALVES ? 2 * NC : NC;  // columns
  constexpr int CH = NC < 32 ? NC : 32;    // columns handled at a time
  constexpr int NCH = NC / CH;
  constexpr int DG = R::dec_groups;
  constexpr int SB = HALVES ? 2 : 4;       // S buffers: two per tile that a softmax group holds
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t row_full[kMaxNS], row_empty[kMaxNS], a_full[2], a_empty[2], v_full[2],
      v_empty[2], s_full[SB], s_empty[SB], p_full[2], p_empty[2], side_full[kSideRing], w_full, w_empty, done_bar;
  __shared__ uint32_t kch[DG][32], vch[DG][32];  // chunk tables of the decoder groups
  // per softmax group and column: offset of the score (c1 - m), m, rescale
  // factor, seen a token; the warps' partial results
  __shared__ __align__(16) float cneg[2][NC];
  __shared__ __align__(16) float corr[2][NC], red[2][4][NC];
  __shared__ __align__(16) float wscale[2][NC];
  __shared__ float mref[2][NC];
  __shared__ int seen[2][NC];  // 0: no token, 1: weights summed, 2: only scores of -inf
  __shared__ __align__(16) unsigned char place_s[(2 + DG) * sizeof(Place)];  // softmax groups, decoder groups
  Place* place = reinterpret_cast<Place*>(place_s);
  __shared__ __align__(16) unsigned short side_s[kSideRing][2][kTile];  // norms, scales
  __shared__ uint32_t tab[KMODE == KVC_MODE_CODEBOOK ? 64 * 32 : 1];  // codebook tables
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag, tiles_done;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* Ws = smem;  // two pieces [N x K] fp16, K-major cores
  unsigned char* Ps = smem + z.off_p;
  unsigned char* Vs = smem + z.off_v;
  unsigned char* Rs = smem + z.off_stage;
  const int w_piece = N * z.K * 2;
  constexpr int p_bytes = kTile * N * 2;  // P: one buffer per group, or one of both halves
  const int v_bytes = z.mt * kTile * 256;

  if (warp == R::score) tmem_alloc(&tmem_base, z.cols);
  if (tid == 0) {
    for (int i = 0; i < z.ns; ++i) { mbar_init(&row_full[i], 1); mbar_init(&row_empty[i], kGroupWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], kGroupWarps);
      mbar_init(&a_empty[i], 1);
      mbar_init(&v_full[i], kGroupWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_empty[i], 1);
    }
    for (int i = 0; i < SB; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], HALVES ? 8 : 4); }
    for (int i = 0; i < kSideRing; ++i) mbar_init(&side_full[i], 1);
    mbar_init(&w_full, 1);
    mbar_init(&w_empty, 1);
    mbar_init(&done_bar, 2);
    fence_mbar_init();
    abort_flag = tiles_done = 0;
  }
  if (tid < 2 + DG) place[tid].w = Walk(t);
  if (KMODE == KVC_MODE_CODEBOOK) {  // pairs of 16 levels, 256 levels, or pairs once per lane
    const int wb = kp.cb_bits, lm = (1 << wb) - 1, n = pair_entries(wb, kp.D) * 32;
    auto half_of = [&](int c) {
      return (uint32_t)__half_as_ushort(__float2half_rn(kp.codebook[c] * t.cb_mul));
    };
    if (wb >= 4) {
      for (int j = tid; j < 256; j += R::threads)
        tab[j] = wb == 4 ? half_of(j & 15) | (half_of(j >> 4) << 16) : half_of(j);
    } else {
      for (int j = tid; j < n; j += R::threads)
        tab[j] = half_of((j >> 5) & lm) | (half_of(j >> (5 + wb)) << 16);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  Walk walk = place[0].w;  // (the MMA warps and the producer walk on their own)
  __syncthreads();
  grid_dependency_wait();  // the key weights come from the launch before

  if (warp >= R::prod) {
    regs_dec<R::ctl_regs>();
    if (warp == R::prod && lane == 0) {
      // ---------------------------------------------------------- producer
      Segment g;
      Ring rr(z.ns);
      int issued = 0, segs = 0;
      while (walk.next(t, kp.H, g)) {
        if (g.tile0 == g.tile1) continue;
        // the job's key weights, once the last segment's scores are done
        if (segs) wait_or_abort(&w_empty, (segs - 1) & 1, &abort_flag);
        if (abort_flag) break;
        mbar_arrive_expect_tx(&w_full, 2 * w_piece);
        bulk_load(Ws, t.w16 + (size_t)g.job * 2 * N * z.K, 2 * w_piece, &w_full);
        ++segs;
        const int Pk = kp.P[kp.basis_of[g.slot]];
        const int Pv = VU ? vp.P[vp.basis_of[g.slot]] : vp.D;
        const unsigned char* ks = kp.store + kp.pay_off[g.slot];
        const unsigned char* vs = vp.store + vp.pay_off[g.slot];
        const unsigned char* kn = kp.store + kp.side_off[g.slot];
        const unsigned char* vsc = vp.store + vp.side_off[g.slot];
        for (int tile = g.tile0; tile < g.tile1; ++tile, ++issued, rr.next()) {
          if (issued >= z.ns) wait_or_abort(&row_empty[rr.slot], rr.phase ^ 1u, &abort_flag);
          if (abort_flag) break;
          const int64_t t0 = (int64_t)tile * kTile;
          const int n = (int)min((int64_t)kTile, t.S - t0);
          const uint32_t kb = (uint32_t)((n * Pk + 15) & ~15), vb = (uint32_t)((n * Pv + 15) & ~15);
          unsigned char* st = Rs + rr.slot * z.stage;
          mbar_arrive_expect_tx(&row_full[rr.slot], kb + vb);
          if (kb) bulk_load(st, ks + t0 * Pk, kb, &row_full[rr.slot]);
          if (vb) bulk_load(st + z.krow, vs + t0 * Pv, vb, &row_full[rr.slot]);
          const int sd = issued & (kSideRing - 1);
          const uint32_t sb = (uint32_t)((2 * n + 15) & ~15);
          mbar_arrive_expect_tx(&side_full[sd], (KMODE == KVC_MODE_CODEBOOK ? sb : 0) + (VU ? 0 : sb));
          if (KMODE == KVC_MODE_CODEBOOK) bulk_load(side_s[sd][0], kn + t0 * 2, sb, &side_full[sd]);
          if (!VU) bulk_load(side_s[sd][1], vsc + t0 * 2, sb, &side_full[sd]);
        }
        if (abort_flag) break;
      }
      // copies still in flight (after a time-out) land before the CTA exits
      if (segs) mbar_wait_bounded(&w_full, (segs - 1) & 1, kWaitNs);
      for (int j = max(0, issued - z.ns); j < issued; ++j)
        mbar_wait_bounded(&row_full[j % z.ns], (j / z.ns) & 1, kWaitNs);
      for (int j = max(0, issued - kSideRing); j < issued; ++j)
        mbar_wait_bounded(&side_full[j & (kSideRing - 1)], (j / kSideRing) & 1, kWaitNs);
    } else if (warp == R::score) {
      // ---------------------------------------------------------- S = A W^T
      // The whole warp walks and waits, one elected lane issues; the two products
      // have a warp each.  (One lane walking and issuing both took 160 cycles per
      // MMA, where the tensor core takes 27 to 64.)
      Segment g;
      const uint32_t lead = elect_one();
      constexpr uint32_t id = idesc_f16(kTile, N, 0);
      const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
      const uint64_t w_desc = desc_kmajor_noswizzle(smem_u32(Ws), 128, (uint32_t)z.KC * 128);
      int it = 0, segs = 0;
      while (walk.next(t, kp.H, g)) {
        const int tiles = __shfl_sync(0xffffffffu, g.tile1 - g.tile0, 0);
        if (tiles == 0) continue;
        wait_or_abort(&w_full, segs & 1, &abort_flag);
        ++segs;
        for (int i = 0; i < tiles; ++i, ++it) {
          const int a = it & 1, s = it % SB;
          if (it >= SB) wait_or_abort(&s_empty[s], (it / SB - 1) & 1, &abort_flag);
          wait_or_abort(&a_full[a], (it >> 1) & 1, &abort_flag);
          __syncwarp();
          tc_fence_after();
          const uint32_t a0 = tmu + a * z.a_cols, d0 = tmu + z.s_col + s * N;
          // both pieces of W; 16 fp16 of K are 8 TMEM columns of A
          for (int p = 0; p < 2; ++p) {
            const uint64_t wd = w_desc + ((p * w_piece) >> 4);
#pragma unroll 4
            for (int ks = 0; ks < z.K / 16; ++ks)
              mma_tmem_a(lead, d0, a0 + ks * 8, wd + ks * 16, id, p + ks > 0);
          }
          commit_if(lead, &s_full[s]);
          commit_if(lead, &a_empty[a]);
          if (i + 1 == tiles) commit_if(lead, &w_empty);
        }
      }
      if (lead) {
        umma_commit(&done_bar);  // TMEM is released only after every MMA has finished
        mbar_wait_bounded(&done_bar, 0, kWaitNs);
      }
      __syncwarp();
    } else if (warp == R::sum) {
      // ---------------------------------------------------------- O += V^T P
      // One product per tile, or, where the groups split the columns, one per
      // group as its weights arrive.
      Segment g;
      const uint32_t lead = elect_one();
      constexpr uint32_t id = idesc_f16(kTile, NC, 0) | kTransposeAB;
      constexpr uint32_t p_k = N * 16;  // bytes between P's cores along the tokens
      const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
      const uint32_t v_k = (uint32_t)z.mt * 2048;
      const uint64_t v_desc = desc_mnmajor(smem_u32(Vs), v_k, 128);
      const uint64_t p_desc = desc_mnmajor(smem_u32(Ps), p_k, 128);
      const uint64_t v_step = (2 * v_k) >> 4;
      constexpr uint64_t p_step = (2 * p_k) >> 4;
      int it = 0;
      Ring rv(z.nv);
      while (walk.next(t, kp.H, g)) {
        const int tiles = __shfl_sync(0xffffffffu, g.tile1 - g.tile0, 0);
        for (int i = 0; i < tiles; ++i, ++it, rv.next()) {
          wait_or_abort(&v_full[rv.slot], rv.phase, &abort_flag);
#pragma unroll
          for (int h = 0; h < (HALVES ? 2 : 1); ++h) {
            const int wg = HALVES ? h : it & 1;
            wait_or_abort(&p_full[wg], (HALVES ? it : it >> 1) & 1, &abort_flag);
            __syncwarp();
            tc_fence_after();
            // the group's first tile of the segment overwrites its O
            const uint32_t add = i >= (HALVES ? 1 : 2);
            for (int m = 0; m < z.mt; ++m) {
              const uint32_t o = tmu + z.o_col + (HALVES ? m * N + h * NC : (wg * z.mt + m) * N);
              const uint64_t vd = v_desc + ((rv.slot * v_bytes + m * 2048) >> 4);
              const uint64_t pd = p_desc + ((HALVES ? h * (NC / 8 * 128) : wg * p_bytes) >> 4);
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                mma_smem(lead, o, vd + ks * v_step, pd + ks * p_step, id, ks ? 1u : add);
            }
            commit_if(lead, &p_empty[wg]);
            if (!HALVES || h == 1) commit_if(lead, &v_empty[rv.slot]);
          }
          tiles_done = it + 1;  // (every lane the same)
        }
      }
      if (lead) {
        umma_commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, kWaitNs);
      }
      __syncwarp();
    } else if (lane == 0) {
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
    regs_dec<R::dec_regs>();
    const int grp = (warp - kSoftWarps) / kGroupWarps;
    const int dtid = tid - (kSoftWarps + grp * kGroupWarps) * 32;
    const int tt = dtid & (kTile - 1), half = dtid >> 7;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // values: eight lanes take eight tokens of one block, each another chunk of
    // the row, so that neither the reads (rows 128 bytes apart) nor the writes
    // (cores 128 bytes apart) meet in a bank
    const int octet = lane >> 3, t8 = lane & 7;
    const int vblk = (dtid >> 5) * 2 + (octet >> 1);
    Levels levels{};
    if (KMODE == KVC_MODE_CODEBOOK && kp.cb_bits <= 3 && kp.D != 128) {
      uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t h =
            j < kp.cb_levels ? __half_as_ushort(__float2half_rn(kp.codebook[j] * t.cb_mul)) : 0u;
        lo[j >> 2] |= (h & 0xffu) << (8 * (j & 3));
        hi[j >> 2] |= (h >> 8) << (8 * (j & 3));
      }
      levels = Levels{lo[0], lo[1], hi[0], hi[1]};
    }
    Ring rr(z.ns), rv(z.nv);
    int it = 0;
    Place& pl = place[2 + grp];
    for (;;) {
      named_bar_sync(kDecBar + grp, kGroupWarps * 32);  // the last segment's tables have been read
      if (dtid == 0) {
        pl.next(t, kp.H);
        if (pl.more) {
          pl.Pk = kp.P[kp.basis_of[pl.g.slot]];
          pl.Pv = VU ? vp.P[vp.basis_of[pl.g.slot]] : vp.D;
        }
      }
      named_bar_sync(kDecBar + grp, kGroupWarps * 32);
      if (!pl.more) break;
      if (dtid < 32) kch[grp][dtid] = chunk_entry(kp, kp.basis_of[pl.g.slot], dtid);
      else if (VU && dtid < 64) vch[grp][dtid - 32] = chunk_entry(vp, vp.basis_of[pl.g.slot], dtid - 32);
      named_bar_sync(kDecBar + grp, kGroupWarps * 32);
      const int Pk = pl.Pk, Pv = pl.Pv;
      int nv = VU ? 0 : vp.D / 8;  // chunks of a value row
      if (VU)
        while (nv < 32 && vch[grp][nv]) ++nv;
      const int vhalf = (nv + 1) / 2;
      const int tile1 = pl.g.tile1;
      for (int tile = pl.g.tile0; tile < tile1; ++tile, ++it, rr.next(), rv.next()) {
        if (DG == 2 && (it & 1) != grp) continue;
        const int a = it & 1;
        wait_or_abort(&row_full[rr.slot], rr.phase, &abort_flag);
        if (it >= 2) wait_or_abort(&a_empty[a], ((it >> 1) - 1) & 1, &abort_flag);
        __syncwarp();
        const unsigned char* st = Rs + rr.slot * z.stage;
        const uint32_t a_tm = tm + lane_base + a * z.a_cols;
        if (KMODE == KVC_MODE_CODEBOOK && kp.cb_bits <= 3 && kp.D == 128) {
          const int W = kp.cb_bits;
          const unsigned char* src = st + tt * Pk + half * 8 * W;
          if (W == 3) codebook64<3>(src, tab, 4 * lane, a_tm + half * 32);
          else if (W == 2) codebook64<2>(src, tab, 4 * lane, a_tm + half * 32);
          else codebook64<1>(src, tab, 4 * lane, a_tm + half * 32);
        } else {
          for (int c = half; c < z.KC; c += 2) {
            const uint32_t ent = kch[grp][c];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (ent) {
              const int w = (int)(ent >> 16);
              const uint2 b = bits_at(st, tt * Pk + (int)(ent & 0xffffu));
              if (KMODE == KVC_MODE_UNIFORM) {
                v = centred_codes(b, w);
              } else if (w <= 3) {
                v = w == 3 ? centroids8<3>(b.x, levels) : w == 2 ? centroids8<2>(b.x, levels)
                                                                 : centroids8<1>(b.x, levels);
              } else {
                const int pair = w == 4;
                auto two = [&](uint32_t x) {
                  return pair ? tab[x & 255u] : tab[x & 255u] | (tab[(x >> 8) & 255u] << 16);
                };
                v = pair ? make_uint4(two(b.x), two(b.x >> 8), two(b.x >> 16), two(b.x >> 24))
                         : make_uint4(two(b.x), two(b.x >> 16), two(b.y), two(b.y >> 16));
              }
            }
            tmem_st4(a_tm + c * 4, v);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[a]);
        if (it >= z.nv) wait_or_abort(&v_empty[rv.slot], rv.phase ^ 1u, &abort_flag);
        __syncwarp();
        {
          const unsigned char* raw = st + z.krow;
          const int tok = vblk * 8 + t8;
          unsigned char* dst = Vs + rv.slot * v_bytes + vblk * z.mt * 2048 + t8 * 16;
          const int c0 = (octet & 1) * vhalf;
          if (!VU && nv == 16) {
            int8_block<16>(raw + tok * 128, dst, c0 + t8);
          } else if (!VU && nv == 8) {
            int8_block<8>(raw + tok * 64, dst, c0 + t8);
          } else {
            const int cend = min(nv, c0 + vhalf);
            for (int j = c0; j < cend; ++j) {
              int c = j + t8;
              while (c >= nv) c -= nv;
              uint4 v;
              if (VU) {
                const uint32_t ent = vch[grp][c];
                v = centred_codes(bits_at(raw, tok * Pv + (int)(ent & 0xffffu)), (int)(ent >> 16));
              } else {
                v = int8_values(*reinterpret_cast<const uint2*>(raw + tok * Pv + c * 8));
              }
              *reinterpret_cast<uint4*>(dst + c * 128) = v;
            }
          }
        }
        fence_proxy_async_smem();  // V is read by the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[rv.slot]);
          mbar_arrive(&row_empty[rr.slot]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<R::soft_regs>();
    const int wg = warp >> 2, quarter = warp & 3, ltid = tid & 127, bar = kSoftBar + wg;
    const int lt = quarter * 32 + lane;  // this lane's token of a tile
    const int col0 = HALVES ? wg * NC : 0;  // the group's first column
    constexpr int kStep = HALVES ? 1 : 2;   // tiles between two of the group's
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_tm = tm + lane_off + z.o_col + (HALVES ? col0 : wg * z.mt * N);
    float* cn = cneg[wg];
    unsigned char* pst = Ps + (HALVES ? 0 : wg * p_bytes) + (lt >> 3) * (N * 16) + col0 * 16 + (lane & 7) * 16;
    int it = 0;  // tiles of the run before the segment
    Place& pl = place[wg];
    for (;;) {
      named_bar_sync(bar, 128);  // the last segment's state has been read
      if (ltid == 0) {
        pl.next(t, kp.H);
        if (pl.more) {
          const int first = t.first ? max(t.first[pl.g.b], 0) : 0;
          pl.first = first;
          pl.plain0 = (int)min(t.tps, ((int64_t)first + kTile - 1) / kTile);
          pl.plain1 = (int)(t.ctx / kTile);
          pl.mask = t.mask ? t.mask_bits + (t.mask_sb ? (size_t)pl.g.b : 0) * t.N * ((t.N + 31) / 32) : nullptr;
        }
      }
      named_bar_sync(bar, 128);
      if (!pl.more) break;
      const int ncol = max(0, min(NC, pl.g.nr - col0));  // rows of this group
      // the rows' factors (0: any will do): one for all goes into the token's norm
      float ws = 0.f, common = 1.f;
      if (ltid < NC) {
        const size_t row = (size_t)pl.g.slot * t.prow + pl.g.r0 + col0 + ltid;
        cn[ltid] = t.c1[row];
        if (ltid < ncol) ws = t.wscale[row];
        mref[wg][ltid] = 0.f;
        seen[wg][ltid] = ltid >= ncol;
      }
      if (KMODE == KVC_MODE_CODEBOOK) {
        const float m = warp_max_redux(ws);
        if (lane == 0) red[wg][quarter][0] = m;
        named_bar_sync(bar, 128);
        const float most = fmaxf(fmaxf(red[wg][0][0], red[wg][1][0]), fmaxf(red[wg][2][0], red[wg][3][0]));
        if (most != 0.f) common = most;
      }
      // wscale is that of a row in jobs of several factors, 1 elsewhere: of uniform
      // keys, whose common factor is 1, known before the vote and ordered by it
      if (KMODE == KVC_MODE_UNIFORM && ltid < NC) wscale[wg][ltid] = ws == 0.f ? 1.f : ws;
      const bool scaled = named_bar_or(bar, 128, ws != 0.f && ws != common);
      if (KMODE == KVC_MODE_CODEBOOK) {
        if (ltid < NC) wscale[wg][ltid] = !scaled ? 1.f : ws == 0.f ? common : ws;
        if (ltid == 0) pl.fold = scaled ? 1.f : common;
        named_bar_sync(bar, 128);
      }
      float2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = make_float2(0.f, 0.f);
      float sref = VU ? 1.f : 0.f, inv_sref = VU ? 1.f : 0.f;
      // the group's tiles of the segment, and its tiles of the run before them
      const int tile_first = pl.g.tile0 + (HALVES ? 0 : (it ^ wg) & 1);
      int j = HALVES ? it : (it + 1 - wg) >> 1;
      // tiles [fast0, fast1) hold visible context alone, of rows that have seen a
      // token already
      int fast0 = pl.plain0, fast1 = 0;
      const int tile1 = pl.g.tile1;
      // this lane's norm and scale, read one tile ahead
      unsigned short nt_next = 0, st_next = 0;
      auto read_side = [&](int gt) {
        const int sd = gt & (kSideRing - 1);
        wait_or_abort(&side_full[sd], (gt / kSideRing) & 1, &abort_flag);
        if (KMODE == KVC_MODE_CODEBOOK) nt_next = side_s[sd][0][lt];
        if (!VU) st_next = side_s[sd][1][lt];
      };
      if (tile_first < tile1) read_side(HALVES ? j : 2 * j + wg);
      for (int tile = tile_first; tile < tile1; tile += kStep, ++j) {
        const int gt = HALVES ? j : 2 * j + wg;        // the tile's number in the run
        const int s = gt % SB;                         // S buffer, and its phase
        const uint32_t s_par = (gt / SB) & 1;
        const uint32_t s_tm = tm + lane_off + z.s_col + s * N + col0;
        float nt = KMODE == KVC_MODE_CODEBOOK ? __half2float(__ushort_as_half(nt_next)) * pl.fold : 1.f;
        const float st = VU ? 1.f : __half2float(__ushort_as_half(st_next));
        if (!VU && st != st) nt = st;  // a scale of NaN: the weights of those who see it
        wait_or_abort(&s_full[s], s_par, &abort_flag);
        __syncwarp();
        tc_fence_after();
        auto scores = [&](int ch, float2 (&x)[CH / 2]) {  // S nt + c1 - m, S times the rows' factors
          uint32_t r[CH];
          tmem_ld_n<CH>(s_tm + ch * CH, r);
          tmem_wait_ld();
          if (scaled) {  // a factor per row
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
              const float4 f = reinterpret_cast<const float4*>(wscale[wg] + ch * CH)[i];
              const float2 a = __fmul2_rn(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])),
                                          make_float2(f.x, f.y));
              const float2 b = __fmul2_rn(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                          make_float2(f.z, f.w));
              r[4 * i] = __float_as_uint(a.x);
              r[4 * i + 1] = __float_as_uint(a.y);
              r[4 * i + 2] = __float_as_uint(b.x);
              r[4 * i + 3] = __float_as_uint(b.y);
            }
          }
          const float2 nt2 = make_float2(nt, nt);
#pragma unroll
          for (int i = 0; i < CH / 4; ++i) {
            const float4 c = reinterpret_cast<const float4*>(cn + ch * CH)[i];
            x[2 * i] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), nt2,
                                  make_float2(c.x, c.y));
            x[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                      nt2, make_float2(c.z, c.w));
          }
        };
        // Tiles of visible context alone only check that no score and no scale is
        // too far above its reference.  The others, and those that fail, first
        // take the general path below, once.
        bool general = tile < fast0 || tile >= fast1;
        uint64_t vis = ~0ull;  // which of the group's rows see this lane's token
        float2 x[CH / 2];
        for (;;) {
          if (general) {
            // Loops are kept rolled: this code runs about twice per job, and its
            // instructions come from L2.
            if (tile < pl.plain0 || tile >= pl.plain1) {
              const int64_t tok = (int64_t)tile * kTile + lt, draft = tok - t.ctx;
              if (draft < 0) {
                vis = tok >= pl.first ? ~0ull : 0ull;
              } else {
                vis = 0ull;
                if (draft < t.N) {
                  // the drafts n that see this one: a bit each, repeated for
                  // every query head of the group's columns
                  const int nc = min(NC, pl.g.nr - col0), words = (t.N + 31) / 32;
                  const uint32_t* bits = pl.mask ? pl.mask + draft * words : nullptr;
                  const uint32_t only = bits && words == 1 ? bits[0] : 0u;
                  int n = (pl.g.r0 + col0) % t.N;
#pragma unroll 1
                  for (int c = 0; c < nc;) {
                    const int take = min(min(t.N - n, nc - c), 32), w = n >> 5, sh = n & 31;
                    uint32_t v;
                    if (!bits) v = draft <= n ? ~0u : draft - n < 32 ? ~0u << (draft - n) : 0u;
                    else if (words == 1) v = only >> sh;
                    else v = __funnelshift_r(bits[w], w + 1 < words ? bits[w + 1] : 0u, sh);
                    if (take < 32) v &= (1u << take) - 1u;
                    vis |= (uint64_t)v << c;
                    c += take;
                    if ((n += take) == t.N) n = 0;
                  }
                }
              }
            }
            float ratio = 1.f;
            if (!VU) {  // the value scales' reference: the next power of two
              const bool up = vis != 0ull && st > 4.f * sref && st <= 65504.f;
              const float m = warp_max_redux(up ? st : 0.f);
              if (lane == 0) red[wg][quarter][0] = m;
              named_bar_sync(bar, 128);
              const float most = fmaxf(fmaxf(red[wg][0][0], red[wg][1][0]), fmaxf(red[wg][2][0], red[wg][3][0]));
              if (most > 0.f) {
                const float to = __int_as_float((__float_as_int(most) & 0x7f800000) + 0x00800000);
                ratio = sref / to;
                sref = to;
                inv_sref = 1.f / to;
              }
              named_bar_sync(bar, 128);
            }
            // the tile's largest score of every column
#pragma unroll 1
            for (int c = 0; c < NC; c += 16) {
              uint32_t r[16];
              tmem_ld16(s_tm + c, r);
              tmem_wait_ld();
              const uint32_t v = (uint32_t)(vis >> c);
              float m[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float f = fmaf(__uint_as_float(r[i]) * wscale[wg][c + i], nt, cn[c + i]);
                m[i] = warp_max_redux(v >> i & 1u ? max_nan(f, kTreeLowest) : -INFINITY);
              }
              if (lane == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  reinterpret_cast<float4*>(&red[wg][quarter][c])[i] =
                      make_float4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
            }
            named_bar_sync(bar, 128);
            bool blind = false;
            if (ltid < NC) {
              const float m = max_nan(max_nan(red[wg][0][ltid], red[wg][1][ltid]),
                                      max_nan(red[wg][2][ltid], red[wg][3][ltid]));
              float d = 0.f, f = 1.f;
              if (m != -INFINITY) {  // (a row with a score of NaN counts as seen and stays NaN)
                if (seen[wg][ltid] != 1) {  // nothing summed yet
                  if (m != kTreeLowest) {
                    d = m - kSet;
                    f = 0.f;
                  }
                  seen[wg][ltid] = m != kTreeLowest ? 1 : 2;
                } else if (m > kMove) {
                  d = m - kSet;
                  f = ex2(-d);
                } else if (m != m) {
                  d = m;
                }
              }
              mref[wg][ltid] += d;
              cn[ltid] -= d;
              corr[wg][ltid] = f;
              blind = seen[wg][ltid] != 1;
            }
            // rows that saw nothing yet keep every tile on this path
            if (!named_bar_or(bar, 128, blind)) fast1 = pl.plain1;
#pragma unroll
            for (int i = 0; i < NC / 4; ++i) {
              const float4 f = reinterpret_cast<const float4*>(corr[wg])[i];
              l[2 * i] = __fmul2_rn(l[2 * i], make_float2(f.x, f.y));
              l[2 * i + 1] = __fmul2_rn(l[2 * i + 1], make_float2(f.z, f.w));
            }
            if (tile != tile_first) {  // O holds sums: rescale it once the last product is done
              wait_or_abort(&p_empty[wg], (j - 1) & 1, &abort_flag);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int m = 0; m < z.mt; ++m)
#pragma unroll 1
                for (int c = 0; c < NC; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(o_tm + m * N + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * (corr[wg][c + i] * ratio));
                  tmem_st16(o_tm + m * N + c, o);
                }
              tmem_wait_st();
            }
            named_bar_sync(bar, 128);  // corr and red have been read
          }
          float mx = -INFINITY;
#pragma unroll
          for (int ch = NCH - 1; ch >= 0; --ch) {  // ends with the first chunk's scores in x
            scores(ch, x);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) mx = max3(mx, x[i].x, x[i].y);
          }
          if (general || !named_bar_or(bar, 128, mx > kMove || (!VU && st > 4.f * sref))) break;
          general = true;
        }
        if (j > 0) wait_or_abort(&p_empty[wg], (j - 1) & 1, &abort_flag);  // P has been read
        __syncwarp();
        if (tile + kStep < tile1) read_side(gt + kStep);
        // a hidden token's scale may be anything: its weights are 0 and stay 0
        // under any finite factor
        const float su = fmaxf(fminf(st * inv_sref, 3e38f), -3e38f);
        const float2 su2 = make_float2(su, su);
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          if (ch) scores(ch, x);
          if (ch == NCH - 1) {  // S has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[s]);
          }
          if (general) {
            const uint32_t v = (uint32_t)(vis >> (ch * CH));
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              if (!(v >> (2 * i) & 1u)) x[i].x = -INFINITY;
              if (!(v >> (2 * i + 1) & 1u)) x[i].y = -INFINITY;
            }
          }
#pragma unroll
          for (int q = 0; q < CH / 8; ++q) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 4 * q + i;
              const float2 p = make_float2(ex2(x[e].x), ex2(x[e].y));
              l[ch * CH / 2 + e] = __fadd2_rn(l[ch * CH / 2 + e], p);
              const float2 u = VU ? p : __fmul2_rn(p, su2);
              h[i] = pack_half2(u.x, u.y);
            }
            *reinterpret_cast<uint4*>(pst + (ch * CH / 8 + q) * 128) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_smem();  // P is read by the tensor core
        tc_fence_before();         // and O, where it was rescaled
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg]);
      }
      // the partial: per row m, l and the weighted sums
      const bool any = tile_first < tile1;
      if (any) {
        wait_or_abort(&p_empty[wg], (j - 1) & 1, &abort_flag);
        __syncwarp();
        tc_fence_after();
      }
      it += tile1 - pl.g.tile0;
      // sums of the weights over the warp's lanes
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += CH) {
        float v[CH];
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          v[2 * i] = l[c0 / 2 + i].x;
          v[2 * i + 1] = l[c0 / 2 + i].y;
        }
        sum_lanes<CH / 2, 16>(v, lane);
        // lane bits 16, 8, .. chose the column's high bits
        const int col = CH == 32 ? lane : lane >> 1;
        if (CH == 32 || !(lane & 1)) red[wg][quarter][c0 + col] = v[0];
      }
      named_bar_sync(bar, 128);
      const size_t prow = (HALVES ? ((size_t)pl.g.job + blockIdx.x) : 2 * ((size_t)pl.g.job + blockIdx.x) + wg) * t.rt + col0;
      // weighted sums by channel, a partial's rows together: [Dvp][rt]
      float* part = t.part + (prow - col0) * t.Dvp + col0;
      if (ltid < ncol) {
        const int sn = seen[wg][ltid];
        t.ml[prow + ltid] = make_float2(
            sn == 1 ? mref[wg][ltid] : sn ? kTreeLowest : -INFINITY,
            sn == 1 ? (red[wg][0][ltid] + red[wg][1][ltid]) + (red[wg][2][ltid] + red[wg][3][ltid]) : 0.f);
      }
      for (int m = 0; m < z.mt; ++m) {
        const int d = m * 128 + lt;
        float4* to = reinterpret_cast<float4*>(part + (size_t)d * t.rt);
        for (int c = 0; c < NC; c += 16) {
          uint32_t o[16];
          if (any) {
            tmem_ld16(o_tm + m * N + c, o);
            tmem_wait_ld();
          }
          if (d < t.Dv) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              to[c / 4 + i] = any ? make_float4(__uint_as_float(o[4 * i]) * sref, __uint_as_float(o[4 * i + 1]) * sref,
                                                __uint_as_float(o[4 * i + 2]) * sref, __uint_as_float(o[4 * i + 3]) * sref)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
      tc_fence_before();  // the next segment's first product overwrites O
    }
  }
  __syncthreads();
  grid_dependents_launch();  // (at the start, the combine's blocks came in the way)
  if (abort_flag && tid == 0) atomicCAS(kp.err, 0, kErrTimeout);
  if (warp == R::score) {
    tc_fence_after();
    tmem_dealloc(tm, z.cols);
  }
}

using TcKernel = void (*)(const Params, const Params, const TreeArgs, const Shape);

template <int KMODE, int VMODE>
TcKernel kernel_for_shape(const Shape& z, int* threads, int* regs) {
  auto use = [&](auto roles) {
    *threads = decltype(roles)::threads;
    *regs = decltype(roles)::launch_regs;
  };
  if (z.halves == 2) {
    use(Roles<64, true>{});
    return tree_tc_kernel<KMODE, VMODE, 64, true>;
  }
  use(Roles<64, false>{});
  switch (z.nc) {
    case 16: return tree_tc_kernel<KMODE, VMODE, 16, false>;
    case 32: return tree_tc_kernel<KMODE, VMODE, 32, false>;
    default: return tree_tc_kernel<KMODE, VMODE, 64, false>;
  }
}

TcKernel kernel_for(int kmode, int vmode, const Shape& z, int* threads, int* regs) {
  if (kmode == KVC_MODE_UNIFORM)
    return vmode == KVC_MODE_UNIFORM
               ? kernel_for_shape<KVC_MODE_UNIFORM, KVC_MODE_UNIFORM>(z, threads, regs)
               : kernel_for_shape<KVC_MODE_UNIFORM, KVC_MODE_INT8>(z, threads, regs);
  return vmode == KVC_MODE_UNIFORM
             ? kernel_for_shape<KVC_MODE_CODEBOOK, KVC_MODE_UNIFORM>(z, threads, regs)
             : kernel_for_shape<KVC_MODE_CODEBOOK, KVC_MODE_INT8>(z, threads, regs);
}

// Layout for nc columns a softmax thread (halves = 2: 2 nc columns in all), or
// false when TMEM or shared memory does not hold it.
bool shape_for(const Params& kp, bool vu, const TreeArgs& t, int nc, int halves, Shape* out) {
  Shape z{};
  z.nc = nc;
  z.halves = halves;
  z.n = nc * halves;
  z.K = (t.NCk + 15) / 16 * 16;
  z.KC = z.K / 8;
  z.mt = (t.Dv + 127) / 128;
  z.a_cols = (z.K / 2 + 31) / 32 * 32;
  z.s_col = 2 * z.a_cols;
  z.o_col = z.s_col + (halves == 2 ? 2 : 4) * z.n;  // S buffers
  const int groups = halves == 2 ? 1 : 2;  // O and P: one of both halves, or one per group
  const int cols = z.o_col + groups * z.mt * z.n;
  if (cols > 512) return false;
  for (z.cols = 32; z.cols < cols; z.cols *= 2) {}
  auto up = [](int v) { return (v + 127) / 128 * 128; };
  z.krow = up(kTile * t.Pk_max + 16);
  z.stage = z.krow + up(kTile * t.Pv_max + (vu ? 16 : 0));
  z.off_p = 2 * z.n * z.K * 2;
  z.off_v = z.off_p + groups * z.n * kTile * 2;
  // two V buffers and four row stages, or what fits
  const int most = 227 * 1024 - 22 * 1024;  // the static arrays take up to 22 KB
  for (z.nv = 2; z.nv >= 1; --z.nv)
    for (z.ns = kMaxNS; z.ns >= 2; --z.ns) {
      z.off_stage = z.off_v + z.nv * z.mt * kTile * 256;
      z.smem = z.off_stage + z.ns * z.stage;
      if (z.smem <= most) {
        *out = z;
        return true;
      }
    }
  return false;
}

bool choose_shape(const Params& kp, const Params& vp, const TreeArgs& t, Shape* z) {
  // The fewest columns that hold all rows, else the most that fit: the softmax
  // works on all columns of a tile, empty ones too, and a tile is decoded once per
  // job.  Measured (us of the whole call): 32 rows 175 with 32 columns, 266 with
  // 64; 8 rows 15.6 with 16, 16.6 with 32, 19.5 with 64; 128 rows 304 in one job
  // of 128, 500 in two of 64.
  static const int kShapes[4][2] = {{16, 1}, {32, 1}, {64, 1}, {64, 2}};
  bool ok = false;
  for (const auto& s : kShapes) {
    Shape c;
    if (!shape_for(kp, vp.mode == KVC_MODE_UNIFORM, t, s[0], s[1], &c)) continue;
    *z = c;
    ok = true;
    if (c.n >= t.rows) break;
  }
  return ok;
}

}  // namespace

// The kernel for a shape, with its shared memory allowed; null where the compiler
// gave it other registers than the roles' split draws on (setmaxnreg would wait
// for ever with fewer): it is never launched then.
static TcKernel ready_kernel(const Params& kp, const Params& vp, const Shape& z, int* threads) {
  int regs = 0, has = 0;
  const TcKernel k = kernel_for(kp.mode, vp.mode, z, threads, &regs);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), z.smem, &has);
  return e == cudaSuccess && has == regs ? k : nullptr;
}

int tree_tc_rows(const Params& kp, const Params& vp, const TreeArgs& t, int* parts, int* K) {
  // Scores of two sums (residual sketches, outliers) take the CUDA-core kernel, and
  // layers for which there is no shape or no ready kernel.  All else goes to the
  // tensor cores at every size (us of the call, CUDA cores and here: 2 slots of 8
  // rows, 84 tokens 29 and 16; 15 slots of 21 rows, 1777 tokens 38 and 27; 64 slots of
  // 64 rows, 4096 tokens 274 and 57; 128 slots of 32 rows, 16384 tokens 5567 and 175).
  if (t.prod) return 0;
  if (vp.mode == KVC_MODE_INT8 && vp.D % 8) return 0;  // value rows are read 8 bytes at a time
  Shape z;
  int threads = 0;
  if (!choose_shape(kp, vp, t, &z) || !ready_kernel(kp, vp, z, &threads)) return 0;
  *parts = z.halves == 2 ? 1 : 2;
  *K = z.K;
  return z.n;
}

cudaError_t launch_tree_tc(const Params& kp, const Params& vp, const TreeArgs& t, cudaStream_t s,
                           int* nk) {
  Shape z;
  if (!choose_shape(kp, vp, t, &z)) return cudaErrorInvalidValue;
  int threads = 0;
  const TcKernel k = ready_kernel(kp, vp, z, &threads);
  if (!k) return cudaErrorLaunchOutOfResources;
  ++*nk;
  return launch_dependent(k, (unsigned)t.grid, threads, (size_t)z.smem, s, kp, vp, t, z);
}

}  // namespace kvc
