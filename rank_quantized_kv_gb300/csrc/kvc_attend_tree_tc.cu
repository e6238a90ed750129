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
//   decoders (8 warps)    key codes -> fp16 A in TMEM (lane = token); value
//                         codes -> fp16 V in shared memory;
//   two MMA warps         S = A W^T, and O += V^T P;
//   softmax (2 groups of 4 warps, each half of the rows' columns; lane = token)
//                         S -> P in fp16 in shared memory, sums of P in fp32.
//
// Precision.  Codes are exact in fp16 (centred codes up to 128, int8 values).
// Centroids are rounded to fp16 after a common scale, chosen at init so that
// they fall nearest to fp16 values.  The key weights W carry two fp16 pieces
// (22 bits).  P is rounded to fp16: one rounding of relative 2^-11 per weight,
// independent between tokens, below the rounding of the 16-bit output.  S, O,
// the sums and the softmax's reference are fp32.
//
// Softmax.  A weight is 2^(s - m) with m a reference per row, not the running
// maximum itself: m is set to the tile's maximum less 6 when the row first sees
// a token, and moves only when a score exceeds m by 12, so that the sums and O
// are rescaled (in registers and TMEM) only then.  Weights reach 2^12 at most,
// fp16's range keeps 2^-14 at full precision, and the sums are 32-bit.  The
// value scales s_t, which multiply the weights, are divided by a power of two
// (sref) that likewise moves only when a scale exceeds it four times.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvc_launch.cuh"
#include "kvc_sm100.cuh"
#include "kvc_tc.h"

namespace kvc {

using namespace sm100;

namespace {

constexpr int kTile = kTreeTile;
constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kProdWarp = kSoftWarps + kDecWarps;
constexpr int kScoreWarp = kProdWarp + 1, kSumWarp = kProdWarp + 2;
// 20 warps: setmaxnreg works on whole groups of four
constexpr int kThreads = (kProdWarp + 4) * 32;
constexpr int kDecThreads = kDecWarps * 32;
// registers per thread: the launch gives 96; producer and MMA warps, decoders
// and softmax groups then hold 48, 72 and 144 (128 (48 + 2 72 + 2 144) = 640 96)
constexpr int kLaunchRegs = 96, kCtlRegs = 48, kDecRegs = 72, kSoftRegs = 144;
static_assert(128 * (kCtlRegs + 2 * kDecRegs + 2 * kSoftRegs) <= kThreads * kLaunchRegs,
              "register split exceeds the launch's registers");
constexpr int kMaxNS = 4;          // row stages
constexpr int kDecBar = 1;         // named barriers: decoders; 2, 3: softmax groups
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kSet = 6.f;        // a reference is set this far below the maximum (log2)
constexpr float kMove = 12.f;      // and moves when a score lies this far above it

struct Shape {
  int nc, nwg, n;        // columns of a softmax group, groups, columns (nc nwg)
  int K, KC;             // K of the score product, its 8-value chunks
  int mt;                // 128-channel tiles of O
  int a_cols, s_col, o_col, cols;  // TMEM layout
  int nv, ns;            // V buffers, row stages
  int krow, stage;       // bytes of a stage's key rows; of a stage
  int off_p, off_v, off_stage, off_tab;  // shared-memory offsets
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
// permute of the levels takes.  No table in shared memory: its bandwidth is
// what the kernel has least of.
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
__device__ __forceinline__ void int8_block(const unsigned char* row, unsigned char* dst, int c0, int t8) {
#pragma unroll
  for (int j = 0; j < NV / 2; j += 4) {
    uint2 b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = *reinterpret_cast<const uint2*>(row + ((c0 + t8 + j + u) & (NV - 1)) * 8);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(dst + ((c0 + t8 + j + u) & (NV - 1)) * 128) = int8_values(b[u]);
  }
}

// 64 consecutive codes (2 W words, 8-byte aligned) of a row of W-bit indices
// into 32 TMEM columns.
template <int W>
__device__ __forceinline__ void codebook64(const unsigned char* src, const Levels& t, uint32_t a_tm) {
  uint32_t w[2 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint2 v = reinterpret_cast<const uint2*>(src)[i];
    w[2 * i] = v.x;
    w[2 * i + 1] = v.y;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int bit = (4 * h + c) * 8 * W, i = bit >> 5, sh = bit & 31;
      const uint32_t x = sh + 8 * W <= 32 ? w[i] >> sh : __funnelshift_r(w[i], w[i + 1], sh);
      const uint4 v = centroids8<W>(x, t);
      r[4 * c] = v.x; r[4 * c + 1] = v.y; r[4 * c + 2] = v.z; r[4 * c + 3] = v.w;
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A CTA's run of tiles, cut at the jobs' ends.
struct Segment {
  int job, slot, r0, nr, b;
  int tile0, tile1;  // tiles of the job (hidden context skipped)
};
struct Walk {
  int64_t at, end;
  __device__ Walk(const TreeArgs& t)
      : at(t.total * blockIdx.x / t.grid), end(t.total * (blockIdx.x + 1) / t.grid) {}
  __device__ bool next(const TreeArgs& t, int H, Segment& g) {
    if (at >= end) return false;
    g.job = (int)(at / t.tps);
    const int64_t a = at - g.job * t.tps;
    const int64_t z = min(t.tps, a + (end - at));
    at += z - a;
    g.slot = g.job / t.row_tiles;
    g.r0 = (g.job - g.slot * t.row_tiles) * t.rt;
    g.nr = min(t.rt, t.rows - g.r0);
    g.b = g.slot / H;
    g.tile0 = (int)a;
    g.tile1 = (int)z;
    if (t.first) {  // tiles of hidden context only
      const int64_t f = min((int64_t)max(t.first[g.b], 0), t.ctx) / kTile;
      g.tile0 = (int)min(z, max(a, f));
    }
    return true;
  }
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

// Wait for a phase.  Once a wait of any role has run out (2 s) every further
// wait returns at once, so that all roles walk to their ends and the named
// barriers stay matched; the results are then undefined and the error word says so.
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!*abort_flag) {
    if (mbar_try_wait_sleep(bar, parity, 100000u)) return;
    if (global_timer_ns() - t0 > kWaitNs) *abort_flag = 1;
  }
}

template <int KMODE, int VMODE, int NC>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const Params kp, const Params vp, const TreeArgs t, const Shape z) {
  constexpr bool VU = VMODE == KVC_MODE_UNIFORM;
  constexpr int CH = NC < 32 ? NC : 32;  // columns handled at a time
  constexpr int NCH = NC / CH;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t row_full[kMaxNS], row_empty[kMaxNS], a_full[2], a_empty[2], v_full[2],
      v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2], w_full, done_bar;
  __shared__ uint32_t kch[32], vch[32];
  // per softmax group and column: offset of the score (c1 - m), m, rescale
  // factor, seen a token; the warps' partial results
  __shared__ __align__(16) float cneg[2][64];
  __shared__ float mref[2][64], corr[2][64], red[2][4][64];
  __shared__ int seen[2][64];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* Ws = smem;  // two pieces [n x K] fp16, K-major cores
  unsigned char* Ps = smem + z.off_p;
  unsigned char* Vs = smem + z.off_v;
  unsigned char* Rs = smem + z.off_stage;
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem + z.off_tab);  // codebooks of 16 or 256 levels
  const int w_piece = z.n * z.K * 2;
  const int v_bytes = z.mt * kTile * 256;

  if (warp == kScoreWarp) tmem_alloc(&tmem_base, z.cols);
  if (tid == 0) {
    for (int i = 0; i < z.ns; ++i) { mbar_init(&row_full[i], 1); mbar_init(&row_empty[i], kDecWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], kDecWarps);
      mbar_init(&a_empty[i], 1);
      mbar_init(&v_full[i], kDecWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], z.nwg * 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(&w_full, z.nwg);
    mbar_init(&done_bar, 2);
    fence_mbar_init();
    abort_flag = 0;
  }
  if (KMODE == KVC_MODE_CODEBOOK && kp.cb_bits >= 4) {  // pairs of 16 levels, or 256 levels
    const int pair = kp.cb_bits == 4;
    auto half_of = [&](int c) {
      return (uint32_t)__half_as_ushort(__float2half_rn(kp.codebook[c] * t.cb_mul));
    };
    for (int j = tid; j < 256; j += kThreads)
      tab[j] = pair ? half_of(j & 15) | (half_of(j >> 4) << 16) : half_of(j);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  Walk walk(t);
  Segment g;
  grid_dependency_wait();  // the key weights come from the launch before

  if (warp >= kProdWarp) {
    regs_dec<kCtlRegs>();
    if (warp == kProdWarp && lane == 0) {
      // ---------------------------------------------------------- producer
      Ring rr(z.ns);
      int issued = 0;
      while (walk.next(t, kp.H, g)) {
        const int Pk = kp.P[kp.basis_of[g.slot]];
        const int Pv = VU ? vp.P[vp.basis_of[g.slot]] : vp.D;
        const unsigned char* ks = kp.store + kp.pay_off[g.slot];
        const unsigned char* vs = vp.store + vp.pay_off[g.slot];
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
        }
        if (abort_flag) break;
      }
      // copies still in flight (after a time-out) land before the CTA exits
      for (int j = max(0, issued - z.ns); j < issued; ++j)
        mbar_wait_bounded(&row_full[j % z.ns], (j / z.ns) & 1, kWaitNs);
    } else if (warp == kScoreWarp) {
      // ---------------------------------------------------------- S = A W^T
      // The whole warp walks and waits, one elected lane issues, so that
      // descriptors stay in uniform registers; the two products have a warp
      // each.  (One lane walking and issuing both took 160 cycles per MMA.)
      const bool leader = elect_one();
      const uint32_t id = idesc_f16(kTile, z.n, 0);
      const uint64_t w_desc = desc_kmajor_noswizzle(smem_u32(Ws), 128, (uint32_t)z.KC * 128);
      int it = 0, segs = 0;
      while (walk.next(t, kp.H, g)) {
        if (g.tile0 == g.tile1) continue;
        wait_or_abort(&w_full, segs & 1, &abort_flag);
        ++segs;
        for (int tile = g.tile0; tile < g.tile1; ++tile, ++it) {
          const int s = it & 1;
          if (it >= 2) wait_or_abort(&s_empty[s], ((it >> 1) - 1) & 1, &abort_flag);
          wait_or_abort(&a_full[s], (it >> 1) & 1, &abort_flag);
          __syncwarp();
          tc_fence_after();
          if (leader) {
            const uint32_t a0 = tm + s * z.a_cols, d0 = tm + z.s_col + s * z.n;
            umma_f16_tmem_a(d0, a0, w_desc, id, 0u);
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // the two pieces of W
              const uint64_t wd = w_desc + ((p * w_piece) >> 4);
#pragma unroll 8
              for (int ks = 1 - p; ks < z.K / 16; ++ks)  // 16 fp16 of K: 8 TMEM columns of A
                umma_f16_tmem_a(d0, a0 + ks * 8, wd + ks * 16, id, 1u);
            }
            umma_commit(&s_full[s]);
            umma_commit(&a_empty[s]);
          }
          __syncwarp();
        }
      }
      if (leader) {
        umma_commit(&done_bar);  // TMEM is released only after every MMA has finished
        mbar_wait_bounded(&done_bar, 0, kWaitNs);
      }
      __syncwarp();
    } else if (warp == kSumWarp) {
      // ---------------------------------------------------------- O += V^T P
      // One product over both groups' columns, or, where the groups hold 64
      // each, one per group as its weights arrive.
      const bool leader = elect_one();
      const int parts = NC == 64 ? z.nwg : 1;
      const uint32_t pn = NC == 64 ? NC : z.n;
      const uint32_t id = idesc_f16(kTile, pn, 0) | kTransposeAB;
      const uint32_t v_k = (uint32_t)z.mt * 2048, p_k = (uint32_t)z.n * 16;
      const uint64_t v_desc = desc_mnmajor(smem_u32(Vs), v_k, 128);
      const uint64_t p_desc = desc_mnmajor(smem_u32(Ps), p_k, 128);
      const uint64_t v_step = (2 * v_k) >> 4, p_step = (2 * p_k) >> 4;
      int it = 0;
      Ring rv(z.nv);
      while (walk.next(t, kp.H, g)) {
        for (int tile = g.tile0; tile < g.tile1; ++tile, ++it, rv.next()) {
          wait_or_abort(&v_full[rv.slot], rv.phase, &abort_flag);
          for (int h = 0; h < parts; ++h) {
            for (int wg = h; wg < (parts == 1 ? z.nwg : h + 1); ++wg)
              wait_or_abort(&p_full[wg], it & 1, &abort_flag);
            __syncwarp();
            tc_fence_after();
            if (leader) {
              for (int m = 0; m < z.mt; ++m) {
                const uint32_t o = tm + z.o_col + m * z.n + h * pn;
                uint64_t vd = v_desc + ((rv.slot * v_bytes + m * 2048) >> 4);
                uint64_t pd = p_desc + h * (NC / 8 * 128 >> 4);
                umma_f16(o, vd, pd, id, tile > g.tile0 ? 1u : 0u);
#pragma unroll
                for (int ks = 1; ks < kTile / 16; ++ks) {
                  vd += v_step;
                  pd += p_step;
                  umma_f16(o, vd, pd, id, 1u);
                }
              }
              for (int wg = h; wg < (parts == 1 ? z.nwg : h + 1); ++wg) umma_commit(&p_empty[wg]);
              if (h == parts - 1) umma_commit(&v_empty[rv.slot]);
            }
            __syncwarp();
          }
        }
      }
      if (leader) {
        umma_commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, kWaitNs);
      }
      __syncwarp();
    }
  } else if (warp >= kSoftWarps) {
    // ------------------------------------------------------------ decoders
    regs_dec<kDecRegs>();
    const int dtid = tid - kSoftWarps * 32;
    const int tt = dtid & (kTile - 1), half = dtid >> 7;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // values: eight lanes take eight tokens of one block, each another chunk of
    // the row, so that neither the reads (rows 128 bytes apart) nor the writes
    // (cores 128 bytes apart) meet in a bank
    const int octet = lane >> 3, t8 = lane & 7;
    const int vblk = (warp - kSoftWarps) * 2 + (octet >> 1);
    Levels levels{};
    if (KMODE == KVC_MODE_CODEBOOK && kp.cb_bits <= 3) {
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
    while (walk.next(t, kp.H, g)) {
      if (g.tile0 == g.tile1) continue;
      const int kbeta = kp.basis_of[g.slot], vbeta = VU ? vp.basis_of[g.slot] : 0;
      named_bar_sync(kDecBar, kDecThreads);  // the last segment's tables have been read
      if (dtid < 32) kch[dtid] = chunk_entry(kp, kbeta, dtid);
      else if (VU && dtid < 64) vch[dtid - 32] = chunk_entry(vp, vbeta, dtid - 32);
      named_bar_sync(kDecBar, kDecThreads);
      const int Pk = kp.P[kbeta], Pv = VU ? vp.P[vbeta] : vp.D;
      int nv = VU ? 0 : vp.D / 8;  // chunks of a value row
      if (VU)
        while (nv < 32 && vch[nv]) ++nv;
      const int vhalf = (nv + 1) / 2;
      for (int tile = g.tile0; tile < g.tile1; ++tile, ++it, rr.next(), rv.next()) {
        const int a = it & 1;
        wait_or_abort(&row_full[rr.slot], rr.phase, &abort_flag);
        if (it >= 2) wait_or_abort(&a_empty[a], ((it >> 1) - 1) & 1, &abort_flag);
        __syncwarp();
        const unsigned char* st = Rs + rr.slot * z.stage;
        const uint32_t a_tm = tm + lane_base + a * z.a_cols;
        if (KMODE == KVC_MODE_CODEBOOK && kp.cb_bits <= 3 && kp.D == 128) {
          const int W = kp.cb_bits;
          const unsigned char* src = st + tt * Pk + half * 8 * W;
          if (W == 3) codebook64<3>(src, levels, a_tm + half * 32);
          else if (W == 2) codebook64<2>(src, levels, a_tm + half * 32);
          else codebook64<1>(src, levels, a_tm + half * 32);
        } else {
#pragma unroll 4
          for (int c = half; c < z.KC; c += 2) {
            const uint32_t ent = kch[c];
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
            int8_block<16>(raw + tok * 128, dst, c0, t8);
          } else if (!VU && nv == 8) {
            int8_block<8>(raw + tok * 64, dst, c0, t8);
          } else {
            const int cend = min(nv, c0 + vhalf);
            for (int j = c0; j < cend; ++j) {
              int c = j + t8;
              while (c >= nv) c -= nv;
              uint4 v;
              if (VU) {
                const uint32_t ent = vch[c];
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
  } else if (warp < z.nwg * 4) {
    // ------------------------------------------------------------ softmax
    regs_inc<kSoftRegs>();
    const int wg = warp >> 2, quarter = warp & 3, ltid = tid & 127, bar = 2 + wg;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_tm = tm + lane_off + z.o_col + wg * NC;
    float* cn = cneg[wg];
    unsigned char* pst = Ps + ((quarter * 32 + lane) >> 3) * (z.n * 16) + wg * (NC / 8 * 128) + (lane & 7) * 16;
    int it = 0;
    while (walk.next(t, kp.H, g)) {
      const int64_t first = t.first ? max(t.first[g.b], 0) : 0;
      const int col0 = wg * NC, ncol = max(0, min(NC, g.nr - col0));  // rows of this group
      const size_t row0 = (size_t)g.slot * t.rows + g.r0 + col0;
      float post = 1.f;
      named_bar_sync(bar, 128);  // the last segment's column state has been read
      if (ltid < NC) {
        cn[ltid] = ltid < ncol ? t.c1[row0 + ltid] : 0.f;
        mref[wg][ltid] = 0.f;
        seen[wg][ltid] = ltid >= ncol;
      }
      if (g.tile0 < g.tile1) {
        // key weights as two fp16 pieces, scaled into fp16's range by a power of two
        const float* w = t.w + row0 * t.NCk;
        float mx = 0.f;
        for (int e = ltid; e < ncol * t.NCk; e += 128) {
          const float v = fabsf(w[e]);
          if (v <= 3.4e38f) mx = fmaxf(mx, v);
        }
        mx = warp_max(mx) * t.w_mul;
        if (lane == 0) red[wg][quarter][0] = mx;
        named_bar_sync(bar, 128);
        mx = fmaxf(fmaxf(red[wg][0][0], red[wg][1][0]), fmaxf(red[wg][2][0], red[wg][3][0]));
        const int ex = max(0, (__float_as_int(mx) >> 23) - 127 - 13);
        post = __int_as_float((127 + ex) << 23);
        const float pre = t.w_mul * __int_as_float((127 - ex) << 23);
        for (int e = ltid; e < NC * z.KC; e += 128) {
          const int r = e / z.KC, c = e - r * z.KC;
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = 0.f;
          if (r < ncol && c * 8 < t.NCk) {
            const float4* src = reinterpret_cast<const float4*>(w + (size_t)r * t.NCk + c * 8);
            const float4 a = src[0], b = src[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
          }
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i] * pre, b = x[2 * i + 1] * pre;
            hi[i] = pack_half2(a, b);
            const __half2 h = *reinterpret_cast<const __half2*>(&hi[i]);
            lo[i] = pack_half2(a - __low2float(h), b - __high2float(h));
          }
          unsigned char* dst = Ws + ((col0 + r) >> 3) * (z.KC * 128) + c * 128 + (r & 7) * 16;
          *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + w_piece) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        named_bar_sync(bar, 128);
        if (ltid == 0) mbar_arrive(&w_full);
      }
      const uint8_t* mask = t.mask ? t.mask + g.b * t.mask_sb : nullptr;
      float2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = make_float2(0.f, 0.f);
      uint32_t unseen = ncol ? (1u << NCH) - 1u : 0u;  // column chunks with rows that saw nothing yet
      float sref = VU ? 1.f : 0.f, inv_sref = VU ? 1.f : 0.f;
      const int lt = quarter * 32 + lane;
      // this lane's norm and scale, loaded one tile ahead and converted at use
      // (converting them at the load would wait for it)
      const unsigned short* knorm = reinterpret_cast<const unsigned short*>(kp.store + kp.side_off[g.slot]);
      const unsigned short* vscale = reinterpret_cast<const unsigned short*>(vp.store + vp.side_off[g.slot]);
      const int live_tiles = (int)((t.S - lt + kTile - 1) / kTile);  // tiles in which this lane has a token
      const unsigned short* kn = knorm + (int64_t)g.tile0 * kTile + lt;
      const unsigned short* vsc = vscale + (int64_t)g.tile0 * kTile + lt;
      unsigned short nt_next = 0, st_next = 0;
      if (g.tile0 < g.tile1 && g.tile0 < live_tiles) {
        if (KMODE == KVC_MODE_CODEBOOK) nt_next = *kn;
        if (!VU) st_next = *vsc;
      }
      // tiles [plain0, plain1) hold visible context alone
      const int plain0 = (int)min((int64_t)t.tps, (first + kTile - 1) / kTile), plain1 = (int)(t.ctx / kTile);
      for (int tile = g.tile0; tile < g.tile1; ++tile, ++it) {
        const int s = it & 1;
        const float nt = KMODE == KVC_MODE_CODEBOOK ? __half2float(__ushort_as_half(nt_next)) * post : post;
        const float st = VU ? 1.f : __half2float(__ushort_as_half(st_next));
        kn += kTile;
        vsc += kTile;
        if (tile + 1 < g.tile1 && tile + 1 < live_tiles) {  // the next tile's norms and scales
          if (KMODE == KVC_MODE_CODEBOOK) nt_next = *kn;
          if (!VU) st_next = *vsc;
        } else {
          nt_next = st_next = 0;
        }
        // which of the group's rows see this lane's token
        const bool special = tile < plain0 || tile >= plain1;
        uint64_t vis = ~0ull;
        if (special) {
          const int64_t tok = (int64_t)tile * kTile + lt, draft = tok - t.ctx;
          if (draft < 0) {
            vis = tok >= first ? ~0ull : 0ull;
          } else {
            vis = 0ull;
            if (draft < t.N) {
              int n = (g.r0 + col0) % t.N;
              for (int c = 0; c < ncol; ++c) {
                if (mask ? mask[(int64_t)n * t.N + draft] != 0 : draft <= n) vis |= 1ull << c;
                if (++n == t.N) n = 0;
              }
            }
          }
        }
        bool up = !VU && vis != 0ull && st > 4.f * sref && st <= 65504.f;
        float su = 0.f;
        wait_or_abort(&s_full[s], (it >> 1) & 1, &abort_flag);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          float2 x[CH / 2];
          bool moved = false;
          for (;;) {
            uint32_t r[CH];
            tmem_ld_n<CH>(tm + lane_off + z.s_col + s * z.n + col0 + ch * CH, r);
            tmem_wait_ld();
            const float2 nt2 = make_float2(nt, nt);
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
              const float4 c = reinterpret_cast<const float4*>(cn + ch * CH)[i];
              x[2 * i] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), nt2,
                                    make_float2(c.x, c.y));
              x[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                        nt2, make_float2(c.z, c.w));
            }
            if (special) {
              const uint32_t v = (uint32_t)(vis >> (ch * CH));
#pragma unroll
              for (int i = 0; i < CH / 2; ++i) {
                if (!(v >> (2 * i) & 1u)) x[i].x = -INFINITY;
                if (!(v >> (2 * i + 1) & 1u)) x[i].y = -INFINITY;
              }
            }
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) mx = fmaxf(mx, fmaxf(x[i].x, x[i].y));
            if (moved || !named_bar_or(bar, 128, mx > kMove || up || (unseen >> ch & 1u))) break;
            moved = true;
            // The references move (rare).  Every thread of the group is here.
            float ratio = 1.f;
            if (!VU) {  // the value scales' reference: the next power of two
              const float m = warp_max(up ? st : 0.f);
              if (lane == 0) red[wg][quarter][0] = m;
              named_bar_sync(bar, 128);
              const float big = fmaxf(fmaxf(red[wg][0][0], red[wg][1][0]), fmaxf(red[wg][2][0], red[wg][3][0]));
              if (big > 0.f) {
                const float to = __int_as_float((__float_as_int(big) & 0x7f800000) + 0x00800000);
                ratio = sref / to;
                sref = to;
                inv_sref = 1.f / to;
              }
              up = false;
              named_bar_sync(bar, 128);
            }
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              const float a = warp_max(x[i].x), b = warp_max(x[i].y);
              if (lane == 0) {
                red[wg][quarter][2 * i] = a;
                red[wg][quarter][2 * i + 1] = b;
              }
            }
            named_bar_sync(bar, 128);
            bool blind = false;
            if (ltid < CH) {
              const int c = ch * CH + ltid;
              const float m = fmaxf(fmaxf(red[wg][0][ltid], red[wg][1][ltid]),
                                    fmaxf(red[wg][2][ltid], red[wg][3][ltid]));
              float d = 0.f, f = 1.f;
              if (m != -INFINITY) {  // (a row of NaN counts as seen and stays NaN)
                if (!seen[wg][c]) {  // nothing summed yet
                  d = m - kSet;
                  f = 0.f;
                  seen[wg][c] = 1;
                } else if (m > kSet) {
                  d = m - kSet;
                  f = ex2(-d);
                }
              }
              mref[wg][c] += d;
              cn[c] -= d;
              corr[wg][c] = f;
              blind = !seen[wg][c];
            }
            if (!named_bar_or(bar, 128, blind)) unseen &= ~(1u << ch);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              l[ch * CH / 2 + i].x *= corr[wg][ch * CH + 2 * i];
              l[ch * CH / 2 + i].y *= corr[wg][ch * CH + 2 * i + 1];
            }
            if (tile > g.tile0) {  // O holds sums: rescale it once the last product is done
              wait_or_abort(&p_empty[wg], (it - 1) & 1, &abort_flag);
              __syncwarp();
              tc_fence_after();
              for (int m = 0; m < z.mt; ++m)
                for (int c = 0; c < NC; c += 16) {
                  const bool mine = c >= ch * CH && c < ch * CH + CH;
                  if (!mine && ratio == 1.f) continue;
                  uint32_t o[16];
                  tmem_ld16(o_tm + m * z.n + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * (mine ? corr[wg][c + i] * ratio : ratio));
                  tmem_st16(o_tm + m * z.n + c, o);
                }
              tmem_wait_st();
            }
            named_bar_sync(bar, 128);  // corr and red have been read
          }
          if (ch == 0) {
            su = vis != 0ull ? st * inv_sref : 0.f;
            if (it > 0) wait_or_abort(&p_empty[wg], (it - 1) & 1, &abort_flag);  // P has been read
            __syncwarp();
          }
          if (ch == NCH - 1) {  // S has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[s]);
          }
          const float2 su2 = make_float2(su, su);
#pragma unroll
          for (int q = 0; q < CH / 8; ++q) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 4 * q + i;
              const float2 p = make_float2(ex2(x[j].x), ex2(x[j].y));
              l[ch * CH / 2 + j] = __fadd2_rn(l[ch * CH / 2 + j], p);
              float2 u = VU ? p : __fmul2_rn(p, su2);
              if (!VU && special) {  // a hidden token's scale may be anything
                const uint32_t v = (uint32_t)(vis >> (ch * CH));
                if (!(v >> (2 * j) & 1u)) u.x = 0.f;
                if (!(v >> (2 * j + 1) & 1u)) u.y = 0.f;
              }
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
      const bool any = g.tile0 < g.tile1;
      if (any) {
        wait_or_abort(&p_empty[wg], (it - 1) & 1, &abort_flag);
        __syncwarp();
        tc_fence_after();
      }
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        const float a = warp_sum(l[i].x), b = warp_sum(l[i].y);
        if (lane == 0) {
          red[wg][quarter][2 * i] = a;
          red[wg][quarter][2 * i + 1] = b;
        }
      }
      named_bar_sync(bar, 128);
      const size_t prow = ((size_t)g.job + blockIdx.x) * t.rt + col0;
      float* part = t.part + prow * t.Dvp;
      if (ltid < ncol) {
        const bool sn = seen[wg][ltid] != 0;
        t.ml[prow + ltid] = make_float2(
            sn ? mref[wg][ltid] : -INFINITY,
            sn ? (red[wg][0][ltid] + red[wg][1][ltid]) + (red[wg][2][ltid] + red[wg][3][ltid]) : 0.f);
      }
      for (int m = 0; m < z.mt; ++m) {
        const int d = m * 128 + quarter * 32 + lane;
        for (int c = 0; c < ncol; c += 16) {
          uint32_t o[16];
          if (any) {
            tmem_ld16(o_tm + m * z.n + c, o);
            tmem_wait_ld();
          }
          if (d < t.Dv) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < ncol)
                part[(size_t)(c + i) * t.Dvp + d] = any ? __uint_as_float(o[i]) * sref : 0.f;
          }
        }
      }
      tc_fence_before();  // the next segment's first product overwrites O
    }
  }
  grid_dependents_launch();
  __syncthreads();
  if (abort_flag && tid == 0) atomicCAS(kp.err, 0, kErrTimeout);
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tm, z.cols);
  }
}

using TcKernel = void (*)(const Params, const Params, const TreeArgs, const Shape);

template <int KMODE, int VMODE>
TcKernel kernel_for_nc(int nc) {
  switch (nc) {
    case 16: return tree_tc_kernel<KMODE, VMODE, 16>;
    case 32: return tree_tc_kernel<KMODE, VMODE, 32>;
    default: return tree_tc_kernel<KMODE, VMODE, 64>;
  }
}

TcKernel kernel_for(int kmode, int vmode, int nc) {
  if (kmode == KVC_MODE_UNIFORM)
    return vmode == KVC_MODE_UNIFORM ? kernel_for_nc<KVC_MODE_UNIFORM, KVC_MODE_UNIFORM>(nc)
                                     : kernel_for_nc<KVC_MODE_UNIFORM, KVC_MODE_INT8>(nc);
  return vmode == KVC_MODE_UNIFORM ? kernel_for_nc<KVC_MODE_CODEBOOK, KVC_MODE_UNIFORM>(nc)
                                   : kernel_for_nc<KVC_MODE_CODEBOOK, KVC_MODE_INT8>(nc);
}

// Layout for n = nc nwg columns, or false when TMEM or shared memory does not hold it.
bool shape_for(const Params& kp, const TreeArgs& t, int nc, int nwg, Shape* out) {
  Shape z{};
  z.nc = nc;
  z.nwg = nwg;
  z.n = nc * nwg;
  z.K = (t.NCk + 15) / 16 * 16;
  z.KC = z.K / 8;
  z.mt = (t.Dv + 127) / 128;
  z.a_cols = (z.K / 2 + 31) / 32 * 32;
  z.s_col = 2 * z.a_cols;
  z.o_col = z.s_col + 2 * z.n;
  const int cols = z.o_col + z.mt * z.n;
  if (cols > 512) return false;
  for (z.cols = 32; z.cols < cols; z.cols *= 2) {}
  auto up = [](int v) { return (v + 127) / 128 * 128; };
  z.krow = up(kTile * t.Pk_max + 16);
  z.stage = z.krow + up(kTile * t.Pv_max + 16);
  z.off_p = 2 * z.n * z.K * 2;
  z.off_v = z.off_p + z.n * kTile * 2;
  int tab = 0;
  if (kp.mode == KVC_MODE_CODEBOOK && kp.cb_bits >= 4) tab = 1024;
  // two V buffers and four row stages, or what fits
  const int most = 220 * 1024;  // of 227 KB: the static arrays take 5
  for (z.nv = 2; z.nv >= 1; --z.nv)
    for (z.ns = kMaxNS; z.ns >= 2; --z.ns) {
      z.off_stage = z.off_v + z.nv * z.mt * kTile * 256;
      z.off_tab = z.off_stage + z.ns * z.stage;
      z.smem = z.off_tab + tab;
      if (z.smem <= most) {
        *out = z;
        return true;
      }
    }
  return false;
}

bool choose_shape(const Params& kp, const TreeArgs& t, Shape* z) {
  // the fewest columns that hold all rows, else the most that fit
  static const int kShapes[4][2] = {{16, 1}, {16, 2}, {32, 2}, {64, 2}};
  bool ok = false;
  for (const auto& s : kShapes) {
    Shape c;
    if (!shape_for(kp, t, s[0], s[1], &c)) break;
    *z = c;
    ok = true;
    if (c.n >= t.rows) break;
  }
  return ok;
}

}  // namespace

int tree_tc_rows(const Params& kp, const Params& vp, const TreeArgs& t) {
  if (t.prod) return 0;
  if (vp.mode == KVC_MODE_INT8 && vp.D % 8) return 0;  // value rows are read 8 bytes at a time
  Shape z;
  return choose_shape(kp, t, &z) ? z.n : 0;
}

cudaError_t launch_tree_tc(const Params& kp, const Params& vp, const TreeArgs& t, cudaStream_t s,
                           int* nk) {
  Shape z;
  if (!choose_shape(kp, t, &z)) return cudaErrorInvalidValue;
  TcKernel k = kernel_for(kp.mode, vp.mode, z.nc);
  // the register split draws on what the launch gives: never launch with less
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, k);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, z.smem);
  if (e != cudaSuccess) return e;
  ++*nk;
  return launch_dependent(k, (unsigned)t.grid, kThreads, (size_t)z.smem, s, kp, vp, t, z);
}

}  // namespace kvc
