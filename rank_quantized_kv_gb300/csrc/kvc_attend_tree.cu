// Attention of N drafted tokens per sequence over the stored codes.  The
// drafted tokens are the last N stored tokens of a key and a value layer; a
// drafted token sees the context (every earlier stored token, from first[b]
// on) and those drafted tokens that the mask gives it, so a whole tree of
// drafts is scored in one pass over the cache.
//
// With centred codes c' = code - 2^(b-1) of a b-bit component, and u = V^T q:
//   scores   uniform keys   q . k_hat = sum_j (u_j step_j) c'_j + c1,
//                           c1 = sum_j u_j (lo_j + 2^(b_j-1) step_j) + q . mean;
//            codebook keys  q . k_hat = n sum_j u_j c[idx_j], with a residual
//                           sketch plus sqrt(pi/2)/m ||r|| sum_j (S q)_j (2 bit_j - 1)
//                           and with an outlier stream plus s sum_l q_{ch_l} o8_l;
//   weights  softmax over the visible tokens, online and in base 2 (scale
//            log2(e) folded into the key weights and c1); a hidden token's
//            weight is 0 whatever its codes, norm or scale hold;
//   output   int8 values    sum_t p_t s_t q8_t;
//            uniform values (lo + 2^(b-1) step + step sum_t p_t c'_t) V^T + mean;
//            zero for a row that sees no token, NaN for one that sees a score
//            of NaN or of +inf, or scores of -inf alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_pipeline.h>

#include <algorithm>

#include "kvc_codes.cuh"
#include "kvc_internal.h"
#include "kvc_launch.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 128;      // 4 warps
constexpr int kRows = 8;           // rows of a job
constexpr int kPrepThreads = 256;
__device__ __forceinline__ float load_q(const TreeArgs& t, int64_t i) {
  if (t.q_dtype == KVC_F32) return static_cast<const float*>(t.q)[i];
  if (t.q_dtype == KVC_F16) return __half2float(static_cast<const __half*>(t.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(t.q)[i]);
}

// ---------------------------------------------------------------- prep

// The mask as bits, transposed: word w of draft j holds the drafts 32 w .. that
// see j.  One block per (mask, w, 256 drafts).
__device__ void pack_mask(const TreeArgs& t, int block) {
  const int words = (t.N + 31) / 32, cols = (t.N + kPrepThreads - 1) / kPrepThreads;
  const int jb = block % cols, w = block / cols % words, b = block / cols / words;
  const int j = jb * kPrepThreads + threadIdx.x;
  grid_dependents_launch();
  if (j >= t.N) return;
  const uint8_t* m = t.mask + b * t.mask_sb + (int64_t)w * 32 * t.N + j;
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (w * 32 + i < t.N && m[(int64_t)i * t.N]) v |= 1u << i;
  t.mask_bits[((size_t)b * t.N + j) * words + w] = v;
}

// The key weights at every packed position, w_j = scale log2(e) u_j coef_j
// (coef = step in uniform mode, 1 for a codebook), and c1, for ROWS rows of a
// slot per block; u = q V in fp32, by the block's 256 threads.
//   64, 32    a register-tiled product, 8 or 4 rows x 4 columns a thread and 128
//   rows      columns a warp, V through shared memory 32 rows at a time: bound by
//             the fp32 FMA pipe (rows D r of them);
//   8 rows    a thread takes one column and a share of the sum over D, V straight
//             from global memory, each element read once: bound by latency.  For
//             bases of up to 64 columns, which leave half of the tiles' columns
//             empty, and for few rows, for which it gives more blocks.
//
// For the tensor cores a row's weights are split into two fp16 pieces and laid
// out as their operand.  They are first divided by a power of two 2^ex that
// brings the row's largest to [2^-6, 2^14), from where the pieces carry 22 bits
// of the large weights and leave at most 2^-25, that is 2^-19 of the largest, of
// any.  The softmax multiplies the products by 2^ex: at no cost where the rows of
// a job have one ex (it goes into the token's norm), so ex is not taken to the
// last bit but in steps of 20, windows that w_shift puts around the usual sizes.
// (Jobs of several take a multiplication more a score: 16 sequences of 8 heads,
// 16384 tokens, 128 rows a head 350 us in place of 316, 32 rows 175 of 173.)
// Uniform keys have no norm that would multiply what the pieces leave, and codes of
// at most 128: their small weights stay as they are (ex >= 0).
constexpr int kPrepCols = 128, kPrepK = 32, kPrepBufs = 2;

template <int ROWS>
constexpr size_t prep_smem(int D, int r) {
  return (size_t)(D * (ROWS + 4) + (ROWS >= 32 ? kPrepBufs * kPrepK * kPrepCols : kPrepThreads * 8) +
                  ROWS * (r | 1)) * sizeof(float);
}

template <int ROWS>
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(const Params kp, const TreeArgs t) {
  constexpr int RT = ROWS / 8;       // rows of a warp
  constexpr int kQ = ROWS + 4;       // stores of q meet four to a bank, not all
  extern __shared__ __align__(16) float sm_f[];
  __shared__ int comp[256];          // packed position: component (-1: padding)
  __shared__ float coef[256];        // component: factor of its weight, 0 when dropped
  __shared__ float off[256];         // component: lo + 2^(b-1) step
  __shared__ int64_t q_row[ROWS];    // first element of a row of q, -1 past the last
  __shared__ float down[ROWS];       // power of two that brings a row into its window
  const int D = kp.D, r = kp.r, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blocks = (t.prow + ROWS - 1) / ROWS;
  if ((int)blockIdx.x >= blocks * kp.n_slots) {
    pack_mask(t, blockIdx.x - blocks * kp.n_slots);
    return;
  }
  grid_dependents_launch();
  const int slot = blockIdx.x / blocks, r0 = (blockIdx.x - slot * blocks) * ROWS;
  const int b = slot / kp.H, h = slot - b * kp.H;
  const int beta = kp.basis_of[slot];
  const int nr = max(0, min(ROWS, t.rows - r0));  // rows of queries
  const int np = min(ROWS, t.prow - r0);          // rows written
  const bool uniform = kp.mode == KVC_MODE_UNIFORM;
  const int us_row = r | 1;           // an odd stride: rows in different banks
  float* qs = sm_f;                   // [D][kQ] rows of q, transposed
  float* vs = qs + D * kQ;            // [2][32][128] rows of V; [share][8][columns] sums
  float* us = vs + (ROWS >= 32 ? kPrepBufs * kPrepK * kPrepCols : kPrepThreads * 8);  // [ROWS][us_row] weights
  const float* V = kp.V + (size_t)beta * D * r;
  const int stages = (D + kPrepK - 1) / kPrepK;
  // rows of V from 32 st, columns c0 ..: asynchronous copies of 16 bytes, or of
  // 4 where a row starts at any multiple of 4
  auto load_v = [&](int st, int c0) {
    const bool wide = (r & 3) == 0;
    const int step = wide ? 4 : 1, buf = st % kPrepBufs;
    for (int e = tid * step; st < stages && e < kPrepK * kPrepCols; e += kPrepThreads * step) {
      const int i = e / kPrepCols, c = e - i * kPrepCols, k = st * kPrepK + i;
      float* dst = vs + buf * kPrepK * kPrepCols + e;
      const float* src = V + (size_t)k * r + c0 + c;
      const bool in = k < D && c0 + c < r;
      if (wide) {
        if (in) __pipeline_memcpy_async(dst, src, 16);
        else *reinterpret_cast<float4*>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        if (in) __pipeline_memcpy_async(dst, src, 4);
        else *dst = 0.f;
      }
    }
    __pipeline_commit();
  };
  if (ROWS >= 32)
    for (int st = 0; st < kPrepBufs - 1; ++st) load_v(st, 0);
  if (tid < ROWS) {
    const int x = r0 + tid, g = x / t.N, n = x - g * t.N;
    q_row[tid] = tid < nr ? b * t.q_sb + (int64_t)(h * t.rep + g) * t.q_sh + n * t.q_st : -1;
  }
  for (int k = tid; k < 256; k += kPrepThreads) {
    int width = 0;
    comp[k] = k < t.NCk ? position_component(kp, beta, k, &width) : -1;
    float c = 0.f, o = 0.f;
    if (k < r) {
      const size_t bk = (size_t)beta * r + k;
      width = kp.bits[bk];
      if (width) c = t.scale_log2 * t.w_mul * (uniform ? kp.step[bk] : 1.f);
      if (width && uniform) o = fmaf((float)(1 << (width - 1)), kp.step[bk], kp.lo[bk]);
    }
    coef[k] = c;
    off[k] = o;
  }
  __syncthreads();
  // a warp takes every eighth row, 64 values at a time, all loads issued before
  // the first is stored
  for (int i0 = 0; i0 < D; i0 += 64) {
    float v[RT][2];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      const int64_t at = q_row[warp + 8 * u] + i0 + lane;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v[u][e] = warp + 8 * u < nr && i0 + lane + 32 * e < D ? load_q(t, at + 32 * e) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (i0 + lane + 32 * e < D) qs[(i0 + lane + 32 * e) * kQ + warp + 8 * u] = v[u][e];
  }
  // rows RT warp ..: largest weight and offset, over the lanes' columns
  float mx[RT], c1[RT];
#pragma unroll
  for (int e = 0; e < RT; ++e) mx[e] = c1[e] = 0.f;
  auto take = [&](int e, int k, float u) {  // column k of the warp's row e
    const float w = u * coef[k];
    us[(RT * warp + e) * us_row + k] = w;
    if (fabsf(w) <= 3.4e38f) mx[e] = fmaxf(mx[e], fabsf(w));  // NaN and infinities stay what they are
    c1[e] = fmaf(u, off[k], c1[e]);
  };
  if constexpr (ROWS >= 32) {
    for (int c0 = 0; c0 < r; c0 += kPrepCols) {
      float2 acc[RT][2];
#pragma unroll
      for (int e = 0; e < RT; ++e) acc[e][0] = acc[e][1] = make_float2(0.f, 0.f);
      if (c0)
        for (int st = 0; st < kPrepBufs - 1; ++st) load_v(st, c0);
      for (int st = 0; st < stages; ++st) {
        load_v(st + kPrepBufs - 1, c0);  // (past the last: an empty group)
        __pipeline_wait_prior(kPrepBufs - 1);
        __syncthreads();
        const float* vb = vs + st % kPrepBufs * kPrepK * kPrepCols + 4 * lane;
        const float* qb = qs + st * kPrepK * kQ + RT * warp;
        const int kn = min(kPrepK, D - st * kPrepK);
#pragma unroll 8
        for (int k = 0; k < kn; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(vb + k * kPrepCols);
          const float4 q0 = *reinterpret_cast<const float4*>(qb + k * kQ);
          const float4 q1 = *reinterpret_cast<const float4*>(qb + k * kQ + RT - 4);
          const float q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
          for (int e = 0; e < RT; ++e) {
            const float2 qq = make_float2(q[e], q[e]);
            acc[e][0] = __ffma2_rn(qq, make_float2(v.x, v.y), acc[e][0]);
            acc[e][1] = __ffma2_rn(qq, make_float2(v.z, v.w), acc[e][1]);
          }
        }
        __syncthreads();  // this buffer is refilled next
      }
      const int c = c0 + 4 * lane;
#pragma unroll
      for (int e = 0; e < RT; ++e) {
        if (c < r) take(e, c, acc[e][0].x);
        if (c + 1 < r) take(e, c + 1, acc[e][0].y);
        if (c + 2 < r) take(e, c + 2, acc[e][1].x);
        if (c + 3 < r) take(e, c + 3, acc[e][1].y);
      }
    }
  } else {
    __syncthreads();
    // columns of a pass: 32, 64 or 128; the rest of the threads share the sum
    const int cols = r <= 32 ? 32 : r <= 64 ? 64 : 128, shares = kPrepThreads / cols;
    const int col = tid & (cols - 1), share = tid / cols;
    const int per = (D + shares - 1) / shares, k0 = share * per, k1 = min(D, k0 + per);
    for (int c0 = 0; c0 < r; c0 += cols) {
      float2 acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
      if (c0 + col < r) {
        const float* vc = V + c0 + col;
        for (int kb = k0; kb < k1; kb += 16) {  // 16 loads in flight
          float v[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) v[u] = kb + u < k1 ? vc[(size_t)(kb + u) * r] : 0.f;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const float* qk = qs + min(kb + u, D - 1) * kQ;
            const float4 q0 = *reinterpret_cast<const float4*>(qk);
            const float4 q1 = *reinterpret_cast<const float4*>(qk + 4);
            const float2 vv = make_float2(v[u], v[u]);
            if (kb + u >= k1) continue;
            acc[0] = __ffma2_rn(vv, make_float2(q0.x, q0.y), acc[0]);
            acc[1] = __ffma2_rn(vv, make_float2(q0.z, q0.w), acc[1]);
            acc[2] = __ffma2_rn(vv, make_float2(q1.x, q1.y), acc[2]);
            acc[3] = __ffma2_rn(vv, make_float2(q1.z, q1.w), acc[3]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vs[(share * 8 + 2 * e) * cols + col] = acc[e].x;
        vs[(share * 8 + 2 * e + 1) * cols + col] = acc[e].y;
      }
      __syncthreads();
      for (int c = lane; c < cols && c0 + c < r; c += 32) {
        float u = 0.f;
        for (int x = 0; x < shares; ++x) u += vs[(x * 8 + warp) * cols + c];
        take(0, c0 + c, u);
      }
      __syncthreads();
    }
  }
  const size_t row0 = (size_t)slot * t.prow + r0;
#pragma unroll
  for (int e = 0; e < RT; ++e) {
    const int row = RT * warp + e;
    if (uniform) {
      for (int i = lane; i < D; i += 32) c1[e] = fmaf(qs[i * kQ + row], kp.mean[(size_t)beta * D + i], c1[e]);
      c1[e] = warp_sum(c1[e]);
    }
    const float most = warp_max(mx[e]);
    if (lane == 0 && row < np) {
      t.c1[row0 + row] = t.scale_log2 * c1[e];
      if (t.tc) {
        const int at = (__float_as_int(most) >> 23) - 127 + t.w_shift + 6;
        const int step = (at >= 0 ? at / 20 : -((19 - at) / 20)) * 20 - t.w_shift;
        const int ex = min(126, max(uniform ? 0 : -126, step));
        t.wscale[row0 + row] = most > 0.f ? __int_as_float((127 + ex) << 23) : 0.f;
        down[row] = most > 0.f ? __int_as_float((127 - ex) << 23) : 1.f;
      }
    }
  }
  __syncthreads();
  if (!t.tc) {
    for (int j = tid; j < t.NCk; j += kPrepThreads)  // this thread's positions of all rows
      for (int row = 0; row < nr; ++row)
        t.w[(row0 + row) * t.NCk + j] = comp[j] < 0 ? 0.f : us[row * us_row + comp[j]];
    return;
  }
  // two fp16 pieces in the layout of a K-major operand without swizzle: cores of
  // 8 rows x 8 positions, 128 contiguous bytes, adjacent along K
  const int KC = t.K / 8;
  for (int e = tid; e < np * KC; e += kPrepThreads) {
    const int c = e / np, row = e - c * np;
    const int x = r0 + row, jt = x / t.rt, rr = x - jt * t.rt;
    uint16_t* dst = t.w16 + ((size_t)slot * t.row_tiles + jt) * 2 * t.rt * t.K +
                    (rr >> 3) * (KC * 64) + c * 64 + (rr & 7) * 8;
    __half hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = comp[8 * c + i];
      const float v = k < 0 || row >= nr ? 0.f : us[row * us_row + k] * down[row];
      hi[i] = __float2half_rn(v);
      lo[i] = __float2half_rn(v - __half2float(hi[i]));
    }
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(hi);
    *reinterpret_cast<uint4*>(dst + t.rt * t.K) = *reinterpret_cast<const uint4*>(lo);
  }
}

// Keys with a residual sketch or an outlier stream: the sketch weights
// sqrt(pi/2)/m (S q)_j and the outlier weights q[ch_l], one block per row.
__global__ void __launch_bounds__(kThreads) tree_prep_prod_kernel(const Params kp, const TreeArgs t) {
  __shared__ float qs[kProdMaxD];
  const int slot = blockIdx.x / t.rows, row = blockIdx.x - slot * t.rows;
  const int b = slot / kp.H, h = slot - b * kp.H, g = row / t.N, n = row - g * t.N;
  const int D = kp.D, nx = t.m + t.n_out;
  for (int i = threadIdx.x; i < D; i += kThreads)
    qs[i] = load_q(t, b * t.q_sb + (int64_t)(h * t.rep + g) * t.q_sh + n * t.q_st + i);
  __syncthreads();
  const float coef = t.m ? 1.2533141373155003f / (float)t.m : 0.f;
  for (int j = threadIdx.x; j < nx; j += kThreads) {
    float u = 0.f;
    if (j < t.m) {
      const float* s = kp.W3 + (size_t)(D + j) * D;
      for (int i = 0; i < D; ++i) u = fmaf(s[i], qs[i], u);
      u *= coef;
    } else {
      u = qs[kp.channels[(size_t)slot * t.n_out + j - t.m]];
    }
    t.wx[(size_t)blockIdx.x * nx + j] = t.scale_log2 * u;
  }
}

// ---------------------------------------------------------------- main

// The run of tiles of CTA c is [total c / grid, total (c + 1) / grid).
__device__ __forceinline__ int64_t run_begin(const TreeArgs& t, int64_t c) {
  return t.total * c / t.grid;
}

// CUDA cores: a warp takes 32 tokens at a time, a lane scores one of them for the
// job's 8 rows (key weights broadcast from shared memory), then the lanes share
// out the value channels.  Bound by shared-memory reads, four fp32 weights to a
// load.  128 slots of 32 rows over 16384 tokens of 3-bit keys and int8 values:
// 5.6 ms (the tensor cores 0.18); 2 slots of 8 rows over 84 tokens in 29 us, launches included.
//
// Dynamic shared memory: ws [NCk][8], wxs [m + n_out][8], per warp krow [32 Pk + 16] and vrow
// [32 Pv + 16] (uniform values) and ps [32][8]; merge [4][8][2 + Dv].
template <int KMODE, int VMODE>
__global__ void __launch_bounds__(kThreads)
    tree_main_kernel(const Params kp, const Params vp, const TreeArgs t, int kstage, int vstage) {
  extern __shared__ __align__(16) unsigned char sm[];
  __shared__ uint32_t kch[32], vch[32];
  __shared__ float cbv[256];
  __shared__ float c1s[kRows];
  constexpr bool VU = VMODE == KVC_MODE_UNIFORM;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NCk = t.NCk, Dv = t.Dv, nx = t.m + t.n_out;
  const int stride = 2 + Dv;
  float* ws = reinterpret_cast<float*>(sm);
  float* wxs = ws + NCk * kRows;
  unsigned char* wbase =
      reinterpret_cast<unsigned char*>(wxs + nx * kRows) + (size_t)warp * (kstage + vstage + 32 * kRows * 4);
  unsigned char* krow = wbase;
  unsigned char* vrow = wbase + kstage;
  float* ps = reinterpret_cast<float*>(wbase + kstage + vstage);
  float* merge = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(wxs + nx * kRows) +
                                          4 * (size_t)(kstage + vstage + 32 * kRows * 4));
  if (KMODE == KVC_MODE_CODEBOOK)
    for (int j = tid; j < kp.cb_levels; j += kThreads) cbv[j] = kp.codebook[j];

  grid_dependency_wait();  // the key weights come from the launch before
  const int64_t run1 = run_begin(t, blockIdx.x + 1);
  for (int64_t at = run_begin(t, blockIdx.x); at < run1;) {
    const int job = (int)(at / t.tps);
    const int64_t tile0 = at - job * t.tps;
    const int64_t tile1 = min(t.tps, tile0 + (run1 - at));
    at += tile1 - tile0;
    const int slot = job / t.row_tiles, r0 = (job - slot * t.row_tiles) * kRows;
    const int nr = min(kRows, t.rows - r0);
    const int b = slot / kp.H;
    const int kbeta = kp.basis_of[slot], vbeta = VU ? vp.basis_of[slot] : 0;
    const int Pk = kp.P[kbeta], Pv = VU ? vp.P[vbeta] : vp.D;
    __syncthreads();  // the previous job's tables and partial have been read
    if (tid < 32) {
      kch[tid] = chunk_entry(kp, kbeta, tid);
      vch[tid] = VU ? chunk_entry(vp, vbeta, tid) : 0u;
    }
    const size_t row0 = (size_t)slot * t.rows + r0;
    for (int e = tid; e < kRows * NCk; e += kThreads) {
      const int j = e / kRows, g = e - j * kRows;
      ws[e] = g < nr ? t.w[(row0 + g) * NCk + j] : 0.f;
    }
    for (int e = tid; e < kRows * nx; e += kThreads) {
      const int j = e / kRows, g = e - j * kRows;
      wxs[e] = g < nr ? t.wx[(row0 + g) * nx + j] : 0.f;
    }
    if (tid < kRows) c1s[tid] = tid < nr ? t.c1[row0 + tid] : 0.f;
    __syncthreads();
    int nchk = 0, nchv = 0;
    while (nchk < 32 && (kch[nchk] >> 31)) ++nchk;
    if (VU)
      while (nchv < 32 && (vch[nchv] >> 31)) ++nchv;
    int LG = 1;  // uniform values: LG chunk lanes x (32 / LG) token groups
    while (LG < nchv) LG *= 2;
    const int vc = lane & (LG - 1), tg = lane / LG, TG = 32 / LG;
    const unsigned char* kbase = kp.store + kp.pay_off[slot];
    const __half* knorm = reinterpret_cast<const __half*>(kp.store + kp.side_off[slot]);
    const unsigned char* vbase = vp.store + vp.pay_off[slot];
    const __half* vscale = reinterpret_cast<const __half*>(vp.store + vp.side_off[slot]);
    const int64_t first = t.first ? t.first[b] : 0;
    const uint8_t* mask = t.mask ? t.mask + b * t.mask_sb : nullptr;

    float m[kRows], l[kRows], acc[kRows][8];
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[g][e] = 0.f;
    }
    const int64_t t1 = min(t.S, tile1 * kTreeTile);
    for (int64_t tb = tile0 * kTreeTile + 32 * warp; tb < t1; tb += kTreeTile) {
      // blocks of hidden context only
      if (tb + 32 <= min(first, t.ctx)) continue;
      const int nrow = (int)min((int64_t)32, t1 - tb);
      {
        const uint4* src = reinterpret_cast<const uint4*>(kbase + tb * Pk);
        const int nv = (nrow * Pk + 15) >> 4;
        for (int i = lane; i < nv; i += 32) reinterpret_cast<uint4*>(krow)[i] = src[i];
        if (VU) {
          const uint4* vs = reinterpret_cast<const uint4*>(vbase + tb * Pv);
          const int nvv = (nrow * Pv + 15) >> 4;
          for (int i = lane; i < nvv; i += 32) reinterpret_cast<uint4*>(vrow)[i] = vs[i];
        }
      }
      __syncwarp();
      const int64_t tok = tb + lane;
      const bool live = lane < nrow;
      float sc[kRows];
#pragma unroll
      for (int g = 0; g < kRows; ++g) sc[g] = 0.f;
      float sv = 1.f;  // value scale
      if (live) {
        const int row = lane * Pk;
        for (int c = 0; c < nchk; ++c) {
          const uint32_t ent = kch[c];
          const int w = (int)((ent >> 16) & 0xfu);
          const uint2 bits = bits_at(krow, row + (int)(ent & 0xffffu));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t code = chunk_code(bits, w, e);
            const float v = KMODE == KVC_MODE_CODEBOOK ? cbv[code] : (float)((int)code - (1 << (w - 1)));
            const float4* wp = reinterpret_cast<const float4*>(ws + (8 * c + e) * kRows);
            const float4 a = wp[0], bb = wp[1];
            sc[0] = fmaf(a.x, v, sc[0]); sc[1] = fmaf(a.y, v, sc[1]);
            sc[2] = fmaf(a.z, v, sc[2]); sc[3] = fmaf(a.w, v, sc[3]);
            sc[4] = fmaf(bb.x, v, sc[4]); sc[5] = fmaf(bb.y, v, sc[5]);
            sc[6] = fmaf(bb.z, v, sc[6]); sc[7] = fmaf(bb.w, v, sc[7]);
          }
        }
        if (KMODE == KVC_MODE_CODEBOOK) {
          const int64_t sw = tok * t.knw;
          const float n = __half2float(knorm[sw]);
#pragma unroll
          for (int g = 0; g < kRows; ++g) sc[g] *= n;
          if (t.m) {  // + ||r|| sum_j w_j (2 bit_j - 1)
            const unsigned char* sb = krow + row + t.kcode;
            float qj[kRows];
#pragma unroll
            for (int g = 0; g < kRows; ++g) qj[g] = 0.f;
            for (int j = 0; j < t.m; ++j) {
              const float f = (sb[j >> 3] >> (j & 7)) & 1u ? 1.f : -1.f;
#pragma unroll
              for (int g = 0; g < kRows; ++g) qj[g] = fmaf(wxs[j * kRows + g], f, qj[g]);
            }
            const float gam = __half2float(knorm[sw + 1]);
#pragma unroll
            for (int g = 0; g < kRows; ++g) sc[g] = fmaf(gam, qj[g], sc[g]);
          }
          if (t.n_out) {  // + s sum_l q[ch_l] o8_l
            const int8_t* o8 = reinterpret_cast<const int8_t*>(krow + row + t.kcode + (t.m >> 3));
            float qo[kRows];
#pragma unroll
            for (int g = 0; g < kRows; ++g) qo[g] = 0.f;
            for (int j = 0; j < t.n_out; ++j) {
              const float v = (float)o8[j];
#pragma unroll
              for (int g = 0; g < kRows; ++g) qo[g] = fmaf(wxs[(t.m + j) * kRows + g], v, qo[g]);
            }
            const float os = __half2float(knorm[sw + t.knw - 1]);
#pragma unroll
            for (int g = 0; g < kRows; ++g) sc[g] = fmaf(os, qo[g], sc[g]);
          }
        }
        if (!VU) sv = __half2float(vscale[tok]);
      }
      // visibility, then the online softmax
      const int64_t draft = tok - t.ctx;
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        bool see = live && g < nr;
        if (draft < 0) {
          see = see && tok >= first;
        } else if (see) {
          const int n = (r0 + g) % t.N;
          see = mask ? mask[(int64_t)n * t.N + draft] != 0 : draft <= n;
        }
        const float s = see ? sc[g] + c1s[g] : -INFINITY;
        const float mn = fmaxf(m[g], warp_max(see ? fmaxf(s, kTreeLowest) : -INFINITY));
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing visible yet
        const float corr = exp2f(m[g] - ref);
        const float pt = see ? exp2f(s - ref) : 0.f;
        l[g] = l[g] * corr + warp_sum(pt);
        m[g] = mn;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[g][e] *= corr;
        ps[lane * kRows + g] = see ? pt * sv : 0.f;
      }
      __syncwarp();
      if (!VU) {
        // lane owns channels lane, lane + 32, ..
        for (int tt = 0; tt < nrow; ++tt) {
          const int8_t* vr = reinterpret_cast<const int8_t*>(vbase + (tb + tt) * (int64_t)Pv) + lane;
          float pv[kRows];
#pragma unroll
          for (int g = 0; g < kRows; ++g) pv[g] = ps[tt * kRows + g];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (lane + 32 * e >= Dv) break;
            const float v = (float)vr[32 * e];
#pragma unroll
            for (int g = 0; g < kRows; ++g) acc[g][e] = fmaf(pv[g], v, acc[g][e]);
          }
        }
      } else if (vc < nchv) {
        const uint32_t ent = vch[vc];
        const int w = (int)((ent >> 16) & 0xfu), off = (int)(ent & 0xffffu);
        for (int tt = tg; tt < nrow; tt += TG) {
          const uint2 bits = bits_at(vrow, tt * Pv + off);
          float pv[kRows];
#pragma unroll
          for (int g = 0; g < kRows; ++g) pv[g] = ps[tt * kRows + g];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = (float)((int)chunk_code(bits, w, e) - (1 << (w - 1)));
#pragma unroll
            for (int g = 0; g < kRows; ++g) acc[g][e] = fmaf(pv[g], v, acc[g][e]);
          }
        }
      }
      __syncwarp();  // staging and ps are rewritten by the next block
    }
    if (VU)
      for (int o = LG; o < 32; o <<= 1)
#pragma unroll
        for (int g = 0; g < kRows; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[g][e] += __shfl_xor_sync(kFull, acc[g][e], o);
    // the warps' states into one partial: [row][m, l, acc[Dv]]
    for (int e = lane; e < kRows * stride; e += 32) merge[(size_t)warp * kRows * stride + e] = 0.f;
    __syncwarp();
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      float* mg = merge + ((size_t)warp * kRows + g) * stride;
      if (lane == 0) {
        mg[0] = m[g];
        mg[1] = l[g];
      }
      if (!VU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (lane + 32 * e < Dv) mg[2 + lane + 32 * e] = acc[g][e];
      } else if (tg == 0 && vc < nchv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mg[2 + vc * 8 + e] = acc[g][e];
      }
    }
    __syncthreads();
    const size_t prow = ((size_t)job + blockIdx.x) * t.rt;
    for (int e = tid; e < nr * stride; e += kThreads) {
      const int g = e / stride, d = e - g * stride;
      float M = -INFINITY;
      for (int w4 = 0; w4 < 4; ++w4) M = fmaxf(M, merge[((size_t)w4 * kRows + g) * stride]);
      float v = d == 0 ? M : 0.f;
      if (d)
        for (int w4 = 0; w4 < 4; ++w4) {
          const float* mg = merge + ((size_t)w4 * kRows + g) * stride;
          // (a warp without tokens has l = 0; one with NaN scores has m = -inf too)
          if (mg[1] != 0.f) v = fmaf(exp2f(mg[0] - M), mg[d], v);
        }
      if (d == 0) t.ml[prow + g].x = v;
      else if (d == 1) t.ml[prow + g].y = v;
      else t.part[prow * t.Dvp + (size_t)(d - 2) * t.rt + g] = v;
    }
  }
}

// ---------------------------------------------------------------- combine

constexpr int kCombineRows = 8, kCombineThreads = 256, kFactors = 64;

// Bound by the latency of the partials' reads, few CTAs being at work: 8 slots of
// 20 rows x 128 channels, about 20 CTAs' partials a slot, take 16 us; 128 slots
// of 128 rows 19 us.
//
// Merge the partials of a job, normalise and write the output rows (uniform
// values: project the weighted mean latent).  One block per (slot, 8 rows);
// thread (d, q) holds channel d of rows 4 q .. 4 q + 3, which lie together in a
// partial.
__global__ void __launch_bounds__(kCombineThreads)
    tree_combine_kernel(const Params kp, const Params vp, const TreeArgs t) {
  __shared__ __align__(16) float fac[kFactors][kCombineRows];  // 2^(m - M) of the partials
  __shared__ __align__(16) float zb[256][kCombineRows];  // uniform values: mean latents
  __shared__ short comp[256];         // component of a packed position
  __shared__ float zs[256], zo[256];  // its step, and its offset lo + 2^(b-1) step
  __shared__ float inv_s[kCombineRows];
  const int blocks = (t.rows + kCombineRows - 1) / kCombineRows;
  const int slot = blockIdx.x / blocks, row0 = (blockIdx.x - slot * blocks) * kCombineRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = slot / kp.H, h = slot - b * kp.H;
  const bool vu = vp.mode == KVC_MODE_UNIFORM;
  const int beta = vu ? vp.basis_of[slot] : 0;
  const int jt = row0 / t.rt, job = slot * t.row_tiles + jt, rr = row0 - jt * t.rt;
  // the CTAs whose runs hold the job's tiles
  const int64_t lo = job * t.tps, hi = lo + t.tps;
  int64_t c0 = lo * t.grid / t.total;
  while (run_begin(t, c0 + 1) <= lo) ++c0;
  while (run_begin(t, c0) > lo) --c0;
  int64_t c1 = c0;
  while (run_begin(t, c1 + 1) < hi) ++c1;
  const int np = ((int)(c1 - c0) + 1) * t.parts;
  const size_t p0 = ((size_t)job + c0) * t.parts;
  if (vu)
    for (int j = tid; j < t.Dv; j += kCombineThreads) {
      int width = 0;
      const int k = position_component(vp, beta, j, &width);
      const size_t bk = (size_t)beta * vp.r + (k < 0 ? 0 : k);
      comp[j] = (short)k;
      zs[j] = vp.step[bk];
      zo[j] = k < 0 ? 0.f : fmaf((float)(1 << (width - 1)), vp.step[bk], vp.lo[bk]);
    }
  grid_dependency_wait();
  // row `warp`: the largest reference
  const float2* ml = t.ml + p0 * t.rt + rr + warp;
  const bool live = row0 + warp < t.rows;
  float M = -INFINITY, L = 0.f;
  if (live)
    for (int s = lane; s < np; s += 32) M = fmaxf(M, ml[(size_t)s * t.rt].x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  const int d0 = tid & 127, q = tid >> 7;  // d0 and d0 + 128; row quad
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = 0; s0 < np; s0 += kFactors) {
    const int n = min(kFactors, np - s0);
    __syncthreads();
    for (int e = lane; e < n; e += 32) {
      const float2 v = live ? ml[(size_t)(s0 + e) * t.rt] : make_float2(0.f, 0.f);
      // a run that saw nothing has l = 0 (and weighted sums of 0)
      const float f = v.y == 0.f ? 0.f : exp2f(v.x - ref);
      if (v.y != 0.f) L = fmaf(f, v.y, L);
      fac[e][warp] = f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d = d0 + 128 * u;
      if (d >= t.Dv) break;
      const float* p = t.part + (p0 + s0) * t.rt * t.Dvp + (size_t)d * t.rt + rr + 4 * q;
#pragma unroll 4
      for (int e = 0; e < n; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(p + (size_t)e * t.rt * t.Dvp);
        const float4 f = *reinterpret_cast<const float4*>(&fac[e][4 * q]);
        acc[u].x = fmaf(f.x, v.x, acc[u].x);
        acc[u].y = fmaf(f.y, v.y, acc[u].y);
        acc[u].z = fmaf(f.z, v.z, acc[u].z);
        acc[u].w = fmaf(f.w, v.w, acc[u].w);
      }
    }
  }
  L = warp_sum(L);
  // nothing visible: zero; scores of -inf alone: NaN
  if (lane == 0) inv_s[warp] = L > 0.f || L != L ? 1.f / L : M == -INFINITY ? 0.f : NAN;
  __syncthreads();
  auto put = [&](int d, float4 v) {  // channel d of the thread's four rows
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = row0 + 4 * q + e;
      if (row >= t.rows) break;
      const int g = row / t.N, n = row - g * t.N;
      const int64_t o = b * t.o_sb + (int64_t)(h * t.rep + g) * t.o_sh + n * t.o_st + d;
      if (t.out_bf16) reinterpret_cast<__nv_bfloat16*>(t.out)[o] = __float2bfloat16_rn(x[e]);
      else reinterpret_cast<__half*>(t.out)[o] = __float2half_rn(x[e]);
    }
  };
  const float4 inv = *reinterpret_cast<const float4*>(&inv_s[4 * q]);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int d = d0 + 128 * u;
    if (d >= t.Dv) break;
    const float4 v = make_float4(acc[u].x * inv.x, acc[u].y * inv.y, acc[u].z * inv.z, acc[u].w * inv.w);
    if (!vu) put(d, v);
    else
      *reinterpret_cast<float4*>(&zb[d][4 * q]) =
          make_float4(fmaf(zs[d], v.x, zo[d]), fmaf(zs[d], v.y, zo[d]), fmaf(zs[d], v.z, zo[d]),
                      fmaf(zs[d], v.w, zo[d]));  // the mean latent
  }
  if (!vu) return;
  __syncthreads();
  for (int i = d0; i < vp.D; i += 128) {
    const float mu = vp.mean[(size_t)beta * vp.D + i];
    float4 v = make_float4(mu, mu, mu, mu);
    const float* Vt = vp.Vt + (size_t)beta * vp.r * vp.D + i;
#pragma unroll 8
    for (int j = 0; j < t.Dv; ++j) {
      const int k = comp[j];
      const float c = k < 0 ? 0.f : Vt[(size_t)k * vp.D];
      const float4 zz = *reinterpret_cast<const float4*>(&zb[j][4 * q]);
      if (k < 0) continue;  // padding: its sums are whatever the codes' padding held
      v.x = fmaf(zz.x, c, v.x);
      v.y = fmaf(zz.y, c, v.y);
      v.z = fmaf(zz.z, c, v.z);
      v.w = fmaf(zz.w, c, v.w);
    }
    auto row = [](float x, float f) { return f == 0.f ? 0.f : f != f ? f : x; };
    put(i, make_float4(row(v.x, inv.x), row(v.y, inv.y), row(v.z, inv.z), row(v.w, inv.w)));
  }
}

using MainKernel = void (*)(const Params, const Params, const TreeArgs, int, int);

MainKernel main_kernel_for(int kmode, int vmode) {
  if (kmode == KVC_MODE_UNIFORM)
    return vmode == KVC_MODE_UNIFORM ? tree_main_kernel<KVC_MODE_UNIFORM, KVC_MODE_UNIFORM>
                                     : tree_main_kernel<KVC_MODE_UNIFORM, KVC_MODE_INT8>;
  return vmode == KVC_MODE_UNIFORM ? tree_main_kernel<KVC_MODE_CODEBOOK, KVC_MODE_UNIFORM>
                                   : tree_main_kernel<KVC_MODE_CODEBOOK, KVC_MODE_INT8>;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// key weights: fp32 (CUDA cores) or two fp16 pieces
size_t w_bytes(const Params& kp, const TreeArgs& t) {
  return align256((size_t)kp.n_slots * t.prow * (t.tc ? t.K : t.NCk) * 4);
}
size_t c1_bytes(const Params& kp, const TreeArgs& t) {  // score offsets; row scales
  return align256((size_t)kp.n_slots * t.prow * 4);
}
size_t ml_bytes(int64_t jobs, const TreeArgs& t) {
  return align256((size_t)(jobs + t.grid - 1) * t.parts * t.rt * 8);
}
size_t mask_bytes(const Params& kp, const TreeArgs& t) {
  return t.tc ? align256((size_t)kp.B * t.N * ((t.N + 31) / 32) * 4) : 0;
}
size_t wx_bytes(const Params& kp, const TreeArgs& t) {
  return align256((size_t)kp.n_slots * t.rows * (t.m + t.n_out) * 4);
}

cudaError_t launch_main(const Params& kp, const Params& vp, const TreeArgs& t, cudaStream_t s,
                        int* nk) {
  const int kstage = (32 * t.Pk_max + 16 + 15) / 16 * 16;
  const int vstage = vp.mode == KVC_MODE_UNIFORM ? (32 * t.Pv_max + 16 + 15) / 16 * 16 : 0;
  const size_t smem = (size_t)kRows * (t.NCk + t.m + t.n_out) * 4 +
                      4 * (size_t)(kstage + vstage + 32 * kRows * 4) +
                      4 * (size_t)kRows * (2 + t.Dv) * 4;
  MainKernel k = main_kernel_for(kp.mode, vp.mode);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), (int)smem);
  if (e != cudaSuccess) return e;
  ++*nk;
  return launch_dependent(k, (unsigned)t.grid, kThreads, smem, s, kp, vp, t, kstage, vstage);
}

}  // namespace

size_t tree_plan(const Params& kp, TreeArgs& t, int sms) {
  t.rt = t.tc ? t.tc : kRows;
  t.row_tiles = (t.rows + t.rt - 1) / t.rt;
  t.prow = t.tc ? t.row_tiles * t.rt : t.rows;
  const int64_t jobs = (int64_t)kp.n_slots * t.row_tiles;
  t.tps = (t.S + kTreeTile - 1) / kTreeTile;
  t.total = jobs * t.tps;
  // one CTA per SM on the tensor cores, else about twelve
  t.grid = (int)std::min<int64_t>(t.total, (t.tc ? 1 : 12) * (int64_t)sms);
  t.Dvp = (t.Dv + 3) / 4 * 4;
  t.sms = sms;
  return w_bytes(kp, t) + 2 * c1_bytes(kp, t) + wx_bytes(kp, t) + mask_bytes(kp, t) +
         ml_bytes(jobs, t) +
         align256((size_t)(jobs + t.grid - 1) * t.parts * t.rt * t.Dvp * 4);
}

cudaError_t launch_attend_tree(const Params& kp, const Params& vp, TreeArgs t, void* workspace,
                               cudaStream_t s, int* nk) {
  auto* ws = static_cast<unsigned char*>(workspace);
  t.w = reinterpret_cast<float*>(ws);
  t.w16 = reinterpret_cast<uint16_t*>(ws);
  ws += w_bytes(kp, t);
  t.c1 = reinterpret_cast<float*>(ws);
  ws += c1_bytes(kp, t);
  t.wscale = reinterpret_cast<float*>(ws);
  ws += c1_bytes(kp, t);
  t.wx = reinterpret_cast<float*>(ws);
  ws += wx_bytes(kp, t);
  t.mask_bits = reinterpret_cast<uint32_t*>(ws);
  ws += mask_bytes(kp, t);
  t.ml = reinterpret_cast<float2*>(ws);
  ws += ml_bytes((int64_t)kp.n_slots * t.row_tiles, t);
  t.part = reinterpret_cast<float*>(ws);
  cudaError_t e;
  if (t.prod) {
    tree_prep_prod_kernel<<<(unsigned)kp.n_slots * t.rows, kThreads, 0, s>>>(kp, t);
    ++*nk;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // rows of a projection block (measured, us: 4096 rows of 128 columns 19 with 32,
  // 26 with 8; 4096 rows of 32 columns 18 and 13; 16384 rows of 128 columns 34
  // with 64, the whole call 8 more with 32)
  const bool few = kp.r <= 64 || t.prow <= 16;
  const bool many = (int64_t)kp.n_slots * ((t.prow + 63) / 64) >= t.sms;
  const int rows = few ? 8 : many ? 64 : 32;
  const size_t smem = few    ? prep_smem<8>(kp.D, kp.r)
                      : many ? prep_smem<64>(kp.D, kp.r)
                             : prep_smem<32>(kp.D, kp.r);
  const auto prep = few ? tree_prep_kernel<8> : many ? tree_prep_kernel<64> : tree_prep_kernel<32>;
  e = prepare_kernel(reinterpret_cast<const void*>(prep), (int)smem);
  if (e != cudaSuccess) return e;
  const int masks = t.tc && t.mask ? (t.mask_sb ? kp.B : 1) : 0;  // blocks that pack the mask
  const int pack = masks * ((t.N + 31) / 32) * ((t.N + kPrepThreads - 1) / kPrepThreads);
  prep<<<(unsigned)kp.n_slots * ((t.prow + rows - 1) / rows) + pack, kPrepThreads, smem, s>>>(kp, t);
  ++*nk;
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = t.tc ? launch_tree_tc(kp, vp, t, s, nk) : launch_main(kp, vp, t, s, nk);
  if (e != cudaSuccess) return e;
  const int blocks = (t.rows + kCombineRows - 1) / kCombineRows;
  ++*nk;
  return launch_dependent(tree_combine_kernel, (unsigned)kp.n_slots * blocks, kCombineThreads, 0, s,
                          kp, vp, t);
}

}  // namespace kvc
