// Attention of the last N stored tokens over a sliding window and the first
// tokens of the cache (sinks), from the codes, and the softmax weights that the
// stored tokens receive.  The query at position p sees the tokens t <= p that lie
// in its window (t > p - window) or among the `sinks` tokens from first[b] on;
// tokens before first[b] are padding.
//
// With centred codes c' = code - 2^(b-1) of a b-bit component, and u = V^T q:
//   scores   uniform keys   q . k_hat = sum_j (u_j step_j) c'_j + c1,
//                           c1 = sum_j u_j (lo_j + 2^(b_j-1) step_j) + q . mean;
//            codebook keys  q . k_hat = n sum_j u_j c[idx_j], with a residual
//                           sketch plus sqrt(pi/2)/m ||r|| sum_j (S q)_j (2 bit_j - 1)
//                           and with an outlier stream plus s sum_l q_{ch_l} o8_l;
//   softmax  over the visible tokens, online and in base 2 (scale log2(e) folded
//            into the key weights and c1);
//   output   int8 values    sum_t p_t s_t q8_t;
//            uniform values (lo + 2^(b-1) step + step sum_t p_t c'_t) V^T + mean;
//            zero for a row that sees no token, NaN for one that sees a score of
//            NaN or of +inf, or scores of -inf alone;
//   weights  w[t] = decay w[t] + sum of p_t over the rows of a slot.  p needs the
//            row's whole sum, so it takes a second pass.  Of at most eight rows the
//            tensor-core kernel keeps its scores for it (16 or 32 bytes a token,
//            mostly still in L2 when they are read: 128 slots, 4 rows, 16384 tokens
//            11.7 us and 3 more in the main kernel; computed again from the 50 bytes of
//            a token's codes 56).  Of more rows, whose scores would outgrow the codes
//            and L2, they are computed again.  Tokens
//            are split over blocks and a token's rows are added in order: no atomics.
//
// This file: the queries' projection, the CUDA-core kernels, which take every layer
// that the entry point takes and compute in fp32, and the joining of partials.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kvc_codes.cuh"
#include "kvc_internal.h"
#include "kvc_launch.cuh"
#include "kvc_window.cuh"

namespace kvc {

namespace {

constexpr int kTcRows = 32;    // more rows of a slot take the tcgen05 kernel
constexpr int kThreads = 128;  // 4 warps
constexpr int kRows = 8;       // rows of a job
constexpr int kTile = 128;     // tokens of a tile: 32 a warp

__device__ __forceinline__ float load_q(const WindowArgs& t, int64_t i) {
  if (t.q_dtype == KVC_F32) return static_cast<const float*>(t.q)[i];
  if (t.q_dtype == KVC_F16) return __half2float(static_cast<const __half*>(t.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(t.q)[i]);
}

// First element of row x of slot (b, h).
__device__ __forceinline__ int64_t q_at(const WindowArgs& t, int b, int h, int x) {
  const int n = x / t.rep, g = x - n * t.rep;
  return b * t.q_sb + (int64_t)(h * t.rep + g) * t.q_sh + n * t.q_st;
}

// ---------------------------------------------------------------- prep

constexpr int kPrepThreads = 256, kPrepCols = 32;

// The key weights w_j = scale log2(e) u_j coef_j (coef = step in uniform mode, 1 for
// a codebook) at 32 packed positions for 8 rows, and their share of c1; the first
// block of a row also takes q . mean.  A thread has one position and an eighth of the
// sum over D.  Bound by latency: one round of loads of V for few rows.
__global__ void __launch_bounds__(kPrepThreads) window_prep_kernel(const Params kp, const WindowArgs t) {
  __shared__ __align__(16) float qs[256][kRows];
  __shared__ float sums[8][kRows][kPrepCols];
  const int row_blocks = (t.rows + kRows - 1) / kRows;
  const int slot = blockIdx.x / row_blocks, r0 = (blockIdx.x - slot * row_blocks) * kRows;
  const int b = slot / kp.H, h = slot - b * kp.H, beta = kp.basis_of[slot];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nr = min(kRows, t.rows - r0), D = kp.D, r = kp.r;
  const bool uniform = kp.mode == KVC_MODE_UNIFORM;
  grid_dependents_launch();
  {
    const int64_t at = warp < nr ? q_at(t, b, h, r0 + warp) : 0;
    for (int i = lane; i < D; i += 32) qs[i][warp] = warp < nr ? load_q(t, at + i) : 0.f;
  }
  const int j = blockIdx.y * kPrepCols + lane;  // this thread's position
  int width = 0;
  const int k = j < t.NCk ? position_component(kp, beta, j, &width) : -1;
  float coef = 0.f, off = 0.f;
  if (k >= 0) {
    const size_t bk = (size_t)beta * r + k;
    coef = t.scale_log2 * (uniform ? kp.step[bk] : 1.f);
    if (uniform) off = t.scale_log2 * fmaf((float)(1 << (width - 1)), kp.step[bk], kp.lo[bk]);
  }
  __syncthreads();
  float acc[kRows];
#pragma unroll
  for (int g = 0; g < kRows; ++g) acc[g] = 0.f;
  if (k >= 0) {
    const int per = (D + 7) / 8, i0 = warp * per, i1 = min(D, i0 + per);
    const float* V = kp.V + (size_t)beta * D * r + k;
    for (int ib = i0; ib < i1; ib += 16) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = ib + u < i1 ? V[(size_t)(ib + u) * r] : 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        if (ib + u >= i1) break;
        const float4 a = *reinterpret_cast<const float4*>(qs[ib + u]);
        const float4 c = *reinterpret_cast<const float4*>(qs[ib + u] + 4);
        acc[0] = fmaf(v[u], a.x, acc[0]); acc[1] = fmaf(v[u], a.y, acc[1]);
        acc[2] = fmaf(v[u], a.z, acc[2]); acc[3] = fmaf(v[u], a.w, acc[3]);
        acc[4] = fmaf(v[u], c.x, acc[4]); acc[5] = fmaf(v[u], c.y, acc[5]);
        acc[6] = fmaf(v[u], c.z, acc[6]); acc[7] = fmaf(v[u], c.w, acc[7]);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kRows; ++g) sums[warp][g][lane] = acc[g];
  __syncthreads();
  if (warp >= nr) return;
  float u = 0.f;  // row `warp`, position j
#pragma unroll
  for (int x = 0; x < 8; ++x) u += sums[x][warp][lane];
  const size_t row = (size_t)slot * t.rows + r0 + warp;
  if (j < t.NCk) t.w[row * t.NCk + j] = k < 0 ? 0.f : u * coef;
  float c1 = k < 0 ? 0.f : u * off;
  if (uniform) {
    if (blockIdx.y == 0)
      for (int i = lane; i < D; i += 32)
        c1 = fmaf(qs[i][warp], t.scale_log2 * kp.mean[(size_t)beta * D + i], c1);
    c1 = warp_sum(c1);
  }
  if (lane == 0) t.c1[row * t.c1_parts + blockIdx.y] = c1;
}

// Keys with a residual sketch or an outlier stream: the sketch weights
// sqrt(pi/2)/m (S q)_j and the outlier weights q[ch_l], one block per row.
__global__ void __launch_bounds__(kThreads) window_prep_prod_kernel(const Params kp, const WindowArgs t) {
  __shared__ float qs[kProdMaxD];
  const int slot = blockIdx.x / t.rows, row = blockIdx.x - slot * t.rows;
  const int b = slot / kp.H, h = slot - b * kp.H, D = kp.D, nx = t.m + t.n_out;
  const int64_t at = q_at(t, b, h, row);
  for (int i = threadIdx.x; i < D; i += kThreads) qs[i] = load_q(t, at + i);
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

// ---------------------------------------------------------------- scores

// What a block holds of a job's rows, in shared memory: weights [NCk][8], sketch
// and outlier weights [m + n_out][8], offsets, the chunk table of the keys' basis.
struct JobTables {
  float *ws, *wxs, *c1s;
  const float* cbv;
  const uint32_t* kch;
  int nchk;
};

__device__ void load_job(const Params& kp, const WindowArgs& t, int slot, int r0, const JobTables& j) {
  const int nr = min(kRows, t.rows - r0), nx = t.m + t.n_out;
  const size_t row0 = (size_t)slot * t.rows + r0;
  for (int e = threadIdx.x; e < kRows * t.NCk; e += blockDim.x) {
    const int c = e / kRows, g = e - c * kRows;
    j.ws[e] = g < nr ? t.w[(row0 + g) * t.NCk + c] : 0.f;
  }
  for (int e = threadIdx.x; e < kRows * nx; e += blockDim.x) {
    const int c = e / kRows, g = e - c * kRows;
    j.wxs[e] = g < nr ? t.wx[(row0 + g) * nx + c] : 0.f;
  }
  if (threadIdx.x < kRows) {
    float c = 0.f;
    if ((int)threadIdx.x < nr)
      for (int x = 0; x < t.c1_parts; ++x) c += t.c1[(row0 + threadIdx.x) * t.c1_parts + x];
    j.c1s[threadIdx.x] = c;
  }
}

// The scores (times log2 e) of a stored token for the job's rows.
template <int KMODE>
__device__ void score_token(const Params& kp, const WindowArgs& t, const JobTables& j,
                            const unsigned char* row, const __half* side, float (&sc)[kRows]) {
#pragma unroll
  for (int g = 0; g < kRows; ++g) sc[g] = 0.f;
  const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 3);
  const unsigned char* base = row - mis;
  for (int c = 0; c < j.nchk; ++c) {
    const uint32_t ent = j.kch[c];
    const int w = (int)((ent >> 16) & 0xfu);
    const uint2 bits = bits_at(base, mis + (int)(ent & 0xffffu));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t code = chunk_code(bits, w, e);
      const float v = KMODE == KVC_MODE_CODEBOOK ? j.cbv[code] : (float)((int)code - (1 << (w - 1)));
      const float4* wp = reinterpret_cast<const float4*>(j.ws + (8 * c + e) * kRows);
      const float4 a = wp[0], b = wp[1];
      sc[0] = fmaf(a.x, v, sc[0]); sc[1] = fmaf(a.y, v, sc[1]);
      sc[2] = fmaf(a.z, v, sc[2]); sc[3] = fmaf(a.w, v, sc[3]);
      sc[4] = fmaf(b.x, v, sc[4]); sc[5] = fmaf(b.y, v, sc[5]);
      sc[6] = fmaf(b.z, v, sc[6]); sc[7] = fmaf(b.w, v, sc[7]);
    }
  }
  if (KMODE == KVC_MODE_CODEBOOK) {
    const float n = __half2float(side[0]);
#pragma unroll
    for (int g = 0; g < kRows; ++g) sc[g] *= n;
    if (t.m) {  // + ||r|| sum_j w_j (2 bit_j - 1)
      float x[kRows];
#pragma unroll
      for (int g = 0; g < kRows; ++g) x[g] = 0.f;
      for (int i = 0; i < t.m; ++i) {
        const float f = (row[t.kcode + (i >> 3)] >> (i & 7)) & 1u ? 1.f : -1.f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) x[g] = fmaf(j.wxs[i * kRows + g], f, x[g]);
      }
      const float gam = __half2float(side[1]);
#pragma unroll
      for (int g = 0; g < kRows; ++g) sc[g] = fmaf(gam, x[g], sc[g]);
    }
    if (t.n_out) {  // + s sum_l q[ch_l] o8_l
      const int8_t* o8 = reinterpret_cast<const int8_t*>(row + t.kcode + (t.m >> 3));
      float x[kRows];
#pragma unroll
      for (int g = 0; g < kRows; ++g) x[g] = 0.f;
      for (int i = 0; i < t.n_out; ++i) {
        const float v = (float)o8[i];
#pragma unroll
        for (int g = 0; g < kRows; ++g) x[g] = fmaf(j.wxs[(t.m + i) * kRows + g], v, x[g]);
      }
      const float os = __half2float(side[t.knw - 1]);
#pragma unroll
      for (int g = 0; g < kRows; ++g) sc[g] = fmaf(os, x[g], sc[g]);
    }
  }
#pragma unroll
  for (int g = 0; g < kRows; ++g) sc[g] += j.c1s[g];
}

// Tables that a block reads codes by: the centroids, the keys' chunks.
template <int KMODE>
__device__ void load_tables(const Params& kp, int beta, float* cbv, uint32_t* kch, JobTables* j) {
  if (KMODE == KVC_MODE_CODEBOOK)
    for (int i = threadIdx.x; i < kp.cb_levels; i += blockDim.x) cbv[i] = kp.codebook[i];
  if (threadIdx.x < 32) kch[threadIdx.x] = chunk_entry(kp, beta, threadIdx.x);
  __syncthreads();
  j->cbv = cbv;
  j->kch = kch;
  j->nchk = 0;
  while (j->nchk < 32 && (kch[j->nchk] >> 31)) ++j->nchk;
}

// ---------------------------------------------------------------- main

// CUDA cores: a warp takes 32 tokens at a time, a lane scores one of them for the
// job's 8 rows (key weights broadcast from shared memory), then the lanes share
// out the value channels.  Bound by shared-memory reads, four fp32 weights to a
// load.
//
// Dynamic shared memory: ws [NCk][8], wxs [m + n_out][8], per warp ps [32][8];
// merge [4][8][2 + Dv].
template <int KMODE, int VMODE>
__global__ void __launch_bounds__(kThreads)
    window_main_kernel(const Params kp, const Params vp, const WindowArgs t) {
  extern __shared__ __align__(16) float smf[];
  __shared__ uint32_t kch[32], vch[32];
  __shared__ float cbv[256];
  __shared__ float c1s[kRows];
  constexpr bool VU = VMODE == KVC_MODE_UNIFORM;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Dv = t.Dv, stride = 2 + Dv;
  JobTables jt;
  jt.ws = smf;
  jt.wxs = jt.ws + t.NCk * kRows;
  jt.c1s = c1s;
  float* ps = jt.wxs + (t.m + t.n_out) * kRows + warp * 32 * kRows;
  float* merge = jt.wxs + (t.m + t.n_out) * kRows + 4 * 32 * kRows;
  grid_dependency_wait();  // the key weights come from the launch before
  const int64_t run1 = window_run(t, blockIdx.x + 1);
  for (int64_t at = window_run(t, blockIdx.x); at < run1;) {
    const int job = (int)(at / t.tps);
    const int64_t a0 = at - job * t.tps, a1 = min(t.tps, a0 + (run1 - at));
    at += a1 - a0;
    const int slot = job / t.row_tiles, r0 = (job - slot * t.row_tiles) * kRows;
    const int nr = min(kRows, t.rows - r0), b = slot / kp.H;
    const int kbeta = kp.basis_of[slot], vbeta = VU ? vp.basis_of[slot] : 0;
    const int64_t Pk = kp.P[kbeta], Pv = VU ? vp.P[vbeta] : vp.D;
    __syncthreads();  // the last job's tables and partial have been read
    if (VU && tid >= 32 && tid < 64) vch[tid - 32] = chunk_entry(vp, vbeta, tid - 32);
    load_tables<KMODE>(kp, kbeta, cbv, kch, &jt);
    load_job(kp, t, slot, r0, jt);
    __syncthreads();
    const unsigned char* kbase = kp.store + kp.pay_off[slot];
    const __half* kside = reinterpret_cast<const __half*>(kp.store + kp.side_off[slot]);
    const unsigned char* vbase = vp.store + vp.pay_off[slot];
    const __half* vscale = reinterpret_cast<const __half*>(vp.store + vp.side_off[slot]);

    float m[kRows], l[kRows], acc[kRows][8];
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[g][e] = 0.f;
    }
    const Sight sight(t, b);
    const Tiles<kTile> tiles(sight, t.ctx + r0 / t.rep, t.ctx + (r0 + nr - 1) / t.rep);
    const int64_t count = tiles.count();
    const int i1 = (int)(count * a1 / t.tps);
    for (int i = (int)(count * a0 / t.tps); i < i1; ++i) {
      const int tb = tiles.tile(i) * kTile + 32 * warp, tok = tb + lane;
      const int n = min(32, t.S - tb);
      if (n <= 0) continue;
      float sc[kRows], sv = 1.f;  // sv: the value's scale
#pragma unroll
      for (int g = 0; g < kRows; ++g) sc[g] = 0.f;
      if (lane < n) {
        score_token<KMODE>(kp, t, jt, kbase + tok * Pk, kside + (int64_t)tok * t.knw, sc);
        if (!VU) sv = __half2float(vscale[tok]);
      }
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        const bool see = lane < n && g < nr && sight.sees(tok, t.ctx + (r0 + g) / t.rep);
        const float mn = fmaxf(m[g], warp_max(see ? fmaxf(sc[g], kWindowLowest) : -INFINITY));
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing visible yet
        const float corr = exp2f(m[g] - ref);
        const float p = see ? exp2f(sc[g] - ref) : 0.f;
        l[g] = l[g] * corr + warp_sum(p);
        m[g] = mn;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[g][e] *= corr;
        ps[lane * kRows + g] = see ? p * sv : 0.f;
      }
      __syncwarp();
      // lane owns channels lane, lane + 32, ..
      for (int tt = 0; tt < n; ++tt) {
        const unsigned char* row = vbase + (tb + tt) * Pv;
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 3);
        float pv[kRows];
#pragma unroll
        for (int g = 0; g < kRows; ++g) pv[g] = ps[tt * kRows + g];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = lane + 32 * e;
          if (d >= Dv) break;
          float v;
          if (VU) {
            const uint32_t ent = vch[d >> 3];
            if (!ent) continue;  // a basis with fewer positions than another one
            const int w = (int)((ent >> 16) & 0xfu);
            v = (float)((int)chunk_code(bits_at(row - mis, mis + (int)(ent & 0xffffu)), w, d & 7) -
                        (1 << (w - 1)));
          } else {
            v = (float)reinterpret_cast<const int8_t*>(row)[d];
          }
#pragma unroll
          for (int g = 0; g < kRows; ++g) acc[g][e] = fmaf(pv[g], v, acc[g][e]);
        }
      }
      __syncwarp();  // ps is rewritten by the next block
    }
    // the warps' states into one partial
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      float* mg = merge + (warp * kRows + g) * stride;
      if (lane == 0) {
        mg[0] = m[g];
        mg[1] = l[g];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < Dv) mg[2 + lane + 32 * e] = acc[g][e];
    }
    __syncthreads();
    for (int e = tid; e < kRows * stride; e += kThreads) {
      const int d = e / kRows, g = e - d * kRows;
      float M = -INFINITY;
      for (int w = 0; w < 4; ++w) M = fmaxf(M, merge[(w * kRows + g) * stride]);
      float v = d == 0 ? M : 0.f;
      if (d)
        for (int w = 0; w < 4; ++w) {
          const float* mg = merge + (w * kRows + g) * stride;
          // (a warp without tokens has l = 0; one with NaN scores has m = -inf too)
          if (mg[1] != 0.f) v = fmaf(exp2f(mg[0] - M), mg[d], v);
        }
      const size_t part = (size_t)job + blockIdx.x;
      if (d == 0) t.ml[part * kRows + g].x = v;
      else if (d == 1) t.ml[part * kRows + g].y = v;
      else t.part[(part * t.Dvp + d - 2) * kRows + g] = v;
    }
  }
}

// ---------------------------------------------------------------- combine

constexpr int kFactors = 64;

// Join the partials of eight rows, normalise and write the output rows (uniform
// values: project the weighted mean latent), and what the weights' pass needs of
// a row.  Thread (d, q) of a group of 256 holds channel d of rows 4 q .. 4 q + 3; the
// groups share the partials and, of uniform values, the sum over components.  Bound by
// the latency of the partials' reads where few blocks are at work: one sequence of 8
// heads, 38 partials a row 9.9 us with four groups, 12 with one.
template <int GROUPS>
__global__ void __launch_bounds__(256 * GROUPS)
    window_combine_kernel(const Params kp, const Params vp, const WindowArgs t) {
  __shared__ __align__(16) float fac[kFactors][kRows];  // 2^(m - M) of the partials
  __shared__ __align__(16) float zb[256][kRows];        // uniform values: mean latents
  __shared__ short comp[256];                           // component of a packed position
  __shared__ float zs[256], zo[256];                    // its step, its offset
  __shared__ __align__(16) float inv_s[kRows];
  __shared__ float4 gsum[GROUPS > 1 ? GROUPS - 1 : 1][2][256];  // the other groups' sums
  constexpr int kCombineThreads = 256 * GROUPS;
  const int blocks = (t.rows + kRows - 1) / kRows;
  int slot = blockIdx.x / blocks, row0 = (blockIdx.x - slot * blocks) * kRows;
  if (t.cuts) {
    // block (cut, 8 rows): the job that the first run after it begins in; the cuts
    // before it must not lie in the same job
    const int per = t.rt / kRows, cut = 1 + blockIdx.x / per;
    const int64_t at = window_run(t, cut), job = at / t.tps, start = job * t.tps;
    slot = (int)(job / t.row_tiles);
    row0 = (int)(job - (int64_t)slot * t.row_tiles) * t.rt + (blockIdx.x % per) * kRows;
    if (at == start || window_run(t, cut - 1) > start || row0 >= t.rows) {
      grid_dependency_wait();  // (who waits for this launch waits for the one before)
      return;
    }
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = slot / kp.H, h = slot - b * kp.H;
  const bool vu = vp.mode == KVC_MODE_UNIFORM;
  const int beta = vu ? vp.basis_of[slot] : 0;
  const int jt = row0 / t.rt, rr = row0 - jt * t.rt;
  // the CTAs whose runs hold the job's tiles
  const int64_t job = (int64_t)slot * t.row_tiles + jt, lo = job * t.tps;
  const int64_t c0 = window_cta(t, lo), c1 = window_cta(t, lo + t.tps - 1);
  const int splits = (int)(c1 - c0) + 1;
  const size_t p0 = (size_t)window_part(t, job, c0);
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
  const float2* ml = t.ml + p0 * t.rt + rr + (warp & 7);
  const bool live = warp < kRows && row0 + warp < t.rows;  // (the first eight warps)
  float M = -INFINITY, L = 0.f;
  if (live)
    for (int s = lane; s < splits; s += 32) M = fmaxf(M, ml[(size_t)s * t.rt].x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  const int group = tid >> 8, d0 = tid & 127, q = (tid >> 7) & 1;  // d0 and d0 + 128; row quad
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = 0; s0 < splits; s0 += kFactors) {
    const int n = min(kFactors, splits - s0);
    __syncthreads();
    for (int e = lane; warp < kRows && e < n; e += 32) {
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
      const float* p = t.part + ((p0 + s0) * t.Dvp + d) * t.rt + rr + 4 * q;
#pragma unroll 4
      for (int e = group; e < n; e += GROUPS) {
        const float4 v = *reinterpret_cast<const float4*>(p + (size_t)e * t.rt * t.Dvp);
        const float4 f = *reinterpret_cast<const float4*>(&fac[e][4 * q]);
        acc[u].x = fmaf(f.x, v.x, acc[u].x);
        acc[u].y = fmaf(f.y, v.y, acc[u].y);
        acc[u].z = fmaf(f.z, v.z, acc[u].z);
        acc[u].w = fmaf(f.w, v.w, acc[u].w);
      }
    }
  }
  if (GROUPS > 1) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (group) gsum[group - 1][u][tid & 255] = acc[u];
  }
  L = warp_sum(L);
  if (lane == 0 && warp < kRows) {
    // nothing visible: zero; scores of -inf alone: NaN
    const float inv = L > 0.f || L != L ? 1.f / L : M == -INFINITY ? 0.f : NAN;
    inv_s[warp] = inv;
    if (t.stats && live) t.stats[(size_t)slot * t.rows + row0 + warp] = make_float2(ref, inv);
  }
  __syncthreads();
  grid_dependents_launch();
  if (GROUPS > 1 && group == 0)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int x = 0; x < GROUPS - 1; ++x) {
        const float4 v = gsum[x][u][tid];
        acc[u].x += v.x;
        acc[u].y += v.y;
        acc[u].z += v.z;
        acc[u].w += v.w;
      }
  auto put = [&](int d, float4 v) {  // channel d of the thread's four rows
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = row0 + 4 * q + e;
      if (row >= t.rows) break;
      const int n = row / t.rep, g = row - n * t.rep;
      const int64_t o = b * t.o_sb + (int64_t)(h * t.rep + g) * t.o_sh + n * t.o_st + d;
      if (t.out_bf16) reinterpret_cast<__nv_bfloat16*>(t.out)[o] = __float2bfloat16_rn(x[e]);
      else reinterpret_cast<__half*>(t.out)[o] = __float2half_rn(x[e]);
    }
  };
  const float4 inv = *reinterpret_cast<const float4*>(&inv_s[4 * q]);
  if (group == 0)
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
#pragma unroll 1
  for (int i0 = 0; i0 < vp.D; i0 += 128) {
    const int i = i0 + d0;
    const bool in = i < vp.D;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* Vt = vp.Vt + (size_t)beta * vp.r * vp.D + (in ? i : 0);
#pragma unroll 8
    for (int j = group; j < t.Dv; j += GROUPS) {
      const int k = comp[j];
      const float c = k < 0 ? 0.f : Vt[(size_t)k * vp.D];
      const float4 zz = *reinterpret_cast<const float4*>(&zb[j][4 * q]);
      if (k < 0) continue;  // padding: its sums are whatever the codes' padding held
      v.x = fmaf(zz.x, c, v.x);
      v.y = fmaf(zz.y, c, v.y);
      v.z = fmaf(zz.z, c, v.z);
      v.w = fmaf(zz.w, c, v.w);
    }
    if (GROUPS > 1) {
      if (group) gsum[group - 1][0][tid & 255] = v;
      __syncthreads();
      if (group == 0)
#pragma unroll
        for (int x = 0; x < GROUPS - 1; ++x) {
          const float4 y = gsum[x][0][tid];
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
      __syncthreads();  // (the next columns' sums take the place)
    }
    if (group == 0 && in) {
      const float mu = vp.mean[(size_t)beta * vp.D + i];
      auto row = [](float x, float f) { return f == 0.f ? 0.f : f != f ? f : x; };
      put(i, make_float4(row(v.x + mu, inv.x), row(v.y + mu, inv.y), row(v.z + mu, inv.z), row(v.w + mu, inv.w)));
    }
  }
}

// ---------------------------------------------------------------- weights

// The weights that 128 tokens of a slot receive, a thread each: the rows' scores
// again, eight at a time, p = 2^(s - m) / l, added up in row order.
template <int KMODE>
__global__ void __launch_bounds__(kThreads)
    window_weights_kernel(const Params kp, const WindowArgs t) {
  extern __shared__ __align__(16) float smf[];
  __shared__ uint32_t kch[32];
  __shared__ float cbv[256];
  __shared__ float c1s[kRows];
  __shared__ float2 st[kRows];
  const int tiles = (t.S + kTile - 1) / kTile;
  const int tid = threadIdx.x, slot = blockIdx.x / tiles, b = slot / kp.H, h = slot - b * kp.H;
  const int t0 = (blockIdx.x - slot * tiles) * kTile, tok = t0 + tid;
  const int kbeta = kp.basis_of[slot];
  const int64_t Pk = kp.P[kbeta];
  JobTables jt;
  jt.ws = smf;
  jt.wxs = jt.ws + t.NCk * kRows;
  jt.c1s = c1s;
  load_tables<KMODE>(kp, kbeta, cbv, kch, &jt);
  grid_dependency_wait();
  const Sight sight(t, b);
  const unsigned char* row = kp.store + kp.pay_off[slot] + tok * Pk;
  const __half* side = reinterpret_cast<const __half*>(kp.store + kp.side_off[slot]) + (int64_t)tok * t.knw;
  float sum = 0.f;
  for (int r0 = 0; r0 < t.rows; r0 += kRows) {
    const int nr = min(kRows, t.rows - r0);
    const int p0 = t.ctx + r0 / t.rep, p1 = t.ctx + (r0 + nr - 1) / t.rep;
    // tokens that no row of these sees
    if (t0 > p1 || t0 + kTile <= sight.first || (t0 + kTile <= p0 - sight.window + 1 && t0 >= sight.sink_end))
      continue;
    __syncthreads();
    load_job(kp, t, slot, r0, jt);
    if (tid < nr) st[tid] = t.stats[(size_t)slot * t.rows + r0 + tid];
    __syncthreads();
    if (tok >= t.S) continue;
    float sc[kRows];
    score_token<KMODE>(kp, t, jt, row, side, sc);
#pragma unroll
    for (int g = 0; g < kRows; ++g)
      if (g < nr && sight.sees(tok, t.ctx + (r0 + g) / t.rep))
        sum = fmaf(exp2f(sc[g] - st[g].x), st[g].y, sum);
  }
  if (tok >= t.S) return;
  float* w = t.weights + b * t.w_sb + h * t.w_sh + tok;
  if (t.decay == 0.f) *w = sum;
  else if (t.decay != 1.f || sum != 0.f) *w = fmaf(t.decay, *w, sum);
}

using MainKernel = void (*)(const Params, const Params, const WindowArgs);

MainKernel main_kernel_for(int kmode, int vmode) {
  if (kmode == KVC_MODE_UNIFORM)
    return vmode == KVC_MODE_UNIFORM ? window_main_kernel<KVC_MODE_UNIFORM, KVC_MODE_UNIFORM>
                                     : window_main_kernel<KVC_MODE_UNIFORM, KVC_MODE_INT8>;
  return vmode == KVC_MODE_UNIFORM ? window_main_kernel<KVC_MODE_CODEBOOK, KVC_MODE_UNIFORM>
                                   : window_main_kernel<KVC_MODE_CODEBOOK, KVC_MODE_INT8>;
}

// Tiles of `tile` tokens that a job of `rows` rows sees at most.
int64_t most_tiles(const WindowArgs& t, int tile, int rows) {
  const int64_t all = (t.S + tile - 1) / tile;
  const int64_t span = (int64_t)t.window + (rows + t.rep - 1) / t.rep + 1;  // the window's tokens
  return std::min<int64_t>(all, (span + tile - 1) / tile + 1 + (t.sinks ? (t.sinks + tile - 1) / tile + 1 : 0));
}

struct Take {
  unsigned char* at;
  size_t used = 0;
  explicit Take(void* p) : at(static_cast<unsigned char*>(p)) {}
  template <class T>
  T* operator()(size_t n) {
    const size_t bytes = (n * sizeof(T) + 255) / 256 * 256;
    T* p = reinterpret_cast<T*>(at + used);
    used += bytes;
    return p;
  }
};

// The workspace's arrays in t; its bytes.
size_t lay_out(const Params& kp, WindowArgs& t, void* workspace) {
  const size_t rows = (size_t)kp.n_slots * t.rows;
  const size_t parts = t.cuts ? 2 * (size_t)t.grid : (size_t)kp.n_slots * t.row_tiles + t.grid - 1;
  Take take(workspace);
  t.w = take.operator()<float>(t.tc && !t.weights ? 0 : rows * t.NCk);
  t.wx = take.operator()<float>(rows * (t.m + t.n_out));
  t.c1 = take.operator()<float>(rows * t.c1_parts);
  t.ml = take.operator()<float2>(parts * t.rt);
  t.part = take.operator()<float>(parts * t.rt * t.Dvp);
  const size_t jobs = t.tc ? (size_t)kp.n_slots * t.row_tiles : 0;
  t.w16 = take.operator()<uint16_t>(jobs * 2 * t.rt * t.K);
  t.wscale = take.operator()<float>(jobs * t.rt);
  t.stats = t.weights ? take.operator()<float2>(rows) : nullptr;
  t.wpart = take.operator()<float>(t.wsplits > 1 ? (size_t)t.wsplits * kp.n_slots * t.S : 0);
  const size_t scores = (size_t)kp.n_slots * t.tps * kWindowTile * (t.rows <= 4 ? 4 : 8);
  t.scores = t.weights && t.mma && t.rows <= 8 ? take.operator()<float>(scores) : nullptr;
  return take.used;
}

}  // namespace

size_t window_plan(const Params& kp, const Params& vp, WindowArgs& t, bool generic, int sms) {
  t.sms = sms;
  t.mma = t.tc = 0;
  int ctas = 12;  // of an SM: the CUDA cores'
  if (!generic && !t.prod) {
    // Small calls are latency: jobs of eight rows while all of their tiles find a warp
    // twice (15 slots of 21 rows, 500 tokens, 4-bit keys: main kernel 13.9 us, 28.7 in
    // jobs of 32).  Many rows: tcgen05, whose jobs cost the same from one row to 128 (32
    // slots of 36 rows, 4096 tokens: 63 us in all, 72 on the warps' tensor cores; of 128
    // rows 69 and 118).  Weights
    // take scores to fp32's precision, which codebooks have in the other kernel alone.
    t.rt = 8;
    const int64_t tiles8 = (int64_t)kp.n_slots * ((t.rows + 7) / 8) * most_tiles(t, kWindowTile, t.rt);
    const bool small = tiles8 <= 2 * 2 * 8 * (int64_t)sms;
    if (!small && t.rows > kTcRows && t.cb_mul > 0.f && (!t.weights || kp.mode == KVC_MODE_UNIFORM))
      t.K = window_tc_k(kp, vp, t);
    if (t.K) {
      t.tc = 1;
      ctas = 1;
    } else {
      const int nt = small || t.rows <= 8 ? 1 : t.rows <= 16 ? 2 : 4;
      const int n = window_mma_ctas(kp, vp, t, nt);
      if (n) {
        t.mma = nt;
        ctas = n;
      }
    }
  }
  t.rt = t.tc ? 128 : t.mma ? 8 * t.mma : kRows;
  t.row_tiles = (t.rows + t.rt - 1) / t.rt;
  t.Dvp = (t.Dv + 3) / 4 * 4;
  t.c1_parts = (t.NCk + kPrepCols - 1) / kPrepCols;
  const int64_t jobs = (int64_t)kp.n_slots * t.row_tiles;
  t.tps = most_tiles(t, t.mma ? kWindowTile : kTile, t.rt);
  t.total = jobs * t.tps;
  // a warp of the tensor-core kernel takes a tile, of the CUDA cores a quarter; jobs of
  // few tiles have a CTA each all the same
  const int64_t runs = t.mma ? std::max<int64_t>(t.total / 8, jobs) : t.total;
  t.grid = (int)std::min<int64_t>(runs, ctas * (int64_t)sms);
  t.cuts = t.tc && vp.mode != KVC_MODE_UNIFORM;
  t.wsplits = t.weights && (t.mma || t.tc) ? window_weights_splits(kp, t) : 1;
  return lay_out(kp, t, nullptr);
}

cudaError_t launch_attend_window(const Params& kp, const Params& vp, WindowArgs t, void* workspace,
                                 cudaStream_t s, int* nk) {
  lay_out(kp, t, workspace);
  t.wtps = t.decay == 1.f && t.wsplits == 1 ? most_tiles(t, kWindowTile, t.rows)
                                            : (t.S + kWindowTile - 1) / kWindowTile;
  cudaError_t e;
  if (t.prod) {
    window_prep_prod_kernel<<<(unsigned)(kp.n_slots * t.rows), kThreads, 0, s>>>(kp, t);
    ++*nk;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const unsigned row_blocks = (unsigned)(kp.n_slots * ((t.rows + kRows - 1) / kRows));
  // (projection of 64 slots of 128 rows, 32 columns: 9.1 us on the tensor cores, 19.5
  // in fp32; few rows are latency, and the fp32 kernel has more blocks for them)
  if (t.tc || (t.mma && t.rows > 32 && (int64_t)kp.n_slots * t.rows >= 4096 && window_projects(kp, t))) {
    e = launch_window_project(kp, t, s, nk);
  } else {
    window_prep_kernel<<<dim3(row_blocks, (unsigned)t.c1_parts), kPrepThreads, 0, s>>>(kp, t);
    ++*nk;
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const size_t tables = (size_t)kRows * (t.NCk + t.m + t.n_out) * 4;
  if (t.tc) {
    e = launch_window_tc(kp, vp, t, s, nk);
  } else if (t.mma) {
    e = launch_window_mma(kp, vp, t, s, nk);
  } else {
    const size_t smem = tables + 4 * 32 * kRows * 4 + 4 * (size_t)kRows * (2 + t.Dv) * 4;
    const MainKernel k = main_kernel_for(kp.mode, vp.mode);
    e = prepare_kernel(reinterpret_cast<const void*>(k), (int)smem);
    if (e != cudaSuccess) return e;
    ++*nk;
    e = launch_dependent(k, (unsigned)t.grid, kThreads, smem, s, kp, vp, t);
  }
  if (e != cudaSuccess) return e;
  const unsigned combines = t.cuts ? (unsigned)(t.grid - 1) * (unsigned)(t.rt / kRows) : row_blocks;
  if (combines) {
    ++*nk;
    // four groups of threads where a row has many partials (at most total / jobs runs)
    const bool many = (int64_t)t.grid > 6 * (int64_t)kp.n_slots * t.row_tiles;
    e = many ? launch_dependent(window_combine_kernel<4>, combines, 1024u, 0, s, kp, vp, t)
             : launch_dependent(window_combine_kernel<1>, combines, 256u, 0, s, kp, vp, t);
    if (e != cudaSuccess) return e;
  }
  if (!t.weights) return cudaSuccess;
  if (t.mma || t.tc) return launch_window_weights_mma(kp, t, s, nk);
  const auto k = kp.mode == KVC_MODE_UNIFORM ? window_weights_kernel<KVC_MODE_UNIFORM>
                                             : window_weights_kernel<KVC_MODE_CODEBOOK>;
  k<<<(unsigned)kp.n_slots * (unsigned)((t.S + kTile - 1) / kTile), kThreads, tables, s>>>(kp, t);
  ++*nk;
  return cudaGetLastError();
}

}  // namespace kvc
