// The windowed attention's kernel for few rows (the mathematics: kvc_window.cu).
//
// A warp takes 32 tokens at a time and is alone with them: it copies their rows to
// its ring in shared memory, decodes the codes into operand registers, and keeps
// references, sums and weighted sums of its own, which the CTA's warps join at the
// end of a job's run.  Tokens lie on the M side of both products, the job's rows (8
// NT) on the N side, so four rows of a decode step fill half of an instruction:
//   S[token][row]   = A[token][K] W[row][K]^T   A: codes
//   O[channel][row] += V[token][channel]^T P[token][row]
// P goes from the layout of a result to that of an operand by movmatrix.
//
// Scores are exact to fp32's rounding (Keys), codes exact in fp16.  Weights times
// value scales are two fp16 pieces (22 bits; 2^-25 of the reference at least).  The
// reference of a row is its first maximum less 4 and moves only when a score exceeds
// it by 8 (in log2); that of the value scales (sref), the row's own too, is the power of
// two above the largest that it sees and moves when one exceeds it four times.  Their sum
// is one exponent: weights times scales stay below 2^10, and nothing of a row depends on
// what other rows see.  The row's constant c1 cancels in the softmax and is left out.
//
// At most four rows (HALF) fill half of the N side: the other half takes the second
// pieces, the weights' in one product and P's in the other, and sums meet by a shuffle
// or at the end.
//
// What bounds it: the instructions of the decoding, on the four warps that a scheduler
// has at 128 registers a thread.  3-bit keys and int8 values of 128 channels take about
// 400 for 16 tokens of up to eight rows: 128 slots, 4 rows, 16384 tokens in 94 us with
// their scores kept, 54 % of the issue slots used, the ALU pipe busy for 46 % of the time,
// shared memory's for 54, the tensor pipe for 25, and HBM at 53 % of its rate.  A window
// of 4096 of them takes 38, of which the decoding is some 24: the rest is a CTA's start,
// changes of jobs and joins.  Uniform codes of 32 components, 8 slots of 100064 tokens, 29
// (40 packed positions in three steps; in four 31).
// Two CTAs per SM of eight warps for one tile of rows (the weights in registers), one
// for more.
#pragma once

#include "kvc_launch.cuh"
#include "kvc_window.cuh"
#include "kvc_window_mma.cuh"

namespace kvc {

namespace {

constexpr int kMmaWarps = 8, kMmaThreads = kMmaWarps * 32;
constexpr int kMmaTile = kWindowTile, kStages = 2;
constexpr float kSet = 4.f, kMove = 8.f;
constexpr float kScaleLowest = -24.f;  // log2 of the smallest positive value scale

// 2^e of a whole number e.
__device__ __forceinline__ float exp2i(float e) { return __int_as_float(((int)e + 127) << 23); }

// VK: head size of int8 values (64 or 128), 0 for uniform ones (up to 128 positions).
template <int VK>
struct Values {
  static constexpr int kTiles = VK ? VK / 16 : 8;      // tiles of 16 channels
  // Pieces of 16 bytes of a row; piece p of a token lies in place p ^ swizzle, so that
  // eight tokens' equal pieces do not meet in a bank.
  static constexpr int kPieces = VK ? VK / 16 : 1;
  static __device__ int swizzle(int token) { return VK == 128 ? token & 7 : (token >> 1) & 3; }
  static constexpr bool kUniform = VK == 0;
};

template <int KB, int KS, int VK, int NT, bool HALF>
__global__ void __launch_bounds__(kMmaThreads, NT == 1 ? 2 : 1)
    window_mma_kernel(const Params kp, const Params vp, const WindowArgs t, const WindowShape z) {
  constexpr bool PAIRED = NT == 1;
  constexpr int HB = NT == 1 ? 2 : 1;  // halves of a tile (16 tokens) handled at a time
  using K = Keys<KB, KS, PAIRED>;
  using V = Values<VK>;
  constexpr int R = 8 * NT;
  constexpr bool WREG = NT == 1;  // weights in registers, else in shared memory
  constexpr int MT = V::kTiles;
  static_assert(!HALF || NT == 1, "half a tile of rows");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(256) unsigned char table[K::kTable ? K::kTable : 16];  // (at an address known to the compiler)
  __shared__ float row_mul[R], row_inv[R];    // 2^x that a row's weights were multiplied by
  __shared__ float wm[kMmaWarps][R], wl[kMmaWarps][R];
  __shared__ uint32_t vch[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int cr = HALF ? 2 * (c & 1) : 2 * c;  // this lane's rows of a result: cr and cr + 1
  uint4* wfrag = reinterpret_cast<uint4*>(smem);  // [step][NT][32], unless in registers
  unsigned char* ring = smem + z.off_ring + warp * kStages * z.stage;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  if (KB) K::fill(kp, table, kMmaThreads);
  K keys;
  keys.begin(table);
  bool waited = false;

  const int64_t run1 = window_run(t, blockIdx.x + 1);
  for (int64_t at = window_run(t, blockIdx.x); at < run1;) {
    const int job = (int)(at / t.tps);
    const int64_t a0 = at - job * t.tps, a1 = min(t.tps, a0 + (run1 - at));
    at += a1 - a0;
    const int slot = job / t.row_tiles, r0 = (job - slot * t.row_tiles) * R;
    const int nr = min(R, t.rows - r0), b = slot / kp.H;
    const int p0 = t.ctx + r0 / t.rep, p1 = t.ctx + (r0 + nr - 1) / t.rep;
    const Sight sight(t, b);
    const Tiles<kMmaTile> tiles(sight, p0, p1);
    const int64_t count = tiles.count();
    const int i0 = (int)(count * a0 / t.tps), i1 = (int)(count * a1 / t.tps);
    const int kbeta = kp.basis_of[slot], vbeta = V::kUniform ? vp.basis_of[slot] : 0;
    const int Pk = kp.P[kbeta], Pv = V::kUniform ? vp.P[vbeta] : VK;
    const unsigned char* kbase = kp.store + kp.pay_off[slot];
    const unsigned char* kside = kp.store + kp.side_off[slot];
    const unsigned char* vbase = vp.store + vp.pay_off[slot];
    const unsigned char* vside = vp.store + vp.side_off[slot];

    // Copies of the tile numbered i into a stage: whole 16-byte pieces that hold rows.
    // Lanes 0 .. 3 take the keys' side words, 4 .. 7 the values'.
    const unsigned char* klane = kbase + 16 * lane;
    const unsigned char* vlane = vbase + 16 * lane;
    const unsigned char* slane = (lane & 4 ? vside : kside) + 16 * (lane & 3);
    const int sdst = (lane & 4 ? z.off_vside : z.off_kside) + 16 * (lane & 3);
    const bool has_side = lane < 8 && (lane & 4 ? !V::kUniform : KB > 0);
    constexpr int kRow = V::kPieces, kRows32 = 32 / kRow;  // rows that the warp's pieces make
    const int vrow = lane / kRow, vpiece = lane % kRow;
    auto load = [&](int i, int st) {
      if (i < i1) {
        const int t0 = tiles.tile(i) * kMmaTile;
        const uint32_t dst = ring_s + st * z.stage;
        const int n = min(kMmaTile, t.S - t0);
        const unsigned char* ks = klane + (int64_t)t0 * Pk;
        if (KB && n == kMmaTile) {
#pragma unroll
          for (int e = 0; e < 4 * KS * KB; e += 32)
            if (e + 32 <= 4 * KS * KB || lane + e < 4 * KS * KB) copy16(dst + 16 * (lane + e), ks + 16 * e);
        } else {
          for (int e = lane; e < (n * Pk + 15) >> 4; e += 32) copy16(dst + 16 * e, ks + 16 * (e - lane));
        }
        if (has_side && 8 * (lane & 3) < n) copy16(dst + sdst, slane + 2 * (int64_t)t0);  // 2 bytes a token
        if (!V::kUniform) {
          const unsigned char* vs = vlane + (int64_t)t0 * VK;
#pragma unroll
          for (int e = 0; e < kRow; ++e) {
            const int row = vrow + kRows32 * e;
            if (n == kMmaTile || row < n)
              copy16(dst + z.off_v + row * VK + 16 * (vpiece ^ V::swizzle(row)), vs + 512 * e);
          }
        } else {
          const unsigned char* vs = vlane + (int64_t)t0 * Pv;
          for (int e = lane; e < (n * Pv + 15) >> 4; e += 32) copy16(dst + z.off_v + 16 * e, vs + 16 * (e - lane));
        }
      }
      copy_commit();
    };
    __syncthreads();  // the last job's partial and weights have been read
    int i = i0 + warp;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(i + s * kMmaWarps, s);
    if (!waited) grid_dependency_wait();  // the key weights come from the launch before
    waited = true;

    // the rows' weights: scaled, split, in the operand's layout
    const float* w0 = t.w + ((size_t)slot * t.rows + r0) * t.NCk;
    {  // NT rows of a warp, their loads first
      float w[NT][(KS + 1) / 2], most[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int j = 0; j < (KS + 1) / 2; ++j) {
          const int r = warp + u * kMmaWarps, k = lane + 32 * j;
          w[u][j] = r < nr && k < t.NCk ? fabsf(w0[(size_t)r * t.NCk + k]) : 0.f;
        }
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        most[u] = 0.f;
#pragma unroll
        for (int j = 0; j < (KS + 1) / 2; ++j)
          if (w[u][j] <= 3.4e38f) most[u] = fmaxf(most[u], w[u][j]);  // NaN and infinities stay what they are
        most[u] = warp_max(most[u]);
      }
      if (lane == 0)
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const float mul = row_scale(most[u]);
          row_mul[warp + u * kMmaWarps] = mul;
          row_inv[warp + u * kMmaWarps] = 1.f / mul;
        }
    }
    if (V::kUniform && tid < 16) vch[tid] = chunk_entry(vp, vbeta, tid);
    __syncthreads();
    auto fragment = [&](int s, int nt) {
      const int r = HALF ? g & 3 : 8 * nt + g, j = K::position(s, c);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nr && j < t.NCk) w = *reinterpret_cast<const float4*>(w0 + (size_t)r * t.NCk + j);
      return weight_pieces(w, row_mul[r]);
    };
    uint4 wreg[WREG && !HALF ? KS : 1];
    uint2 whalf[HALF ? KS : 1];
    if (HALF) {
#pragma unroll
      for (int s = 0; s < KS; ++s) whalf[HALF ? s : 0] = one_piece(fragment(s, 0), g >= 4);
    } else if (WREG) {
#pragma unroll
      for (int s = 0; s < KS; ++s) wreg[WREG && !HALF ? s : 0] = fragment(s, 0);
    } else {
#pragma unroll
      for (int e0 = 0; e0 < KS * NT; e0 += kMmaWarps)
        if (const int e = e0 + warp; e < KS * NT) wfrag[e * 32 + lane] = fragment(e / NT, e % NT);
      __syncthreads();
    }
    const float tab_inv = KB ? 1.f / K::table_scale(kp) : 1.f;
    float rs[NT][2], negm[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rs[nt][j] = row_inv[8 * nt + cr + j] * tab_inv;
        negm[nt][j] = INFINITY;  // the reference is -inf: nothing seen
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][m][e] = 0.f;
    }
    keys.basis(kp, kbeta, Pk);
    // uniform values: a lane has chunks g and 8 + g of tokens 2 c and 2 c + 1 (and 8 more)
    constexpr int SETS = V::kUniform ? 2 : 1;
    Width vwidth[SETS];
    ChunkPlace vplace[SETS][2];
    bool vwide[SETS];
    const bool two = V::kUniform && vch[8];
    if (V::kUniform)
#pragma unroll
      for (int e = 0; e < SETS; ++e) {
        const uint32_t x = vch[8 * e + g];
        vwidth[e].set(x);
        vwide[e] = __any_sync(kFull, vwidth[e].w == 8);
        vplace[e][0].set(2 * c * Pv + (int)(x & 0xffffu));
        vplace[e][1].set((2 * c + 1) * Pv + (int)(x & 0xffffu));
      }
    // A row's l and o are in units of 2^(score reference + sref), sref (log2) being that of
    // its value scales; negm is minus their sum.  Above high[j] in log2 and above limit a
    // score or a scale may have to move the reference of one of the lane's rows.
    float sref[NT][2], high[2], limit = INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      high[j] = kMove;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sref[nt][j] = V::kUniform ? 0.f : kScaleLowest;
    }
    // tiles that all rows see whole: t0 >= see0 and t0 <= see1, and t0 > see2 or t0 < see3
    const int see0 = sight.first, see1 = p0 - (kMmaTile - 1), see2 = p1 - sight.window,
              see3 = sight.sink_end - (kMmaTile - 1);
    // ldmatrix: this lane's row and piece
    const uint32_t vmat = (uint32_t)((lane & 15) * VK), vflip = (uint32_t)((V::swizzle(lane & 15) ^ (lane >> 4)) * 16);

    int st = 0;
    for (; i < i1; i += kMmaWarps) {
      copy_wait<kStages - 2>();
      __syncwarp();
      const unsigned char* sp = ring + st * z.stage;
      load(i + (kStages - 1) * kMmaWarps, st ^ 1);
      const int t0 = tiles.tile(i) * kMmaTile;
      const bool all = t0 >= see0 && t0 <= see1 && (t0 > see2 || t0 < see3);
#pragma unroll 1
      for (int h0 = 0; h0 < 2; h0 += HB) {  // halves of the tile
        // ---- scores: s[half][rows][e], token 16 half + g + 8 (e >> 1), row cr + (e & 1)
        float s[HB][NT][4];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          const int tok = 16 * (h0 + h) + g;
          const typename K::Row ra = keys.row(sp, 16 * (h0 + h), Pk), rb = keys.row(sp, 16 * (h0 + h) + 8, Pk);
          if constexpr (PAIRED && KB) {
            float d[2][4], small[2][4];  // of tokens g, of tokens g + 8: both pieces of their codes
#pragma unroll
            for (int e = 0; e < 4; ++e) d[0][e] = d[1][e] = small[0][e] = small[1][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t hi[2], lo[2];
                keys.step(q ? rb : ra, k, hi, lo);
                const uint32_t a[4] = {hi[0], lo[0], hi[1], lo[1]};
                if (HALF) {
                  mma_f16(d[q], a, whalf[HALF ? k : 0].x, whalf[HALF ? k : 0].y);
                } else {
                  const uint4 w = wreg[HALF || !WREG ? 0 : k];
                  mma_f16(d[q], a, w.x, w.y);
                  mma_f16(small[q], a, w.z, w.w);
                }
              }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int q = e >> 1, j = e & 1;
              s[h][0][e] = d[q][j] + (HALF ? d[q][2 + j] : d[q][2 + j] + small[q][j] + small[q][2 + j]);
              if (HALF) s[h][0][e] += __shfl_xor_sync(kFull, s[h][0][e], 2);  // the weights' second pieces
            }
          } else {
            float small[NT][4], other[NT][4];  // (sums apart: shorter chains)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[h][nt][e] = small[nt][e] = other[nt][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t ha[2], la[2], hb[2], lb[2];
              keys.step(ra, k, ha, la);
              keys.step(rb, k, hb, lb);
              const uint32_t hi[4] = {ha[0], hb[0], ha[1], hb[1]}, lo[4] = {la[0], lb[0], la[1], lb[1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (HALF) {
                  mma_f16(s[h][nt], hi, whalf[HALF ? k : 0].x, whalf[HALF ? k : 0].y);
                } else {
                  const uint4 w = WREG ? wreg[WREG && !HALF ? k : 0] : wfrag[(k * NT + nt) * 32 + lane];
                  mma_f16(s[h][nt], hi, w.x, w.y);
                  mma_f16(small[nt], hi, w.z, w.w);
                  if (KB) mma_f16(other[nt], lo, w.x, w.y);
                }
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (HALF) s[h][nt][e] += __shfl_xor_sync(kFull, s[h][nt][e], 2);
                else s[h][nt][e] += KB ? small[nt][e] + other[nt][e] : small[nt][e];
              }
          }
          if (KB) {  // norms
            const __half* nm = reinterpret_cast<const __half*>(sp + z.off_kside) + tok;
            const float na = __half2float(nm[0]), nb = __half2float(nm[8]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              s[h][nt][0] *= na; s[h][nt][1] *= na;
              s[h][nt][2] *= nb; s[h][nt][3] *= nb;
            }
          }
        }
        // ---- softmax: x = s rs - m
        float sv[HB][2];  // value scales
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          sv[h][0] = sv[h][1] = 1.f;
          if (!V::kUniform) {
            const __half* vs = reinterpret_cast<const __half*>(sp + z.off_vside) + 16 * (h0 + h) + g;
            sv[h][0] = __half2float(vs[0]);
            sv[h][1] = __half2float(vs[8]);
          }
        }
        if constexpr (NT == 1)
          if (t.scores) {  // kept for the weights' pass: [token][R or 4 rows]
            float* at = t.scores + (((size_t)slot * t.tps + i) * kMmaTile + g) * (HALF ? 4 : 8) + cr;
#pragma unroll
            for (int h = 0; h < HB; ++h) {
              if (HALF) {  // (lanes c and c + 2 hold the same: a token each)
                const bool q = c & 2;
                const float2 y = make_float2((q ? s[h][0][2] : s[h][0][0]) * rs[0][0], (q ? s[h][0][3] : s[h][0][1]) * rs[0][1]);
                *reinterpret_cast<float2*>(at + 4 * (16 * h + 4 * (c & 2))) = y;
              } else {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  *reinterpret_cast<float2*>(at + 8 * (16 * h + 8 * q)) =
                      make_float2(s[h][0][2 * q] * rs[0][0], s[h][0][2 * q + 1] * rs[0][1]);
              }
            }
          }
        uint32_t seen = ~0u;  // bit 4 (h NT + nt) + e
        float x[HB][NT][4];
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[h][nt][e] = fmaf(s[h][nt][e], rs[nt][e & 1], negm[nt][e & 1]);
        if (!all) {
          seen = 0u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = r0 + 8 * nt + cr + j;
              const int pos = t.ctx + r / t.rep;
              if (r < t.rows)
#pragma unroll
                for (int h = 0; h < HB; ++h)
#pragma unroll
                  for (int q = 0; q < 2; ++q)
                    if (sight.sees(t0 + 16 * (h0 + h) + g + 8 * q, pos)) seen |= 1u << (4 * (h * NT + nt) + 2 * q + j);
            }
#pragma unroll
          for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!(seen >> (4 * (h * NT + nt) + e) & 1u)) x[h][nt][e] = -INFINITY;
        }
        float top[2] = {-INFINITY, -INFINITY}, most = 0.f;
#pragma unroll
        for (int h = 0; h < HB; ++h) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            top[0] = max_nan(top[0], x[h][nt][0], x[h][nt][2]);
            top[1] = max_nan(top[1], x[h][nt][1], x[h][nt][3]);
          }
          most = fmaxf(most, fmaxf(sv[h][0], sv[h][1]));
        }
        bool move = !(top[0] <= high[0]) || !(top[1] <= high[1]);
        if (!V::kUniform) move |= most > limit;
        if (__any_sync(kFull, move)) {  // (a row's first token, too: its reference is -inf)
          limit = INFINITY;
          high[0] = high[1] = INFINITY;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // the row's largest visible score and scale (finite)
              float m = -INFINITY, big = 0.f;
#pragma unroll
              for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int e = j; e < 4; e += 2)
                  if (seen >> (4 * (h * NT + nt) + e) & 1u) {
                    m = fmaxf(m, fmaxf(s[h][nt][e] * rs[nt][j], kWindowLowest));
                    if (!V::kUniform && sv[h][e >> 1] <= 65504.f) big = fmaxf(big, sv[h][e >> 1]);
                  }
#pragma unroll
              for (int d = 4; d < 32; d *= 2) {
                m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
                if (!V::kUniform) big = fmaxf(big, __shfl_xor_sync(kFull, big, d));
              }
              const float old = -negm[nt][j], was = sref[nt][j];
              if (!V::kUniform && big > exp2i(was + 2.f))  // the next power of two
                sref[nt][j] = (float)((__float_as_int(big) >> 23) - 126);
              float now = old + (sref[nt][j] - was);
              if (m != -INFINITY && (m - old > kMove - was || !(old > kWindowLowest))) {
                // the first reference, or a new one (the lowest: scores of -inf alone so far)
                now = m > kWindowLowest ? m - kSet + sref[nt][j] : fmaxf(old, m);
                if (m - now > kMove - sref[nt][j]) now = m;  // (past 2^27 fp32 has no such steps)
              }
              const float f = old == now ? 1.f : ex2(old - now);
              l[nt][j] *= f;
#pragma unroll
              for (int q = 0; q < MT; ++q) {
                o[nt][q][j] *= f;
                o[nt][q][2 + j] *= f;
              }
              if (!V::kUniform && now != -INFINITY) limit = fminf(limit, exp2i(sref[nt][j] + 2.f));
              high[j] = fminf(high[j], kMove - sref[nt][j]);
              negm[nt][j] = -now;
#pragma unroll
              for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int e = j; e < 4; e += 2)
                  x[h][nt][e] = seen >> (4 * (h * NT + nt) + e) & 1u ? fmaf(s[h][nt][e], rs[nt][j], -now) : -INFINITY;
            }
        }
        uint32_t ph[HB][NT][2], pl[HB][NT][2];  // P as an operand, in two fp16 pieces
#pragma unroll
        for (int h = 0; h < HB; ++h) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ex2(x[h][nt][e]);
              l[nt][e & 1] += p[e];
              if (!V::kUniform) p[e] *= sv[h][e >> 1];
            }
            if (!V::kUniform && !all) {  // a hidden token's scale may be anything
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!(seen >> (4 * (h * NT + nt) + e) & 1u)) p[e] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const __half2 hi = __floats2half2_rn(p[2 * q], p[2 * q + 1]);
              const float2 back = __half22float2(hi);
              const uint32_t large = *reinterpret_cast<const uint32_t*>(&hi);
              const uint32_t rest = pack_f16(p[2 * q] - back.x, p[2 * q + 1] - back.y);
              if (HALF) {
                ph[h][nt][q] = transpose8(c < 2 ? large : rest);
              } else {
                ph[h][nt][q] = transpose8(large);
                pl[h][nt][q] = transpose8(rest);
              }
            }
          }
        }
        // ---- values: tokens 2 c, 2 c + 1 and 8 more of a half are this lane's K indices
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          auto product = [&](int m, const uint32_t (&a)[4]) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(o[nt][m], a, ph[h][nt][0], ph[h][nt][1]);
              if (!HALF) mma_f16(o[nt][m], a, pl[h][nt][0], pl[h][nt][1]);
            }
          };
          if constexpr (!V::kUniform) {
            // two bytes of a token make a 16-bit element: its low bytes are rows g of a
            // tile of 16 channels, its high bytes rows g + 8
            const uint32_t va0 = ring_s + st * z.stage + z.off_v + vmat + 16 * (h0 + h) * VK;
#pragma unroll
            for (int q = 0; q < VK / 32; ++q) {
              uint32_t v[4];
              load_transposed(v, va0 + (vflip ^ (32 * q)));
              const uint32_t a0[4] = {int8_f16(v[0]), int8_f16(v[0] >> 8), int8_f16(v[1]), int8_f16(v[1] >> 8)};
              product(2 * q, a0);
              const uint32_t a1[4] = {int8_f16(v[2]), int8_f16(v[2] >> 8), int8_f16(v[3]), int8_f16(v[3] >> 8)};
              product(2 * q + 1, a1);
            }
          } else {
            const unsigned char* vr = sp + z.off_v + 16 * (h0 + h) * Pv;
#pragma unroll
            for (int e = 0; e < SETS; ++e) {
              if (e && !two) break;
              uint2 v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                v[q] = vwidth[e].split(vplace[e][q & 1].read(vr + (q >> 1) * 8 * Pv, vwide[e]));
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                uint32_t a[4];
                vwidth[e].both(v[0], v[1], m, &a[0], &a[1]);
                vwidth[e].both(v[2], v[3], m, &a[2], &a[3]);
                product(4 * e + m, a);
              }
            }
          }
        }
      }
      st ^= 1;
    }
    copy_wait<0>();

    // ---- the warps' states into one partial
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = l[nt][j];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        if (g == 0 && (!HALF || c < 2)) {
          wm[warp][8 * nt + cr + j] = -negm[nt][j];
          wl[warp][8 * nt + cr + j] = v;
        }
      }
    __syncthreads();
    const size_t part = (size_t)job + blockIdx.x;
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * nt + cr + j;
        float M = -INFINITY;
        for (int w = 0; w < kMmaWarps; ++w) M = fmaxf(M, wm[w][r]);
        // (a warp that summed nothing has l = 0)
        f[nt][j] = wl[warp][r] == 0.f ? 0.f : ex2(wm[warp][r] - M);
      }
    if (tid < (HALF ? 4 : R)) {
      float M = -INFINITY, L = 0.f;
      for (int w = 0; w < kMmaWarps; ++w) M = fmaxf(M, wm[w][tid]);
      for (int w = 0; w < kMmaWarps; ++w)
        if (wl[w][tid] != 0.f) L = fmaf(ex2(wm[w][tid] - M), wl[w][tid], L);
      t.ml[part * R + tid] = make_float2(M, L);
    }
    // [warp][channel][8] in the ring's place
    float* ob = reinterpret_cast<float*>(smem + z.off_ring);
    constexpr int OW = MT * 16 * 8;
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();
#pragma unroll
      for (int n2 = 0; n2 < NT; ++n2)
        if (n2 == nt)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // channel of row g + 8 (e >> 1) of tile m
              const int d = VK ? 16 * m + 2 * g + (e >> 1)
                               : 8 * (8 * (m >> 2) + g) + 2 * (m & 3) + (e >> 1);
              ob[warp * OW + d * 8 + 2 * c + (e & 1)] = o[n2][m][e] * f[n2][e & 1];
            }
      __syncthreads();
      for (int e = tid; e < t.Dv * 8; e += kMmaThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) v += ob[w * OW + e];
        if (HALF) {
          if (e & 4) continue;
#pragma unroll
          for (int w = 0; w < kMmaWarps; ++w) v += ob[w * OW + e + 4];
        }
        t.part[(part * t.Dvp + (e >> 3)) * R + 8 * nt + (e & 7)] = v;
      }
    }
  }
  grid_dependents_launch();
}

template <int KB, int KS, int NT, bool HALF>
WindowKernel mma_kernel_for_values(bool uniform, int D) {
  if (uniform) return window_mma_kernel<KB, KS, 0, NT, HALF>;
  if constexpr (KB == 0 || KS == 4)
    if (D == 64) return window_mma_kernel<KB, KS, 64, NT, HALF>;
  if constexpr (KB == 0 || KS == 8)
    if (D == 128) return window_mma_kernel<KB, KS, 128, NT, HALF>;
  return nullptr;
}

// The kernel for these layers, null where there is none, and the bytes of its table
// and weights in shared memory.
template <int NT, bool HALF>
WindowKernel mma_kernel_for(const Params& kp, const Params& vp, int NCk, int* tables) {
  const bool vu = vp.mode == KVC_MODE_UNIFORM;
  const int D = kp.D;
  auto of = [&](auto keys, WindowKernel k) {
    using K = decltype(keys);
    *tables = NT == 1 ? 0 : K::kSteps * NT * 512;
    return k;
  };
  if (kp.mode == KVC_MODE_UNIFORM) {
    if (NCk <= 32) return of(Keys<0, 2, NT == 1>{}, mma_kernel_for_values<0, 2, NT, HALF>(vu, D));
    if (NCk <= 48) return of(Keys<0, 3, NT == 1>{}, mma_kernel_for_values<0, 3, NT, HALF>(vu, D));
    if (NCk <= 64) return of(Keys<0, 4, NT == 1>{}, mma_kernel_for_values<0, 4, NT, HALF>(vu, D));
    if (NCk <= 128) return of(Keys<0, 8, NT == 1>{}, mma_kernel_for_values<0, 8, NT, HALF>(vu, D));
    return nullptr;
  }
  switch (kp.cb_bits * 1000 + D) {
    case 2064: return of(Keys<2, 4, NT == 1>{}, mma_kernel_for_values<2, 4, NT, HALF>(vu, D));
    case 3064: return of(Keys<3, 4, NT == 1>{}, mma_kernel_for_values<3, 4, NT, HALF>(vu, D));
    case 4064: return of(Keys<4, 4, NT == 1>{}, mma_kernel_for_values<4, 4, NT, HALF>(vu, D));
    case 2128: return of(Keys<2, 8, NT == 1>{}, mma_kernel_for_values<2, 8, NT, HALF>(vu, D));
    case 3128: return of(Keys<3, 8, NT == 1>{}, mma_kernel_for_values<3, 8, NT, HALF>(vu, D));
    case 4128: return of(Keys<4, 8, NT == 1>{}, mma_kernel_for_values<4, 8, NT, HALF>(vu, D));
    default: return nullptr;
  }
}

}  // namespace

}  // namespace kvc
