// The windowed attention's kernel for few rows (the mathematics: kvc_window.cu).
//
// A warp takes 16 tokens at a time and is alone with them: it copies their rows to
// its ring in shared memory, decodes the codes into operand registers, and keeps
// references, sums and weighted sums of its own, which the CTA's warps join at the
// end of a job's run.  Tokens lie on the M side of both products, the job's rows (8
// NT) on the N side, so four rows of a decode step fill half of an instruction:
//   S[token][row]   = A[token][K] W[row][K]^T   A: codes
//   O[channel][row] += V[token][channel]^T P[token][row]
// P goes from the layout of a result to that of an operand by movmatrix.
//
// Scores are exact to fp32's rounding (Keys); weights are bf16 pairs (16 bits at
// least, fp32's range, so no value scale can overflow them); codes are exact.
// The reference of a row moves only when a score exceeds it by 60 (in log2): bf16
// and fp32 hold weights up to 2^127.  The row's constant c1 cancels in the softmax
// and is left out.
//
// What bounds it: see window_mma_rows().
#pragma once

#include "kvc_launch.cuh"
#include "kvc_window.cuh"
#include "kvc_window_mma.cuh"

namespace kvc {

namespace {

constexpr int kMmaWarps = 8, kMmaThreads = kMmaWarps * 32;
constexpr int kMmaTile = kWindowTile, kStages = 3;
constexpr float kMove = 60.f;

// VK: head size of int8 values (64 or 128), 0 for uniform ones (up to 128 positions).
template <int VK>
struct Values {
  static constexpr int kBytes = VK / 8;                // a lane's bytes of an int8 row
  static constexpr int kTiles = VK ? VK / 16 : 8;      // tiles of 16 channels
  static constexpr int kStride = VK + 16;              // rows in shared memory, no bank conflicts
  static constexpr bool kUniform = VK == 0;
};

template <int KB, int KS, int VK, int NT>
__global__ void __launch_bounds__(kMmaThreads, NT == 1 ? 2 : 1)
    window_mma_kernel(const Params kp, const Params vp, const WindowArgs t, const WindowShape z) {
  using K = Keys<KB, KS>;
  using V = Values<VK>;
  constexpr int R = 8 * NT;
  constexpr bool WREG = NT == 1;  // weights in registers, else in shared memory
  constexpr int MT = V::kTiles;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float row_mul[R], row_inv[R];    // 2^x that a row's weights were multiplied by
  __shared__ float wm[kMmaWarps][R], wl[kMmaWarps][R];
  __shared__ uint32_t vch[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  unsigned char* table = smem;
  uint4* wfrag = reinterpret_cast<uint4*>(smem + K::kTable);  // [step][NT][32], unless in registers
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

    // copies of the tile numbered i into a stage: whole 16-byte pieces that hold rows
    auto load = [&](int i, int st) {
      if (i < i1) {
        const int64_t t0 = (int64_t)tiles.tile(i) * kMmaTile;
        const int n = (int)min((int64_t)kMmaTile, t.S - t0);
        const uint32_t dst = ring_s + st * z.stage;
        const unsigned char* src = kbase + t0 * Pk;
        for (int e = lane; e < (n * Pk + 15) >> 4; e += 32) copy16(dst + 16 * e, src + 16 * e);
        const int words = (2 * n + 15) >> 4;  // side words: 2 bytes a token
        if (KB && lane < words) copy16(dst + z.off_kside + 16 * lane, kside + 2 * t0 + 16 * lane);
        if (!V::kUniform) {
          if (lane >= 2 && lane - 2 < words)
            copy16(dst + z.off_vside + 16 * (lane - 2), vside + 2 * t0 + 16 * (lane - 2));
          constexpr int kRow = VK ? VK / 16 : 1;  // pieces of a row
          const unsigned char* vs = vbase + t0 * VK;
#pragma unroll
          for (int e = 0; e < kRow / 2; ++e) {
            const int x = lane + 32 * e, row = x / kRow, piece = x - row * kRow;
            if (row < n) copy16(dst + z.off_v + row * V::kStride + 16 * piece, vs + 16 * x);
          }
        } else {
          const unsigned char* vs = vbase + t0 * Pv;
          for (int e = lane; e < (n * Pv + 15) >> 4; e += 32) copy16(dst + z.off_v + 16 * e, vs + 16 * e);
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
    for (int r = warp; r < R; r += kMmaWarps) {
      float most = 0.f;
      if (r < nr)
        for (int j = lane; j < t.NCk; j += 32) {
          const float w = fabsf(w0[(size_t)r * t.NCk + j]);
          if (w <= 3.4e38f) most = fmaxf(most, w);  // NaN and infinities stay what they are
        }
      const float mul = row_scale(warp_max(most));
      if (lane == 0) {
        row_mul[r] = mul;
        row_inv[r] = 1.f / mul;
      }
    }
    if (V::kUniform && tid < 16) vch[tid] = chunk_entry(vp, vbeta, tid);
    __syncthreads();
    auto fragment = [&](int s, int nt) {
      const int r = 8 * nt + g, j = K::position(s, c);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nr && j < t.NCk) w = *reinterpret_cast<const float4*>(w0 + (size_t)r * t.NCk + j);
      return weight_pieces(w, row_mul[r]);
    };
    uint4 wreg[WREG ? KS : 1];
    if (WREG) {
#pragma unroll
      for (int s = 0; s < KS; ++s) wreg[WREG ? s : 0] = fragment(s, 0);
    } else {
      for (int e = warp; e < KS * NT; e += kMmaWarps) wfrag[e * 32 + lane] = fragment(e / NT, e % NT);
      __syncthreads();
    }
    const float tab_inv = KB ? 1.f / K::table_scale(kp) : 1.f;
    float rs[NT][2], negm[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rs[nt][j] = row_inv[8 * nt + 2 * c + j] * tab_inv;
        negm[nt][j] = INFINITY;  // the reference is -inf: nothing seen
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][m][e] = 0.f;
    }
    keys.basis(kp, kbeta);
    uint32_t vent[V::kUniform ? 2 : 1];
    if (V::kUniform) {
      vent[0] = vch[g];
      vent[V::kUniform ? 1 : 0] = vch[8 + g];
    }

    int st = 0;
    for (; i < i1; i += kMmaWarps) {
      copy_wait<kStages - 2>();
      __syncwarp();
      const unsigned char* sp = ring + st * z.stage;
      {
        int to = st + kStages - 1;
        if (to >= kStages) to -= kStages;
        load(i + (kStages - 1) * kMmaWarps, to);
      }
      // ---- scores
      float s[NT][4];
      {
        const typename K::Row ra = keys.row(sp, g, Pk), rb = keys.row(sp, g + 8, Pk);
        float small[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = small[nt][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t ha[2], la[2], hb[2], lb[2];
          keys.step(ra, k, ha, la);
          keys.step(rb, k, hb, lb);
          const uint32_t hi[4] = {ha[0], hb[0], ha[1], hb[1]}, lo[4] = {la[0], lb[0], la[1], lb[1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 w = WREG ? wreg[WREG ? k : 0] : wfrag[(k * NT + nt) * 32 + lane];
            mma_f16(s[nt], hi, w.x, w.y);
            mma_f16(small[nt], hi, w.z, w.w);
            if (KB) mma_f16(small[nt], lo, w.x, w.y);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] += small[nt][e];
      }
      if (KB) {  // norms
        const __half* nm = reinterpret_cast<const __half*>(sp + z.off_kside);
        const float na = __half2float(nm[g]), nb = __half2float(nm[g + 8]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] *= na; s[nt][1] *= na;
          s[nt][2] *= nb; s[nt][3] *= nb;
        }
      }
      // ---- softmax: x = s rs - m
      const int t0 = tiles.tile(i) * kMmaTile;
      const bool all = sight.all(t0, t0 + kMmaTile - 1, p0, p1);
      uint32_t seen = ~0u;  // bit 4 nt + e
      if (!all) {
        seen = 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = r0 + 8 * nt + 2 * c + j;
            const int pos = t.ctx + r / t.rep;
            if (r < t.rows) {
              if (sight.sees(t0 + g, pos)) seen |= 1u << (4 * nt + j);
              if (sight.sees(t0 + g + 8, pos)) seen |= 1u << (4 * nt + 2 + j);
            }
          }
      }
      float x[NT][4];
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = fmaf(s[nt][e], rs[nt][e & 1], negm[nt][e & 1]);
          x[nt][e] = all || (seen >> (4 * nt + e) & 1u) ? v : -INFINITY;
          move |= !(x[nt][e] <= kMove);
        }
      if (__any_sync(kFull, move)) {  // (a row's first token, too: its reference is -inf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float va = s[nt][j] * rs[nt][j], vb = s[nt][2 + j] * rs[nt][j];
            const bool sa = seen >> (4 * nt + j) & 1u, sb = seen >> (4 * nt + 2 + j) & 1u;
            float m = fmaxf(sa ? fmaxf(va, kWindowLowest) : -INFINITY, sb ? fmaxf(vb, kWindowLowest) : -INFINITY);
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            const float old = -negm[nt][j], now = fmaxf(old, m);
            const float f = now == -INFINITY ? 1.f : ex2(old - now);
            l[nt][j] *= f;
#pragma unroll
            for (int q = 0; q < MT; ++q) {
              o[nt][q][j] *= f;
              o[nt][q][2 + j] *= f;
            }
            negm[nt][j] = -now;
            x[nt][j] = sa ? fmaf(s[nt][j], rs[nt][j], -now) : -INFINITY;
            x[nt][2 + j] = sb ? fmaf(s[nt][2 + j], rs[nt][j], -now) : -INFINITY;
          }
      }
      uint32_t ph[NT][2], pl[NT][2];  // P as an operand, in two bf16 pieces
      {
        float va = 1.f, vb = 1.f;
        if (!V::kUniform) {
          const __half* vs = reinterpret_cast<const __half*>(sp + z.off_vside);
          va = __half2float(vs[g]);
          vb = __half2float(vs[g + 8]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(x[nt][e]);
            l[nt][e & 1] += p[e];
            if (!V::kUniform) p[e] *= e < 2 ? va : vb;
            // a hidden token's scale may be anything
            if (!V::kUniform && !all && !(seen >> (4 * nt + e) & 1u)) p[e] = 0.f;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t hi = pack_bf16(p[2 * h], p[2 * h + 1]);
            const uint32_t lo = pack_bf16(p[2 * h] - __uint_as_float(hi << 16),
                                          p[2 * h + 1] - __uint_as_float(hi & 0xffff0000u));
            ph[nt][h] = transpose8(hi);
            pl[nt][h] = transpose8(lo);
          }
        }
      }
      // ---- values: tokens 2 c, 2 c + 1 and 8 more are this lane's K indices
      auto product = [&](int m, const uint32_t (&a)[4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16(o[nt][m], a, ph[nt][0], ph[nt][1]);
          mma_bf16(o[nt][m], a, pl[nt][0], pl[nt][1]);
        }
      };
      const unsigned char* vr = sp + z.off_v;
      if constexpr (!V::kUniform) {
        constexpr int W = VK ? V::kBytes / 4 : 1;
        uint32_t v[4][W];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const unsigned char* p = vr + (2 * c + (q & 1) + 8 * (q >> 1)) * V::kStride + g * V::kBytes;
          if (W == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(p);
            v[q][0] = y.x; v[q][1 % W] = y.y; v[q][2 % W] = y.z; v[q][3 % W] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(p);
            v[q][0] = y.x; v[q][1 % W] = y.y;
          }
        }
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const uint32_t a01[4] = {int8_bf16(bytes_of<0>(v[0][q], v[1][q])), int8_bf16(bytes_of<1>(v[0][q], v[1][q])),
                                   int8_bf16(bytes_of<0>(v[2][q], v[3][q])), int8_bf16(bytes_of<1>(v[2][q], v[3][q]))};
          product(2 * q, a01);
          const uint32_t a23[4] = {int8_bf16(bytes_of<2>(v[0][q], v[1][q])), int8_bf16(bytes_of<3>(v[0][q], v[1][q])),
                                   int8_bf16(bytes_of<2>(v[2][q], v[3][q])), int8_bf16(bytes_of<3>(v[2][q], v[3][q]))};
          product(2 * q + 1, a23);
        }
      } else {
#pragma unroll
        for (int set = 0; set < 2; ++set) {
          if (!vch[8 * set]) break;  // (the same for all lanes)
          const uint32_t e = vent[V::kUniform ? set : 0];
          uint2 v[4];
          const int w = e ? (int)((e >> 16) & 0xfu) : 1;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = e ? bits_at(vr, (2 * c + (q & 1) + 8 * (q >> 1)) * Pv + (int)(e & 0xffffu)) : make_uint2(0u, 0u);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t a[4] = {centred_bf16(v[0], v[1], w, 2 * m), centred_bf16(v[0], v[1], w, 2 * m + 1),
                                   centred_bf16(v[2], v[3], w, 2 * m), centred_bf16(v[2], v[3], w, 2 * m + 1)};
            product(4 * set + m, a);
          }
        }
      }
      if (++st == kStages) st = 0;
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
        if (g == 0) {
          wm[warp][8 * nt + 2 * c + j] = -negm[nt][j];
          wl[warp][8 * nt + 2 * c + j] = v;
        }
      }
    __syncthreads();
    const size_t part = (size_t)job + blockIdx.x;
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * nt + 2 * c + j;
        float M = -INFINITY;
        for (int w = 0; w < kMmaWarps; ++w) M = fmaxf(M, wm[w][r]);
        // (a warp that summed nothing has l = 0)
        f[nt][j] = wl[warp][r] == 0.f ? 0.f : ex2(wm[warp][r] - M);
      }
    if (tid < R) {
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
              const int d = VK ? g * V::kBytes + 2 * m + (e >> 1)
                               : 8 * (8 * (m >> 2) + g) + 2 * (m & 3) + (e >> 1);
              ob[warp * OW + d * 8 + 2 * c + (e & 1)] = o[n2][m][e] * f[n2][e & 1];
            }
      __syncthreads();
      for (int e = tid; e < t.Dv * 8; e += kMmaThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) v += ob[w * OW + e];
        t.part[(part * t.Dvp + (e >> 3)) * R + 8 * nt + (e & 7)] = v;
      }
    }
  }
  grid_dependents_launch();
}

template <int KB, int KS, int NT>
WindowKernel mma_kernel_for_values(bool uniform, int D) {
  if (uniform) return window_mma_kernel<KB, KS, 0, NT>;
  if constexpr (KB == 0 || KS == 4)
    if (D == 64) return window_mma_kernel<KB, KS, 64, NT>;
  if constexpr (KB == 0 || KS == 8)
    if (D == 128) return window_mma_kernel<KB, KS, 128, NT>;
  return nullptr;
}

// The kernel for these layers, null where there is none, and the bytes of its table
// and weights in shared memory.
template <int NT>
WindowKernel mma_kernel_for(const Params& kp, const Params& vp, int NCk, int* tables) {
  const bool vu = vp.mode == KVC_MODE_UNIFORM;
  const int D = kp.D;
  auto of = [&](auto keys, WindowKernel k) {
    using K = decltype(keys);
    *tables = K::kTable + (NT == 1 ? 0 : K::kSteps * NT * 512);
    return k;
  };
  if (kp.mode == KVC_MODE_UNIFORM) {
    if (NCk <= 64) return of(Keys<0, 4>{}, mma_kernel_for_values<0, 4, NT>(vu, D));
    if (NCk <= 128) return of(Keys<0, 8>{}, mma_kernel_for_values<0, 8, NT>(vu, D));
    return nullptr;
  }
  switch (kp.cb_bits * 1000 + D) {
    case 2064: return of(Keys<2, 4>{}, mma_kernel_for_values<2, 4, NT>(vu, D));
    case 3064: return of(Keys<3, 4>{}, mma_kernel_for_values<3, 4, NT>(vu, D));
    case 4064: return of(Keys<4, 4>{}, mma_kernel_for_values<4, 4, NT>(vu, D));
    case 2128: return of(Keys<2, 8>{}, mma_kernel_for_values<2, 8, NT>(vu, D));
    case 3128: return of(Keys<3, 8>{}, mma_kernel_for_values<3, 8, NT>(vu, D));
    case 4128: return of(Keys<4, 8>{}, mma_kernel_for_values<4, 8, NT>(vu, D));
    default: return nullptr;
  }
}

}  // namespace

}  // namespace kvc
