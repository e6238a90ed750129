// The windowed attention's queries in the keys' basis for many rows: u = V^T q on the
// warps' tensor cores, as fp32 key weights or as the operand of kvc_window_tc.cu.
//
// Both factors are two fp16 pieces of values that powers of two bring into fp16's upper
// range (a row of q by its largest, a column of V by its norm), so three products keep
// 22 bits of what an fp32 sum would; the small ones are summed apart.
//
// A CTA takes runs of 128 rows of a slot, a warp 16 of them with all columns; V lies in
// shared memory, a column's values together, until another basis is needed.  Bound by
// latency: a warp loads, converts, multiplies and stores in turn, so that a second CTA
// on an SM counts for most (8 heads of 8192 rows, 128 x 128, bf16: 28 us, one CTA 45;
// the fp32 product took 225).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kvc_launch.cuh"
#include "kvc_window.cuh"
#include "kvc_window_mma.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 256, kRows = 128;

__device__ __forceinline__ float load_q(const WindowArgs& t, int64_t i) {
  if (t.q_dtype == KVC_F32) return static_cast<const float*>(t.q)[i];
  if (t.q_dtype == KVC_F16) return __half2float(static_cast<const __half*>(t.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(t.q)[i]);
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}
// The largest finite magnitude.
__device__ __forceinline__ float larger(float most, float v) {
  v = fabsf(v);
  return v <= 3.4e38f ? fmaxf(most, v) : most;  // NaN and infinities stay what they are
}

// KD: steps of 16 over the head size.  OPERAND: two fp16 pieces in the layout of a
// K-major operand without swizzle (cores of 8 rows x 8 positions, 128 contiguous bytes,
// adjacent along K), per row a power of two, the only factor from its products to its
// scores, so that these are exact; else fp32 weights.  REST:
// fp32 queries; those of 16 bits have no second piece to speak of.
template <int KD, bool OPERAND, bool REST>
__global__ void __launch_bounds__(kThreads, REST ? 1 : 2) window_project_kernel(const Params kp, const WindowArgs t) {
  constexpr int D = 16 * KD, kStride = D + 8;  // (padding: a step's columns in different banks)
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int comp[128];
  __shared__ float up[128], down[128];  // factor of a column of V; of a weight
  __half* bh = reinterpret_cast<__half*>(smem);  // [column][D]
  __half* bl = bh + t.NCk * kStride;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const bool uniform = kp.mode == KVC_MODE_UNIFORM;
  // pairs of 16-bit queries that lie on word boundaries are loaded as words
  const bool words = t.q_dtype != KVC_F32 && !(reinterpret_cast<uintptr_t>(t.q) & 3) && !((t.q_sb | t.q_sh | t.q_st) & 1);
  grid_dependents_launch();
  const int blocks = (t.rows + kRows - 1) / kRows;
  const int64_t jobs = (int64_t)kp.n_slots * blocks;
  const int job1 = (int)(jobs * (blockIdx.x + 1) / gridDim.x);
  int loaded = -1;  // the basis in shared memory
  for (int job = (int)(jobs * blockIdx.x / gridDim.x); job < job1; ++job) {
    const int slot = job / blocks, r0 = (job - slot * blocks) * kRows;
    const int b = slot / kp.H, h = slot - b * kp.H, beta = kp.basis_of[slot];
    // this lane's rows of q: 16 warp + g and 8 more
    uint32_t ah[KD][4], al[REST ? KD : 1][4];
    float inv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = r0 + 16 * warp + g + 8 * e, n = x / t.rep;
      const bool in = x < t.rows;
      const int64_t at = b * t.q_sb + (int64_t)(h * t.rep + x - n * t.rep) * t.q_sh + n * t.q_st + 2 * c;
      float v[KD][4], most = 0.f;
      if (words) {
        uint32_t w[KD][2];
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __half*>(t.q) + at);
#pragma unroll
        for (int k = 0; k < KD; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u) w[k][u] = in ? q[8 * k + 4 * u] : 0u;
#pragma unroll
        for (int k = 0; k < KD; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float2 f;
            if (t.q_dtype == KVC_F16) f = __half22float2(*reinterpret_cast<const __half2*>(&w[k][u]));
            else f = make_float2(__uint_as_float(w[k][u] << 16), __uint_as_float(w[k][u] & 0xffff0000u));
            v[k][2 * u] = f.x;
            v[k][2 * u + 1] = f.y;
          }
      } else {
#pragma unroll
        for (int k = 0; k < KD; ++k)
#pragma unroll
          for (int u = 0; u < 4; ++u) v[k][u] = in ? load_q(t, at + 16 * k + (u & 1) + 8 * (u >> 1)) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < KD; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u) most = larger(most, v[k][u]);
      const float mul = row_scale(quad_max(most));
      inv[e] = 1.f / mul;
#pragma unroll
      for (int k = 0; k < KD; ++k) {
        const uint4 p = weight_pieces(make_float4(v[k][0], v[k][1], v[k][2], v[k][3]), mul);
        ah[k][e] = p.x; ah[k][2 + e] = p.y;
        if (REST) {
          al[REST ? k : 0][e] = p.z; al[REST ? k : 0][2 + e] = p.w;
        }
      }
    }
    if (beta != loaded) {
      __syncthreads();  // the last basis has been read
      loaded = beta;
      for (int j = tid; j < t.NCk; j += kThreads) {
        int width = 0;
        const int k = position_component(kp, beta, j, &width);
        comp[j] = k;
        float s = 1.f, f = 0.f;
        if (k >= 0) {
          const size_t bk = (size_t)beta * kp.r + k;
          s = row_scale(kp.vnorm[bk]);
          f = t.scale_log2 * (uniform ? kp.step[bk] : 1.f) / s;
          if (OPERAND) f *= t.w_frac;  // (the fraction here, so that a row's factor is a power of two)
        }
        up[j] = s;
        down[j] = f;
      }
      __syncthreads();
      // a warp takes every eighth column, all loads of four of them first
      for (int j0 = warp; j0 < t.NCk; j0 += 32) {
        float2 v[4][D / 64];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = j0 + 8 * q, k = j < t.NCk ? comp[j] : -1;
#pragma unroll
          for (int i = 0; i < D / 64; ++i)
            v[q][i] = k < 0 ? make_float2(0.f, 0.f)
                            : *reinterpret_cast<const float2*>(kp.Vt + ((size_t)beta * kp.r + k) * D + 64 * i + 2 * lane);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = j0 + 8 * q;
          if (j >= t.NCk) break;
          const float s = up[j];
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const __half2 hi = __floats2half2_rn(v[q][i].x * s, v[q][i].y * s);
            const float2 f = __half22float2(hi);
            *reinterpret_cast<__half2*>(bh + j * kStride + 64 * i + 2 * lane) = hi;
            *reinterpret_cast<__half2*>(bl + j * kStride + 64 * i + 2 * lane) =
                __floats2half2_rn(v[q][i].x * s - f.x, v[q][i].y * s - f.y);
          }
        }
      }
      __syncthreads();
    }
    const int tiles = t.NCk / 8;
    float u[16][4], most[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
      if (nt < tiles) {
#pragma unroll
        for (int k = 0; k < KD; ++k) {
          const int at = (8 * nt + g) * kStride + 16 * k + 2 * c;
          const uint32_t h0 = *reinterpret_cast<const uint32_t*>(bh + at), h1 = *reinterpret_cast<const uint32_t*>(bh + at + 8);
          const uint32_t l0 = *reinterpret_cast<const uint32_t*>(bl + at), l1 = *reinterpret_cast<const uint32_t*>(bl + at + 8);
          mma_f16(acc, ah[k], h0, h1);
          mma_f16(small, ah[k], l0, l1);
          if (REST) mma_f16(small, al[REST ? k : 0], h0, h1);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = nt < tiles ? down[(8 * nt + 2 * c + (e & 1)) & 127] : 0.f;
        u[nt][e] = nt < tiles ? (acc[e] + small[e]) * inv[e >> 1] * f : 0.f;
        most[e >> 1] = larger(most[e >> 1], u[nt][e]);
      }
    }
    if (!OPERAND || t.weights) {  // (the weights' pass takes them in fp32)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = r0 + 16 * warp + g + 8 * e;
        if (x >= t.rows) continue;
        float* w = t.w + ((size_t)slot * t.rows + x) * t.NCk + 2 * c;
#pragma unroll
        for (int nt = 0; nt < 16; ++nt)
          if (nt < tiles) *reinterpret_cast<float2*>(w + 8 * nt) = make_float2(u[nt][2 * e], u[nt][2 * e + 1]);
      }
    }
    if (!OPERAND) continue;
    const int KC = t.K / 8;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float mul = row_scale(quad_max(most[e]));
      const int r = 16 * warp + g + 8 * e;
      if (c == 0) t.wscale[(size_t)job * kRows + r] = t.w_pow / mul;
      uint32_t* w = reinterpret_cast<uint32_t*>(t.w16 + (size_t)job * 2 * kRows * t.K) + (r >> 3) * (KC * 32) + (r & 7) * 4 + c;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt)
        if (nt < KC) {
          const uint4 p = weight_pieces(make_float4(u[nt][2 * e], u[nt][2 * e + 1], 0.f, 0.f), mul);
          w[nt * 32] = p.x;
          w[nt * 32 + kRows * t.K / 2] = p.z;
        }
    }
  }
}

}  // namespace

bool window_projects(const Params& kp, const WindowArgs& t) {
  return (kp.D == 64 || kp.D == 128) && t.NCk <= 128;
}

cudaError_t launch_window_project(const Params& kp, const WindowArgs& t, cudaStream_t s, int* nk) {
  const int smem = 2 * t.NCk * (kp.D + 8) * 2;
  const bool operand = t.tc != 0, rest = t.q_dtype == KVC_F32;
  const auto k = kp.D == 64 ? operand ? rest ? window_project_kernel<4, true, true> : window_project_kernel<4, true, false>
                                      : rest ? window_project_kernel<4, false, true> : window_project_kernel<4, false, false>
                 : operand  ? rest ? window_project_kernel<8, true, true> : window_project_kernel<8, true, false>
                            : rest ? window_project_kernel<8, false, true> : window_project_kernel<8, false, false>;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  ++*nk;
  const int64_t jobs = (int64_t)kp.n_slots * ((t.rows + kRows - 1) / kRows);
  k<<<(unsigned)std::min<int64_t>(jobs, (rest ? 1 : 2) * t.sms), kThreads, smem, s>>>(kp, t);
  return cudaGetLastError();
}

}  // namespace kvc
