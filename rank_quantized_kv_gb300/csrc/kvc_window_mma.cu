// The windowed attention's warp-level tensor-core kernels: their choice and launch,
// and the kernel for the weights that the tokens receive.
#include <algorithm>

#include "kvc_launch.cuh"
#include "kvc_window.cuh"
#include "kvc_window_mma.cuh"

namespace kvc {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32, kTile = kWindowTile, kStages = 2;
constexpr int kManyWarps = 16;   // of the weights' kernel for many rows: one CTA per SM
constexpr int kChunkTiles = 16;  // 8-row tiles whose weights are in shared memory at a time

// The weights that the tokens of a slot receive: the scores again, p = 2^(s - m) / l.
// A warp decodes the keys of 16 tokens at a time into operand registers once and meets all rows
// of a chunk with them, whose weights lie in shared memory; a token's sums stay in two
// registers of four lanes.  CTAs take runs of the slots' tiles.  Where there are more
// rows than a chunk the keys are decoded again for the next one, by the same warp, which
// then adds to what it wrote.  Bound by its products and exponentials: 64 slots, 128 rows,
// 4096 tokens of 32 components 50 us (40 positions in three steps; in four 54), of which
// the exponentials alone would take 7.
template <int KB, int KS>
__global__ void __launch_bounds__(kManyWarps * 32, 1)
    window_weights_mma_kernel(const Params kp, const WindowArgs t, const WindowShape z) {
  using K = Keys<KB, KS, false>;
  constexpr int NT = kChunkTiles, WARPS = kManyWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(256) unsigned char table[K::kTable ? K::kTable : 16];
  __shared__ __align__(16) float4 rowc[8 * NT];  // per row: score factor, -m, 1 / l, position
  __shared__ float row_mul[8 * NT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int cr = 2 * c;
  uint4* wfrag = reinterpret_cast<uint4*>(smem);  // [NT][step][32]
  unsigned char* ring = smem + z.off_ring + warp * kStages * z.stage;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  if (KB) K::fill(kp, table, WARPS * 32);
  K keys;
  keys.begin(table);
  // the tiles that some row sees; all of them where the old weights are scaled
  const bool every = t.decay != 1.f || t.wsplits > 1;
  const int64_t tps = t.wtps, total = tps * kp.n_slots;
  const int ctas = gridDim.x / t.wsplits, share = blockIdx.x / ctas, cta = blockIdx.x - share * ctas;
  const int chunks = (t.rows + 8 * NT - 1) / (8 * NT);
  const int row0 = (int)((int64_t)chunks * share / t.wsplits) * 8 * NT;
  const int row1 = min(t.rows, (int)((int64_t)chunks * (share + 1) / t.wsplits) * 8 * NT);
  const int64_t run1 = total * (cta + 1) / ctas;
  bool waited = false;
  for (int64_t at = total * cta / ctas; at < run1;) {
    const int slot = (int)(at / tps);
    const int64_t a0 = at - slot * tps, a1 = min(tps, a0 + (run1 - at));
    at += a1 - a0;
    const int b = slot / kp.H, h = slot - b * kp.H, kbeta = kp.basis_of[slot], Pk = kp.P[kbeta];
    const unsigned char* kbase = kp.store + kp.pay_off[slot];
    const unsigned char* kside = kp.store + kp.side_off[slot];
    float* wout = t.wsplits > 1 ? t.wpart + ((size_t)share * kp.n_slots + slot) * t.S : t.weights + b * t.w_sb + h * t.w_sh;
    const Sight sight(t, b);
    const Tiles<kTile> tiles_seen(sight, t.ctx, t.S - 1);
    const int64_t count = every ? tps : tiles_seen.count();
    const int i0 = (int)(count * a0 / tps), i1 = (int)(count * a1 / tps);
    auto tile_of = [&](int i) { return every ? i : tiles_seen.tile(i); };
    keys.basis(kp, kbeta, Pk);
    for (int r0 = row0; r0 < row1; r0 += 8 * NT) {
      const int nr = min(8 * NT, row1 - r0), tiles = (nr + 7) / 8;
      const int p0 = t.ctx + r0 / t.rep, p1 = t.ctx + (r0 + nr - 1) / t.rep;
      const float decay = r0 > row0 ? 1.f : t.wsplits > 1 ? 0.f : t.decay;
      // tiles that no row of the chunk sees, and those that all see whole
      const int last = p1, hidden = sight.first - kTile, gap0 = sight.sink_end, gap1 = p0 - sight.window + 1 - kTile;
      const int see0 = sight.first, see1 = p0 - (kTile - 1), see2 = p1 - sight.window,
                see3 = sight.sink_end - (kTile - 1);
      const unsigned char* klane = kbase + 16 * lane;
      auto load = [&](int i, int st) {
        if (i < i1) {
          const int t0 = tile_of(i) * kTile, n = min(kTile, t.S - t0);
          const uint32_t dst = ring_s + st * z.stage + 16 * lane;
          const unsigned char* ks = klane + (int64_t)t0 * Pk;
          if (KB && n == kTile) {
#pragma unroll
            for (int e = 0; e < 4 * KS * KB; e += 32)
              if (e + 32 <= 4 * KS * KB || lane + e < 4 * KS * KB) copy16(dst + 16 * e, ks + 16 * e);
          } else {
            for (int e = lane; e < (n * Pk + 15) >> 4; e += 32) copy16(dst + 16 * (e - lane), ks + 16 * (e - lane));
          }
          if (KB && lane < 4 && 8 * lane < n) copy16(dst + z.off_kside, kside + 2 * (int64_t)t0 + 16 * lane);
        }
        copy_commit();
      };
      __syncthreads();  // the last chunk's rows have been read
      int i = i0 + warp;
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) load(i + s * WARPS, s);
      if (!waited) grid_dependency_wait();
      waited = true;
      const float tab_inv = KB ? 1.f / K::table_scale(kp) : 1.f;
      const float* w0 = t.w + ((size_t)slot * t.rows + r0) * t.NCk;
      // four rows of a warp at a time, their loads first
#pragma unroll 1
      for (int rb = warp; rb < 8 * tiles; rb += 4 * WARPS) {
        float w[4][(KS + 1) / 2], most[4];
        float2 st[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = rb + u * WARPS;
          st[u] = r < nr ? t.stats[(size_t)slot * t.rows + r0 + r] : make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < (KS + 1) / 2; ++j)
            w[u][j] = r < nr && lane + 32 * j < t.NCk ? fabsf(w0[(size_t)r * t.NCk + lane + 32 * j]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          most[u] = 0.f;
#pragma unroll
          for (int j = 0; j < (KS + 1) / 2; ++j)
            if (w[u][j] <= 3.4e38f) most[u] = fmaxf(most[u], w[u][j]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) most[u] = warp_max(most[u]);
        if (lane == 0)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = rb + u * WARPS;
            if (r >= 8 * tiles) break;
            const float mul = row_scale(most[u]);
            row_mul[r] = mul;
            rowc[r] = make_float4(tab_inv / mul, -st[u].x, st[u].y,
                                  __int_as_float(r < nr ? t.ctx + (r0 + r) / t.rep : -1));
          }
      }
      __syncthreads();
      auto fragment = [&](int s, int nt) {
        const int r = 8 * nt + g, j = K::position(s, c);
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nr && j < t.NCk) w = *reinterpret_cast<const float4*>(w0 + (size_t)r * t.NCk + j);
        return weight_pieces(w, row_mul[r]);
      };
#pragma unroll 4
      for (int e = warp; e < KS * tiles; e += WARPS) wfrag[e * 32 + lane] = fragment(e % KS, e / KS);
      __syncthreads();
      int st = 0;
      for (; i < i1; i += WARPS) {
        copy_wait<kStages - 2>();
        __syncwarp();
        const unsigned char* sp = ring + st * z.stage;
        load(i + (kStages - 1) * WARPS, st ^ 1);
        const int t0 = tile_of(i) * kTile;
        // lanes of a quad write tokens g, g + 8, g + 16 and g + 24: what is there, in time
        const int tok = t0 + g + 8 * c;
        const float old = tok < t.S && decay != 0.f ? wout[tok] : 0.f;
        float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // halves of the tile: tokens g and g + 8
        if (t0 <= last && t0 > hidden && (t0 > gap1 || t0 < gap0)) {
          const bool all = t0 >= see0 && t0 <= see1 && (t0 > see2 || t0 < see3);
          auto add = [&](int h, int nt, const float (&s)[4], float na, float nb) {  // the weights of a tile of rows
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 rc = rowc[8 * nt + cr + j];
              const float pa = ex2(fmaf(s[j] * na, rc.x, rc.y)) * rc.z;
              const float pb = ex2(fmaf(s[2 + j] * nb, rc.x, rc.y)) * rc.z;
              if (all) {
                sum[h][0] += pa;
                sum[h][1] += pb;
              } else {
                const int pos = __float_as_int(rc.w);
                if (sight.sees(t0 + 16 * h + g, pos)) sum[h][0] += pa;
                if (sight.sees(t0 + 16 * h + g + 8, pos)) sum[h][1] += pb;
              }
            }
          };
          auto half = [&](int h) {
            const int tk = 16 * h + g;
            const typename K::Row ra = keys.row(sp, 16 * h, Pk), rb = keys.row(sp, 16 * h + 8, Pk);
            float na = 1.f, nb = 1.f;
            if (KB) {
              const __half* nm = reinterpret_cast<const __half*>(sp + z.off_kside) + tk;
              na = __half2float(nm[0]);
              nb = __half2float(nm[8]);
            }
            uint32_t hi[KS][4], lo[KS][4];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t ha[2], la[2], hb[2], lb[2];
              keys.step(ra, k, ha, la);
              keys.step(rb, k, hb, lb);
              hi[k][0] = ha[0]; hi[k][1] = hb[0]; hi[k][2] = ha[1]; hi[k][3] = hb[1];
              lo[k][0] = la[0]; lo[k][1] = lb[0]; lo[k][2] = la[1]; lo[k][3] = lb[1];
            }
#pragma unroll 2
            for (int nt = 0; nt < tiles; ++nt) {
              float s[4], small[4], other[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) s[e] = small[e] = other[e] = 0.f;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                const uint4 w = wfrag[(nt * KS + k) * 32 + lane];
                mma_f16(s, hi[k], w.x, w.y);
                mma_f16(small, hi[k], w.z, w.w);
                if (KB) mma_f16(other, lo[k], w.x, w.y);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) s[e] += KB ? small[e] + other[e] : small[e];
              add(h, nt, s, na, nb);
            }
          };
          half(0);
          half(1);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            sum[h][j] += __shfl_xor_sync(kFull, sum[h][j], 1);
            sum[h][j] += __shfl_xor_sync(kFull, sum[h][j], 2);
          }
        const float add = c < 2 ? c ? sum[0][1] : sum[0][0] : c == 2 ? sum[1][0] : sum[1][1];
        if (tok < t.S && (decay != 1.f || add != 0.f)) wout[tok] = fmaf(decay, old, add);
        st ^= 1;
      }
      copy_wait<0>();
    }
  }
}

// The weights from the scores that the main kernel kept, of R rows at most: a lane has a
// token of each of four tiles.  Bound by the scores' bytes, most of which still lie in L2:
// 128 slots, 4 rows, 16384 tokens, 34 MB of scores and 17 of weights, in 11.7 us.
constexpr int kKeptTiles = 4;

template <int R>
__global__ void __launch_bounds__(256) window_weights_kept_kernel(const Params kp, const WindowArgs t) {
  const int chunks = (int)((t.wtps + kKeptTiles - 1) / kKeptTiles);
  const int64_t at = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int slot = (int)(at / chunks), i0 = (int)(at - (int64_t)slot * chunks) * kKeptTiles, lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (slot >= kp.n_slots) return;
  const int b = slot / kp.H, h = slot - b * kp.H;
  const bool every = t.decay != 1.f;  // the old weights of all tokens are scaled
  const Sight sight(t, b);
  const Tiles<kTile> seen(sight, t.ctx, t.S - 1);
  float* wout = t.weights + b * t.w_sb + h * t.w_sh;
  const float4* scores = reinterpret_cast<const float4*>(t.scores) + (size_t)slot * t.tps * kTile * (R / 4);
  int tok[kKeptTiles];
  float4 y[kKeptTiles][R / 4];
  float old[kKeptTiles], sum[kKeptTiles];
  bool any[kKeptTiles];
#pragma unroll
  for (int u = 0; u < kKeptTiles; ++u) {
    const int e = i0 + u, tile = every ? e : seen.tile(e), i = every ? seen.index(e) : e < seen.count() ? e : -1;
    tok[u] = tile * kTile + lane;
    any[u] = i >= 0 && tok[u] < t.S;
    old[u] = (every || any[u]) && tok[u] < t.S && t.decay != 0.f ? wout[tok[u]] : 0.f;
#pragma unroll
    for (int x = 0; x < R / 4; ++x)
      y[u][x] = any[u] ? scores[((size_t)i * kTile + lane) * (R / 4) + x] : make_float4(0.f, 0.f, 0.f, 0.f);
    sum[u] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < t.rows) {
      const float2 st = t.stats[(size_t)slot * t.rows + r];
      const int pos = t.ctx + r / t.rep;
#pragma unroll
      for (int u = 0; u < kKeptTiles; ++u) {
        const float4 v = y[u][r / 4];
        const float s = r % 4 == 0 ? v.x : r % 4 == 1 ? v.y : r % 4 == 2 ? v.z : v.w;
        if (any[u] && sight.sees(tok[u], pos)) sum[u] = fmaf(ex2(s - st.x), st.y, sum[u]);
      }
    }
#pragma unroll
  for (int u = 0; u < kKeptTiles; ++u)
    if ((every || any[u]) && tok[u] < t.S && (every || sum[u] != 0.f)) wout[tok[u]] = fmaf(t.decay, old[u], sum[u]);
}

// The shares' weights added up.
__global__ void __launch_bounds__(256) window_add_weights_kernel(const Params kp, const WindowArgs t) {
  grid_dependency_wait();
  const int64_t words = (int64_t)kp.n_slots * t.S;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) {
    const int slot = (int)(i / t.S), tok = (int)(i - (int64_t)slot * t.S), b = slot / kp.H, h = slot - b * kp.H;
    float v = 0.f;
    for (int x = 0; x < t.wsplits; ++x) v += t.wpart[x * words + i];
    float* w = t.weights + b * t.w_sb + h * t.w_sh + tok;
    if (t.decay == 0.f) *w = v;
    else if (t.decay != 1.f || v != 0.f) *w = fmaf(t.decay, *w, v);
  }
}

using WeightsKernel = void (*)(const Params, const WindowArgs, const WindowShape);

WeightsKernel weights_kernel_for(const Params& kp, int NCk, int* tables) {
  auto of = [&](auto keys, WeightsKernel k) {
    using K = decltype(keys);
    *tables = K::kSteps * kChunkTiles * 512;
    return k;
  };
  if (kp.mode == KVC_MODE_UNIFORM) {
    if (NCk <= 32) return of(Keys<0, 2, false>{}, window_weights_mma_kernel<0, 2>);
    if (NCk <= 48) return of(Keys<0, 3, false>{}, window_weights_mma_kernel<0, 3>);
    if (NCk <= 64) return of(Keys<0, 4, false>{}, window_weights_mma_kernel<0, 4>);
    return of(Keys<0, 8, false>{}, window_weights_mma_kernel<0, 8>);
  }
  switch (kp.cb_bits * 1000 + kp.D) {
    case 2064: return of(Keys<2, 4, false>{}, window_weights_mma_kernel<2, 4>);
    case 3064: return of(Keys<3, 4, false>{}, window_weights_mma_kernel<3, 4>);
    case 4064: return of(Keys<4, 4, false>{}, window_weights_mma_kernel<4, 4>);
    case 2128: return of(Keys<2, 8, false>{}, window_weights_mma_kernel<2, 8>);
    case 3128: return of(Keys<3, 8, false>{}, window_weights_mma_kernel<3, 8>);
    default: return of(Keys<4, 8, false>{}, window_weights_mma_kernel<4, 8>);
  }
}

WindowKernel main_kernel(const Params& kp, const Params& vp, int rows, int NCk, int nt, int* tables) {
  return rows <= 4 ? window_kernel_4(kp, vp, NCk, tables)
         : nt == 1 ? window_kernel_8(kp, vp, NCk, tables)
         : nt == 2 ? window_kernel_16(kp, vp, NCk, tables)
                   : window_kernel_32(kp, vp, NCk, tables);
}

// The layout of the rings behind `tables` bytes; the dynamic shared memory.
int lay_out(const Params& kp, const Params* vp, const WindowArgs& t, int tables, int warps, WindowShape* z) {
  auto up = [](int v) { return (v + 15) / 16 * 16; };
  int at = up(kTile * t.Pk_max) + 16;  // (words are read past a row's end)
  z->off_kside = at;
  at += kTile * 2;
  if (vp) {
    z->off_v = at;
    at += vp->mode == KVC_MODE_UNIFORM ? up(kTile * t.Pv_max) + 16 : kTile * vp->D;
    z->off_vside = at;
    at += kTile * 2;
  }
  z->stage = (at + 127) / 128 * 128;
  z->off_ring = (tables + 127) / 128 * 128;
  // the join of the warps' sums takes the rings' place
  const int join = vp ? kWarps * (vp->mode == KVC_MODE_UNIFORM ? 128 : vp->D) * 32 : 0;
  return z->off_ring + std::max(warps * kStages * z->stage, join);
}

}  // namespace

int window_mma_ctas(const Params& kp, const Params& vp, const WindowArgs& t, int nt) {
  if (kp.prod || kp.D > 128) return 0;
  if (vp.mode == KVC_MODE_UNIFORM ? t.Dv > 128 : vp.D != 64 && vp.D != 128) return 0;
  int tables = 0;
  const WindowKernel k = main_kernel(kp, vp, t.rows, t.NCk, nt, &tables);
  if (!k) return 0;
  WindowShape z;
  const int smem = lay_out(kp, &vp, t, tables, kWarps, &z);
  if (smem > 200 * 1024) return 0;
  return nt == 1 && 2 * smem <= 188 * 1024 ? 2 : 1;
}

cudaError_t launch_window_mma(const Params& kp, const Params& vp, const WindowArgs& t, cudaStream_t s, int* nk) {
  int tables = 0;
  const WindowKernel k = main_kernel(kp, vp, t.rows, t.NCk, t.mma, &tables);
  WindowShape z;
  const int smem = lay_out(kp, &vp, t, tables, kWarps, &z);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  ++*nk;
  return launch_dependent(k, (unsigned)t.grid, kThreads, (size_t)smem, s, kp, vp, t, z);
}

// CTAs that share out the tokens of the weights' pass.  Of many rows a chunk takes
// about 10 us to bring in, so that a warp should have four tiles for it.
static int weights_ctas(const Params& kp, const WindowArgs& t, int64_t tiles) {
  const int64_t total = tiles * kp.n_slots;
  const int64_t per = (t.rows > 8 * kChunkTiles ? 4 : 1) * kManyWarps;
  return (int)std::min<int64_t>(std::max<int64_t>(total / per, kp.n_slots), t.sms);
}

int window_weights_splits(const Params& kp, const WindowArgs& t) {
  if (t.rows <= 8 * kChunkTiles) return 1;
  const int ctas = weights_ctas(kp, t, (t.S + kTile - 1) / kTile);
  const int chunks = (t.rows + 8 * kChunkTiles - 1) / (8 * kChunkTiles);
  return std::max(1, std::min(chunks, t.sms / ctas));
}

cudaError_t launch_window_weights_mma(const Params& kp, const WindowArgs& t, cudaStream_t s, int* nk) {
  if (t.scores) {
    const int64_t warps = kp.n_slots * ((t.wtps + kKeptTiles - 1) / kKeptTiles);
    ++*nk;
    return launch_dependent(t.rows <= 4 ? window_weights_kept_kernel<4> : window_weights_kept_kernel<8>,
                            (unsigned)((warps + 7) / 8), 256u, 0, s, kp, t);
  }
  int tables = 0;
  const WeightsKernel k = weights_kernel_for(kp, t.NCk, &tables);
  WindowShape z;
  const int smem = lay_out(kp, nullptr, t, tables, kManyWarps, &z);
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  const int grid = weights_ctas(kp, t, t.wtps) * t.wsplits;
  ++*nk;
  const cudaError_t f = launch_dependent(k, (unsigned)grid, kManyWarps * 32u, (size_t)smem, s, kp, t, z);
  if (f != cudaSuccess || t.wsplits == 1) return f;
  ++*nk;
  const int64_t words = (int64_t)kp.n_slots * t.S;
  return launch_dependent(window_add_weights_kernel, (unsigned)std::min<int64_t>((words + 255) / 256, 8 * t.sms), 256u, 0, s,
                          kp, t);
}

}  // namespace kvc
