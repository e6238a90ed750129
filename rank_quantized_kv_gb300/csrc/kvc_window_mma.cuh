// Pieces of the windowed attention's warp-level tensor-core kernels: matrix
// instructions, decoding of codes straight into their operand registers.
//
// m16n8k16 with tokens on the M side: lane (g, c) = (lane / 4, lane % 4) holds of A
// rows g and g + 8, of B and of the result columns g and 2 c, 2 c + 1.  The order of
// the K axis is free as long as both operands agree, so a lane takes a stretch of a
// token's packed row and decodes it into the registers where it is needed.
#pragma once

#include <cuda_fp16.h>

#include "kvc_codes.cuh"
#include "kvc_internal.h"

namespace kvc {

namespace {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, two neighbours of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 matrices of 16-bit values from shared memory, transposed: lane i gives the
// address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The larger of two and three, NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Codes as fp16: 0x6400 | c is 1024 + c exactly, less 1024 + the centre.
constexpr uint32_t kMagic = 0x64006400u;

// (a & b) ^ c in one instruction (with two constants the compiler makes two of it).
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// int8 values in the low bytes of the halves (the high bytes hold anything).
__device__ __forceinline__ uint32_t int8_f16(uint32_t x) {
  return sub_f16x2(and_xor(x, 0x00ff00ffu, kMagic | 0x00800080u), kMagic | 0x00800080u);
}

// A chunk's width as the decoders use it: eight codes of w bits, of which b.x holds
// the first four and, after split(), b.y the others in its low bits, at any width.
struct Width {
  uint32_t w, mask, centre;  // mask: in both halves; centre: 1024 + 2^(w-1), in both
  __device__ void set(uint32_t entry) {
    w = entry ? (entry >> 16) & 0xfu : 1u;
    mask = ((1u << w) - 1u) * 0x10001u;
    centre = kMagic | ((1u << (w - 1)) * 0x10001u);
  }
  __device__ uint2 split(uint2 b) const { return make_uint2(b.x, w == 8 ? b.y : b.x >> (4 * w & 31)); }
  // Codes 2 q and 2 q + 1 of split bits, centred.
  __device__ uint32_t pair(uint2 b, int q) const {
    uint32_t x = q < 2 ? b.x : b.y;
    if (q & 1) x >>= 2 * w;
    const uint32_t lo = (x & (mask & 0xffffu)) | kMagic;
    return sub_f16x2(((x << (16 - w)) & (mask & 0xffff0000u)) | lo, centre);
  }
  // Codes 2 q and 2 q + 1 of two tokens, split: one code of both, then the other.
  __device__ void both(uint2 a, uint2 b, int q, uint32_t* first, uint32_t* second) const {
    uint32_t x = q < 2 ? a.x : a.y, y = q < 2 ? b.x : b.y;
    if (q & 1) {
      x >>= 2 * w;
      y >>= 2 * w;
    }
    const uint32_t z = __byte_perm(x, y, 0x5410);
    *first = sub_f16x2((z & mask) | kMagic, centre);
    *second = sub_f16x2(((z >> w) & mask) | kMagic, centre);
  }
};

// Where a lane reads a chunk of a token's row: words from byte `at` on, shifted right by
// `shift`.  Tokens eight further on lie 8 P bytes further on, a multiple of 4, so that
// neither depends on them.  A chunk that does not exist reads the row's first bytes:
// what it gives meets weights of zero, or a sum that nobody reads.
struct ChunkPlace {
  uint32_t at, shift;
  __device__ void set(int byte) {
    at = (uint32_t)byte & ~3u;
    shift = 8 * ((uint32_t)byte & 3u);
  }
  // wide: the chunk may have eight bytes.
  __device__ uint2 read(const unsigned char* rows, bool wide) const {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(rows + at);
    uint2 b;
    const uint32_t w1 = p[1];
    b.x = __funnelshift_r(p[0], w1, shift);
    b.y = 0u;
    if (wide) b.y = __funnelshift_r(w1, p[2], shift);
    return b;
  }
};

// ---------------------------------------------------------------- keys

// How a warp reads the keys of 16 tokens: KB > 0, a codebook of KB bits over 16 KS
// components, else centred codes of up to 2 KS chunks (KS steps of 16): two steps take
// a chunk of each of four lanes, the last of an odd number the halves of two chunks.
//
// Scores carry fp32's precision: weights are two fp16 pieces of values that a power
// of two per row brings up to 2^13 .. 2^14 (22 bits and more), uniform codes are
// exact, and centroids two fp16 pieces of values in 8 .. 16; the products of the
// small pieces are summed apart.
//
// PAIRED: the two pieces of a token's codes are rows g and g + 8 of one operand, so
// that a lookup of both lands in neighbouring registers of it; else a lookup for each,
// and tokens g and g + 8 make an operand of either piece (for many rows: three
// products of 16 tokens in place of four).
template <int KB, int KS, bool PAIRED>
struct Keys {
  static constexpr int kCodes = 4 * KS;                 // a lane's codes of a token
  static constexpr int kSteps = KS;
  static constexpr int kPlaces = (KS + 1) / 2;          // a lane's chunks (uniform)
  static_assert(!KB || KS % 2 == 0, "codebooks: 64 or 128 components");
  static constexpr int kWords = KB ? (kCodes * KB + 31) / 32 : 1;
  static constexpr bool kPairs = KB && KB <= 3;         // the table holds pairs of centroids
  // The table, once per lane (no bank conflicts): pairs of centroids up to 3 bits, both
  // pieces together (PAIRED) or all first ones before the second ones; at 4 bits single
  // ones, both pieces in a word.
  static constexpr int kTable = !KB ? 0 : kPairs ? (1 << (2 * KB)) * 32 * 8 : 16 * 32 * 4;
  static constexpr int kShift = PAIRED && kPairs ? 8 : 7;  // log2 of the bytes of an entry's copies

  const unsigned char* tab;  // the table in shared memory
  uint32_t lane_at;     // where this lane's copy starts in an entry
  ChunkPlace place[kPlaces];  // uniform: the lane's chunks of token g
  Width width[kPlaces];
  bool wide[kPlaces];   // some lane's has eight-bit codes

  // The scale of the centroids: a power of two that brings the largest to [8, 16).
  static __device__ float table_scale(const Params& kp) {
    const float big = fmaxf(fabsf(kp.codebook[0]), fabsf(kp.codebook[kp.cb_levels - 1]));
    if (!(big > 0.f) || big > 3.4e38f) return 1.f;
    const int e = ((__float_as_int(big) >> 23) & 0xff) - 127;  // big in [2^e, 2^(e + 1))
    return __int_as_float((min(126, max(-126, 3 - e)) + 127) << 23);
  }
  // Fill the table (all threads).
  static __device__ void fill(const Params& kp, unsigned char* table, int threads) {
    const float mul = table_scale(kp);
    auto pieces = [&](int c, uint32_t* hi, uint32_t* lo) {
      const float v = kp.codebook[c] * mul;
      const __half h = __float2half_rn(v);
      *hi = __half_as_ushort(h);
      *lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
    };
    constexpr int lm = KB ? (1 << KB) - 1 : 0;
    for (int i = threadIdx.x; i < kTable / (kPairs ? 8 : 4); i += threads) {
      const int x = i >> 5;
      uint32_t h0, l0, h1, l1;
      pieces(x & lm, &h0, &l0);
      if (kPairs) {
        pieces(x >> KB, &h1, &l1);
        const uint32_t hi = h0 | (h1 << 16), lo = l0 | (l1 << 16);
        if (PAIRED) {
          reinterpret_cast<uint2*>(table)[i] = make_uint2(hi, lo);
        } else {
          reinterpret_cast<uint32_t*>(table)[i] = hi;
          reinterpret_cast<uint32_t*>(table + kTable / 2)[i] = lo;
        }
      } else {
        reinterpret_cast<uint32_t*>(table)[i] = h0 | (l0 << 16);
      }
    }
  }

  __device__ void begin(const unsigned char* table) {
    tab = table;
    lane_at = (threadIdx.x & 31) * (kShift == 8 ? 8 : 4);
  }
  // A job's basis (uniform keys): rows of Pk bytes.
  __device__ void basis(const Params& kp, int beta, int Pk) {
    if (!KB)
#pragma unroll
      for (int s = 0; s < kPlaces; ++s) {
        const int c = threadIdx.x & 3;
        const uint32_t e = chunk_entry(kp, beta, 4 * s + (2 * s + 1 < KS ? c : c >> 1));
        place[s].set((int)((threadIdx.x & 31) >> 2) * Pk + (int)(e & 0xffffu));
        width[s].set(e);
        wide[s] = __any_sync(kFull, width[s].w == 8);
      }
  }
  // The packed position of the first of the four codes that lane c has of step s.
  static __device__ int position(int s, int c) {
    if (KB) return c * kCodes + 4 * s;
    return (s | 1) < KS ? 8 * (4 * (s / 2) + c) + 4 * (s & 1) : 16 * s + 4 * c;
  }

  // What a lane holds of a token's row: the words of its codes (codebook).
  struct Row { uint32_t w[kWords]; const unsigned char* rows; };
  // (token g + `ahead`, a multiple of 8)
  __device__ Row row(const unsigned char* rows, int ahead, int Pk) const {
    Row r;
    if (KB) {
      const int a = (ahead + (int)((threadIdx.x & 31) >> 2)) * (2 * KS * KB) + (threadIdx.x & 3) * (kCodes * KB / 8);
      if ((kCodes * KB / 8) % 4 == 0) {
        const unsigned char* p = rows + a;
        if (kWords == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          r.w[0] = v.x; r.w[1 % kWords] = v.y; r.w[2 % kWords] = v.z; r.w[3 % kWords] = v.w;
        } else if (kWords == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          r.w[0] = v.x; r.w[1 % kWords] = v.y;
        } else {
#pragma unroll
          for (int i = 0; i < kWords; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
      } else {  // 6 bytes
        const uint2 v = bits_at(rows, a);
        r.w[0] = v.x; r.w[1 % kWords] = v.y;
      }
    } else {
      r.rows = rows + ahead * Pk;
    }
    return r;
  }
  // The lane's four codes of step s of a token as fp16 pairs: hi[0] the first two,
  // hi[1] the others; their second pieces in lo.
  __device__ void step(const Row& r, int s, uint32_t (&hi)[2], uint32_t (&lo)[2]) const {
    if constexpr (KB == 0) {
      const Width& w = width[s / 2];
      uint2 b = w.split(place[s / 2].read(r.rows, wide[s / 2]));
      if ((s | 1) >= KS && (threadIdx.x & 1)) b.x = b.y;  // (odd lanes: the chunk's second half)
      hi[0] = w.pair(b, 2 * (s & 1));
      hi[1] = w.pair(b, 2 * (s & 1) + 1);
      lo[0] = lo[1] = 0u;
    } else if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // the pair's field (2 KB bits) shifted to where it is an offset
        constexpr uint32_t mask = ((1u << (2 * KB)) - 1u) << kShift;
        const int bit = KB * (4 * s + 2 * i) - kShift, at = bit >> 5, sh = bit & 31;
        uint32_t v;
        if (bit < 0) v = r.w[0] << -bit;
        else if (sh + 2 * KB + kShift <= 32 || at + 1 >= kWords) v = r.w[at] >> sh;
        else v = __funnelshift_r(r.w[at], r.w[(at + 1) % kWords], sh);
        const unsigned char* p = tab + ((v & mask) | lane_at);
        if (PAIRED) {
          const uint2 both = *reinterpret_cast<const uint2*>(p);
          hi[i] = both.x;
          lo[i] = both.y;
        } else {
          hi[i] = *reinterpret_cast<const uint32_t*>(p);
          lo[i] = *reinterpret_cast<const uint32_t*>(p + kTable / 2);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = r.w[s / 2] >> (16 * (s & 1) + 8 * i);  // two codes in the low byte
        const uint32_t a = *reinterpret_cast<const uint32_t*>(tab + (((x & 15u) << 7) | lane_at));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(tab + (((x & 0xf0u) << 3) | lane_at));
        hi[i] = __byte_perm(a, b, 0x5410);
        lo[i] = __byte_perm(a, b, 0x7632);
      }
    }
  }
};

// The power of two by which a row's weights are multiplied (largest to [2^13, 2^14)),
// given the largest of their magnitudes (finite ones).
__device__ __forceinline__ float row_scale(float most) {
  const int e = ((__float_as_int(most) >> 23) & 0xff) - 127;
  return most > 0.f ? __int_as_float((min(126, 13 - e) + 127) << 23) : 1.f;
}

// Four weights of a row as fp16 pieces: {hi01, hi23, lo01, lo23}, the operand
// registers of a step.
__device__ __forceinline__ uint4 weight_pieces(float4 w, float scale) {
  w.x *= scale; w.y *= scale; w.z *= scale; w.w *= scale;
  const __half2 h0 = __floats2half2_rn(w.x, w.y), h1 = __floats2half2_rn(w.z, w.w);
  const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
  return make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                    pack_f16(w.x - f0.x, w.y - f0.y), pack_f16(w.z - f1.x, w.w - f1.y));
}

// Of four weights' pieces the large or the small ones.
__device__ __forceinline__ uint2 one_piece(uint4 w, bool small) { return small ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y); }

}  // namespace

}  // namespace kvc
