// Which tokens a query of the windowed attention sees, and the tiles of them
// that a job walks.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// The run of tiles of CTA c is [window_run(t, c), window_run(t, c + 1)).
__device__ __forceinline__ int64_t window_run(const WindowArgs& t, int64_t c) { return t.total * c / t.grid; }
// The CTA whose run holds place `at` of the line.
__device__ inline int64_t window_cta(const WindowArgs& t, int64_t at) {
  int64_t c = at * t.grid / t.total;
  while (window_run(t, c + 1) <= at) ++c;
  while (window_run(t, c) > at) --c;
  return c;
}
// Number of the first partial of a job whose tiles begin in CTA c0; those of the CTAs
// after it follow.  Where only cut jobs leave partials they are numbered by CTA: one that
// begins behind another job's end takes the odd number, and a job that begins in the CTA
// where the last one ended always does.
__device__ __forceinline__ int64_t window_part(const WindowArgs& t, int64_t job, int64_t c0) {
  return t.cuts ? 2 * c0 + (window_run(t, c0) < job * t.tps) : job + c0;
}

// The tokens visible to a query at position pos of a batch entry: those of
// [first, pos] within the window or before sink_end.
struct Sight {
  int first, sink_end, window;
  __device__ Sight(const WindowArgs& t, int b) {
    first = t.first ? min(max(t.first[b], 0), t.S) : 0;
    sink_end = (int)min((int64_t)first + t.sinks, (int64_t)t.S);
    window = t.window;
  }
  __device__ bool sees(int tok, int pos) const {
    return tok >= first && tok <= pos && (tok > pos - window || tok < sink_end);
  }
  // Whether queries p0 .. p1 all see tokens t0 .. t1.
  __device__ bool all(int t0, int t1, int p0, int p1) const {
    return t0 >= first && t1 <= p0 && (t0 > p1 - window || t1 < sink_end);
  }
};

// The tiles of T tokens that hold what some query of p0 .. p1 sees: the sinks'
// [a, a + na), then the window's [b, b + nb); one range where they meet.
template <int T>
struct Tiles {
  int a = 0, na = 0, b = 0, nb = 0;
  __device__ Tiles(const Sight& s, int p0, int p1) {
    if (s.first > p1) return;
    a = s.first / T;
    const int sink_end = min(s.sink_end, p1 + 1);
    if (sink_end > s.first) na = (sink_end + T - 1) / T - a;
    b = max(s.first, p0 - s.window + 1) / T;
    nb = p1 / T + 1 - b;
    if (a + na >= b) {  // (no sinks: where the window starts with the first token)
      nb += b - a;
      b = a;
      na = 0;
    }
  }
  __device__ int count() const { return na + nb; }
  __device__ int tile(int i) const { return i < na ? a + i : b + i - na; }
  // Tile t's place among them, -1: not one of them.
  __device__ int index(int t) const {
    return t >= b && t < b + nb ? na + t - b : t >= a && t < a + na ? t - a : -1;
  }
};

}  // namespace kvc
