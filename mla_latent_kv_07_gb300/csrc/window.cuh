// window.cuh -- which positions a token of a windowed call sees, and the run of
// positions that is loaded for it.
//
// The token at position t = end - 1 sees positions below `sinks` and those from
// low = end - window on.  Both ranges are widened to whole boxes of 16 positions,
// the unit in which rows are loaded (a page holds a multiple of 16), and laid
// side by side: place v of the run is position v, or v + gap from place `cut` on.
// Splits, tiles and lookups count places; at most 30 of them are not seen (15
// behind the sinks, 15 before low), and every box of 16 holds one that is.
#pragma once

#include "common.cuh"
#include "schedule.cuh"

namespace mla {

constexpr unsigned kFew = 16;   // positions up to which a token sees few

struct WindowSpan {
  int sinks, low, end, cut, gap;
  __device__ __forceinline__ int places() const { return end - gap; }
  __device__ __forceinline__ int pos(int v) const { return v + (v >= cut ? gap : 0); }
  // the positions p .. p + 15 that are seen, as bits
  __device__ __forceinline__ uint32_t seen16(int p) const {
    auto below = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u; };
    return below(sinks - p) | (below(end - p) & ~below(low - p));
  }
};

// of `end` positions
__device__ __forceinline__ WindowSpan window_span(int end, int window, int sinks) {
  WindowSpan w;
  w.end = end;
  w.sinks = min(sinks, end);
  w.low = end > window ? end - window : 0;
  w.cut = (w.sinks + 15) & ~15;
  w.gap = max(0, (w.low & ~15) - w.cut);
  return w;
}

// of sequence (token) b of a windowed call
__device__ __forceinline__ WindowSpan window_span(const DenseSchedule& s, int b, uint32_t* flags) {
  return window_span(dense_len(s, b >> s.halves, flags), s.window, s.sinks);
}

// Unit u of a windowed call whose chunks are fixed, with the token's span; b = -1
// where the token has fewer.  writer: the lane that also writes the combine's entry
// of a token (its first unit does).
__device__ __forceinline__ Unit window_unit(const DenseSchedule& s, int u, bool writer, int2* seq, WindowSpan* span, uint32_t* flags) {
  const int b = u / s.per_token, i = u - b * s.per_token;
  *span = window_span(s, b, flags);
  const int places = span->places(), n = (places + s.chunk - 1) / s.chunk;
  if (writer && i == 0) seq[b] = make_int2(u, n == 1 ? -1 : n);
  const int t0 = i * s.chunk;
  return t0 >= places ? Unit{-1, 0, 0, 0} : Unit{b, t0, min(t0 + s.chunk, places), n == 1 ? kUnitDirect : 0};
}

}  // namespace mla
