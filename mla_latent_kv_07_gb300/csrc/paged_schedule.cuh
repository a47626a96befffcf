// paged_schedule.cuh -- the split schedule of a paged decode: which run of
// positions each CTA (or CTA pair) takes.
//
// A sequence is cut into units of `chunk` positions and a last one of what is
// left.  With one unit per CTA, ragged lengths leave CTAs with short last units
// idle for much of the call (a quarter of the GPU's time at 32 sequences of
// uniform lengths on 76 pairs).  So there may be more units than CTAs at a
// time: the whole chunks come first, one for each, and the short units after
// them, longest first, for CTAs as they become free.  chunk is the smallest
// (by steps) at which the short units fit: either each has a place of its own,
// or those above half a place do and all together leave a fifth of their places
// free, a unit's start and end counted as kUnitCost positions.
// Measured against one unit per CTA: 32 sequences of 1024 to 16384 positions, 128
// heads, FP8, 147 -> 129 us; 32 of 8192, 16 heads, 63 -> 57 us; 4 equal ones the
// same to 0.3 us.
#pragma once

#include "append_row.cuh"
#include "common.cuh"
#include "schedule.cuh"
#include "window.cuh"

namespace mla {

// The work of a unit beyond its positions, in positions: schedule, lookups,
// first load and outputs take about 9 us, in which a CTA (64 heads, bf16) or a
// pair (128 heads) takes some 320 positions.
constexpr unsigned kUnitCost = 320;

// Run by one whole warp, s.B <= 32 kBlk, dense lengths.  Returns unit
// `want` in the order of launch (b = -1 if there are fewer), whose flags carry
// its place in its sequence's partial results (kUnitSlot); the status bits and
// the number of units; with `seq` the combine's table, with `all` every unit.
template <int kBlk, bool kWin>
__device__ __forceinline__ Unit packed_units(const DenseSchedule& s, int want, uint32_t* flags_out, int* units_out, int2* seq,
                                             Unit* all) {
  const int lane = threadIdx.x & 31;
  unsigned len[kBlk];
  uint32_t flags = 0, valid = 0;   // valid: the new row is written (bit r)
  unsigned hi = 0, lo = 0, longest = 0;
#pragma unroll
  for (int r = 0; r < kBlk; ++r) {
    len[r] = 0;
    const int b = lane + 32 * r;
    if (b < s.B) {
      len[r] = (unsigned)(kWin ? window_span(s, b, &flags).places() : dense_len(s, b, &flags));
      if (s.append) {
        const bool v = append_row_valid(s.end_pos[b], s.max_end_pos);
        valid |= (uint32_t)v << r;
        if (!v) flags |= kDevAppendSkipped;
      }
    }
    hi += len[r] >> 12;
    lo += len[r] & 4095;
    longest = max(longest, len[r]);
  }
  hi = __reduce_add_sync(0xffffffffu, hi);
  lo = __reduce_add_sync(0xffffffffu, lo);
  longest = __reduce_max_sync(0xffffffffu, longest);
  flags = __reduce_or_sync(0xffffffffu, flags);
  const unsigned long long total = (unsigned long long)hi * 4096u + lo;
  const unsigned g = (unsigned)s.granule, places = (unsigned)s.target;
  const unsigned cap = longest > g ? (longest + g - 1) / g * g : g;
  const unsigned long long c0 = ((total + places - 1) / places + g - 1) / g * g;
  unsigned chunk = c0 < g ? g : c0 > cap ? cap : (unsigned)c0;
  unsigned nfull = 0;
#pragma unroll 1
  for (int iter = 0; iter < 64; ++iter) {
    unsigned full = 0, rest = 0, big = 0, rhi = 0, rlo = 0;
#pragma unroll
    for (int r = 0; r < kBlk; ++r) {
      const unsigned n = len[r] / chunk, left = len[r] - n * chunk;
      full += n;
      rest += left > 0;
      big += left > 0 && 2 * left + kUnitCost > chunk;
      rhi += left >> 12;
      rlo += left & 4095;
    }
    nfull = __reduce_add_sync(0xffffffffu, full);
    if (chunk >= cap) break;
    const unsigned counts = __reduce_add_sync(0xffffffffu, rest | big << 16);
    rhi = __reduce_add_sync(0xffffffffu, rhi);
    rlo = __reduce_add_sync(0xffffffffu, rlo);
    rest = counts & 0xffff;
    big = counts >> 16;
    if (nfull <= places) {
      const unsigned free = places - nfull;
      const unsigned long long load = (unsigned long long)rhi * 4096u + rlo + (unsigned long long)rest * kUnitCost;
      if (rest <= free || (big <= free && load * 5 <= (unsigned long long)free * (chunk + kUnitCost) * 4)) break;
    }
    // by 1/64, later by more, so that a few dozen steps reach any length
    const int shift = 6 - (iter >> 3) < 1 ? 1 : 6 - (iter >> 3);
    const unsigned grown = (chunk + (chunk >> shift)) / g * g;
    chunk = grown > chunk ? grown : chunk + g;
    chunk = chunk > cap || iter == 62 ? cap : chunk;
  }
  // short units by size in eighths of a chunk, largest first
  unsigned rank[kBlk];
  {
    const unsigned eighth = (chunk + 7) / 8;
    unsigned at = nfull;
    int size[kBlk];
#pragma unroll
    for (int r = 0; r < kBlk; ++r) {
      const unsigned left = len[r] % chunk;
      size[r] = left > 0 ? (int)(left / eighth) : -1;
      rank[r] = 0xffffffffu;
    }
#pragma unroll 1
    for (int c = 7; c >= 0; --c) {
#pragma unroll
      for (int r = 0; r < kBlk; ++r) {
          const uint32_t m = __ballot_sync(0xffffffffu, size[r] == c);
        if (size[r] == c) rank[r] = at + __popc(m & ((1u << lane) - 1));
        at += __popc(m);
      }
    }
  }
  // walk the sequences in order: places in the partial results, whole chunks
  Unit found{-1, 0, 0, 0};
  unsigned slots = 0, fulls = 0;
#pragma unroll
  for (int r = 0; r < kBlk; ++r) {
    const int b = lane + 32 * r;
    const unsigned nf = len[r] / chunk, n = nf + (rank[r] != 0xffffffffu);
    unsigned in = n, inf = nf;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, in, o), z = __shfl_up_sync(0xffffffffu, inf, o);
      if (lane >= o) in += y, inf += z;
    }
    const unsigned u0 = slots + in - n, f0 = fulls + inf - nf;
    const bool one = s.direct && n == 1;
    auto unit = [&](unsigned i) {
      const unsigned t0 = i * chunk, t1 = i < nf ? t0 + chunk : len[r];
      const int app = i + 1 == n && (valid >> r & 1) ? kUnitAppend : 0;
      return Unit{b, (int)t0, (int)t1, (one ? kUnitDirect : 0) | app | kUnitSlot | (int)((u0 + i) << kUnitSlotShift)};
    };
    if (b < s.B) {
      if (seq) seq[b] = make_int2((int)u0, one ? -1 : (int)n);
      if ((unsigned)want - f0 < nf) found = unit((unsigned)want - f0);
      if ((unsigned)want == rank[r]) found = unit(nf);
      if (all) {
        for (unsigned i = 0; i < nf; ++i) all[f0 + i] = unit(i);
        if (n > nf) all[rank[r]] = unit(nf);
      }
    }
    slots += __shfl_sync(0xffffffffu, in, 31);
    fulls += __shfl_sync(0xffffffffu, inf, 31);
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, found.b >= 0);
  if (hit) {   // the lane that found the unit broadcasts it
    const int src = __ffs(hit) - 1;
    found.b = __shfl_sync(0xffffffffu, found.b, src);
    found.t0 = __shfl_sync(0xffffffffu, found.t0, src);
    found.t1 = __shfl_sync(0xffffffffu, found.t1, src);
    found.flags = __shfl_sync(0xffffffffu, found.flags, src);
  }
  *flags_out = flags;
  *units_out = (int)slots;
  return found;
}

// s.B <= kWarpScheduleMaxB.  (Few sequences: a quarter of the code, which a
// schedule runs through once, at the rate it is fetched.)
template <bool kWin = false>
__device__ inline Unit packed_schedule(const DenseSchedule& s, int want, uint32_t* flags_out, int* units_out, int2* seq,
                                       Unit* all) {
  static_assert(kWarpScheduleMaxB <= 128, "four blocks of 32");
  return s.B <= 32 ? packed_units<1, kWin>(s, want, flags_out, units_out, seq, all)
                   : packed_units<4, kWin>(s, want, flags_out, units_out, seq, all);
}

}  // namespace mla
