// ring.cuh -- which load a slot of the latent ring received last.  (Plain C++ as
// well, so that the arithmetic is tested without a GPU.)
//
// Pair m (0 .. per - 1) of tile i is load n = per i + m.  Producer m makes it,
// into slot n % slots, once load n - slots has been read; a slot's loads, which
// several producers may make, are so made in order.
#pragma once

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ inline
#else
#define MLA_HD inline
#endif

namespace mla {
namespace paged {

// The last load made into slot s when producer m has made those of issued[m]
// tiles; -1: none.  Every other load into the slot has been read, so this one
// alone may be in flight.
MLA_HD int last_load(const int* issued, int per, int slots, int s) {
  int last = -1;
  for (int m = 0; m < per; ++m) {
    int n = per * (issued[m] - 1) + m;
    for (int k = 0; k < slots && n >= 0 && n % slots != s; ++k) n -= per;   // (slots steps pass every slot m uses)
    if (n >= 0 && n % slots == s && n > last) last = n;
  }
  return last;
}

}  // namespace paged
}  // namespace mla
