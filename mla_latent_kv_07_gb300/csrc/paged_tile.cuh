// paged_tile.cuh -- what the tensor-memory kernels over a paged cache share: the
// tile of 64 positions they work on, how its rows come in through the page
// table, and bounded waits.
//
// A tile is 64 positions x 576 columns in bf16, as nine blocks of 64 columns
// (64 rows x 128 bytes, 128-byte swizzle, 8 KB): eight latent blocks, taken
// as four pairs of 128 columns (an FP8 scale's block), and the rotary block.
// The tile is an MMA's A operand either way it is read: K-major, 64 positions
// x columns, for the scores, and MN-major, 128 latent columns x positions, for
// the value sum.  Rows come in boxes of `box` positions (the largest power of
// two up to 64 that divides the page size), which lie on one page each: bf16
// boxes by TMA straight into the blocks; FP8 codes through registers (16-byte
// loads, converted, stored swizzled), the rotary columns by TMA.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "window.cuh"

namespace mla {
namespace paged {

using namespace ptx;

constexpr int kTile = 64;
constexpr int kBlock = kTile * 128;     // 64 rows x 64 columns
constexpr int kPair = 2 * kBlock;       // 128 latent columns
constexpr int kPairsPerTile = 4;
// FP8: warps that load and convert, in four teams, one for each pair of a tile.
// (All sixteen on one pair at a time spend a pair's time on its barriers and
// latencies: 0.75 us a pair, where a team takes about as long for a tile.)
constexpr int kTeamWarps = 4, kConvWarps = kPairsPerTile * kTeamWarps;
constexpr int kConvEach = kTile * 8 / (32 * kTeamWarps);   // rows of a thread
constexpr uint32_t kWaitNs = 2000000000u;      // nanoseconds a wait may take
constexpr uint32_t kSelftestWaitNs = 1000000u;   // the same in the self-tests of the waits

// Bounded waits on this CTA's barriers; on expiry every wait of the CTA gives
// up at once and the timeout flag is raised.  The probe may suspend the thread:
// with up to 28 warps waiting, polling without a pause takes issue slots from
// those that work (FP8 at 128 heads, 131072 positions: 286 -> 260 us).
struct Wait {
  volatile int* abort;
  uint32_t* flags;   // shared memory: the CTA's MLA_DEV_* bits, then the limit in nanoseconds
  __device__ __forceinline__ bool operator()(uint64_t* b, uint32_t parity) const {
    if (bar_try_suspend(b, parity)) return true;
    const uint64_t t0 = now();
    while (!bar_try_suspend(b, parity)) {
      if (*abort) return false;
      if (now() - t0 > flags[1]) {
        *abort = 1;
        atomicOr(flags, kDevTimeout);
        return false;
      }
    }
    return true;
  }
  static __device__ __forceinline__ uint64_t now() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
  }
  // by a whole warp: the same answer in every lane
  __device__ __forceinline__ bool warp(uint64_t* b, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(b, parity));
  }
  // for operations in flight that land in any case: ignores the abort flag
  __device__ __forceinline__ void drain(uint64_t* b, uint32_t parity) const {
    const uint64_t t0 = now();
    while (!bar_try_suspend(b, parity)) {
      if (now() - t0 > flags[1]) {
        atomicOr(flags, kDevTimeout);
        return;
      }
    }
  }
};

// Eight e4m3 codes times their scale, as bf16(fp32(code) * scale).
__device__ __forceinline__ uint4 dequant8(uint2 v, float sc) {
  const uint32_t w[2] = {v.x, v.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t pair = (__nv_fp8x2_storage_t)((w[i >> 1] >> ((i & 1) * 16)) & 0xffffu);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    const __nv_bfloat162 bb = __float22bfloat162_rn(__fmul2_rn(f, make_float2(sc, sc)));
    o[i] = *reinterpret_cast<const uint32_t*>(&bb);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The producer warp's view of a tile: lane l stands for box l % boxes.  kWin (a
// windowed call): places e0 .. of the token's run, in boxes of 16.
template <bool kWin>
struct BoxesOf {
  int page, off;   // page (-1: nothing to load) and first row in it
  int live;        // boxes of the tile that are loaded
  uint32_t seen;   // kWin: the box's positions that are seen
  __device__ __forceinline__ void find(const PagedTable& pt, int b, int e0, int t1, int box, const WindowSpan& w = {}) {
    const int n = kTile / box, v = e0 + ((threadIdx.x & 31) % n) * box, e = kWin ? w.pos(v) : v;
    page = -1;
    off = 0;
    seen = 0;
    if (v < t1) {
      const int pg = pt.page_of(e);
      const int id = pt.table[(size_t)b * pt.stride + pg];
      off = e - pg * pt.page_size;
      page = id < 0 || id >= pt.num_pages ? -1 : id;
      if (kWin) seen = w.seen16(e);
    }
    live = __popc(__ballot_sync(0xffffffffu, page >= 0 && (threadIdx.x & 31) < n));
  }
  // the tile's positions that have a row, as bits (warp-collective); *bad: one
  // below t1 has none
  __device__ __forceinline__ uint64_t rows(int e0, int t1, int box, bool* bad) const {
    const int n = kTile / box;
    const uint32_t have = __ballot_sync(0xffffffffu, page >= 0 && (threadIdx.x & 31) < n);
    uint64_t mask = 0;
    if constexpr (kWin) {
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        if (const uint32_t bits = __shfl_sync(0xffffffffu, seen, k); have >> k & 1) mask |= (uint64_t)bits << (16 * k);
      *bad = __any_sync(0xffffffffu, seen != 0 && page < 0);
      return mask;
    } else {
      for (int k = 0; k < n; ++k)
        if (have >> k & 1) mask |= (box == 64 ? ~0ull : (1ull << box) - 1) << (k * box);
      const uint64_t want = t1 - e0 >= kTile ? ~0ull : (1ull << (t1 - e0)) - 1;
      *bad = (want & ~mask) != 0;
      return mask & want;
    }
  }
};
using Boxes = BoxesOf<false>;

// `blocks` blocks of 64 columns from column c0 on into dst (warp-collective);
// the phase of `full` completes when they have landed.
template <bool kWin>
__device__ __forceinline__ void load_blocks(const BoxesOf<kWin>& bx, int box, uint8_t* dst, const CUtensorMap* m, int c0,
                                            int blocks, uint64_t* full) {
  const int lane = threadIdx.x & 31, n = kTile / box;
  if (lane == 0) bar_expect_tx(full, (uint32_t)(bx.live * blocks * box * 128));
  __syncwarp();
  const int blk = lane / n, k = lane % n;
  if (blk < blocks && bx.page >= 0)
    tma3(dst + blk * kBlock + k * box * 128, m, c0 + 64 * blk, bx.off, bx.page, full);
}

// A tile's latent rows (and FP8 scales) towards L2, ahead of the loads into the
// SM (a box's rows are contiguous in its page).
template <int kFmt, bool kWin>
__device__ __forceinline__ void prefetch_rows(const BoxesOf<kWin>& bx, int box, int page_size, const void* kv, const float* kv_scale) {
  if (bx.page < 0 || (int)(threadIdx.x & 31) >= kTile / box) return;
  constexpr int kRow = kFmt == 0 ? 2 * kDc : kDc;
  const size_t row = (size_t)bx.page * page_size + bx.off;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const uint8_t*>(kv) + row * kRow), "r"(box * kRow));
  if (kFmt != 0)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(kv_scale + row * kNblk), "r"(box * kNblk * 4));
}

// The converter's view: thread t of a team takes 16 of the pair's 128 columns
// (t % 8) of rows conv_row(t) + 16 k, k = 0..3.  Threads of the pair's second
// block take the neighbouring row: chunk 2 c of row r lies at chunk position
// 2 c ^ (r % 8), so the eight threads of a quarter warp then store to all eight
// positions at a time, free of bank conflicts.
__device__ __forceinline__ int conv_row(int t) { return (t >> 3) ^ ((t >> 2) & 1); }
// The 16 rows of a k lie on one page, which lane l looks up for k = l % 4.
template <bool kWin>
struct ConvRowsOf {
  int id, off;   // page table entry (-1: no position), as fetched, and the first row in the page
  int left;      // the thread's positions below the end, from its first row on (kWin: all; the softmax tells them apart)
  // (fetch only issues the table's load; at() uses it)
  __device__ __forceinline__ void fetch(const PagedTable& pt, int b, int e0, int t1, int t, const WindowSpan& w = {}) {
    static_assert(4 * kTeamWarps == 16 && kConvEach == 4, "rows of a thread 16 apart");
    const int v = e0 + 16 * (t & 3), e = kWin ? w.pos(v) : v, pg = pt.page_of(e);
    id = -1;
    off = e - pg * pt.page_size;
    if (v < t1) id = pt.table[(size_t)b * pt.stride + pg];
    left = kWin ? 16 * kConvEach : t1 - e0 - conv_row(t);
  }
  // pool row of the lane's 16; -1: none
  __device__ __forceinline__ int at(const PagedTable& pt) const {
    return (uint32_t)id < (uint32_t)pt.num_pages ? id * pt.page_size + off : -1;
  }
};
using ConvRows = ConvRowsOf<false>;
struct ConvData {
  uint4 v[kConvEach];
  float sc[kConvEach];
  // kZero: rows that are not there as zeros (else as any row)
  template <bool kZero, bool kWin>
  __device__ __forceinline__ void load(const ConvRowsOf<kWin>& r, const PagedTable& pt, const void* kv, const float* kv_scale,
                                       int m, int t) {
    const uint8_t* base = static_cast<const uint8_t*>(kv) + 128 * m + 16 * (t & 7);
    const int mine = r.at(pt);
#pragma unroll
    for (int k = 0; k < kConvEach; ++k) {
      const int row = __shfl_sync(0xffffffffu, mine, k);
      if (kZero) {
        v[k] = make_uint4(0, 0, 0, 0);
        sc[k] = 0.f;
      }
      if (!kZero || (row >= 0 && 16 * k < r.left)) {
        const size_t at = (kZero ? row : max(row, 0)) + conv_row(t);
        v[k] = __ldcg(reinterpret_cast<const uint4*>(base + at * kDc));
        sc[k] = __ldcg(kv_scale + at * kNblk + m);
      }
    }
  }
};
// Two of a thread's four rows, converted.
struct ConvOut {
  uint4 x[2][2];
  __device__ __forceinline__ void convert(const ConvData& d, int k0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k][0] = dequant8(make_uint2(d.v[k0 + k].x, d.v[k0 + k].y), d.sc[k0 + k]);
      x[k][1] = dequant8(make_uint2(d.v[k0 + k].z, d.v[k0 + k].w), d.sc[k0 + k]);
    }
  }
  __device__ __forceinline__ void store(uint8_t* pair, int t, int k0) const {
    const int row = conv_row(t), ch = 2 * (t & 3);
    uint8_t* dst = pair + ((t >> 2) & 1) * kBlock + k0 * 2048;
    const int one = swz_chunk(row, ch), two = swz_chunk(row, ch + 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // (16 rows on: the same place in the swizzle)
      *reinterpret_cast<uint4*>(dst + k * 2048 + one) = x[k][0];
      *reinterpret_cast<uint4*>(dst + k * 2048 + two) = x[k][1];
    }
  }
};

// Largest power of two up to 64 that divides the page size (a multiple of 16).
inline int box_rows(int page_size) {
  int r = 16;
  while (r < 64 && page_size % (2 * r) == 0) r *= 2;
  return r;
}

// 3-D map of [outer][rows][inner] elements of `esize` bytes, box `box0` x
// `box1` rows, 128-byte swizzle (paged_decode.cu)
bool encode_rows(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t outer, uint32_t box1);

}  // namespace paged
}  // namespace mla
