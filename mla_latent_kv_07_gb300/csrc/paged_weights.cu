// paged_weights.cu -- the attention weight one decode step gave every row of a
// paged cache, summed over the heads and added to the row's total:
//   weight[row(b, t)] += sum_h exp(s[b, h, t] - lse[b, h])
// on the 5th-generation tensor cores, for 16, 32, 64 and 128 heads.
//
// With the log-sum-exp given, a position's weight needs no other position's:
// one pass over the rows forms the scores S[t, h] = c[t] . q_latent[h] + kR[t] .
// q_pe[h] (cache rows on the MMA's M side, heads its N, as in the paged
// decode), and a thread sums exp over its quarter of the heads of two
// positions.  36 MMAs of 32 cycles (64 at 128 heads) for 64 positions take 0.6
// (1.1) us, the 72 KB of a bf16 tile 1.6 us at an SM's share of the HBM rate.
// Measured at 128 heads: bf16, 8 x 4096 positions 14.0 us (2.7 TB/s; an SM has
// three tiles, so the first one's latency and the launch are half of it); FP8,
// 32 sequences of up to 16384, 59 us (3.2 TB/s): 1.7 us a tile, of which the
// MMAs are 1.2 and the rows' HBM time 0.9; the issuer's waits and commits fill
// the rest.  (A second issuer for the odd tiles took 1 us off, and put 0.2 on
// the 5.6 of 2 sequences of 1001 positions.)
//
// The tiles of all sequences, in order, are cut into equal runs, one per SM, so
// an SM changes its queries only where a sequence ends in its run.
//
// Warps: 0 producer of the queries and rotary columns; 1 issues the MMAs and
// owns tensor memory; 4-7 and 8-11 take the even and the odd tiles' scores (a
// buffer each, so a group has two tiles' time); 12-15 (bf16) producers of the
// latent columns, one pair each; 12-27 (FP8) load and convert them.  Waits are
// bounded; on expiry the CTA flags it, stops issuing and tears down.
#include <cuda.h>
#include <cuda_bf16.h>

#include <string.h>

#include "common.cuh"
#include "paged_tile.cuh"
#include "ring.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace paged {
namespace {

template <int kFmt, int kH>
struct WCfg {
  static constexpr int kPairs = kH == 128 ? 4 : kH == 64 ? 8 : 10;   // latent ring
  static constexpr int kRopes = kH == 128 ? 2 : 3;
  static constexpr int kThreads = 32 * (12 + (kFmt == 0 ? 4 : kConvWarps));
  static constexpr int kQBlk = kH * 128;
  static constexpr int kRopeOff = kPairs * kPair;
  static constexpr int kQOff = kRopeOff + kRopes * kBlock;
  static constexpr int kBarOff = kQOff + 9 * kQBlk;
  static constexpr int kSmem = kBarOff + 2048 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kH;
  static_assert(kSmem <= 232448, "shared memory");
};

struct WParams {
  CUtensorMap m_kv, m_pe, m_ql, m_qp;   // as the paged decode's
  const void* kv;
  const float* kv_scale;
  float* weight;
  PagedTable pt;
  const float* lse;
  const int* end_pos;
  int max_end_pos, B, box;
  float scale_log2;
  uint32_t* status;
  int selftest;          // self-test of the waits: the first rotary block of CTA 0 never counts as loaded
};

struct __align__(16) WShared {
  uint64_t full[10], empty[10];
  uint64_t rfull[3], rempty[3];
  uint64_t sfull[2], sfree[2], gbar[2];
  uint64_t qfull, qempty, drain;
  long long scan[32];          // tiles before a warp's sequences
  long long left;              // tiles of this CTA's run
  int b0, t0;                  // where it begins: sequence, tile
  uint32_t tmem, flags, limit;   // (the last two as Wait has them)
  volatile int abort;
  int issued[kPairsPerTile];   // bf16: tiles whose pair each latent producer has loaded
  int ropes, segs;             // rotary blocks and segments' queries loaded
  int base[3][4];              // per rotary slot: pool row of the tile's boxes (-1: none)
  __align__(16) float nl[2][128];   // per group: -lse (log2 units) of its sequence's heads
};
static_assert(sizeof(WShared) <= 2048, "barrier block");

// The run of tiles, walked by every role on its own.
struct Walk {
  const int* end_pos;
  int max_end, b, t, len;   // sequence, tile, the sequence's positions
  long long left;
  __device__ __forceinline__ int length(int i) const {
    const int e = end_pos[i];
    return e < 0 ? 0 : (e > max_end ? max_end : e);
  }
  __device__ __forceinline__ void start(const WParams& p, const WShared* sh) {
    end_pos = p.end_pos;
    max_end = p.max_end_pos;
    b = sh->b0;
    t = sh->t0;
    left = sh->left;
    len = left > 0 ? length(b) : 0;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ int e0() const { return t * kTile; }
  // the sequence's last tile in this run
  __device__ __forceinline__ bool last() const { return left == 1 || (t + 1) * (long long)kTile >= len; }
  __device__ __forceinline__ void step() {
    --left;
    ++t;
    if (left > 0 && (long long)t * kTile >= len) {
      t = 0;
      do len = length(++b);   // (tiles are left, so a sequence with positions follows)
      while (len == 0);
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The copies of a CTA that gave up land before its shared memory goes away: the
// last queries, and the last one into each slot of the rings (by one warp, once
// no producer starts another).  (Out of line: 59.1 us for 60.4, 128 heads, FP8,
// 32 sequences of 1k-16k.)
template <int kFmt, int kH>
__device__ __noinline__ void drain_copies(WShared* sh) {
  using C = WCfg<kFmt, kH>;
  constexpr int kPairs = C::kPairs, kRopes = C::kRopes;
  const Wait wait{&sh->abort, &sh->flags};
  const int lane = threadIdx.x & 31;
  if (lane < kPairs) {
    const int n = kFmt == 0 ? last_load(sh->issued, kPairsPerTile, kPairs, lane) : -1;
    if (n >= 0) wait.drain(&sh->full[lane], (n / kPairs) & 1);
  } else if (lane < kPairs + kRopes) {
    const int s = lane - kPairs, n = last_load(&sh->ropes, 1, kRopes, s);
    if (n >= 0) wait.drain(&sh->rfull[s], (n / kRopes) & 1);
  } else if (lane == 31 && sh->segs > 0) {
    wait.drain(&sh->qfull, (sh->segs - 1) & 1);
  }
  __syncwarp();
}

template <int kFmt, int kH>
__global__ void __launch_bounds__(WCfg<kFmt, kH>::kThreads, 1) weights_kernel(const __grid_constant__ WParams p) {
  using C = WCfg<kFmt, kH>;
  constexpr int kPairs = C::kPairs, kRopes = C::kRopes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WShared* sh = reinterpret_cast<WShared*>(sm + C::kBarOff);
  auto pair = [&](int s) { return sm + s * kPair; };
  auto rope = [&](int s) { return sm + C::kRopeOff + s * kBlock; };
  uint8_t* qs = sm + C::kQOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Wait wait{&sh->abort, &sh->flags};

  // ---------------------------------------------------------------- set-up
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairs; ++s) {
      bar_init(&sh->full[s], kFmt == 0 ? 1 : kTeamWarps);
      bar_init(&sh->empty[s], 1);
    }
    for (int s = 0; s < kRopes; ++s) {
      bar_init(&sh->rfull[s], s == 0 && p.selftest && blockIdx.x == 0 ? 2 : 1);   // (self-test: one arrival never comes)
      bar_init(&sh->rempty[s], 5);   // the MMAs' commit, and the group's warps have read base
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(&sh->sfull[s], 1);
      bar_init(&sh->sfree[s], 4);
      bar_init(&sh->gbar[s], 4);
    }
    bar_init(&sh->qfull, 1);
    bar_init(&sh->qempty, 1);
    bar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->flags = 0;
    sh->limit = p.selftest ? kSelftestWaitNs : kWaitNs;
    sh->left = 0;
    for (int m = 0; m < kPairsPerTile; ++m) sh->issued[m] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    constexpr uint32_t cols = C::kTmemCols;
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&sh->tmem)), "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  // The CTA's run: tiles [total c / G, total (c + 1) / G) of all sequences'.
  // Every thread takes a run of sequences; their tiles, scanned over the
  // block, say which thread's hold the beginning.
  {
    const int nw = C::kThreads / 32, per = (p.B + C::kThreads - 1) / C::kThreads, first = threadIdx.x * per;
    long long mine = 0;
    uint32_t flags = 0;
    for (int b = first; b < first + per && b < p.B; ++b) {
      int e = p.end_pos[b];
      if (e < 0 || e > p.max_end_pos) {
        flags = kDevEndPosClamped;
        e = e < 0 ? 0 : p.max_end_pos;
      }
      mine += (e + (long long)kTile - 1) / kTile;
    }
    if (flags && blockIdx.x == 0 && p.status) atomicOr(p.status, flags);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
      before += w < warp ? sh->scan[w] : 0;
      total += sh->scan[w];
    }
    const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    long long at = before + incl - mine;   // tiles before this thread's sequences
    if (lo < hi && lo >= at && lo < at + mine) {
      for (int b = first;; ++b) {
        int e = p.end_pos[b];
        e = e < 0 ? 0 : (e > p.max_end_pos ? p.max_end_pos : e);
        const long long n = (e + (long long)kTile - 1) / kTile;
        if (lo < at + n) {
          sh->b0 = b;
          sh->t0 = (int)(lo - at);
          sh->left = hi - lo;
          break;
        }
        at += n;
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh->tmem;
  Walk w;
  w.start(p, sh);

  // FP8: registers to where they are needed: 28 warps x 72 at launch = 4 x 56
  // + 8 x 64 + 16 x 80
  static_assert(kFmt == 0 || 4 * 56 + 8 * 64 + kConvWarps * 80 <= C::kThreads / 32 * 72, "register split");
  if (warp < 4) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    // ------------------------------------- queries and rotary columns
    Walk ahead = w;   // the tile looked up: two tiles on, and its rows towards L2
    Boxes bx, b1, b2;
    auto look = [&](bool fetch) {
      bx = b1;
      b1 = b2;
      if (!ahead.more()) return;
      b2.find(p.pt, ahead.b, ahead.e0(), ahead.len, p.box);
      if (fetch) prefetch_rows<kFmt>(b2, p.box, p.pt.page_size, p.kv, p.kv_scale);
      ahead.step();
    };
    // (bf16's own loads run as far ahead, and would only be delayed)
    look(kFmt != 0);
    look(kFmt != 0);
    int seq = -1, segs = 0, ropes = 0;   // segments' queries loaded, rotary blocks loaded
    for (; w.more(); w.step()) {
      if (w.b != seq) {
        seq = w.b;
        if (!wait.warp(&sh->qempty, (segs & 1) ^ 1)) break;
        if (lane == 0) {
          bar_expect_tx(&sh->qfull, 9 * C::kQBlk);
          for (int k = 0; k < 8; ++k) tma3(qs + k * C::kQBlk, &p.m_ql, 64 * k, 0, w.b, &sh->qfull);
          tma3(qs + 8 * C::kQBlk, &p.m_qp, 0, 0, w.b, &sh->qfull);
        }
        __syncwarp();
        ++segs;
      }
      look(kFmt != 0);
      const int s = ropes % kRopes, n = kTile / p.box;
      if (!wait.warp(&sh->rempty[s], ((ropes / kRopes) & 1) ^ 1)) break;
      if (lane < n) sh->base[s][lane] = bx.page < 0 ? -1 : bx.page * p.pt.page_size + bx.off;
      bool bad;
      bx.rows(w.e0(), w.len, p.box, &bad);
      if (bad && lane == 0) atomicOr(&sh->flags, kDevBadPage);
      __syncwarp();
      load_blocks(bx, p.box, rope(s), &p.m_pe, 0, 1, &sh->rfull[s]);
      ++ropes;
    }
    if (lane == 0) {
      sh->ropes = ropes;
      sh->segs = segs;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id = idesc(kTile, kH, false, false);
    const bool el = elect_one();
    const uint64_t d_kv = sdesc(sa(pair(0)), 16, 1024), d_pe = sdesc(sa(rope(0)), 16, 1024);
    const uint64_t d_q = sdesc(sa(qs), 16, 1024);
    int s = 0, ph = 0, seq = -1, segs = 0;
    bool ok = true;
    for (int i = 0; w.more() && ok; ++i, w.step()) {
      if (w.b != seq) {
        seq = w.b;
        ok = wait.warp(&sh->qfull, segs++ & 1);
      }
      const int sb = i & 1;
      ok = wait.warp(&sh->sfree[sb], ((i >> 1) & 1) ^ 1) && ok;
      if (!ok) break;
      const uint32_t ds = tmem + sb * kH;
      uint64_t q = d_q;
#pragma unroll 1
      for (int m = 0; m < kPairsPerTile; ++m) {
        ok = wait.warp(&sh->full[s], ph) && ok;
        tc_after();
        const uint64_t a = sdesc_at(d_kv, s * kPair);
        mma_ss4_if<2>(el, ds, a, q, id, m);
        mma_ss4_if<2>(el, ds, sdesc_at(a, kBlock), sdesc_at(q, C::kQBlk), id, 1);
        mma_commit_if(el, &sh->empty[s]);
        q = sdesc_at(q, 2 * C::kQBlk);
        if (++s == kPairs) s = 0, ph ^= 1;
      }
      const int rs = i % kRopes;
      ok = wait.warp(&sh->rfull[rs], (i / kRopes) & 1) && ok;
      tc_after();
      mma_ss4_if<2>(el, ds, sdesc_at(d_pe, rs * kBlock), q, id, 1);
      mma_commit_if(el, &sh->rempty[rs]);
      if (w.last()) mma_commit_if(el, &sh->qempty);
      mma_commit_if(el, &sh->sfull[sb]);
    }
    mma_commit_if(el, &sh->drain);
    wait.drain(&sh->drain, 0);
  }
  } else if (warp < 12) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ weights
    // thread: positions fl and fl + 8 of the quadrant's 16, heads 8 k + 2 fc
    // and 8 k + 2 fc + 1
    const int g = (warp - 4) >> 2, quad = warp & 3, fl = lane >> 2, fc = lane & 3;
    const int row0 = 16 * quad + fl, row1 = row0 + 8;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16) + g * kH;
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    const float* nl = sh->nl[g];
    int gph = 0, seq = -1;
    bool ok = true;
    // among the group's four warps (bounded)
    auto group_sync = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->gbar[g]);
      ok = wait.warp(&sh->gbar[g], gph) && ok;
      gph ^= 1;
    };
    if (g == 1 && w.more()) w.step();
    for (int i = g; w.more() && ok; i += 2) {
      if (w.b != seq) {
        seq = w.b;
        group_sync();   // the group is done with the sequence before
        const int t = threadIdx.x - 128 - 128 * g;
        if (t < kH) {
          // -inf (no sum) gives weight 0, as does +inf
          const float l = p.lse[(size_t)w.b * kH + t];
          sh->nl[g][t] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
        }
        group_sync();
      }
      const int rs = i % kRopes;
      ok = ok && wait.warp(&sh->rfull[rs], (i / kRopes) & 1);   // (for base; long complete)
      const volatile int* base = sh->base[rs];
      const int lim = w.len - w.e0(), b0 = base[row0 / p.box], b1 = base[row1 / p.box];
      const int at0 = row0 < lim && b0 >= 0 ? b0 + row0 % p.box : -1, at1 = row1 < lim && b1 >= 0 ? b1 + row1 % p.box : -1;
      ok = ok && wait.warp(&sh->sfull[g], (i >> 1) & 1);
      tc_after();
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
      for (int c = 0; c < kH; c += 32) {
        constexpr int kN = kH < 32 ? kH / 8 : 4;
        uint32_t r[4 * kN];
        if constexpr (kN == 2) {
          TC_LD16L_X2(tl + c, r);
        } else {
          TC_LD16L_X4(tl + c, r);
        }
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const float2 m = *reinterpret_cast<const float2*>(nl + c + 8 * k + 2 * fc);
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1])), sl2, m);
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])), sl2, m);
          s0 = __fadd2_rn(s0, make_float2(ex2(x.x), ex2(x.y)));
          s1 = __fadd2_rn(s1, make_float2(ex2(y.x), ex2(y.y)));
        }
      }
      tc_before();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(&sh->sfree[g]);
        bar_arrive(&sh->rempty[rs]);
      }
      float a = s0.x + s0.y, b = s1.x + s1.y;
      a += __shfl_xor_sync(0xffffffffu, a, 1);
      b += __shfl_xor_sync(0xffffffffu, b, 1);
      a += __shfl_xor_sync(0xffffffffu, a, 2);
      b += __shfl_xor_sync(0xffffffffu, b, 2);
      // (an atomic: other sequences may share the row; one addition from this
      // one, so the sum's value does not depend on timing otherwise)
      if (ok && fc == 0) {
        if (at0 >= 0) atomicAdd(p.weight + at0, a);
        if (at1 >= 0) atomicAdd(p.weight + at1, b);
      }
      w.step();
      if (w.more()) w.step();
    }
  } else {
    if constexpr (kFmt == 0) {
      // ----------------------------------- producers of the latent columns
      const int m = warp - 12;
      int i = 0;
      Boxes bx, next;
      if (w.more()) next.find(p.pt, w.b, w.e0(), w.len, p.box);
      while (w.more()) {
        bx = next;
        w.step();
        if (w.more()) next.find(p.pt, w.b, w.e0(), w.len, p.box);
        const int n = kPairsPerTile * i + m, s = n % kPairs;
        if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) break;
        load_blocks(bx, p.box, pair(s), &p.m_kv, 128 * m, 2, &sh->full[s]);
        ++i;
      }
      if (lane == 0) sh->issued[m] = i;
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
      // ------------------------------------------------------ converter
      const int m = (warp - 12) / kTeamWarps, t = threadIdx.x - 384 - m * 32 * kTeamWarps;
      ConvRows next;
      ConvData d;
      Walk on = w;   // the tile whose rows are looked up
      auto look = [&]() {
        if (!on.more()) return;
        next.fetch(p.pt, on.b, on.e0(), on.len, t);
        on.step();
      };
      next.id = -1;
      next.off = next.left = 0;
      look();
      d.load<false>(next, p.pt, p.kv, p.kv_scale, m, t);
      look();
      const int tiles = (int)w.left;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        ConvOut o0, o1;
        o0.convert(d, 0);
        o1.convert(d, 2);
        d.load<false>(next, p.pt, p.kv, p.kv_scale, m, t);   // (past the run's end: any row again)
        look();
        const int n = kPairsPerTile * i + m, s = n % kPairs;
        if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) break;
        o0.store(pair(s), t, 0);
        o1.store(pair(s), t, 2);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh->full[s]);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_before();
  __syncthreads();
  if (warp == 0 && sh->abort) drain_copies<kFmt, kH>(sh);
  if (threadIdx.x == 0 && sh->flags && p.status) atomicOr(p.status, sh->flags);
  if (warp == 1) {
    tc_after();
    constexpr uint32_t cols = C::kTmemCols;
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
}

template <int kFmt, int kH>
cudaError_t launch(const WParams& p, int sms, cudaStream_t s) {
  using C = WCfg<kFmt, kH>;
  cudaError_t e = ensure_smem<weights_kernel<kFmt, kH>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(weights_kernel<kFmt, kH>, dim3((unsigned)sms), dim3(C::kThreads), C::kSmem, s, p);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_weights(const WeightsParams& d, int sms, cudaStream_t s) {
  using namespace paged;
  WParams p;
  memset(&p, 0, sizeof(p));
  const uint64_t pages = (uint64_t)d.pt.num_pages, rows = (uint64_t)d.pt.page_size, B = (uint64_t)d.B, H = (uint64_t)d.H;
  p.box = box_rows(d.pt.page_size);
  if ((d.fmt == 0 && !encode_rows(&p.m_kv, d.kv, kDc, rows, pages, p.box)) ||
      !encode_rows(&p.m_pe, d.pe, kDr, rows, pages, p.box) || !encode_rows(&p.m_ql, d.q_latent, kDc, H, B, d.H) ||
      !encode_rows(&p.m_qp, d.q_pe, kDr, H, B, d.H))
    return cudaErrorInvalidValue;
  p.kv = d.kv;
  p.kv_scale = d.kv_scale;
  p.weight = d.weight;
  p.pt = d.pt;
  p.lse = d.lse;
  p.end_pos = d.end_pos;
  p.max_end_pos = d.max_end_pos;
  p.B = d.B;
  p.scale_log2 = d.scale_log2;
  p.status = d.status;
  p.selftest = d.withhold_tile >= 0 ? 1 : 0;
  if (d.fmt == 0)
    return d.H == 16   ? launch<0, 16>(p, sms, s)
           : d.H == 32 ? launch<0, 32>(p, sms, s)
           : d.H == 64 ? launch<0, 64>(p, sms, s)
                       : launch<0, 128>(p, sms, s);
  return d.H == 16   ? launch<1, 16>(p, sms, s)
         : d.H == 32 ? launch<1, 32>(p, sms, s)
         : d.H == 64 ? launch<1, 64>(p, sms, s)
                     : launch<1, 128>(p, sms, s);
}

}  // namespace mla
