// paged_chunk.cu -- windowed attention of many tokens over a paged cache: a
// prompt's chunk, or the drafted tokens of many sequences.
//
// What is computed is paged_decode.cu's, with its tile (64 positions), its
// layout (cache rows on the MMA's M side, 64 columns on the N side) and its
// softmax; what differs is what many tokens allow:
//   * The 64 columns are (token, head) pairs in order: the heads of four tokens of
//     16, two of 32, one of 64, or half of one of 128.  A tile's rows are loaded,
//     converted and multiplied once for all of them; each column's scores are
//     masked by what its token sees, and the tile's run is the union of the
//     tokens' (consecutive ones: their windows overlap in all but a few rows).
//   * A CTA per SM takes units one after another, and nothing is torn down in
//     between: the tiles of all its units are one sequence through the rings, so
//     the next unit's rows come in while the last one's outputs leave.  Between
//     two units only the queries change (once the last scores are issued) and the
//     accumulators (once they are read).
//
// Rows that some of a unit's tokens see and others do not: P is 0 for the latter,
// and 0 times a row that holds NaN or an infinity must not reach them.  Such a row
// shows in its scores (every column's is non-finite then); where one does, the
// row's pieces that are non-finite are zeroed before the value sum.  The tokens
// that see the row are NaN all the same, by their scores; with a score of
// -infinity it weighs 0, and NaN (0 times an infinite value) is left only in tiles
// that all tokens see.  (Zeros in every row that is not seen, without looking: 254 us for the
// first case below.)
//
// Measured, 1000 tokens of two sequences, window 512: 128 heads bf16 216 us (665
// TFLOP/s; a pair per token, decode_tc.cu, took 318), FP8 269; 64 heads 113 and
// 142, 32 heads 68 and 86, 16 heads 37 and 50 (a CTA per token: 120 and 151).  The sum
// of the rounded weights is 0 to 7% of that (214 and 264 us without).  A unit
// takes 16 us: nine tiles of 1.3 us, the time of a tile's 52 MMAs of about 48 cycles
// (36 of them 64 rows high, which take no less than 128), and 4 us in which the
// last value sum ends and the outputs leave.  FP8 tiles take 1.7 us: the conversion's
// instructions (the SM issues in 70% of its cycles).  Rows that are not seen are
// converted like others (testing every row instead: 285 us, 268 without).
//
// Warps as in paged_decode.cu: 0 producer of the rotary columns, queries and
// masks; 1 (which owns tensor memory) and 3 issue the scores' MMAs; 2 the value
// sum's; 4-7 and 8-11 softmax and outputs of the lower and upper 32 columns; 12-15
// (bf16) producers of the latent columns; 12-27 (FP8) load and convert them.
//
// Waits are bounded; on expiry the CTA flags it, stops issuing and tears down.
#include <cuda.h>
#include <cuda_bf16.h>

#include <float.h>
#include <string.h>

#include "common.cuh"
#include "paged_tile.cuh"
#include "ring.cuh"
#include "schedule.cuh"
#include "tc_ptx.cuh"
#include "window.cuh"

namespace mla {
namespace paged {
namespace {

constexpr float kRaise = 24.0f;   // (paged_decode.cu)
constexpr int kCols = 64;         // columns of a unit
constexpr int kHT = kCols / 2;    // of a softmax thread's group
constexpr int kK = kHT / 8;

template <int kFmt>
struct Cfg {
  static constexpr int kPairs = 8;     // latent ring: pairs of blocks (two tiles)
  static constexpr int kRopes = 3;     // rotary blocks (and P)
  static constexpr int kThreads = 32 * (12 + (kFmt == 0 ? 4 : kConvWarps));
  static constexpr int kQBlk = kCols * 128;
  static constexpr int kRopeOff = kPairs * kPair;
  static constexpr int kQOff = kRopeOff + kRopes * kBlock;
  static constexpr int kBarOff = kQOff + 9 * kQBlk;
  static constexpr int kSmem = kBarOff + 2048 + 1024;
  static constexpr uint32_t kTmemS = 4 * kCols;   // S: [buffer][issuer] of kCols columns
  static_assert(kSmem <= 232448, "shared memory");
};

struct Params {
  CUtensorMap m_kv;   // bf16: latent [pages][rows][512] (box 64 x 16)
  CUtensorMap m_pe;   // rotary [pages][rows][64] (box 64 x 16)
  CUtensorMap m_ql;   // q_latent [B][s H][512] (box 64 x 64)
  CUtensorMap m_qp;   // q_pe [B][s H][64] (box 64 x 64)
  const void* kv;
  const float* kv_scale;
  PagedTable pt;
  const int* end_pos;
  int max_end_pos, s, log_h, window, sinks;
  int per_seq, units;   // units of a sequence and in all
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;     // cleared before the launch
  int selftest;         // self-test of the waits: the first rotary block of CTA 0 never counts as loaded
};

struct __align__(16) Shared {
  uint64_t full[8], empty[8];      // latent pair landed / read by its value sum
  uint64_t rfull[3], rempty[3];    // rotary block landed / tile's value sum done (P and rotary free)
  uint64_t sfull[2], sfree[2];
  uint64_t pfull[3];               // P written
  uint64_t pfix[2];                // P corrected by a group that raised its references
  uint64_t gbar[2];                // among a group's warps
  uint64_t qbar, qfree;            // the unit's queries landed / read by both issuers
  uint64_t ofree;                  // the unit's accumulators read
  uint64_t drain, drain_pv;
  uint32_t tmem;
  uint32_t flags, limit;   // (as Wait has them)
  volatile int abort;
  int issued[kPairsPerTile];   // bf16: tiles whose pair each latent producer has loaded
  int ropes, qloads;           // rotary blocks and queries loaded
  volatile int need[3][2];     // [rotary slot][group]: tile number + 1 if references must be raised
  __align__(8) uint16_t seen[3][4][4];   // per rotary slot: what each token sees of the tile's four boxes
  __align__(16) float alpha[kCols];      // factor of the last raise
  __align__(16) float inv[kCols];        // minus the unit's last references, then the inverse sums
  float part[2][4][32];  // per group and lane quadrant: tile maxima, then row sums
};
static_assert(sizeof(Shared) <= 2048, "barrier block");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A unit's tokens and the run of places loaded for them.
struct ChunkUnit {
  int b, col0, ntiles;
  int end0;          // positions of the first token (those of the next: one more each)
  WindowSpan span;   // of all its tokens
};
template <int kTok>
__device__ __forceinline__ ChunkUnit unit_of(const Params& p, int u, uint32_t* flags) {
  ChunkUnit c;
  c.b = u / p.per_seq;
  c.col0 = (u - c.b * p.per_seq) * kCols;
  int end = p.end_pos[c.b];
  if (end < 0 || end > p.max_end_pos) {
    *flags |= kDevEndPosClamped;
    end = end < 0 ? 0 : p.max_end_pos;
  }
  const int j0 = c.col0 >> p.log_h, more = min(kTok, p.s - j0) - 1;
  c.end0 = end - p.s + j0 + 1;
  c.span = window_span(max(0, c.end0 + more), p.window + more, p.sinks);
  c.ntiles = (c.span.places() + kTile - 1) / kTile;
  return c;
}

// whether one of eight bf16 values is NaN or infinite
__device__ __forceinline__ bool non_finite(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

template <int kFmt, int kTok>
__global__ void __launch_bounds__(Cfg<kFmt>::kThreads, 1) chunk_kernel(const __grid_constant__ Params p) {
  using C = Cfg<kFmt>;
  constexpr int kPairs = C::kPairs, kRopes = C::kRopes, kMine = kTok == 4 ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared* sh = reinterpret_cast<Shared*>(sm + C::kBarOff);
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
      bar_init(&sh->rempty[s], 1);
      bar_init(&sh->pfull[s], 8);
      sh->need[s][0] = sh->need[s][1] = 0;
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(&sh->sfull[s], 2);
      bar_init(&sh->sfree[s], 8);
      bar_init(&sh->pfix[s], 4);
      bar_init(&sh->gbar[s], 4);
    }
    bar_init(&sh->qbar, 1);
    bar_init(&sh->qfree, 2);
    bar_init(&sh->ofree, 8);
    bar_init(&sh->drain, 2);
    bar_init(&sh->drain_pv, 1);
    sh->abort = 0;
    sh->flags = 0;
    sh->limit = p.selftest ? kSelftestWaitNs : kWaitNs;
    for (int m = 0; m < kPairsPerTile; ++m) sh->issued[m] = 0;
    sh->ropes = sh->qloads = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sa(&sh->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh->tmem;
  pdl_wait();
  pdl_trigger();

  // Every role walks the CTA's units and their tiles; g counts tiles over all of
  // them and gives the rings' slots and phases.
  uint32_t unused = 0;
  // FP8: registers to where they are needed: 28 warps x 72 at launch = 4 x 40
  // + 8 x 72 + 16 x 80 (4 x 56 + 8 x 64: 285 -> 302 us, 1000 tokens of 128 heads)
  static_assert(kFmt == 0 || 4 * 40 + 8 * 72 + kConvWarps * 80 <= C::kThreads / 32 * 72, "register split");
  if (warp < 4) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      int g = 0, n = 0;   // tiles, units with tiles
      bool ok = true;
      uint32_t flags = 0;
      for (int u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const ChunkUnit c = unit_of<kTok>(p, u, &flags);
        if (c.ntiles == 0) continue;
        const int t1 = c.span.places();
        BoxesOf<true> bx, next, after;
        next.find(p.pt, c.b, 0, t1, 16, c.span);
        after.find(p.pt, c.b, kTile, t1, 16, c.span);
        if (kFmt != 0) {
          prefetch_rows<kFmt>(next, 16, p.pt.page_size, p.kv, p.kv_scale);
          prefetch_rows<kFmt>(after, 16, p.pt.page_size, p.kv, p.kv_scale);
        }
        if (n > 0 && !wait.warp(&sh->qfree, (n - 1) & 1)) break;
        if (lane == 0) {
          bar_expect_tx(&sh->qbar, 9 * C::kQBlk);
          for (int k = 0; k < 8; ++k) tma3(qs + k * C::kQBlk, &p.m_ql, 64 * k, c.col0, c.b, &sh->qbar);
          tma3(qs + 8 * C::kQBlk, &p.m_qp, 0, c.col0, c.b, &sh->qbar);
          sh->qloads = n + 1;
        }
        __syncwarp();
        ++n;
        for (int i = 0; i < c.ntiles; ++i, ++g) {
          bx = next;
          next = after;
          after.find(p.pt, c.b, (i + 2) * kTile, t1, 16, c.span);
          if (kFmt != 0) prefetch_rows<kFmt>(after, 16, p.pt.page_size, p.kv, p.kv_scale);
          const int s = g % kRopes;
          if (!wait.warp(&sh->rempty[s], ((g / kRopes) & 1) ^ 1)) {
            ok = false;
            break;
          }
          // lane 4 t + k: what token t sees of box k
          if (lane < 4 * kTok) {
            const int v = i * kTile + 16 * (lane & 3), end = max(0, c.end0 + (lane >> 2));
            const bool live = v < t1 && bx.page >= 0 && (c.col0 >> p.log_h) + (lane >> 2) < p.s;
            sh->seen[s][lane >> 2][lane & 3] =
                live ? (uint16_t)window_span(end, p.window, p.sinks).seen16(c.span.pos(v)) : (uint16_t)0;
          }
          if (__any_sync(0xffffffffu, bx.seen != 0 && bx.page < 0) && lane == 0) flags |= kDevBadPage;
          __syncwarp();   // (the arrival of load_blocks releases the masks)
          load_blocks(bx, 16, rope(s), &p.m_pe, 0, 1, &sh->rfull[s]);
          if (lane == 0) sh->ropes = g + 1;
        }
      }
      if (lane == 0 && flags) atomicOr(&sh->flags, flags);
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------- scores' issuers
      const int half = warp >> 1;
      constexpr uint32_t id = idesc(kTile, kCols, false, false);
      const bool el = elect_one();
      const uint64_t d_kv = sdesc(sa(pair(0)), 16, 1024), d_pe = sdesc(sa(rope(0)), 16, 1024);
      const uint64_t d_q = sdesc(sa(qs), 16, 1024);
      bool ok = true;
      int g = 0, n = 0, s = 2 * half, ph = 0;   // s, ph: the ring's slot and phase
      for (int u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const int ntiles = unit_of<kTok>(p, u, &unused).ntiles;
        if (ntiles == 0) continue;
        ok = wait.warp(&sh->qbar, n++ & 1);
        for (int i = 0; i < ntiles && ok; ++i, ++g) {
          const int sb = g & 1;
          ok = wait.warp(&sh->sfree[sb], ((g >> 1) & 1) ^ 1);
          if (!ok) break;
          const uint32_t ds = tmem + C::kTmemS + (2 * sb + half) * kCols;
          uint64_t q = sdesc_at(d_q, half * 4 * C::kQBlk);
#pragma unroll 1
          for (int m = 0; m < 2; ++m) {
            ok = wait.warp(&sh->full[s], ph) && ok;
            tc_after();
            const uint64_t a = sdesc_at(d_kv, s * kPair);
            mma_ss4_if<2>(el, ds, a, q, id, m);
            mma_ss4_if<2>(el, ds, sdesc_at(a, kBlock), sdesc_at(q, C::kQBlk), id, 1);
            q = sdesc_at(q, 2 * C::kQBlk);
            if (++s == kPairs) s = 0, ph ^= 1;
          }
          if (half == 1) {
            const int rs = g % kRopes;
            ok = wait.warp(&sh->rfull[rs], (g / kRopes) & 1) && ok;
            tc_after();
            mma_ss4_if<2>(el, ds, sdesc_at(d_pe, rs * kBlock), q, id, 1);
          }
          mma_commit_if(el, &sh->sfull[sb]);
          s += 2;   // the other warp's pairs
          if (s >= kPairs) s -= kPairs, ph ^= 1;
        }
        mma_commit_if(el, &sh->qfree);
      }
      mma_commit_if(el, &sh->drain);
      wait.drain(&sh->drain, 0);
    } else {
      // ----------------------------------------------------- value sum's issuer
      constexpr uint32_t id = idesc(128, kCols, true, true);
      const bool el = elect_one();
      const uint64_t d_v = sdesc(sa(pair(0)), kBlock, 1024), d_p = sdesc(sa(rope(0)), kBlock, 1024);
      bool ok = true;
      int g = 0, n = 0, s = 0, fixed0 = 0, fixed1 = 0;
      for (int u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const int ntiles = unit_of<kTok>(p, u, &unused).ntiles;
        if (ntiles == 0) continue;
        for (int i = 0; i < ntiles && ok; ++i, ++g) {
          const int rs = g % kRopes;
          ok = wait.warp(&sh->pfull[rs], (g / kRopes) & 1);
          if (ok && sh->need[rs][0] == g + 1) ok = wait.warp(&sh->pfix[0], fixed0++ & 1);
          if (ok && sh->need[rs][1] == g + 1) ok = wait.warp(&sh->pfix[1], fixed1++ & 1);
          if (ok && i == 0 && n > 0) ok = wait.warp(&sh->ofree, (n - 1) & 1);
          if (!ok) break;
          tc_after();
          const uint64_t pd = sdesc_at(d_p, rs * kBlock);
#pragma unroll 1
          for (int m = 0; m < kPairsPerTile; ++m) {
            static_assert(kTile == 64, "four steps of 16 positions");
            mma_ss4_if<128>(el, tmem + m * kCols, sdesc_at(d_v, s * kPair), pd, id, i);
            mma_commit_if(el, &sh->empty[s]);
            if (++s == kPairs) s = 0;
          }
          mma_commit_if(el, &sh->rempty[rs]);
        }
        ++n;
      }
      mma_commit_if(el, &sh->drain_pv);
      wait.drain(&sh->drain_pv, 0);
    }
  } else if (warp < 12) {

    // ------------------------------------------------------------ softmax
    // thread: positions fl and fl + 8 of the quadrant's 16, columns 8 k + 2 fc
    // and 8 k + 2 fc + 1 of the group's (see paged_decode.cu), which belong to
    // token 2 grp + k / 2 (four tokens), grp (two) or 0 (one)
    const int grp = (warp - 4) >> 2, quad = warp & 3, fl = lane >> 2, fc = lane & 3;
    const int row0 = 16 * quad + fl, row1 = row0 + 8;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    const int tok0 = kTok == 4 ? 2 * grp : kTok == 2 ? grp : 0;
    constexpr int kPer = kK / kMine;   // k of a token
    int gph = 0, g = 0;
    bool ok = true;
    auto group_sync = [&]() -> bool {   // among the group's four warps
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->gbar[grp]);
      const bool all = wait.warp(&sh->gbar[grp], gph);
      gph ^= 1;
      return all;
    };
    auto scores = [&](uint32_t at, float2 (&r)[2 * kK]) {   // the sum of what the two issuers' columns gave
      uint32_t a[4 * kK], b[4 * kK];
      TC_LD16L_X4(at, a);
      TC_LD16L_X4(at + kCols, b);
      tc_wait_ld();
#pragma unroll
      for (int k = 0; k < 2 * kK; ++k)
        r[k] = __fadd2_rn(make_float2(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1])),
                          make_float2(__uint_as_float(b[2 * k]), __uint_as_float(b[2 * k + 1])));
    };
    // The lane's column, hl, summed over the eight lanes that have values of it.  (A
    // register for a sum instead of eight: with eight for each of the two sums the FP8
    // variant spills: 1000 tokens of 128 heads, window 2048, 757 and 824 us.)
    const int hl = 8 * (fl >> 1) + 2 * fc + (fl & 1);
    auto column_of = [&](const float2 (&v)[kK]) -> float {
      static_assert(kK == 4, "two columns of each of four groups of eight");
      float2 a[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 mine = fl & 4 ? v[k + 2] : v[k], send = fl & 4 ? v[k] : v[k + 2];
        a[k] = __fadd2_rn(mine, make_float2(__shfl_xor_sync(0xffffffffu, send.x, 16), __shfl_xor_sync(0xffffffffu, send.y, 16)));
      }
      const float2 mine = fl & 2 ? a[1] : a[0], send = fl & 2 ? a[0] : a[1];
      const float2 b = __fadd2_rn(mine, make_float2(__shfl_xor_sync(0xffffffffu, send.x, 8), __shfl_xor_sync(0xffffffffu, send.y, 8)));
      return (fl & 1 ? b.y : b.x) + __shfl_xor_sync(0xffffffffu, fl & 1 ? b.x : b.y, 4);
    };
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
      const ChunkUnit c = unit_of<kTok>(p, u, &unused);
      const int cols = min(kCols, (p.s << p.log_h) - c.col0);
      const size_t out0 = (size_t)c.b * (p.s << p.log_h) + c.col0;
      if (c.ntiles == 0) {   // no position: zeros
        for (int e = threadIdx.x - 128; e < cols * (kDc / 8); e += 256)
          reinterpret_cast<uint4*>(p.out + out0 * kDc)[e] = make_uint4(0, 0, 0, 0);
        if (const int h = threadIdx.x - 128; p.lse && h < cols) p.lse[out0 + h] = -INFINITY;
        continue;
      }
      float2 nref[kK];          // minus the reference (log2 units)
      // Sums of the warp's p of column hl: of p, for the log-sum-exp, and of p as
      // rounded for the value sum, which the output is divided by, so that a lone large
      // weight's rounding leaves it (paged_decode.cu).
      float l = 0.f, lr = 0.f;
#pragma unroll
      for (int k = 0; k < kK; ++k) nref[k] = make_float2(0.f, 0.f);
      // a token of mine sees few positions: its largest p is then 1, which bf16 holds exactly (paged_decode.cu)
      auto few = [&](int t) { return (unsigned)p.window + (unsigned)p.sinks <= kFew || c.end0 + tok0 + t <= (int)kFew; };
      bool begun[kMine];   // the token has seen a position
#pragma unroll
      for (int t = 0; t < kMine; ++t) begun[t] = false;
      for (int i = 0; i < c.ntiles; ++i, ++g) {
        const int sb = g & 1, rs = g % kRopes;
        ok = ok && wait.warp(&sh->rfull[rs], (g / kRopes) & 1);   // (for the masks; long complete)
        uint64_t all = ~0ull;
        bool v0[kMine], v1[kMine], fresh[kMine];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
          const uint64_t m = *reinterpret_cast<const volatile uint64_t*>(sh->seen[rs][t]);
          all &= m;
          const int mine = t - tok0;
          if (mine >= 0 && mine < kMine) {
#pragma unroll
            for (int q = 0; q < kMine; ++q)
              if (q == mine) {
                v0[q] = m >> row0 & 1;
                v1[q] = m >> row1 & 1;
                fresh[q] = !begun[q] && m != 0;
              }
          }
        }
        const uint32_t ts = tl + C::kTmemS + 2 * sb * kCols + grp * kHT;
        volatile int* need = &sh->need[rs][grp];
        ok = ok && wait.warp(&sh->sfull[sb], (g >> 1) & 1);
        tc_after();
        float2 x[2 * kK];   // scores relative to their column's reference
        float2 tsum[kK];    // the thread's p, summed
        uint32_t pw[2 * kK];   // and as stored
        bool over, odd = false;     // odd: some score is NaN or infinite (where a row is not seen by all)
        auto refer = [&]() {
          float2 r[2 * kK];
          scores(ts, r);
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            x[2 * k] = __ffma2_rn(r[2 * k], sl2, nref[k]);
            x[2 * k + 1] = __ffma2_rn(r[2 * k + 1], sl2, nref[k]);
          }
          over = false;
#pragma unroll
          for (int t = 0; t < kMine; ++t)
            if (fresh[t]) {   // a token's first positions: also if some score is far below, or few are seen (paged_decode.cu)
              float low = INFINITY;
#pragma unroll
              for (int k = t * kPer; k < (t + 1) * kPer; ++k) {
                if (v0[t]) low = fminf(fminf(low, x[2 * k].x), x[2 * k].y);
                if (v1[t]) low = fminf(fminf(low, x[2 * k + 1].x), x[2 * k + 1].y);
              }
              over |= few(t) || !(low >= -kRaise);
            }
          if (all != ~0ull) {   // (the same way for the whole CTA; most tiles are seen whole)
            float2 none = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 2 * kK; ++k) none = __ffma2_rn(x[k], make_float2(0.f, 0.f), none);   // (0 times a finite value is 0)
            odd = none.x != 0.f || none.y != 0.f;
#pragma unroll
            for (int k = 0; k < kK; ++k) {
              if (!v0[k / kPer]) x[2 * k] = make_float2(-INFINITY, -INFINITY);
              if (!v1[k / kPer]) x[2 * k + 1] = make_float2(-INFINITY, -INFINITY);
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kK; ++k)
            top = fmaxf(fmaxf(fmaxf(top, x[2 * k].x), fmaxf(x[2 * k].y, x[2 * k + 1].x)), x[2 * k + 1].y);
          over |= top > kRaise;
        };
        // P over the rotary block, whose scores are done
        uint8_t* pb = rope(rs);
        auto put = [&]() {
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int ch = grp * kK + k;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 y = make_float2(ex2(x[2 * k + j].x), ex2(x[2 * k + j].y));
              const __nv_bfloat162 w = __float22bfloat162_rn(y);
              pw[2 * k + j] = *reinterpret_cast<const uint32_t*>(&w);
              *reinterpret_cast<uint32_t*>(pb + swz_chunk(j ? row1 : row0, ch) + 4 * fc) = pw[2 * k + j];
              tsum[k] = j ? __fadd2_rn(tsum[k], y) : y;
            }
          }
        };
        refer();
        over = __any_sync(0xffffffffu, over);
        if (over && lane == 0) *need = g + 1;
        put();
        // A row that some token does not see may hold non-finite values (one that
        // none sees anything: bf16, it may not even have been loaded): zeros in
        // their place, so that P = 0 never meets one.
        if (odd && !(all >> row0 & all >> row1 & 1)) {
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const int q = fc + 4 * (e & 7), row = e < 8 ? row0 : row1;
            uint4* at = reinterpret_cast<uint4*>(pair((kPairsPerTile * g + 2 * grp + (q >> 4)) % kPairs) + ((q >> 3) & 1) * kBlock +
                                                 swz_chunk(row, q & 7));
            if (!(all >> row & 1) && non_finite(*at)) *at = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh->pfull[rs]);
        // The value sum starts at once unless some warp's scores exceed their
        // reference by too much: then it waits (pfix) for this group's new P.
        ok = ok && wait.warp(&sh->pfull[rs], (g / kRopes) & 1);
        if (ok && *need == g + 1) {
          // raise the references of this group's columns to the tile's maxima
          float2 r[2 * kK];
          scores(ts, r);
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const bool w0 = v0[k / kPer], w1 = v1[k / kPer];
            float2 m;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a = (j ? r[2 * k].y : r[2 * k].x) * sl2.x, b = (j ? r[2 * k + 1].y : r[2 * k + 1].x) * sl2.x;
              float t = fmaxf(w0 ? a : -INFINITY, w1 ? b : -INFINITY);   // (fmaxf drops NaN)
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              (j ? m.y : m.x) = t;
            }
            if (fl == 0) *reinterpret_cast<float2*>(&sh->part[grp][quad][8 * k + 2 * fc]) = m;
          }
          ok = group_sync();
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int h = 8 * k + 2 * fc;
            const bool had = begun[k / kPer];
            // (a token's first maxima replace the 0s, below them too)
            float2 m = had ? make_float2(-nref[k].x, -nref[k].y) : make_float2(-FLT_MAX, -FLT_MAX);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 t = *reinterpret_cast<const float2*>(&sh->part[grp][q][h]);
              m = make_float2(fmaxf(m.x, t.x), fmaxf(m.y, t.y));
            }
            if (!had && !fresh[k / kPer]) m = make_float2(0.f, 0.f);   // (it has seen nothing yet)
            const float2 al = had ? make_float2(exp2f(-nref[k].x - m.x), exp2f(-nref[k].y - m.y)) : make_float2(1.f, 1.f);
            nref[k] = make_float2(-m.x, -m.y);
            if (quad == 0 && fl == 0) *reinterpret_cast<float2*>(&sh->alpha[grp * kHT + h]) = al;
          }
          ok = group_sync() && ok;
          l *= sh->alpha[grp * kHT + hl];
          lr *= sh->alpha[grp * kHT + hl];
          refer();
          put();
          fence_async_smem();
          if (i > 0) {   // O holds the tiles before this one
            ok = ok && wait.warp(&sh->rempty[(g - 1) % kRopes], ((g - 1) / kRopes) & 1);
            tc_after();
            const float* alpha = sh->alpha + grp * kHT;
#pragma unroll 1
            for (int e = 0; e < 4 * kHT; e += 8) {
              const int at = (e / kHT) * kCols + grp * kHT + e % kHT;
              uint32_t o[8];
              TC_LD8(tl + at, o);
              tc_wait_ld();
#pragma unroll
              for (int h = 0; h < 8; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * alpha[e % kHT + h]);
              TC_ST8(tl + at, o);
            }
            tc_wait_st();
          }
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sh->pfix[grp]);
        }
        if (lane == 0) bar_arrive(&sh->sfree[sb]);
        l += column_of(tsum);
#pragma unroll
        for (int k = 0; k < kK; ++k) tsum[k] = add_bf16(add_bf16(make_float2(0.f, 0.f), pw[2 * k]), pw[2 * k + 1]);
        lr += column_of(tsum);
#pragma unroll
        for (int t = 0; t < kMine; ++t) begun[t] |= fresh[t];
      }
      // ---------------------------------------------------------- outputs
      // (The last raise's reads of `part` precede its second barrier, the last
      // unit's of `inv` this unit's P, which every warp has written.  A raise's
      // factors may still be read here: `alpha` stays as it is.)
      // The two sums go through `part` one after the other.
      auto column_sum = [&](float v) -> float {   // of all rows, of column threadIdx.x - 128 below kCols
        sh->part[grp][quad][hl] = v;
        softmax_sync();
        const int h = min((int)threadIdx.x - 128, kCols - 1), hg = h / kHT, t = h % kHT;
        return (sh->part[hg][0][t] + sh->part[hg][1][t]) + (sh->part[hg][2][t] + sh->part[hg][3][t]);
      };
#pragma unroll
      for (int k = 0; k < kK; ++k)
        if (quad == 0 && fl == 0) *reinterpret_cast<float2*>(&sh->inv[grp * kHT + 8 * k + 2 * fc]) = nref[k];
      const float sum = column_sum(l);
      softmax_sync();
      const float by = column_sum(lr);
      if (const int h = threadIdx.x - 128; h < kCols) {
        const bool fin = ok && !sh->abort;
        if (p.lse && h < cols) p.lse[out0 + h] = fin && sum != 0.f ? (log2f(sum) - sh->inv[h]) * 0.69314718055994531f : -INFINITY;
        sh->inv[h] = fin && sum != 0.f ? 1.f / by : 0.f;
      }
      softmax_sync();
      // (the last value sum meanwhile)
      ok = ok && wait.warp(&sh->rempty[(g - 1) % kRopes], ((g - 1) / kRopes) & 1);
      tc_after();
      // A warp's 32 lanes are 32 consecutive latent columns of one head; lanes 2 i
      // and 2 i + 1 exchange heads, so that each stores two columns of one.
      const int col = 32 * quad + (lane & ~1), odd_lane = lane & 1;
      constexpr int kRead = kFmt == 0 ? 64 : 32;   // columns read at a time, as registers hold
#pragma unroll 1
      for (int e = 0; e < 2 * kCols; e += kRead) {
        const int m = 2 * grp + e / kCols, hb = e % kCols;
        uint32_t o[kRead];
#pragma unroll
        for (int k = 0; k < kRead; k += 16) TC_LD16(tl + m * kCols + hb + k, (o + k));
        tc_wait_ld();
        if (e + kRead == 2 * kCols) {   // the next unit's value sum may begin
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sh->ofree);
        }
        // (the factors first: no load then waits for a store that might be to its address)
#pragma unroll
        for (int k = 0; k < kRead; k += 4) {
          const float4 inv = *reinterpret_cast<const float4*>(&sh->inv[hb + k]);
          const float f[4] = {inv.x, inv.y, inv.z, inv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) o[k + j] = ok ? __float_as_uint(__uint_as_float(o[k + j]) * f[j]) : 0u;   // (a wait that ran out: zeros)
        }
        __nv_bfloat16* dst = p.out + (out0 + hb + odd_lane) * kDc + 128 * m + col;
#pragma unroll
        for (int k = 0; k < kRead; k += 2) {
          const float a = __uint_as_float(o[k]), b = __uint_as_float(o[k + 1]);
          const float got = __shfl_xor_sync(0xffffffffu, odd_lane ? a : b, 1);
          const __nv_bfloat162 two = odd_lane ? __floats2bfloat162_rn(got, b) : __floats2bfloat162_rn(a, got);
          if (hb + k + odd_lane < cols) *reinterpret_cast<__nv_bfloat162*>(dst + k * kDc) = two;
        }
      }
    }
  } else if constexpr (kFmt == 0) {
    // ------------------------------------- producers of the latent columns
    const int m = warp - 12;
    int g = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const ChunkUnit c = unit_of<kTok>(p, u, &unused);
      const int t1 = c.span.places();
      BoxesOf<true> bx, next;
      next.find(p.pt, c.b, 0, t1, 16, c.span);
      for (int i = 0; i < c.ntiles; ++i, ++g) {
        bx = next;
        next.find(p.pt, c.b, (i + 1) * kTile, t1, 16, c.span);
        const int n = kPairsPerTile * g + m, s = n % kPairs;
        if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) {
          ok = false;
          break;
        }
        load_blocks(bx, 16, pair(s), &p.m_kv, 128 * m, 2, &sh->full[s]);
      }
    }
    if (lane == 0) sh->issued[m] = g;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ------------------------------------------------------------ converter
    // A team holds its pair of the next tile converted, and loads the one after
    // it (of the next unit, behind the last): when the value sum frees the slot,
    // only the stores are left to do.
    const int m = (warp - 12) / kTeamWarps, t = threadIdx.x - 384 - m * 32 * kTeamWarps;
    ConvRowsOf<true> next;   // of the tile whose loads go out next
    ConvData d;
    int lu = blockIdx.x, li = 0;   // that tile: of unit lu, its li-th
    ChunkUnit lc{};
    auto settle = [&]() {          // at a tile that there is, or behind all units
      while (lu < p.units && li >= lc.ntiles) {
        lu += gridDim.x;
        li = 0;
        if (lu < p.units) lc = unit_of<kTok>(p, lu, &unused);
      }
    };
    auto fetch = [&]() {
      if (lu < p.units) next.fetch(p.pt, lc.b, li * kTile, lc.span.places(), t, lc.span);
    };
    auto load = [&]() {
      if (lu >= p.units) return;
      d.load<false>(next, p.pt, p.kv, p.kv_scale, m, t);
      ++li;
      settle();
      fetch();
    };
    if (lu < p.units) lc = unit_of<kTok>(p, lu, &unused);
    settle();
    fetch();
    bool more = lu < p.units;   // d holds a tile that is not converted yet
    load();
#pragma unroll 1
    for (int g = 0; more; ++g) {
      ConvOut o0, o1;
      o0.convert(d, 0);
      o1.convert(d, 2);
      more = lu < p.units;
      load();
      const int n = kPairsPerTile * g + m, s = n % kPairs;
      if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) break;
      o0.store(pair(s), t, 0);
      o1.store(pair(s), t, 2);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->full[s]);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_before();
  __syncthreads();
  // The copies of a CTA that gave up land before its shared memory goes away: the
  // queries, and the last one into each slot of the rings.
  if (warp == 0 && sh->abort) {
    if (lane < kPairs) {
      const int n = kFmt == 0 ? last_load(sh->issued, kPairsPerTile, kPairs, lane) : -1;
      if (n >= 0) wait.drain(&sh->full[lane], (n / kPairs) & 1);
    } else if (lane < kPairs + kRopes) {
      const int s = lane - kPairs, n = last_load(&sh->ropes, 1, kRopes, s);
      if (n >= 0) wait.drain(&sh->rfull[s], (n / kRopes) & 1);
    } else if (lane == 31 && sh->qloads > 0) {
      wait.drain(&sh->qbar, (sh->qloads - 1) & 1);
    }
  }
  __syncwarp();
  if (threadIdx.x == 0 && sh->flags) atomicOr(p.status, sh->flags);
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int kFmt, int kTok>
cudaError_t launch(const Params& p, int ctas, cudaStream_t s) {
  using C = Cfg<kFmt>;
  cudaError_t e = ensure_smem<chunk_kernel<kFmt, kTok>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_kernel<kFmt, kTok>, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, s, p);
}

}  // namespace
}  // namespace paged

int chunk_units(int B, int s, int H) { return B * ((s * H + paged::kCols - 1) / paged::kCols); }

cudaError_t launch_paged_chunk(const DecodeParams& d, int sms, cudaStream_t s) {
  using namespace paged;
  Params p;
  memset(&p, 0, sizeof(p));
  const int B = d.B / d.mtp_s;
  const uint64_t pages = (uint64_t)d.pt.num_pages, rows = (uint64_t)d.pt.page_size, q = (uint64_t)d.mtp_s * d.H;
  if ((d.fmt == 0 && !encode_rows(&p.m_kv, d.kv, kDc, rows, pages, 16)) || !encode_rows(&p.m_pe, d.pe, kDr, rows, pages, 16) ||
      !encode_rows(&p.m_ql, d.q_latent, kDc, q, B, kCols) || !encode_rows(&p.m_qp, d.q_pe, kDr, q, B, kCols))
    return cudaErrorInvalidValue;
  p.kv = d.kv;
  p.kv_scale = d.kv_scale;
  p.pt = d.pt;
  p.end_pos = d.sched.end_pos;
  p.max_end_pos = d.sched.max_end_pos;
  p.s = d.mtp_s;
  for (p.log_h = 4; (1 << p.log_h) < d.H; ++p.log_h) {}
  p.window = d.sched.window;
  p.sinks = d.sched.sinks;
  p.units = chunk_units(B, d.mtp_s, d.H);
  p.per_seq = p.units / B;
  p.scale_log2 = d.scale_log2;
  p.out = static_cast<__nv_bfloat16*>(d.out);
  p.lse = d.lse;
  p.status = d.ws.status;
  p.selftest = d.withhold_tile >= 0 ? 1 : 0;
  const int ctas = p.units < sms ? p.units : sms;
  if (d.fmt == 0) return d.H == 16 ? launch<0, 4>(p, ctas, s) : d.H == 32 ? launch<0, 2>(p, ctas, s) : launch<0, 1>(p, ctas, s);
  return d.H == 16 ? launch<1, 4>(p, ctas, s) : d.H == 32 ? launch<1, 2>(p, ctas, s) : launch<1, 1>(p, ctas, s);
}

}  // namespace mla
