// paged_decode.cu -- absorbed MLA decode over a paged latent cache on the
// 5th-generation tensor cores, for 16, 32 and 64 heads (128: decode_tc.cu).
//
// What is computed, per unit (a run of positions of one sequence):
//   S[t, h] = c[t] . q_latent[h] + kR[t] . q_pe[h]        (64 positions a tile)
//   online softmax over t
//   O[c, h] = sum_t c[t, c] p[t, h]                       (512 latent columns)
// The cache rows are the MMA's M side in both products and the heads its N: a
// decode step has few heads, so the wide side goes to what there is much of,
// and no row of the tensor core idles at 16 heads.  It also lays the
// accumulators out so that one SM holds them: O takes 4 blocks of 128 latent
// columns x heads (256 of the 512 tensor-memory columns at 64 heads), S two
// buffers of two halves of 64 positions x heads.  (128 heads as two CTAs that read the same
// rows: 248 us where the pair kernel takes 207, FP8, 4 x 131072 positions.)
//
// One pass: a tile is loaded once, read as a K-major operand for the scores
// and as an MN-major one for the value sum.  P (bf16, positions x heads) takes
// the place of the tile's rotary block, which the scores alone need.  Two
// tiles fit beside 64 heads' queries, so one is loaded and scored while the
// other waits for its softmax and value sum.  (128-position tiles cost the
// tensor pipe less, 68 MMAs of 48 cycles for 128 positions against 104, but
// only one fits, and load, scores, softmax and value sum then follow one
// another: 4.6 to 5.1 us per 128 positions.)
//
// Softmax: a quarter warp of tensor-memory lanes is 16 positions; a thread
// holds two of them at a quarter of its group's heads.  What a head's scores are
// referred to need not be their maximum: bf16 and fp32 have the exponents to
// spare.  The reference is 0 unless a score of the first tile is further than
// 2^24 from it, and is raised only when a later score exceeds it by that, so a
// tile hardly ever needs an exchange; the sums stay per thread until the unit
// ends.
//
// Warps: 0 producer of the rotary columns and queries (TMA); 1 (which owns tensor
// memory) and 3 issue the scores' MMAs, half of the columns each into an
// accumulator of its own: the 36 MMAs of a tile took one warp 1.5 us beside the
// others (FP8, 64 heads, 4 x 65536 positions: 75.3 -> 70.9 us); 2 issues the
// value sum's MMAs (and works out the unit first); 4-7 and 8-11
// softmax of the lower and upper half of the heads (warp & 3 = tensor-memory
// lane quadrant); 12-15 (bf16) producers of the latent columns, one pair each: a warp issues a
// TMA box in about 100 cycles whatever its size, so one warp would need longer
// for a tile's boxes than the tile takes; 12-27 (FP8) load and convert them.
//
// Measured: 64 heads, bf16, 4 x 40000 positions 47.7 us (3.9 TB/s of rows, 0.57
// of a copy's rate): each further row costs its HBM time, and 20 us go to the
// launch, the first tile, the partial outputs and the combine.  FP8, 4 x 65536,
// 67 us (2.6 TB/s); 16 heads, FP8, 32 x 8192, 57 us: a tile takes 1.8 times its
// HBM time on its way through the SM (load and conversion, 52 MMAs of about 1 us,
// softmax, value sum), of which 2 (64 heads) to 2.5 are in shared memory.
//
// Waits are bounded; on expiry the CTA flags it, stops issuing and tears down.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <float.h>


#include <mutex>
#include <string.h>

#include "common.cuh"
#include "paged_schedule.cuh"
#include "paged_tile.cuh"
#include "ring.cuh"
#include "schedule.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace paged {
namespace {

// References start at 0 and stay while the first tile's scores lie within
// 2^+-24 of it and no later one exceeds its reference by more (log2 units): p
// then stays below 2^24 and the largest of the first tile above 2^-24.
constexpr float kRaise = 24.0f;

template <int kFmt, int kH>
struct Cfg {
  static constexpr int kHalf = kH / 2;                 // heads per softmax thread
  static constexpr int kPairs = kH == 64 ? 8 : 10;     // latent ring: pairs of blocks
  static constexpr int kRopes = kH == 16 ? 4 : 3;      // rotary blocks (and P)
  static constexpr int kThreads = 32 * (12 + (kFmt == 0 ? 4 : kConvWarps));
  static constexpr int kQBlk = kH * 128;               // 64 columns of the group's queries
  static constexpr int kRopeOff = kPairs * kPair;
  static constexpr int kQOff = kRopeOff + kRopes * kBlock;
  static constexpr int kBarOff = kQOff + 9 * kQBlk;
  static constexpr int kSmem = kBarOff + 2048 + 1024;
  static constexpr uint32_t kTmemS = 4 * kH;   // S: [buffer][issuer] of kH columns
  static constexpr uint32_t kTmemCols = kH == 64 ? 512 : kH == 32 ? 256 : 128;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Params {
  CUtensorMap m_kv;   // bf16: latent [pages][rows][512] (box 64 x box)
  CUtensorMap m_pe;   // rotary [pages][rows][64] (box 64 x box)
  CUtensorMap m_ql;   // q_latent [B][H][512] (box 64 x kH)
  CUtensorMap m_qp;   // q_pe [B][H][64] (box 64 x kH)
  const void* kv;
  const float* kv_scale;
  PagedTable pt;
  int box;
  float scale_log2;
  void* out;
  float* lse;
  Workspace ws;
  DenseSchedule sched;   // B == 0: the schedule kernel wrote the units
  int whole;             // CTA b takes all of sequence b (sched.B sequences); no combine follows
  AppendRows ap;         // new rows (kv_new null: none), which the unit that reads them writes
  float* ap_weight;
  int selftest;          // self-test of the waits: the first rotary block of CTA 0 never counts as loaded
};

struct __align__(16) Shared {
  uint64_t full[10], empty[10];    // latent pair landed / read by its value sum
  uint64_t rfull[4], rempty[4];    // rotary block landed / tile's value sum done (P and rotary free)
  uint64_t sfull[2], sfree[2];
  uint64_t pfull[4];               // P written
  uint64_t pfix[2];                // P corrected by a group that raised its references
  uint64_t gbar[2];                // among a group's warps
  uint64_t qbar, drain, drain_pv;
  uint64_t appended;               // the new row is in the pool
  uint64_t rows[4];                // per rotary slot: the tile's positions that are attended to
  Unit unit;
  uint32_t tmem;
  uint32_t flags, limit;   // (as Wait has them)
  volatile int abort;
  int issued[kPairsPerTile];   // bf16: tiles whose pair each latent producer has loaded
  int ropes;                   // rotary blocks loaded
  volatile int need[4][2];   // [rotary slot][group]: tile number + 1 if references must be raised

  __align__(16) float alpha[64];       // factor of the last raise, then minus the last reference
  float inv[64];
  float part[2][4][32];  // per group and lane quadrant: tile maxima, then row sums
};
static_assert(sizeof(Shared) <= 2048, "barrier block");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 16 lanes x 8 N columns, see TC_LD16L_X4
template <int N>
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[4 * N]) {
  if constexpr (N == 1) {
    TC_LD16L_X1(addr, r);
  } else if constexpr (N == 2) {
    TC_LD16L_X2(addr, r);
  } else {
    TC_LD16L_X4(addr, r);
  }
  tc_wait_ld();
}

// The new row (see append_row), out of line: its code among the hot loops
// costs their instruction fetch.
__device__ __noinline__ void append_new_row(const Params& p, int b, int pos, int t, uint32_t* flags) {
  append_paged_row(p.ap, p.pt, p.ap_weight, b, pos, t, true, flags);
}

// The status word of a call without a combine, by one warp: what the sequences'
// lengths and tables raise.
__device__ __noinline__ void whole_status(const Params& p) {
  uint32_t flags = 0;
  for (int b = threadIdx.x & 31; b < p.sched.B; b += 32) {
    const int len = dense_len(p.sched, b, &flags);
    bool bad = false;
    for (int t = 0; t < len; t += p.pt.page_size) bad |= p.pt.row(b, t) < 0;
    if (bad) flags |= kDevBadPage;
    if (p.sched.append && !(append_row_valid(p.sched.end_pos[b], p.sched.max_end_pos) && p.pt.row(b, len - 1) >= 0))
      flags |= kDevAppendSkipped;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if ((threadIdx.x & 31) == 0) *p.ws.status = flags;
}

template <int kFmt, int kH>
__global__ void __launch_bounds__(Cfg<kFmt, kH>::kThreads, 1) decode_kernel(const __grid_constant__ Params p) {
  using C = Cfg<kFmt, kH>;
  constexpr int kHT = C::kHalf, kPairs = C::kPairs, kRopes = C::kRopes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared* sh = reinterpret_cast<Shared*>(sm + C::kBarOff);
  auto pair = [&](int s) { return sm + s * kPair; };
  auto rope = [&](int s) { return sm + C::kRopeOff + s * kBlock; };
  uint8_t* qs = sm + C::kQOff;

  const int unit_id = blockIdx.x;
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
    bar_init(&sh->drain, 2);
    bar_init(&sh->drain_pv, 1);
    bar_init(&sh->appended, 4);
    sh->abort = 0;
    sh->flags = 0;
    sh->limit = p.selftest ? kSelftestWaitNs : kWaitNs;
    for (int m = 0; m < kPairsPerTile; ++m) sh->issued[m] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&sh->tmem)),
                 "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {
    Unit mine;
    if (p.whole) {
      uint32_t flags = 0;   // (whole_status reports them)
      mine = Unit{unit_id, 0, dense_len(p.sched, unit_id, &flags), kUnitDirect};
      if (p.sched.append && append_row_valid(p.sched.end_pos[unit_id], p.sched.max_end_pos)) mine.flags |= kUnitAppend;
    } else if (p.sched.B == 0) {
      mine = p.ws.units[unit_id];
    } else {
      const bool writer = blockIdx.x == 0;
      uint32_t flags = 0;
      int units = 0;
      mine = packed_schedule(p.sched, unit_id, &flags, &units, writer ? p.ws.seq : nullptr, nullptr);
      if (writer && lane == 0) {
        *p.ws.status = flags;
        *p.ws.n_units = units;
      }
    }
    if (lane == 0) sh->unit = mine;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh->tmem;
  const Unit u = sh->unit;
  const int slot = u.flags & kUnitSlot ? u.flags >> kUnitSlotShift : unit_id;
  const int ntiles = u.b < 0 ? 0 : (u.t1 - u.t0 + kTile - 1) / kTile;
  const bool append = (u.flags & kUnitAppend) && p.ap.kv_new != nullptr;   // (row t1 - 1, in the last tile)
  if (p.whole) {
    if (warp == 3 && unit_id == 0) whole_status(p);
    if (ntiles == 0) {   // (elsewhere a unit has a position, and the combine writes the others)
      uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)u.b * kH * kDc);
      for (int i = threadIdx.x; i < kH * kDc / 8; i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
      if (p.lse && threadIdx.x < kH) p.lse[(size_t)u.b * kH + threadIdx.x] = -INFINITY;
    }
  }

  // FP8: registers to where they are needed: 28 warps x 72 at launch = 4 x 56
  // + 8 x 64 + 16 x 80
  static_assert(kFmt == 0 || 4 * 56 + 8 * 64 + kConvWarps * 80 <= C::kThreads / 32 * 72, "register split");
  if (ntiles == 0) {
  } else if (warp < 4) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bar_expect_tx(&sh->qbar, 9 * C::kQBlk);
      for (int k = 0; k < 8; ++k) tma3(qs + k * C::kQBlk, &p.m_ql, 64 * k, 0, u.b, &sh->qbar);
      tma3(qs + 8 * C::kQBlk, &p.m_qp, 0, 0, u.b, &sh->qbar);
    }
    __syncwarp();
    Boxes bx, next, after;
    next.find(p.pt, u.b, u.t0, u.t1, p.box);
    after.find(p.pt, u.b, u.t0 + kTile, u.t1, p.box);
    // FP8: the rows go towards L2 two tiles ahead (64 heads, 4 x 65536
    // positions: 81 us without, 75 so); bf16's own loads run that far ahead,
    // and are only delayed by it (64 heads, 4 x 40000: 49.5 and 52.4 us)
    if (kFmt != 0) {
      prefetch_rows<kFmt>(next, p.box, p.pt.page_size, p.kv, p.kv_scale);
      prefetch_rows<kFmt>(after, p.box, p.pt.page_size, p.kv, p.kv_scale);
    }
    int ropes = 0;   // issued
    for (int i = 0; i < ntiles; ++i) {
      bx = next;
      next = after;
      after.find(p.pt, u.b, u.t0 + (i + 2) * kTile, u.t1, p.box);
      if (kFmt != 0) prefetch_rows<kFmt>(after, p.box, p.pt.page_size, p.kv, p.kv_scale);
      const int s = i % kRopes;
      if (append && i == ntiles - 1 && !wait.warp(&sh->appended, 0)) break;
      if (!wait.warp(&sh->rempty[s], ((i / kRopes) & 1) ^ 1)) break;
      bool bad;
      const uint64_t rows = bx.rows(u.t0 + i * kTile, u.t1, p.box, &bad);
      if (lane == 0) {
        sh->rows[s] = rows;   // (the arrival of load_blocks releases it)
        if (bad) atomicOr(&sh->flags, kDevBadPage);
      }
      load_blocks(bx, p.box, rope(s), &p.m_pe, 0, 1, &sh->rfull[s]);
      ++ropes;
    }
    if (lane == 0) sh->ropes = ropes;
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------- scores' issuers
    const int half = warp >> 1;
    constexpr uint32_t id = idesc(kTile, kH, false, false);
    const bool el = elect_one();
    const uint64_t d_kv = sdesc(sa(pair(0)), 16, 1024), d_pe = sdesc(sa(rope(0)), 16, 1024);
    const uint64_t d_q = sdesc(sa(qs), 16, 1024);
    bool ok = wait.warp(&sh->qbar, 0);
    int s = 2 * half, ph = 0;   // the ring's slot and phase
    for (int i = 0; i < ntiles && ok; ++i) {
      const int sb = i & 1;
      ok = wait.warp(&sh->sfree[sb], ((i >> 1) & 1) ^ 1);
      if (!ok) break;
      const uint32_t ds = tmem + C::kTmemS + (2 * sb + half) * kH;
      // (rolled loops: straight-line code of a tile's MMAs runs at the rate
      // instructions are fetched, which the CTA's many warps share)
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
        const int rs = i % kRopes;
        ok = wait.warp(&sh->rfull[rs], (i / kRopes) & 1) && ok;
        tc_after();
        mma_ss4_if<2>(el, ds, sdesc_at(d_pe, rs * kBlock), q, id, 1);
      }
      mma_commit_if(el, &sh->sfull[sb]);
      s += 2;   // the other warp's pairs
      if (s >= kPairs) s -= kPairs, ph ^= 1;
    }
    mma_commit_if(el, &sh->drain);
    wait.drain(&sh->drain, 0);
  } else if (warp == 2) {
    // ----------------------------------------------------- value sum's issuer
    constexpr uint32_t id = idesc(128, kH, true, true);
    const bool el = elect_one();
    const uint64_t d_v = sdesc(sa(pair(0)), kBlock, 1024), d_p = sdesc(sa(rope(0)), kBlock, 1024);
    int s = 0, fixed0 = 0, fixed1 = 0;
    for (int i = 0; i < ntiles; ++i) {
      const int rs = i % kRopes;
      if (!wait.warp(&sh->pfull[rs], (i / kRopes) & 1)) break;
      if (sh->need[rs][0] == i + 1 && !wait.warp(&sh->pfix[0], fixed0++ & 1)) break;
      if (sh->need[rs][1] == i + 1 && !wait.warp(&sh->pfix[1], fixed1++ & 1)) break;
      tc_after();
      const uint64_t pd = sdesc_at(d_p, rs * kBlock);
#pragma unroll 1
      for (int m = 0; m < kPairsPerTile; ++m) {
        static_assert(kTile == 64, "four steps of 16 positions");
        mma_ss4_if<128>(el, tmem + m * kH, sdesc_at(d_v, s * kPair), pd, id, i);
        mma_commit_if(el, &sh->empty[s]);
        if (++s == kPairs) s = 0;
      }
      mma_commit_if(el, &sh->rempty[rs]);
    }
    mma_commit_if(el, &sh->drain_pv);
    wait.drain(&sh->drain_pv, 0);
  }
  } else if (warp < 12) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ softmax
    // thread: positions fl and fl + 8 of the quadrant's 16, heads 8 k + 2 fc
    // and 8 k + 2 fc + 1 of the group's (values 4 k .. 4 k + 3: both heads at
    // the first position, then at the second)
    const int g = (warp - 4) >> 2, quad = warp & 3, fl = lane >> 2, fc = lane & 3;
    const int row0 = 16 * quad + fl, row1 = row0 + 8;
    if (append && g == 0) {   // while the first scores are computed
      append_new_row(p, u.b, u.t1 - 1, threadIdx.x - 128, &sh->flags);
      fence_async_global();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->appended);
    }
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    constexpr int kK = kHT / 8;
    float2 nref[kK], l[kK];   // minus the reference maximum (log2 units), sum of p
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      nref[k] = make_float2(0.f, 0.f);
      l[k] = make_float2(0.f, 0.f);
    }
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    int gph = 0;
    // among the group's four warps (bounded, so an aborted CTA never stays here)
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->gbar[g]);
      const bool all = wait.warp(&sh->gbar[g], gph);
      gph ^= 1;
      return all;
    };
    // the tile's scores: the sum of what the two issuers' columns gave
    auto scores = [&](uint32_t at, float2 (&r)[2 * kK]) {
      uint32_t a[4 * kK], b[4 * kK];
      tmem_ld16<kK>(at, a);
      tmem_ld16<kK>(at + kH, b);
#pragma unroll
      for (int k = 0; k < 2 * kK; ++k)
        r[k] = __fadd2_rn(make_float2(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1])),
                          make_float2(__uint_as_float(b[2 * k]), __uint_as_float(b[2 * k + 1])));
    };
    bool ok = true;
    for (int i = 0; i < ntiles; ++i) {
      const int sb = i & 1, rs = i % kRopes;
      ok = ok && wait.warp(&sh->rfull[rs], (i / kRopes) & 1);   // (for rows; long complete)
      const uint64_t rows = *const_cast<volatile uint64_t*>(&sh->rows[rs]);
      const bool v0 = rows >> row0 & 1, v1 = rows >> row1 & 1;
      const uint32_t ts = tl + C::kTmemS + 2 * sb * kH + g * kHT;
      volatile int* need = &sh->need[rs][g];
      ok = ok && wait.warp(&sh->sfull[sb], (i >> 1) & 1);
      tc_after();
      float2 x[2 * kK];   // scores relative to their head's reference, then p
      float top, low;
      auto refer = [&]() {
        float2 r[2 * kK];
        scores(ts, r);
        top = -INFINITY;
        low = INFINITY;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          x[2 * k] = __ffma2_rn(r[2 * k], sl2, nref[k]);
          x[2 * k + 1] = __ffma2_rn(r[2 * k + 1], sl2, nref[k]);
          low = fminf(fminf(fminf(low, x[2 * k].x), fminf(x[2 * k].y, x[2 * k + 1].x)), x[2 * k + 1].y);
          if (!v0) x[2 * k] = make_float2(-INFINITY, -INFINITY);
          if (!v1) x[2 * k + 1] = make_float2(-INFINITY, -INFINITY);
          top = fmaxf(fmaxf(fmaxf(top, x[2 * k].x), fmaxf(x[2 * k].y, x[2 * k + 1].x)), x[2 * k + 1].y);
        }
      };
      // P over the rotary block, whose scores are done
      uint8_t* pb = rope(rs);
      auto put = [&]() {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const int c = g * kK + k;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2& y = x[2 * k + j];
            y = make_float2(ex2(y.x), ex2(y.y));
            *reinterpret_cast<__nv_bfloat162*>(pb + swz_chunk(j ? row1 : row0, c) + 4 * fc) = __float22bfloat162_rn(y);
          }
        }
      };
      refer();
      // (the first tile: also if some score is far below, NaN, or not there)
      const bool over = __any_sync(0xffffffffu, top > kRaise || (i == 0 && !(v0 && v1 && low >= -kRaise)));
      if (over && lane == 0) *need = i + 1;
      put();
      if (kFmt == 0 && !(v0 && v1)) {
        // a row that is not attended to holds anything, or nothing was loaded
        // there: zeros, so that P = 0 never meets a non-finite value
#pragma unroll 1
        for (int c = 0; c < 16; ++c) {
          const int q = fc + 4 * (c & 7), row = c < 8 ? row0 : row1;
          if (c < 8 ? !v0 : !v1)
            *reinterpret_cast<uint4*>(pair((kPairsPerTile * i + 2 * g + (q >> 4)) % kPairs) + ((q >> 3) & 1) * kBlock +
                                      swz_chunk(row, q & 7)) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async_smem();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->pfull[rs]);
      // The value sum starts at once unless some warp's scores exceed their
      // reference by too much: then it waits (pfix) for this group's new P.
      ok = ok && wait.warp(&sh->pfull[rs], (i / kRopes) & 1);
      if (ok && *need == i + 1) {
        // raise the references of this group's heads to the tile's maxima
        float2 r[2 * kK];
        scores(ts, r);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          float2 m;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float a = (j ? r[2 * k].y : r[2 * k].x) * sl2.x, b = (j ? r[2 * k + 1].y : r[2 * k + 1].x) * sl2.x;
            float t = fmaxf(v0 ? a : -INFINITY, v1 ? b : -INFINITY);   // (fmaxf drops NaN)
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            (j ? m.y : m.x) = t;
          }
          if (fl == 0) *reinterpret_cast<float2*>(&sh->part[g][quad][8 * k + 2 * fc]) = m;
        }
        ok = group_sync();
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const int h = 8 * k + 2 * fc;
          // (the first tile's maxima replace the 0s, below them too)
          float2 m = i > 0 ? make_float2(-nref[k].x, -nref[k].y) : make_float2(-FLT_MAX, -FLT_MAX);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 t = *reinterpret_cast<const float2*>(&sh->part[g][q][h]);
            m = make_float2(fmaxf(m.x, t.x), fmaxf(m.y, t.y));
          }
          // (the first tile has no sums to scale, and may lower a reference)
          const float2 al = i > 0 ? make_float2(exp2f(-nref[k].x - m.x), exp2f(-nref[k].y - m.y)) : make_float2(1.f, 1.f);
          l[k] = make_float2(l[k].x * al.x, l[k].y * al.y);
          nref[k] = make_float2(-m.x, -m.y);
          if (quad == 0 && fl == 0) *reinterpret_cast<float2*>(&sh->alpha[g * kHT + h]) = al;
        }
        ok = group_sync() && ok;
        refer();
        put();
        fence_async_smem();
        if (i > 0) {   // O holds the tiles before this one
          ok = ok && wait.warp(&sh->rempty[(i - 1) % kRopes], ((i - 1) / kRopes) & 1);
          tc_after();
          const float* alpha = sh->alpha + g * kHT;
#pragma unroll 1
          for (int c = 0; c < 4 * kHT; c += 8) {
            const int at = (c / kHT) * kH + g * kHT + c % kHT;
            uint32_t o[8];
            TC_LD8(tl + at, o);
            tc_wait_ld();
#pragma unroll
            for (int h = 0; h < 8; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * alpha[c % kHT + h]);
            TC_ST8(tl + at, o);
          }
          tc_wait_st();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh->pfix[g]);
      }
      if (lane == 0) bar_arrive(&sh->sfree[sb]);
      // l sums the fp32 values (P's rounding to bf16, 2^-8 relative, then
      // averages out of the output)
#pragma unroll
      for (int k = 0; k < kK; ++k) l[k] = __fadd2_rn(l[k], __fadd2_rn(x[2 * k], x[2 * k + 1]));
    }
    // ------------------------------------------------------------ epilogue
    // (the last raise's reads of `part` precede its second barrier)
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      float2 t = l[k];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
      }
      if (fl == 0) *reinterpret_cast<float2*>(&sh->part[g][quad][8 * k + 2 * fc]) = t;
    }
    ok = ok && wait.warp(&sh->rempty[(ntiles - 1) % kRopes], ((ntiles - 1) / kRopes) & 1);
    if (quad == 0 && fl == 0) {   // (every raise of the group is done)
#pragma unroll
      for (int k = 0; k < kK; ++k) *reinterpret_cast<float2*>(&sh->alpha[g * kHT + 8 * k + 2 * fc]) = nref[k];
    }
    softmax_sync();
    const bool direct = (u.flags & kUnitDirect) != 0;
    if (const int h = threadIdx.x - 128; h < kH) {
      const bool fin = ok && !sh->abort;
      const int hg = h / kHT, t = h % kHT;
      const float sum = (sh->part[hg][0][t] + sh->part[hg][1][t]) + (sh->part[hg][2][t] + sh->part[hg][3][t]);
      sh->inv[h] = fin && sum != 0.f ? 1.f / sum : 0.f;
      const float lse = fin && sum != 0.f ? (log2f(sum) - sh->alpha[h]) * 0.69314718055994531f : -INFINITY;
      if (!direct)
        p.ws.part_lse[(size_t)slot * kH + h] = lse;
      else if (p.lse)
        p.lse[(size_t)u.b * kH + h] = lse;
    }
    softmax_sync();
    tc_after();
    // a warp's 32 lanes are 32 consecutive latent columns of one head
    const int row = 32 * quad + lane;
#pragma unroll 1
    for (int m = 2 * g; m < 2 * g + 2; ++m) {
      const int col = 128 * m + row;
#pragma unroll 1
      for (int hb = 0; hb < kH; hb += 16) {
        uint32_t o[16];
        TC_LD16(tl + m * kH + hb, o);
        tc_wait_ld();
        if (direct) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((size_t)u.b * kH + hb) * kDc + col;
#pragma unroll
          for (int k = 0; k < 16; ++k) dst[k * kDc] = __float2bfloat16_rn(__uint_as_float(o[k]) * sh->inv[hb + k]);
        } else {
          float* dst = p.ws.part_o + ((size_t)slot * kH + hb) * kDc + col;
#pragma unroll
          for (int k = 0; k < 16; ++k) dst[k * kDc] = __uint_as_float(o[k]) * sh->inv[hb + k];
        }
      }
    }
  } else if constexpr (kFmt == 0) {
    // ------------------------------------- producers of the latent columns
    const int m = warp - 12;
    Boxes bx, next;
    next.find(p.pt, u.b, u.t0, u.t1, p.box);
    int i = 0;   // tiles issued
    for (; i < ntiles; ++i) {
      bx = next;
      next.find(p.pt, u.b, u.t0 + (i + 1) * kTile, u.t1, p.box);
      const int n = kPairsPerTile * i + m, s = n % kPairs;
      if (append && i == ntiles - 1 && !wait.warp(&sh->appended, 0)) break;
      if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) break;
      load_blocks(bx, p.box, pair(s), &p.m_kv, 128 * m, 2, &sh->full[s]);
    }
    if (lane == 0) sh->issued[m] = i;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ------------------------------------------------------------ converter
    // A team holds its pair of the next tile converted, and loads the one after
    // it: when the value sum frees the slot, only the stores are left to do.
    const int m = (warp - 12) / kTeamWarps, t = threadIdx.x - 384 - m * 32 * kTeamWarps;
    ConvRows next;   // of the tile whose loads go out next
    ConvData d;
    auto load = [&](int i) -> bool {   // tile i's
      if (append && i == ntiles - 1 && !wait.warp(&sh->appended, 0)) return false;
      d.load<true>(next, p.pt, p.kv, p.kv_scale, m, t);
      next.fetch(p.pt, u.b, u.t0 + (i + 1) * kTile, u.t1, t);
      return true;
    };
    next.fetch(p.pt, u.b, u.t0, u.t1, t);
    bool ok = load(0);
#pragma unroll 1
    for (int i = 0; i < ntiles && ok; ++i) {
      ConvOut o0, o1;
      o0.convert(d, 0);
      o1.convert(d, 2);
      ok = load(i + 1);
      const int n = kPairsPerTile * i + m, s = n % kPairs;
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
  // The copies of a CTA that gave up land before its shared memory goes away:
  // the queries, and the last one into each slot of the rings (no producer
  // starts another).  (Out of line: 26.4 us for 25.8, 16 heads, bf16, 8 x 10000.)
  if (warp == 0 && sh->abort && ntiles > 0) {
    if (lane < kPairs) {
      const int n = kFmt == 0 ? last_load(sh->issued, kPairsPerTile, kPairs, lane) : -1;
      if (n >= 0) wait.drain(&sh->full[lane], (n / kPairs) & 1);
    } else if (lane < kPairs + kRopes) {
      const int s = lane - kPairs, n = last_load(&sh->ropes, 1, kRopes, s);
      if (n >= 0) wait.drain(&sh->rfull[s], (n / kRopes) & 1);
    } else if (lane == 31) {
      wait.drain(&sh->qbar, 0);
    }
  }
  __syncwarp();
  if (threadIdx.x == 0 && u.b >= 0) {
    if (!p.whole)
      p.ws.unit_flags[unit_id] = sh->flags;
    else if (sh->flags & kDevTimeout)   // (the others are whole_status's)
      atomicOr(p.ws.status, kDevTimeout);
  }
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
  }
}

// ---------------------------------------------------------------- combine
// out = sum_i w_i O_i / sum_i w_i, w_i = exp(lse_i - max lse), over a sequence's
// units.  CTA (h, y) takes head h of sequences y, y + gridDim.y, ...: kTeams teams
// of 128 threads (4 latent columns each) take every kTeams-th unit, eight partial
// rows in flight each, and join through shared memory; a sequence of one unit
// was finished by the decode.
template <int kTeams>
__global__ void __launch_bounds__(128 * kTeams) combine_kernel(Workspace ws, int H, int B, __nv_bfloat16* __restrict__ out,
                                                               float* __restrict__ lse_out, int groups) {
  __shared__ float4 acc_s[kTeams][128];
  __shared__ float w_s[kTeams];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) {   // the units' status bits
    const int n = *ws.n_units * groups;
    uint32_t f = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) f |= ws.unit_flags[i];
    f = __reduce_or_sync(0xffffffffu, f);
    if (f && (threadIdx.x & 31) == 0) atomicOr(ws.status, f);
  }
  const int h = blockIdx.x, team = threadIdx.x >> 7, t = threadIdx.x & 127;
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    const int2 sq = ws.seq[b];   // (first unit, units; -1: finished)
    const int n = sq.y;
    if (n < 0) continue;
    const float* pl = ws.part_lse + (size_t)sq.x * H + h;
    const float* po = ws.part_o + ((size_t)sq.x * H + h) * kDc + 4 * t;
    constexpr int kBatch = 8;
    float4 o[kBatch];
    float l[kBatch];
    auto bring = [&](int i0) {   // units i0, i0 + kTeams, ...
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kTeams;
        l[k] = -INFINITY;
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          o[k] = *reinterpret_cast<const float4*>(po + (size_t)i * H * kDc);
          l[k] = pl[(size_t)i * H];
        }
      }
    };
    bring(team);
    float m = -INFINITY;
    for (int i = threadIdx.x & 31; i < n; i += 32) m = fmaxf(m, pl[(size_t)i * H]);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float ref = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    for (int i0 = team; i0 < n; i0 += kBatch * kTeams) {
      if (i0 > team) bring(i0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = expf(l[k] - ref);
        acc.x += w * o[k].x;
        acc.y += w * o[k].y;
        acc.z += w * o[k].z;
        acc.w += w * o[k].w;
        wsum += w;
      }
    }
    if (kTeams > 1) {
      acc_s[team][t] = acc;
      if (t == 0) w_s[team] = wsum;
      __syncthreads();
    }
    if (team == 0) {
#pragma unroll
      for (int k = 1; k < kTeams; ++k) {
        const float4 a = acc_s[k][t];
        acc.x += a.x;
        acc.y += a.y;
        acc.z += a.z;
        acc.w += a.w;
        wsum += w_s[k];
      }
      const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(out + ((size_t)b * H + h) * kDc + 4 * t) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if (lse_out && t == 0) lse_out[(size_t)b * H + h] = wsum != 0.f ? ref + logf(wsum) : -INFINITY;
    }
    if (kTeams > 1) __syncthreads();
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

template <int kFmt, int kH>
cudaError_t launch(const Params& p, int units, cudaStream_t s) {
  using C = Cfg<kFmt, kH>;
  cudaError_t e = ensure_smem<decode_kernel<kFmt, kH>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_kernel<kFmt, kH>, dim3((unsigned)units), dim3(C::kThreads), C::kSmem, s, p);
}

}  // namespace

// bf16 [outer][rows][inner], box 64 x box1, 128-byte swizzle
bool encode_rows(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t outer, uint32_t box1) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {inner, rows, outer};
  cuuint64_t strides[2] = {inner * 2, inner * 2 * rows};
  cuuint32_t box[3] = {64, box1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace paged

__global__ void __launch_bounds__(32) paged_schedule_kernel(Workspace ws, const DenseSchedule d) {
  pdl_wait();
  pdl_trigger();
  uint32_t flags = 0;
  int units = 0;
  packed_schedule(d, -1, &flags, &units, ws.seq, ws.units);
  for (int i = units + (int)threadIdx.x; i < ws.max_units; i += 32) ws.units[i] = Unit{-1, 0, 0, 0};
  if (threadIdx.x == 0) {
    *ws.n_units = units;
    *ws.status = flags;
  }
}

cudaError_t launch_paged_schedule(const Workspace& ws, const DenseSchedule& d, cudaStream_t s) {
  return launch_pdl(paged_schedule_kernel, dim3(1), dim3(32), 0, s, ws, d);
}

cudaError_t launch_paged_combine(const Workspace& ws, int B, int H, void* out, float* lse, int groups, cudaStream_t s) {
  // Four teams where sequences have more units than one team keeps in flight
  // twice over (a decode with 38 units a sequence, 64 heads: one team 64.8 us,
  // four 57.9; equal at 19 units).  Otherwise the teams' joining costs more than
  // they save (9 units: 30.6 and 34.1).
  const int seqs = B < 32 ? B : 32;
  if (ws.max_units - B > 16 * B)
    return launch_pdl(paged::combine_kernel<4>, dim3(H, seqs), dim3(512), 0, s, ws, H, B, static_cast<__nv_bfloat16*>(out), lse,
                      groups);
  return launch_pdl(paged::combine_kernel<1>, dim3(H, seqs), dim3(128), 0, s, ws, H, B, static_cast<__nv_bfloat16*>(out), lse,
                    groups);
}

cudaError_t launch_paged_decode(const DecodeParams& d, bool whole, cudaStream_t s) {
  using namespace paged;
  Params p;
  memset(&p, 0, sizeof(p));
  const int kh = d.H;
  const uint64_t pages = (uint64_t)d.pt.num_pages, rows = (uint64_t)d.pt.page_size, B = (uint64_t)d.B, H = (uint64_t)d.H;
  p.box = box_rows(d.pt.page_size);
  if ((d.fmt == 0 && !encode_rows(&p.m_kv, d.kv, kDc, rows, pages, p.box)) ||
      !encode_rows(&p.m_pe, d.pe, kDr, rows, pages, p.box) || !encode_rows(&p.m_ql, d.q_latent, kDc, H, B, kh) ||
      !encode_rows(&p.m_qp, d.q_pe, kDr, H, B, kh))
    return cudaErrorInvalidValue;
  p.kv = d.kv;
  p.kv_scale = d.kv_scale;
  p.pt = d.pt;
  p.scale_log2 = d.scale_log2;
  p.out = d.out;
  p.lse = d.lse;
  p.ws = d.ws;
  p.sched = d.sched;
  p.whole = whole ? 1 : 0;
  p.ap = d.ap;
  p.ap_weight = d.ap_weight;
  p.selftest = d.withhold_tile >= 0 ? 1 : 0;
  const int units = whole ? d.B : d.ws.max_units;
  if (d.fmt == 0)
    return kh == 16 ? launch<0, 16>(p, units, s) : kh == 32 ? launch<0, 32>(p, units, s) : launch<0, 64>(p, units, s);
  return kh == 16 ? launch<1, 16>(p, units, s) : kh == 32 ? launch<1, 32>(p, units, s) : launch<1, 64>(p, units, s);
}

}  // namespace mla
