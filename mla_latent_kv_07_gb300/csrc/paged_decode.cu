// paged_decode.cu -- absorbed MLA decode over a paged latent cache on the
// 5th-generation tensor cores, for 16, 32, 64 and 128 heads.
//
// What is computed, per unit (a run of positions of one sequence) and per
// group of up to 64 heads:
//   S[t, h] = c[t] . q_latent[h] + kR[t] . q_pe[h]        (128 positions a tile)
//   online softmax over t
//   O[c, h] = sum_t c[t, c] p[t, h]                       (512 latent columns)
// The cache rows are the MMA's M side in both products and the heads its N: a
// decode step has few heads, so the 128-row side goes to what there is much
// of, and no row of the tensor core idles at 16 heads.  It also lays the
// accumulators out so that one SM holds a whole group: O takes 4 blocks of 128
// latent columns x heads (256 of the 512 tensor-memory columns at 64 heads),
// S two buffers of 128 positions x heads; 128 heads are two groups, two CTAs
// that read the same rows (the second finds them in L2).
//
// One pass: a tile is loaded once, read as a K-major operand for the scores
// and as an MN-major one for the value sum.  P (bf16, positions x heads) takes
// the place of the tile's rotary block, which the scores alone need.
//
// Softmax with one row per thread: tensor-memory lane t is position t, so a
// thread holds its position's scores of half of the group's heads and no
// exchange is needed within a tile.  The reference maximum of a head need not
// be its maximum: it is raised only when a score exceeds it by 2^16 (one vote
// per tile), which keeps p below 2^16 in bf16 and its sum in fp32 exact enough,
// and the sums stay per thread until the unit ends.
//
// Warps: 0 producer of the rotary columns and queries (TMA); 1 issues the scores' MMAs and owns tensor memory; 2
// issues the value sum's MMAs (and works out the unit first); 4-7 and 8-11
// softmax of the lower and upper half of the heads (warp & 3 = tensor-memory
// lane quadrant); 12-15 (bf16) producers of the latent columns, one pair each: a warp issues a
// TMA box in about 100 cycles whatever its size, so one warp would need longer
// for a tile's boxes than the tile takes; 12-27 (FP8) load and convert them.
//
// Waits are bounded; on expiry the CTA flags it, stops issuing and tears down.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <float.h>


#include <mutex>
#include <string.h>

#include "common.cuh"
#include "paged_tile.cuh"
#include "schedule.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace paged {
namespace {

// Raising a reference rescales O: at most once per factor of 2^16.
constexpr float kRaise = 16.0f;

template <int kFmt, int kH>
struct Cfg {
  static constexpr int kHalf = kH / 2;                 // heads per softmax thread
  static constexpr int kPairs = kH == 64 ? 4 : 5;      // latent ring: pairs of blocks
  static constexpr int kRopes = kH == 16 ? 2 : 1;      // rotary blocks (and P)
  static constexpr int kThreads = 32 * (12 + (kFmt == 0 ? 4 : kConvWarps));
  static constexpr int kQBlk = kH * 128;               // 64 columns of the group's queries
  static constexpr int kRopeOff = kPairs * kPair;
  static constexpr int kQOff = kRopeOff + kRopes * kBlock;
  static constexpr int kBarOff = kQOff + 9 * kQBlk;
  static constexpr int kSmem = kBarOff + 4096 + 1024;
  static constexpr uint32_t kTmemS = 4 * kH;
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
  int box, H, groups;
  float scale_log2;
  void* out;
  float* lse;
  Workspace ws;
  DenseSchedule sched;   // B == 0: the schedule kernel wrote the units
};

struct __align__(16) Shared {
  uint64_t full[5], empty[5];      // latent pair landed / read by its value sum
  uint64_t rfull[2], rempty[2];    // rotary block landed / tile's value sum done (P and rotary free)
  uint64_t sfull[2], sfree[2];
  uint64_t pfull[2], pfix[2];      // P written / corrected by a group that raised its references
  uint64_t gbar[2];                // among a group's warps
  uint64_t qbar, drain, drain_pv;
  Unit unit;
  uint32_t tmem;
  uint32_t flags;
  volatile int abort;
  volatile int need[2][2];   // [tile parity][group]: tile number + 1 if references must be raised

  __align__(16) float nref[64];        // minus the reference maximum of each head (log2 units)
  float alpha[64];       // factor of the last raise
  float inv[64];
  float part[2][4][32];  // per group and lane quadrant: tile maxima, then row sums
};
static_assert(sizeof(Shared) <= 4096, "barrier block");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// N (8, 16 or 32) consecutive columns of this thread's lane
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 8) {
    TC_LD8(addr, r);
  } else if constexpr (N == 16) {
    TC_LD16(addr, r);
  } else {
    TC_LD16(addr, r);
    TC_LD16(addr + 16, (r + 16));
  }
  tc_wait_ld();
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) {
    TC_ST8(addr, r);
  } else if constexpr (N == 16) {
    TC_ST16(addr, r);
  } else {
    TC_ST16(addr, r);
    TC_ST16(addr + 16, (r + 16));
  }
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

  const int unit_id = blockIdx.x / p.groups, h0 = (blockIdx.x - unit_id * p.groups) * kH;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Wait wait{&sh->abort, &sh->flags};

  // ---------------------------------------------------------------- set-up
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairs; ++s) {
      bar_init(&sh->full[s], kFmt == 0 ? 1 : kConvWarps);
      bar_init(&sh->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(&sh->rfull[s], 1);
      bar_init(&sh->rempty[s], 1);
      bar_init(&sh->sfull[s], 1);
      bar_init(&sh->sfree[s], 8);
      bar_init(&sh->pfull[s], 8);
      bar_init(&sh->pfix[s], 4);
      bar_init(&sh->gbar[s], 4);
      sh->need[s][0] = sh->need[s][1] = 0;
    }
    bar_init(&sh->qbar, 1);
    bar_init(&sh->drain, 1);
    bar_init(&sh->drain_pv, 1);
    sh->abort = 0;
    sh->flags = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < kH) sh->nref[threadIdx.x] = FLT_MAX;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&sh->tmem)),
                 "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {
    Unit mine;
    if (p.sched.B == 0) {
      mine = p.ws.units[unit_id];
    } else {
      const bool writer = blockIdx.x == 0;
      uint32_t flags = 0;
      int units = 0;
      mine = warp_schedule(p.sched, unit_id, &flags, &units, writer ? p.ws.seq : nullptr);
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
  const int ntiles = u.b < 0 ? 0 : (u.t1 - u.t0 + kTile - 1) / kTile;
  // (a unit that exists has at least one position)

  // FP8: registers to where they are needed: 28 warps x 72 at launch = 4 x 56
  // + 8 x 96 + 16 x 64
  static_assert(kFmt == 0 || 32 * (4 * 56 + 8 * 96 + kConvWarps * 64) <= C::kThreads * 72, "register split");
  if (ntiles == 0) {
  } else if (warp < 4) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bar_expect_tx(&sh->qbar, 9 * C::kQBlk);
      for (int k = 0; k < 8; ++k) tma3(qs + k * C::kQBlk, &p.m_ql, 64 * k, h0, u.b, &sh->qbar);
      tma3(qs + 8 * C::kQBlk, &p.m_qp, 0, h0, u.b, &sh->qbar);
    }
    __syncwarp();
    Boxes bx, next, after;
    next.find(p.pt, u.b, u.t0, u.t1, p.box);
    after.find(p.pt, u.b, u.t0 + kTile, u.t1, p.box);
    if (kFmt != 0) prefetch_rows<kFmt>(next, p.box, p.pt.page_size, p.kv, p.kv_scale);
    prefetch_rows<kFmt>(after, p.box, p.pt.page_size, p.kv, p.kv_scale);
    int ropes = 0;   // issued
    for (int i = 0; i < ntiles; ++i) {
      bx = next;
      next = after;
      after.find(p.pt, u.b, u.t0 + (i + 2) * kTile, u.t1, p.box);
      prefetch_rows<kFmt>(after, p.box, p.pt.page_size, p.kv, p.kv_scale);
      const int s = i % kRopes;
      if (!wait.warp(&sh->rempty[s], ((i / kRopes) & 1) ^ 1)) break;
      load_blocks(bx, p.box, rope(s), &p.m_pe, 0, 1, &sh->rfull[s]);
      ++ropes;
    }
    // an aborted CTA's copies land before its shared memory goes away
    if (lane == 0 && sh->abort) {
      wait.drain(&sh->qbar, 0);
      for (int n = ropes > kRopes ? ropes - kRopes : 0; n < ropes; ++n) wait.drain(&sh->rfull[n % kRopes], (n / kRopes) & 1);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- scores' issuer
    constexpr uint32_t id = idesc(128, kH, false, false);
    const bool el = elect_one();
    const uint64_t d_kv = sdesc(sa(pair(0)), 16, 1024), d_pe = sdesc(sa(rope(0)), 16, 1024);
    const uint64_t d_q = sdesc(sa(qs), 16, 1024);
    bool ok = wait.warp(&sh->qbar, 0);
    int s = 0, ph = 0;   // the ring's slot and phase
    for (int i = 0; i < ntiles && ok; ++i) {
      const int sb = i & 1;
      ok = wait.warp(&sh->sfree[sb], ((i >> 1) & 1) ^ 1);
      if (!ok) break;
      const uint32_t ds = tmem + C::kTmemS + sb * kH;
#pragma unroll
      for (int m = 0; m < kPairsPerTile; ++m) {
        ok = ok && wait.warp(&sh->full[s], ph);
        if (ok) {
          tc_after();
          const uint64_t a = sdesc_at(d_kv, s * kPair);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_if(el, ds, sdesc_at(a, (kk >> 2) * kBlock + (kk & 3) * 32),
                      sdesc_at(d_q, (2 * m + (kk >> 2)) * C::kQBlk + (kk & 3) * 32), id, m > 0 || kk > 0);
        }
        if (++s == kPairs) s = 0, ph ^= 1;
      }
      const int rs = i % kRopes;
      ok = ok && wait.warp(&sh->rfull[rs], (i / kRopes) & 1);
      if (!ok) break;
      tc_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ss_if(el, ds, sdesc_at(d_pe, rs * kBlock + kk * 32), sdesc_at(d_q, 8 * C::kQBlk + kk * 32), id, 1);
      mma_commit_if(el, &sh->sfull[sb]);
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
      if (sh->need[i & 1][0] == i + 1 && !wait.warp(&sh->pfix[0], fixed0++ & 1)) break;
      if (sh->need[i & 1][1] == i + 1 && !wait.warp(&sh->pfix[1], fixed1++ & 1)) break;
      tc_after();
      const uint64_t pd = sdesc_at(d_p, rs * kBlock);
#pragma unroll
      for (int m = 0; m < kPairsPerTile; ++m) {
        const uint64_t v = sdesc_at(d_v, s * kPair);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss_if(el, tmem + m * kH, sdesc_at(v, kk * 2048), sdesc_at(pd, kk * 2048), id, i > 0 || kk > 0);
        mma_commit_if(el, &sh->empty[s]);
        if (++s == kPairs) s = 0;
      }
      mma_commit_if(el, &sh->rempty[rs]);
    }
    mma_commit_if(el, &sh->drain_pv);
    wait.drain(&sh->drain_pv, 0);
  }
  } else if (warp < 12) {
    if constexpr (kFmt != 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    // ------------------------------------------------------------ softmax
    const int g = (warp - 4) >> 2, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    float l[kHT];
#pragma unroll
    for (int h = 0; h < kHT; ++h) l[h] = 0.f;
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    const float* nref = sh->nref + g * kHT;
    int gph = 0;
    // among the group's four warps (bounded, so an aborted CTA never stays here)
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->gbar[g]);
      const bool all = wait.warp(&sh->gbar[g], gph);
      gph ^= 1;
      return all;
    };
    bool ok = true;
    for (int i = 0; i < ntiles; ++i) {
      const int e = u.t0 + i * kTile + row;
      bool valid = e < u.t1;
      if (valid && p.pt.row(u.b, e) < 0) {
        valid = false;
        if (g == 0) atomicOr(&sh->flags, kDevBadPage);
      }
      const int sb = i & 1, rs = i % kRopes;
      const uint32_t ts = tl + C::kTmemS + sb * kH + g * kHT;
      volatile int* need = &sh->need[i & 1][g];
      ok = ok && wait.warp(&sh->sfull[sb], (i >> 1) & 1);
      tc_after();
      uint32_t r[kHT];
      tmem_ld<kHT>(ts, r);
      // scores relative to their head's reference
      float top = -INFINITY;
      auto refer = [&]() {
#pragma unroll
        for (int h = 0; h < kHT; h += 4) {
          const float4 m = *reinterpret_cast<const float4*>(nref + h);   // minus the references
          const float2 a = __ffma2_rn(make_float2(__uint_as_float(r[h]), __uint_as_float(r[h + 1])), sl2,
                                      make_float2(m.x, m.y));
          const float2 b = __ffma2_rn(make_float2(__uint_as_float(r[h + 2]), __uint_as_float(r[h + 3])), sl2,
                                      make_float2(m.z, m.w));
          r[h] = __float_as_uint(a.x);
          r[h + 1] = __float_as_uint(a.y);
          r[h + 2] = __float_as_uint(b.x);
          r[h + 3] = __float_as_uint(b.y);
          top = fmaxf(fmaxf(top, fmaxf(a.x, a.y)), fmaxf(b.x, b.y));
        }
      };
      // P over the rotary block, whose scores are done (r becomes p)
      uint8_t* pb = rope(rs);
      auto put = [&]() {
#pragma unroll
        for (int c = 0; c < kHT / 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int h = 8 * c + 2 * k;
            float a = ex2(__uint_as_float(r[h])), b = ex2(__uint_as_float(r[h + 1]));
            a = valid ? a : 0.f;
            b = valid ? b : 0.f;
            r[h] = __float_as_uint(a);
            r[h + 1] = __float_as_uint(b);
            const __nv_bfloat162 ab = __floats2bfloat162_rn(a, b);
            w[k] = *reinterpret_cast<const uint32_t*>(&ab);
          }
          *reinterpret_cast<uint4*>(pb + swz_chunk(row, g * (kHT / 8) + c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      };
      refer();
      const bool over = __any_sync(0xffffffffu, valid && top > kRaise);
      if (over && lane == 0) *need = i + 1;
      put();
      if (kFmt == 0 && !valid) {
        // a row that is not attended to holds anything, or nothing was loaded
        // there: zeros, so that P = 0 never meets a non-finite value
#pragma unroll 1
        for (int m = 2 * g; m < 2 * g + 2; ++m) {
          uint8_t* v = pair((kPairsPerTile * i + m) % kPairs);
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(v + (c >> 3) * kBlock + swz_chunk(row, c & 7)) = make_uint4(0, 0, 0, 0);
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
        tmem_ld<kHT>(ts, r);
        float mine = -INFINITY;
#pragma unroll
        for (int h = 0; h < kHT; ++h) {
          const float x = __uint_as_float(r[h]) * sl2.x;
          int k = __float_as_int(valid && x == x ? x : -INFINITY);
          k ^= (k >> 31) & 0x7fffffff;   // ordered as signed integers
          k = __reduce_max_sync(0xffffffffu, k);
          if (lane == h) mine = __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
        }
        if (lane < kHT) sh->part[g][quad][lane] = mine;
        ok = group_sync();
        if (quad == 0 && lane < kHT) {
          const float old = -nref[lane];
          const float m = fmaxf(fmaxf(fmaxf(sh->part[g][0][lane], sh->part[g][1][lane]),
                                      fmaxf(sh->part[g][2][lane], sh->part[g][3][lane])), old);
          sh->alpha[g * kHT + lane] = exp2f(old - m);
          sh->nref[g * kHT + lane] = -m;
        }
        ok = group_sync() && ok;
        const float* alpha = sh->alpha + g * kHT;
#pragma unroll
        for (int h = 0; h < kHT; ++h) l[h] *= alpha[h];
        refer();
        put();
        fence_async_smem();
        if (i > 0) {   // O holds the tiles before this one
          ok = ok && wait.warp(&sh->rempty[(i - 1) % kRopes], ((i - 1) / kRopes) & 1);
          tc_after();
#pragma unroll 1
          for (int c = 0; c < 4 * kHT; c += 8) {
            const int at = (c / kHT) * kH + g * kHT + c % kHT;
            uint32_t o[8];
            tmem_ld<8>(tl + at, o);
#pragma unroll
            for (int h = 0; h < 8; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * alpha[c % kHT + h]);
            tmem_st<8>(tl + at, o);
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
      for (int h = 0; h < kHT; h += 2) {
        const float2 s2 = __fadd2_rn(make_float2(l[h], l[h + 1]), make_float2(__uint_as_float(r[h]), __uint_as_float(r[h + 1])));
        l[h] = s2.x;
        l[h + 1] = s2.y;
      }
    }
    // ------------------------------------------------------------ epilogue
    float mine = 0.f;
#pragma unroll
    for (int h = 0; h < kHT; ++h) {
      float x = l[h];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == h) mine = x;
    }
    // (the last raise's reads of `part` precede its second barrier)
    if (lane < kHT) sh->part[g][quad][lane] = mine;
    ok = ok && wait.warp(&sh->rempty[(ntiles - 1) % kRopes], ((ntiles - 1) / kRopes) & 1);
    softmax_sync();
    const bool direct = (u.flags & kUnitDirect) != 0;
    if (quad == 0 && lane < kHT) {
      const int h = g * kHT + lane;
      const float sum = (sh->part[g][0][lane] + sh->part[g][1][lane]) + (sh->part[g][2][lane] + sh->part[g][3][lane]);
      const bool fin = ok && !sh->abort;
      sh->inv[h] = fin && sum != 0.f ? 1.f / sum : 0.f;
      const float lse = fin && sum != 0.f ? (log2f(sum) - sh->nref[h]) * 0.69314718055994531f : -INFINITY;
      if (!direct)
        p.ws.part_lse[(size_t)unit_id * p.H + h0 + h] = lse;
      else if (p.lse)
        p.lse[(size_t)u.b * p.H + h0 + h] = lse;
    }
    softmax_sync();
    tc_after();
    // a warp's 32 lanes are 32 consecutive latent columns of one head
#pragma unroll 1
    for (int m = 2 * g; m < 2 * g + 2; ++m) {
      const int col = 128 * m + row;
#pragma unroll 1
      for (int hb = 0; hb < kH; hb += 16) {
        uint32_t o[16];
        tmem_ld<16>(tl + m * kH + hb, o);
        if (direct) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((size_t)u.b * p.H + h0 + hb) * kDc + col;
#pragma unroll
          for (int k = 0; k < 16; ++k) dst[k * kDc] = __float2bfloat16_rn(__uint_as_float(o[k]) * sh->inv[hb + k]);
        } else {
          float* dst = p.ws.part_o + ((size_t)unit_id * p.H + h0 + hb) * kDc + col;
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
      if (!wait.warp(&sh->empty[s], ((n / kPairs) & 1) ^ 1)) break;
      load_blocks(bx, p.box, pair(s), &p.m_kv, 128 * m, 2, &sh->full[s]);
    }
    if (lane == 0 && sh->abort && i > 0) {
      const int n = kPairsPerTile * (i - 1) + m;
      wait.drain(&sh->full[n % kPairs], (n / kPairs) & 1);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ converter
    // A tile's pairs 0 and 1 are converted in registers while the tile before
    // it is still in use, and pair 2 loaded; as the value sum frees the slots,
    // the first two need their stores only.
    const int t = threadIdx.x - 384;
    ConvRows next;   // of the tile after the one in registers
    int rows[kConvEach];
    ConvData raw[2];
    ConvOut out[2];
    auto bring = [&](int e_next) {
#pragma unroll
      for (int k = 0; k < kConvEach; ++k) rows[k] = next.row(p.pt, k);
      next.fetch(p.pt, u.b, e_next, u.t1, t);
      raw[0].load(rows, p.kv, p.kv_scale, 0, t);
      raw[1].load(rows, p.kv, p.kv_scale, 1, t);
      out[0].convert(raw[0]);
      raw[0].load(rows, p.kv, p.kv_scale, 2, t);
      out[1].convert(raw[1]);
    };
    next.fetch(p.pt, u.b, u.t0, u.t1, t);
    bring(u.t0 + kTile);
    int s = 0, ph = 1;   // the ring's slot, and the phase that frees it
    for (int i = 0; i < ntiles; ++i) {
      bool ok = true;
#pragma unroll
      for (int m = 0; m < kPairsPerTile; ++m) {
        if (m >= 2) out[m & 1].convert(raw[m & 1]);
        ok = ok && wait.warp(&sh->empty[s], ph);
        if (ok) {
          out[m & 1].store(pair(s), t);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(&sh->full[s]);
        }
        if (m == 0) raw[1].load(rows, p.kv, p.kv_scale, 3, t);
        if (++s == kPairs) s = 0, ph ^= 1;
      }
      if (!ok) break;
      if (i + 1 < ntiles) bring(u.t0 + (i + 2) * kTile);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_before();
  __syncthreads();
  if (threadIdx.x == 0 && u.b >= 0) p.ws.unit_flags[blockIdx.x] = sh->flags;
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
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
  return launch_pdl(decode_kernel<kFmt, kH>, dim3((unsigned)units * p.groups), dim3(C::kThreads), C::kSmem, s, p);
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

cudaError_t launch_paged_decode(const DecodeParams& d, cudaStream_t s) {
  using namespace paged;
  Params p;
  memset(&p, 0, sizeof(p));
  const int kh = d.H < 64 ? d.H : 64;   // heads per CTA
  const uint64_t pages = (uint64_t)d.pt.num_pages, rows = (uint64_t)d.pt.page_size, B = (uint64_t)d.B, H = (uint64_t)d.H;
  p.box = box_rows(d.pt.page_size);
  if ((d.fmt == 0 && !encode_rows(&p.m_kv, d.kv, kDc, rows, pages, p.box)) ||
      !encode_rows(&p.m_pe, d.pe, kDr, rows, pages, p.box) || !encode_rows(&p.m_ql, d.q_latent, kDc, H, B, kh) ||
      !encode_rows(&p.m_qp, d.q_pe, kDr, H, B, kh))
    return cudaErrorInvalidValue;
  p.kv = d.kv;
  p.kv_scale = d.kv_scale;
  p.pt = d.pt;
  p.H = d.H;
  p.groups = d.H / kh;
  p.scale_log2 = d.scale_log2;
  p.out = d.out;
  p.lse = d.lse;
  p.ws = d.ws;
  p.sched = d.sched;
  const int units = d.ws.max_units;
  if (d.fmt == 0)
    return kh == 16 ? launch<0, 16>(p, units, s) : kh == 32 ? launch<0, 32>(p, units, s) : launch<0, 64>(p, units, s);
  return kh == 16 ? launch<1, 16>(p, units, s) : kh == 32 ? launch<1, 32>(p, units, s) : launch<1, 64>(p, units, s);
}

}  // namespace mla
