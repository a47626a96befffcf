// topk.cuh -- selection of the K largest of a sequence's keys by a cluster of
// CTAs, shared by the top-k position selection (per-position scores) and the
// eviction (accumulated attention weights).
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace mla {

// A cluster of kTopkCtas CTAs per sequence selects, among positions
// 0 .. T-1, the K with the largest key (equal keys: the lower position) and
// writes them in increasing order, then -1.  Keys are order-preserving 32-bit
// words (score_key); CTA r of the cluster holds the keys of the r-th of
// kTopkCtas equal runs of positions in shared memory (read once).  A
// radix select over the key's four bytes (most significant first) finds the
// K-th largest key t and how many keys equal to t belong to the selection:
// per pass every CTA builds a 256-bin histogram of its run, and after one
// cluster barrier each CTA sums the kTopkCtas histograms through distributed
// shared memory and takes the same decision (histograms alternate between
// two buffers by pass, so none is cleared while a peer still reads it).  A
// last pass counts, per CTA and per warp, the keys above and equal to t,
// turns the counts into offsets (the peers' through distributed shared
// memory) and writes the selected positions in order.
constexpr int kTopkCtas = 8;
constexpr int kTopkThreads = 512;
constexpr int kTopkSmemKeys = 55296;   // runs up to this many positions are staged (216 KB)

__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;                             // NaN: below every number
  const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);   // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <bool kSmem, class Src>
__device__ __forceinline__ void topk_select_body(const Src& src, int T, int K, int* o) {
  extern __shared__ uint32_t keys_smem[];   // kSmem: this CTA's run of keys
  __shared__ uint32_t hist[2][256];
  __shared__ uint32_t ghist[256];
  __shared__ int wgt[kTopkThreads / 32], weq[kTopkThreads / 32];
  __shared__ int cta_cnt[2];   // this CTA's keys above / equal to t (read by the peers)
  __shared__ uint32_t s_prefix;
  __shared__ int s_krem, s_all;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kTopkThreads / 32;
  if (T <= K) {   // every valid position is selected (the same test in every CTA of the cluster)
    if (rank == 0)
      for (int k = tid; k < K; k += kTopkThreads) o[k] = k < T ? k : -1;
    return;
  }
  // this CTA's run [c0, c1): a multiple of 4 positions long except the last
  const int per = ((T + kTopkCtas - 1) / kTopkCtas + 3) & ~3;
  const int c0 = min((int)rank * per, T), c1 = min(c0 + per, T), n = c1 - c0;
  if (kSmem) src.stage(keys_smem, c0, n);
  // key of the run's i-th position
  auto key_at = [&](int i) -> uint32_t { return kSmem ? keys_smem[i] : src.key(c0 + i); };

  uint32_t prefix = 0u, mask = 0u;
  int krem = K;   // selected positions still to place at or below the current prefix
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* h = hist[pass & 1];
    for (int i = tid; i < 256; i += kTopkThreads) h[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kTopkThreads) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) atomicAdd(&h[(key >> shift) & 255u], 1u);
    }
    ptx::cluster_sync();   // every CTA's histogram of this pass is complete
    for (int i = tid; i < 256; i += kTopkThreads) {
      uint32_t sum = 0;
#pragma unroll
      for (int r = 0; r < kTopkCtas; ++r) sum += ld_cluster_u32(ptx::mapa(&h[i], r));
      ghist[i] = sum;
    }
    __syncthreads();
    if (tid < 32) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l (largest first)
      uint32_t cnt[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cnt[e] = ghist[255 - 8 * lane - e];
        sum += cnt[e];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o2 = 1; o2 < 32; o2 <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o2);
        if (lane >= o2) incl += y;
      }
      const uint32_t before = incl - sum;   // keys in the bins above this lane's
      if (before < (uint32_t)krem && (uint32_t)krem <= incl) {
        uint32_t acc = before;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (acc + cnt[e] >= (uint32_t)krem) {
            s_prefix = prefix | ((uint32_t)(255 - 8 * lane - e) << shift);
            s_krem = krem - (int)acc;
            s_all = acc + cnt[e] == (uint32_t)krem;
            break;
          }
          acc += cnt[e];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    krem = s_krem;
    mask |= 255u << shift;
    // Every key of the bin is selected, so the lower bytes decide nothing: take
    // the keys above prefix - 1.  (prefix > 0: the keys from 0 on are all T > K.)
    // With distinct scores one pass of four is left out (an eviction of 2048 of
    // 4096 rows 11.4 -> 10.4 us).
    if (s_all) {
      --prefix;
      krem = 0;
      break;
    }
  }

  // The keys above prefix are selected, and krem of those equal to it.
  // Warp w owns run positions [w R, w R + R), R a multiple of 32.
  const int R = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int q0 = warp * R, q1 = min(q0 + R, n);
  int ngt = 0, neq = 0;
  for (int i = q0 + lane; i < q1; i += 32) {
    const uint32_t key = key_at(i);
    ngt += key > prefix;
    neq += key == prefix;
  }
  ngt = __reduce_add_sync(0xffffffffu, ngt);
  neq = __reduce_add_sync(0xffffffffu, neq);
  if (lane == 0) {
    wgt[warp] = ngt;
    weq[warp] = neq;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive scans of the warps' counts; this CTA's totals
    const int g = lane < kWarps ? wgt[lane] : 0, e = lane < kWarps ? weq[lane] : 0;
    int gi = g, ei = e;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const int yg = __shfl_up_sync(0xffffffffu, gi, o2), ye = __shfl_up_sync(0xffffffffu, ei, o2);
      if (lane >= o2) {
        gi += yg;
        ei += ye;
      }
    }
    if (lane < kWarps) {
      wgt[lane] = gi - g;
      weq[lane] = ei - e;
    }
    if (lane == kWarps - 1) {
      cta_cnt[0] = gi;
      cta_cnt[1] = ei;
    }
  }
  ptx::cluster_sync();   // every CTA's totals are in place
  int gbase = 0, ebase = 0;   // keys above / equal to t in the runs of the lower ranks
  for (int r = 0; r < (int)rank; ++r) {
    gbase += (int)ld_cluster_u32(ptx::mapa(&cta_cnt[0], r));
    ebase += (int)ld_cluster_u32(ptx::mapa(&cta_cnt[1], r));
  }
  int gt = gbase + wgt[warp], eq = ebase + weq[warp];   // before this warp's next step
  const uint32_t lt = (1u << lane) - 1u;
  for (int i0 = q0; i0 < q1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < q1 ? key_at(i) : 0u;
    const bool is_gt = i < q1 && key > prefix, is_eq = i < q1 && key == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const int g_before = gt + __popc(bg & lt), e_before = eq + __popc(be & lt);
    if (is_gt) o[g_before + min(e_before, krem)] = c0 + i;
    if (is_eq && e_before < krem) o[g_before + e_before] = c0 + i;
    gt += __popc(bg);
    eq += __popc(be);
  }
  ptx::cluster_sync();   // no peer reads this CTA's counts any more
}

}  // namespace mla
