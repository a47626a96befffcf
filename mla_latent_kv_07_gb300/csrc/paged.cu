// paged.cu -- the operators of a paged cache beside its decode: the cache write
// of new rows through the page table, and the eviction of the rows that drew
// the least attention weight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cuda.h>

#include "append_row.cuh"
#include "common.cuh"
#include "paged_tile.cuh"
#include "topk.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------- append
// kRows new rows per CTA of four warps (a warp per latent block), all loaded
// before the first is stored.  A position below 0 or past the table, and one
// on a page that is not in the pool, is left out and flagged.
template <int kRows>
__global__ void __launch_bounds__(128) paged_append_kernel(const PagedAppend p) {
  pdl_wait();
  pdl_trigger();
  __shared__ int rows[kRows];
  const int n = p.B * p.s, i0 = blockIdx.x * kRows;
  AppendPiece x[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) x[k] = append_load(p.rows, min(i0 + k, n - 1), threadIdx.x);
  if (threadIdx.x < kRows) {
    const int i = i0 + threadIdx.x;
    int row = -1;
    if (i < n) {
      const int b = i / p.s;
      const long long pos = (long long)p.end_pos[b] - p.s + (i - b * p.s);
      uint32_t flags = kDevAppendSkipped;
      if (pos >= 0 && pos < p.max_pos) {
        row = p.pt.row(b, (int)pos);
        if (row < 0) flags |= kDevBadPage;
      }
      if (row >= 0 && p.weight) p.weight[row] = 0.f;
      if (row < 0 && p.status) atomicOr(p.status, flags);
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int row = rows[k];
    if (row >= 0) append_store(p.rows, (size_t)row, threadIdx.x, x[k]);   // (the same way for the whole CTA)
  }
}

// ------------------------------------------------------------------ read
// kRows packed rows per CTA: the first warp finds their pool rows (-1: zeros, -2:
// behind the last sequence, left as it is) by searches whose steps grow with the
// logarithm of the sequences' number, empty ones included, then every 16-byte piece of output is
// loaded (bf16: 16 bytes; FP8: 8 codes and their scale) before the first is
// stored.  Bound by the rows' bytes, read and written.
constexpr int kReadThreads = 256;

template <int kFmt, int kRows>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const PagedRead p) {
  static_assert(kRows <= 32 && kRows * 64 % kReadThreads == 0, "a lane per row, whole rounds");
  __shared__ int rows[kRows];
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * kRows;
  if (threadIdx.x < 32) {
    // the last b with offsets[b] <= n0, 32 candidates at a time
    const int lane = threadIdx.x;
    int b = 0, len = p.B + 1;
    while (len > 1) {
      const int step = (len + 31) / 32, i = lane * step;
      const int below = __popc(__ballot_sync(0xffffffffu, i < len && p.offsets[b + i] <= n0));
      const int skip = below > 0 ? (below - 1) * step : 0;
      b += skip;
      len = min(step, len - skip);
    }
    const int n = n0 + lane;
    if (lane < kRows) {
      // its own sequence: this one or one of the next, unless many are empty
#pragma unroll 1
      for (int k = 0; b < p.B && p.offsets[b + 1] <= n; ++k) {
        ++b;
        if (k < 4) continue;
        for (int hi = p.B; b < hi;) {   // the last with offsets[.] <= n is in b .. hi
          const int mid = b + (hi - b + 1) / 2;
          if (p.offsets[mid] <= n)
            b = mid;
          else
            hi = mid - 1;
        }
        break;
      }
      int row = -2;
      if (n < p.total && b < p.B && n >= p.offsets[b]) {
        const long long t = (long long)(p.first ? p.first[b] : 0) + (n - p.offsets[b]);
        row = t >= 0 && t < p.max_pos ? p.pt.row(b, (int)t) : -1;
        if (row < 0 && p.status) atomicOr(p.status, kDevBadPage);
      }
      rows[lane] = row;
    }
  }
  __syncthreads();
  constexpr int kEach = kRows * 64 / kReadThreads;   // 64 pieces of a latent row
  uint4 v[kEach];
  float sc[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int c = threadIdx.x + e * kReadThreads, row = rows[c >> 6], k = c & 63;
    v[e] = make_uint4(0, 0, 0, 0);
    sc[e] = 0.f;
    if (row >= 0) {
      if (kFmt == 0) {
        v[e] = __ldcs(static_cast<const uint4*>(p.kv) + (size_t)row * 64 + k);
      } else {
        const uint2 w = __ldcs(static_cast<const uint2*>(p.kv) + (size_t)row * 64 + k);
        v[e].x = w.x, v[e].y = w.y;
        sc[e] = p.kv_scale[(size_t)row * kNblk + (k >> 4)];
      }
    }
  }
  // the rotary columns: 8 pieces a row
  uint4 r = make_uint4(0, 0, 0, 0);
  const int rr = threadIdx.x >> 3, rk = threadIdx.x & 7;
  const int rrow = rr < kRows ? rows[rr] : -2;
  if (rrow >= 0) r = __ldcs(static_cast<const uint4*>(p.pe) + (size_t)rrow * 8 + rk);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int c = threadIdx.x + e * kReadThreads, m = c >> 6, k = c & 63;
    const uint4 o = kFmt == 0 ? v[e] : paged::dequant8(make_uint2(v[e].x, v[e].y), sc[e]);
    if (rows[m] > -2) reinterpret_cast<uint4*>(p.out_kv + (n0 + m) * p.kv_stride)[k] = o;
  }
  if (rrow > -2) reinterpret_cast<uint4*>(p.out_pe + (n0 + rr) * p.pe_stride)[rk] = r;
}

// ----------------------------------------------------------------- evict
// Keys of the selection: the accumulated weight of the position's row (NaN
// lowest, score_key), and the largest key there is for the first `sinks` and
// the last `recent` positions, which are always kept.
struct WeightRows {
  const float* weight;
  const PagedTable& pt;
  int b, sinks, tail;
  __device__ __forceinline__ uint32_t key_of(int i, float w) const {
    return i < sinks || i >= tail ? 0xffffffffu : score_key(w);
  }
  __device__ __forceinline__ uint32_t key(int i) const { return key_of(i, weight[pt.row(b, i)]); }
  // (a thread's table entries, then its weights, four loads in flight: 2 x 65536
  // positions 31.8 -> 25.3 us, eight 24.6; 32 x 8192 45.7 -> 44.1, 44.6)
  __device__ __forceinline__ void stage(uint32_t* keys, int c0, int n) const {
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kTopkThreads) {
      int row[kAhead];
      float w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kTopkThreads;
        if (i < n) row[k] = pt.row(b, c0 + i);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * kTopkThreads < n) w[k] = weight[row[k]];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kTopkThreads;
        if (i < n) keys[i] = key_of(c0 + i, w[k]);
      }
    }
  }
};

__device__ __forceinline__ int clamped_end(int end, int max_end_pos) {
  return end < 0 ? 0 : (end > max_end_pos ? max_end_pos : end);
}

// The kept positions of every sequence and their count, by a cluster of CTAs
// per sequence (topk.cuh); bound by the latency of its passes (4096 positions:
// about 8 us of an eviction's 10.4).  A sequence one of whose pages (old or new) is not in the pool keeps nothing and is flagged.
template <bool kSmem>
__global__ void __launch_bounds__(kTopkThreads, 2) evict_select_kernel(const EvictParams p) {
  __shared__ int s_bad;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / kTopkCtas, rank = blockIdx.x % kTopkCtas;
  const int end = p.end_pos[b], T = clamped_end(end, p.max_end_pos), n = min(T, p.keep);
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  // every CTA of the cluster looks at all pages, so all take the same way
  bool bad = false;
  const int np = (T + p.pt.page_size - 1) / p.pt.page_size, nq = (n + p.to.page_size - 1) / p.to.page_size;
  for (int i = threadIdx.x; i < np + nq; i += kTopkThreads) {
    const int id = i < np ? p.pt.table[(size_t)b * p.pt.stride + i] : p.to.table[(size_t)b * p.to.stride + i - np];
    bad |= id < 0 || id >= p.pt.num_pages;
  }
  if (bad) s_bad = 1;
  __syncthreads();
  int* kept = p.kept + (size_t)b * p.keep;
  const bool skip = s_bad != 0;
  if (rank == 0 && threadIdx.x == 0) {
    const uint32_t flags = (T != end ? kDevEndPosClamped : 0u) | (skip ? kDevBadPage : 0u);
    if (flags && p.status) atomicOr(p.status, flags);
  }
  if (skip) {
    if (rank == 0)
      for (int i = threadIdx.x; i < p.keep; i += kTopkThreads) kept[i] = -1;
    return;
  }
  topk_select_body<kSmem>(WeightRows{p.weight, p.pt, b, p.sinks, T - p.recent}, T, p.keep, kept);
}

// Kept row i of every sequence -> row i of its new pages: kCopyRows rows per
// CTA, every 16-byte piece loaded before the first is stored.  Bound by the
// rows' bytes, read and written: 32 sequences of up to 4096 kept FP8 rows (162
// MB) in 30 us (5.4 TB/s), 40.8 us with their selection.  The count of the kept
// rows is written here, since every CTA of the selection's clusters reads end_pos
// when it comes to it, and the new lengths may take its place.
constexpr int kCopyThreads = 288;

template <int kFmt, int kCopyRows>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p) {
  __shared__ int src[kCopyRows], dst[kCopyRows];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, i0 = blockIdx.x * kCopyRows;
  if (threadIdx.x < kCopyRows) {
    const int i = i0 + threadIdx.x;
    const int* kept = p.kept + (size_t)b * p.keep;   // (positions, then -1)
    const int at = i < p.keep ? kept[i] : -1, after = i + 1 < p.keep ? kept[i + 1] : -1;
    if (after < 0 && (at >= 0 || i == 0)) p.new_end[b] = at >= 0 ? i + 1 : 0;
    const int from = at < 0 ? -1 : p.pt.row(b, at), to = at < 0 ? -1 : p.to.row(b, i);
    src[threadIdx.x] = from;
    dst[threadIdx.x] = to;
    if (from >= 0) p.weight[to] = p.weight[from];
  }
  __syncthreads();
  constexpr int kKv = (kFmt == 0 ? kDc * 2 : kDc) / 16, kPe = kDr * 2 / 16, kSc = kFmt == 0 ? 0 : 1;
  constexpr int kChunks = kKv + kPe + kSc;   // 16-byte pieces of a row
  constexpr int kEach = (kCopyRows * kChunks + kCopyThreads - 1) / kCopyThreads;
  uint4 v[kEach];
  uint4* to[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int c = threadIdx.x + e * kCopyThreads, r = c / kChunks, k = c % kChunks;
    to[e] = nullptr;
    if (r < kCopyRows && src[r] >= 0) {
      uint4* base = static_cast<uint4*>(p.kv);
      int width = kKv, off = k;
      if (k >= kKv + kPe) {
        base = reinterpret_cast<uint4*>(p.kv_scale), width = 1, off = 0;
      } else if (k >= kKv) {
        base = static_cast<uint4*>(p.pe), width = kPe, off = k - kKv;
      }
      v[e] = base[(size_t)src[r] * width + off];
      to[e] = base + (size_t)dst[r] * width + off;
    }
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (to[e]) *to[e] = v[e];
}

template <bool kSmem>
cudaError_t launch_select(const EvictParams& p, size_t smem, cudaStream_t s) {
  if (kSmem) {
    cudaError_t e = ensure_smem<evict_select_kernel<kSmem>>((size_t)kTopkSmemKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((unsigned)p.B * kTopkCtas);
  cfg.blockDim = dim3(kTopkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kTopkCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<kSmem>, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppend& p, cudaStream_t s) {
  const unsigned n = (unsigned)p.B * p.s;
  // A row per CTA until they fill the GPU (16 CTAs on each of 152 SMs), then
  // four, so that a prompt's rows do not come in many waves of one load each.
  // One and four, FP8: 32 rows 1.8 and 2.8 us, 2432 rows 3.0 and 3.3, 4864 rows
  // 5.3 and 4.8, 16000 rows 16.6 and 10.3 (29 MB: 2.8 TB/s); bf16, 16000 rows:
  // 16.9 and 7.6 (37 MB: 4.9 TB/s).  The FP8 codes' arithmetic bounds the former.
  if (n <= 2432) return launch_pdl(paged_append_kernel<1>, dim3(n), dim3(128), 0, s, p);
  return launch_pdl(paged_append_kernel<4>, dim3((n + 3) / 4), dim3(128), 0, s, p);
}

cudaError_t launch_paged_read(const PagedRead& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.total + 15) / 16)), block(kReadThreads);
  return p.fmt == 0 ? launch_pdl(paged_read_kernel<0, 16>, grid, block, 0, s, p)
                    : launch_pdl(paged_read_kernel<1, 16>, grid, block, 0, s, p);
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t s) {
  const int per = ((p.max_end_pos + kTopkCtas - 1) / kTopkCtas + 3) & ~3;   // longest run of a CTA
  cudaError_t e = per <= kTopkSmemKeys ? launch_select<true>(p, (size_t)per * 4, s) : launch_select<false>(p, 0, s);
  if (e != cudaSuccess) return e;
  // 16 rows per CTA (18 KB in bf16), and 32 of FP8's where they fill the GPU.
  // 16 and 32 rows: FP8, 1 x 4096 10.4 and 11.0 us, 32 x 4096 44.1 and 42.6;
  // bf16, 8 x 2048 16.9 and 17.7, 32 x 8192 104.7 and 105.5.
  const int rows = p.fmt == 0 || (int64_t)p.B * p.keep < 16384 ? 16 : 32;
  const dim3 grid((unsigned)((p.keep + rows - 1) / rows), (unsigned)p.B), block(kCopyThreads);
  if (p.fmt == 0) return launch_pdl(evict_copy_kernel<0, 16>, grid, block, 0, s, p);
  return rows == 16 ? launch_pdl(evict_copy_kernel<1, 16>, grid, block, 0, s, p)
                    : launch_pdl(evict_copy_kernel<1, 32>, grid, block, 0, s, p);
}

}  // namespace mla
