// paged_rotary.cu -- a token's way into a paged cache from the projections'
// outputs, in one launch: RMSNorm of the latent, rotation of the rotary key and
// of every head's rotary query by the token's position, quantisation, and the
// write through the page table.
//
//   y_c = x_c * w_c / sqrt(mean(x^2) + eps)                       (512 latent columns)
//   (u, v) -> gain * (u cos a - v sin a, v cos a + u sin a),  a = pos * freq_i
//                                        (32 pairs of columns, of the key and of each query)
//
// Angles.  A position may be 10^6 and a frequency 1, so pos * freq in 32 bits is
// off by hundredths of a radian.  The frequency is held as a fraction of a turn
// in 64-bit fixed point (2^64 = one turn): pos * turn modulo 2^64 is then the
// angle's fraction of a turn, exact but for the frequency's own rounding (2^-64
// turns a position), in one integer multiplication, at any position.  Its upper
// 32 bits, as a signed fraction of a half turn, go to sincospif: 2^-24 of a half turn.
//
// Two kinds of CTA.  Rows (the first `row_ctas`): a warp takes a new row, four
// values of each of the four scale blocks a lane, so the norm's sum and the
// blocks' maxima are warp reductions and nothing crosses warps.  Queries: a CTA
// takes 64 head rows of 192 values, six 16-byte pieces a thread, all loaded before
// the first is stored (32 rows 128, 128 rows 124, 64 rows 122 us at 8192 tokens of
// 128 heads; 12.1, 13.6 and 11.6 at 5105 of 16).  A thread's two rotary pieces hold both columns of
// its pairs in either layout.  The cosines of the CTA's tokens (at most four) are worked out
// once, a lane a pair, while the loads are under way.
//
// Bound by the bytes: 8192 tokens of 128 heads, FP8, 122.8 us (820 MB, 6.7 TB/s,
// 0.98 of a copy's rate); 5105 of 16 heads, bf16, 11.8 us (6.3 TB/s); 32 of 128 heads
// 3.3 us and one 2.5, launch and three dependent reads (position, table, row).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "append_row.cuh"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeadRows = 64, kTokens = kHeadRows / 16;   // of a query CTA; tokens that they are of at most
constexpr int kDn = 128;   // content columns of a head's query, before its 64 rotary ones

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// gain * (cos, sin) of a position's angle
__device__ __forceinline__ float2 turn_of(int pos, uint64_t turn, float gain) {
  const uint64_t phase = (uint64_t)(int64_t)pos * turn;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(gain * c, gain * s);
}
__device__ __forceinline__ float2 rotated(float2 uv, float2 cs) {
  return make_float2(uv.x * cs.x - uv.y * cs.y, uv.y * cs.x + uv.x * cs.y);
}

// New row i (token i % s of sequence i / s), by one warp.
__device__ __forceinline__ void write_row(const RotaryAppend& p, int i, int lane) {
  const int b = i / p.s, j = i - b * p.s;
  const __nv_bfloat16* x = p.kv_a + b * p.kv_sb + j * p.kv_ss;
  uint2 raw[kNblk];
#pragma unroll
  for (int k = 0; k < kNblk; ++k) raw[k] = *reinterpret_cast<const uint2*>(x + k * kBlk + 4 * lane);
  // the lane's pair of rotary columns: 2 lane and 2 lane + 1, or lane and lane + 32
  uint32_t kr;
  if (p.halves) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(x + kDc);
    kr = h[lane] | (uint32_t)h[lane + 32] << 16;
  } else {
    kr = reinterpret_cast<const uint32_t*>(x + kDc)[lane];
  }
  float2 w[kNblk][2];
#pragma unroll
  for (int k = 0; k < kNblk; ++k) {
    if (p.norm_f32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.norm) + k * kBlk + 4 * lane);
      w[k][0] = make_float2(f.x, f.y), w[k][1] = make_float2(f.z, f.w);
    } else {
      const uint2 f = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.norm) + k * kBlk + 4 * lane);
      w[k][0] = unpack(f.x), w[k][1] = unpack(f.y);
    }
  }
  const int angle_pos = p.pos[i];
  const uint64_t turn = p.turns[lane];
  const long long at = (long long)p.end_pos[b] - p.s + j;
  uint32_t flags = kDevAppendSkipped;
  int row = -1;
  if (at >= 0 && at < p.max_pos) {
    row = p.pt.row(b, (int)at);
    if (row < 0) flags |= kDevBadPage;
  }
  if (row < 0) {
    if (lane == 0 && p.status) atomicOr(p.status, flags);
    return;
  }
  float2 y[kNblk][2];
  auto squares = [&]() {
    float2 a = make_float2(0.f, 0.f), c = a;
#pragma unroll
    for (int k = 0; k < kNblk; ++k) {
      a = __ffma2_rn(y[k][0], y[k][0], a);
      c = __ffma2_rn(y[k][1], y[k][1], c);
    }
    float s = (a.x + a.y) + (c.x + c.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
#pragma unroll
  for (int k = 0; k < kNblk; ++k) y[k][0] = unpack(raw[k].x), y[k][1] = unpack(raw[k].y);
  float sum = squares(), eps = p.eps;
  // squares that leave the 32-bit range (|x| from 2^59 on; below 2^-48, where eps
  // does not cover them): the row is scaled by a power of two, and so is eps
  if (sum >= 0x1p127f || (sum < 0x1p-96f && eps < 0x1p-70f)) {
    const float f = sum < 1.f ? 0x1p80f : 0x1p-70f;
#pragma unroll
    for (int k = 0; k < kNblk; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m) y[k][m] = __fmul2_rn(y[k][m], make_float2(f, f));
    sum = squares();
    eps = eps * f * f;
  }
  const float r = __frsqrt_rn(sum * (1.0f / kDc) + eps);
#pragma unroll
  for (int k = 0; k < kNblk; ++k)
#pragma unroll
    for (int m = 0; m < 2; ++m) y[k][m] = __fmul2_rn(__fmul2_rn(y[k][m], make_float2(r, r)), w[k][m]);
  const AppendRows& c = p.rows;
  if (c.fmt == 0) {
#pragma unroll
    for (int k = 0; k < kNblk; ++k)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(c.kv) + (size_t)row * kDc + k * kBlk + 4 * lane) =
          make_uint2(pack(y[k][0].x, y[k][0].y), pack(y[k][1].x, y[k][1].y));
  } else {
    // quantised from the 32-bit values: each is rounded once
    float scale[kNblk];
#pragma unroll
    for (int k = 0; k < kNblk; ++k) {
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(c.kv) + (size_t)row * kDc + k * kBlk + 4 * lane) =
          quantize4(y[k][0], y[k][1], c.fmt, &scale[k]);
    }
    if (lane == 0) *reinterpret_cast<float4*>(c.kv_scale + (size_t)row * kNblk) = make_float4(scale[0], scale[1], scale[2], scale[3]);
  }
  const float2 z = rotated(unpack(kr), turn_of(angle_pos, turn, p.gain));
  const uint32_t o = pack(z.x, z.y);
  __nv_bfloat16* pe = static_cast<__nv_bfloat16*>(c.pe) + (size_t)row * kDr;
  if (p.halves) {
    reinterpret_cast<uint16_t*>(pe)[lane] = (uint16_t)o;
    reinterpret_cast<uint16_t*>(pe)[lane + 32] = (uint16_t)(o >> 16);
  } else {
    reinterpret_cast<uint32_t*>(pe)[lane] = o;
  }
  if (lane == 0 && p.weight) p.weight[row] = 0.f;
}

// Head rows r0 .. r0 + 63 (row r: head r % H of token r / H).
__device__ __forceinline__ void turn_queries(const RotaryAppend& p, int r0) {
  __shared__ const __nv_bfloat16* src[kTokens];
  __shared__ float4 cs[kTokens][kDr / 4];   // cosine and sine of two pairs
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int tok0 = r0 >> p.log_h, n = p.B * p.s, last = min(n, ((r0 + kHeadRows - 1) >> p.log_h) + 1) - tok0;
  int pos = 0;
  if (warp < last) {
    const int tok = tok0 + warp, b = tok / p.s;
    pos = p.pos[tok];
    if (lane == 0) src[warp] = p.q + b * p.q_sb + (tok - b * p.s) * p.q_ss;
  }
  __syncthreads();
  const int total = n << p.log_h, mask = (1 << p.log_h) - 1;
  auto from = [&](int r) { return reinterpret_cast<const uint4*>(src[(r >> p.log_h) - tok0] + (r & mask) * p.q_sh); };
  // two of the eight pieces of a row's rotary part, which hold the pairs' both
  // columns: 2 c and 2 c + 1, or c and c + 4
  const int rr = r0 + (t >> 2), c0 = p.halves ? t & 3 : 2 * (t & 3), c1 = p.halves ? c0 + 4 : c0 + 1;
  uint4 a[4], v0, v1;
  if (rr < total) {
    v0 = __ldcs(from(rr) + kDn / 8 + c0);
    v1 = __ldcs(from(rr) + kDn / 8 + c1);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = r0 + (t >> 4) + 16 * k;
    if (r < total) a[k] = __ldcs(from(r) + (t & 15));
  }
  if (warp < last) reinterpret_cast<float2*>(cs[warp])[lane] = turn_of(pos, p.turns[lane], p.gain);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = r0 + (t >> 4) + 16 * k;
    if (r < total) reinterpret_cast<uint4*>(p.q_nope + (size_t)r * kDn)[t & 15] = a[k];
  }
  if (rr >= total) return;
  const float4* tab = cs[(rr >> p.log_h) - tok0] + 4 * (t & 3);   // of the eight pairs
  uint32_t x[4] = {v0.x, v0.y, v0.z, v0.w}, y[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    if (p.halves) {   // pairs 2 m and 2 m + 1: one column in x, the other in y
      const float4 f = tab[m];
      const float2 u = unpack(x[m]), v = unpack(y[m]);
      const float2 e = rotated(make_float2(u.x, v.x), make_float2(f.x, f.y)), o = rotated(make_float2(u.y, v.y), make_float2(f.z, f.w));
      x[m] = pack(e.x, o.x);
      y[m] = pack(e.y, o.y);
    } else {          // pair m of either piece
      const float2 f = reinterpret_cast<const float2*>(tab)[m], g = reinterpret_cast<const float2*>(tab)[4 + m];
      const float2 e = rotated(unpack(x[m]), f), o = rotated(unpack(y[m]), g);
      x[m] = pack(e.x, e.y);
      y[m] = pack(o.x, o.y);
    }
  }
  uint4* out = reinterpret_cast<uint4*>(p.q_pe + (size_t)rr * kDr);
  out[c0] = make_uint4(x[0], x[1], x[2], x[3]);
  out[c1] = make_uint4(y[0], y[1], y[2], y[3]);
}

__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const RotaryAppend p) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < p.row_ctas) {
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i < p.B * p.s) write_row(p, i, threadIdx.x & 31);
  } else {
    turn_queries(p, (blockIdx.x - p.row_ctas) * kHeadRows);
  }
}

}  // namespace

cudaError_t launch_append_rotary(RotaryAppend p, cudaStream_t s) {
  const int n = p.B * p.s;
  p.row_ctas = (n + kWarps - 1) / kWarps;
  const int64_t heads = p.q ? (int64_t)n << p.log_h : 0;
  const unsigned grid = (unsigned)(p.row_ctas + (heads + kHeadRows - 1) / kHeadRows);
  return launch_pdl(append_rotary_kernel, dim3(grid), dim3(kThreads), 0, s, p);
}

}  // namespace mla
