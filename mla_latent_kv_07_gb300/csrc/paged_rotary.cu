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
// takes 32 kU head rows of 192 values, twelve 16-byte pieces a thread (kU = 4)
// all loaded before the first is stored; the cosines of its tokens (at most
// eight) are worked out once, a lane a pair, while the loads are under way.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "append_row.cuh"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

// Head rows r0 .. r0 + 32 kU - 1 (row r: head r % H of token r / H).
template <int kU>
__device__ __forceinline__ void turn_queries(const RotaryAppend& p, int r0) {
  constexpr int kRows = 32 * kU, kMaxTokens = kRows / 16;
  static_assert(kMaxTokens <= kWarps, "a warp per token");
  __shared__ const __nv_bfloat16* src[kMaxTokens];
  __shared__ float2 cs[kMaxTokens][kDr / 2];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int tok0 = r0 >> p.log_h, n = p.B * p.s, last = min(n, ((r0 + kRows - 1) >> p.log_h) + 1) - tok0;
  int pos = 0;
  if (warp < last) {
    const int tok = tok0 + warp, b = tok / p.s;
    pos = p.pos[tok];
    if (lane == 0) src[warp] = p.q + b * p.q_sb + (tok - b * p.s) * p.q_ss;
  }
  __syncthreads();
  const int total = n << p.log_h, mask = (1 << p.log_h) - 1;
  uint4 a[2 * kU], v[kU];
  auto from = [&](int r) { return src[(r >> p.log_h) - tok0] + (r & mask) * p.q_sh; };
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int r = r0 + (t >> 3) + 32 * k;
    if (r < total) v[k] = __ldcs(reinterpret_cast<const uint4*>(from(r) + kDn) + (t & 7));
  }
#pragma unroll
  for (int k = 0; k < 2 * kU; ++k) {
    const int r = r0 + (t >> 4) + 16 * k;
    if (r < total) a[k] = __ldcs(reinterpret_cast<const uint4*>(from(r)) + (t & 15));
  }
  if (warp < last) cs[warp][lane] = turn_of(pos, p.turns[lane], p.gain);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2 * kU; ++k) {
    const int r = r0 + (t >> 4) + 16 * k;
    if (r < total) reinterpret_cast<uint4*>(p.q_nope + (size_t)r * kDn)[t & 15] = a[k];
  }
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int r = r0 + (t >> 3) + 32 * k, c = t & 7;
    const bool live = r < total;
    const float2* tab = cs[live ? (r >> p.log_h) - tok0 : 0];
    uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, out[4];
    if (p.halves) {
      // values 8 c .. 8 c + 7; the other half of their pairs is four lanes away
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 own = unpack(in[m]), other = unpack(__shfl_xor_sync(0xffffffffu, in[m], 4));
        const float2 c0 = tab[8 * (c & 3) + 2 * m], c1 = tab[8 * (c & 3) + 2 * m + 1];
        out[m] = c < 4 ? pack(rotated(make_float2(own.x, other.x), c0).x, rotated(make_float2(own.y, other.y), c1).x)
                       : pack(rotated(make_float2(other.x, own.x), c0).y, rotated(make_float2(other.y, own.y), c1).y);
      }
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 z = rotated(unpack(in[m]), tab[4 * c + m]);
        out[m] = pack(z.x, z.y);
      }
    }
    if (live) reinterpret_cast<uint4*>(p.q_pe + (size_t)r * kDr)[c] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <int kU>
__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const RotaryAppend p) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < p.row_ctas) {
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i < p.B * p.s) write_row(p, i, threadIdx.x & 31);
  } else {
    turn_queries<kU>(p, (blockIdx.x - p.row_ctas) * 32 * kU);
  }
}

}  // namespace

cudaError_t launch_append_rotary(RotaryAppend p, cudaStream_t s) {
  const int n = p.B * p.s;
  p.row_ctas = (n + kWarps - 1) / kWarps;
  const int64_t heads = p.q ? (int64_t)n << p.log_h : 0;
  const int u = heads <= 32 * 8 * 152 ? 1 : 4;
  const unsigned grid = (unsigned)(p.row_ctas + (heads + 32 * u - 1) / (32 * u));
  if (u == 1) return launch_pdl(append_rotary_kernel<1>, dim3(grid), dim3(kThreads), 0, s, p);
  return launch_pdl(append_rotary_kernel<4>, dim3(grid), dim3(kThreads), 0, s, p);
}

}  // namespace mla
