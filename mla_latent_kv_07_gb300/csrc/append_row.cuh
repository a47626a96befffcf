// append_row.cuh -- the cache-write step of "DeepSeek-V3.2-Exp . KV cache"
// (cache-write excerpt) for one row, as device code shared by the append
// kernels, the sparse prep kernel and the dense decode kernel (which writes
// the new row itself inside the unit that reads it).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace mla {

// Smallest power of two >= s, for s > 0 or +inf (returned unchanged).  A
// normal s with a zero fraction is already one; otherwise the next exponent.
// A subnormal s is m * 2^-149 with m in [1, 2^23): the answer is 2^ceil(log2 m)
// units of 2^-149, whose bit pattern is that single bit (2^23 units = the
// smallest normal, bit 23, comes out the same way).
__device__ __forceinline__ float pow2_at_least(float s) {
  const uint32_t u = __float_as_uint(s);
  const uint32_t e = u >> 23, m = u & 0x7fffffu;
  if (e == 0) return __uint_as_float(1u << (32 - __clz(m - 1)));
  return (m == 0 || e == 0xffu) ? s : __uint_as_float((e + 1) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}
// The e4m3 codes of fp32(x / scale) for four values.  Products with the
// reciprocal lie within a few steps of the quotients (half a step each for the
// reciprocal, the product and the quotient itself; four more if the reciprocal
// is subnormal).  Where the products moved 2^-20 (eight steps) down and up have
// the same codes, so have the quotients in between; only where a border
// between codes is that near, and where the reciprocal overflows, are the
// divisions made.
__device__ __forceinline__ uint32_t e4m3_quotients(float2 x01, float2 x23, float scale) {
  const float r = __fdiv_rn(1.0f, scale);
  const float2 rr = make_float2(r, r), dn = make_float2(1.0f - 0x1p-20f, 1.0f - 0x1p-20f),
               up = make_float2(1.0f + 0x1p-20f, 1.0f + 0x1p-20f);
  const float2 y01 = __fmul2_rn(x01, rr), y23 = __fmul2_rn(x23, rr);
  const uint32_t lo = e4m3x4(__fmul2_rn(y01, dn), __fmul2_rn(y23, dn));
  const uint32_t hi = e4m3x4(__fmul2_rn(y01, up), __fmul2_rn(y23, up));
  if (lo == hi && r < INFINITY) return lo;
  return e4m3x4(make_float2(__fdiv_rn(x01.x, scale), __fdiv_rn(x01.y, scale)),
                make_float2(__fdiv_rn(x23.x, scale), __fdiv_rn(x23.y, scale)));
}

// A latent block of 128 values, four per lane of the calling warp: the lane's
// four codes, and the block's scale.  A block whose scale is 0 has codes 0: one of
// zeros, and one whose largest value, below 2^-141, is less than half of 448
// times the smallest fp32 number (bf16 holds none so small; normalised rows may).
__device__ __forceinline__ uint32_t quantize4(float2 x01, float2 x23, int fmt, float* scale_out) {
  float amax = fmaxf(fmaxf(fabsf(x01.x), fabsf(x01.y)), fmaxf(fabsf(x23.x), fabsf(x23.y)));
  // (non-negative floats order as their bits; NaN counts as nothing unless
  // all are)
  const uint32_t bits = __reduce_max_sync(0xffffffffu, amax == amax ? __float_as_uint(amax) + 1u : 0u);
  amax = bits ? __uint_as_float(bits - 1u) : __uint_as_float(0x7fffffffu);
  float scale = __fdiv_rn(amax, 448.0f);
  if (fmt == 2 && scale > 0.0f) scale = pow2_at_least(scale);
  *scale_out = scale;
  return scale > 0.0f ? e4m3_quotients(x01, x23, scale) : 0u;
}

// Row b of the new rows into cache row `row` of slot b, by 128 threads of
// the calling CTA that form four whole warps; t in [0, 128) is the thread's
// index among them.  Warp t / 32 owns latent block t / 32 (128 values, 4 per
// lane): amax by shuffle, scale = amax / 448 (IEEE fp32 division; format 2
// rounds it up to a power of two), codes = e4m3 of x / scale with
// round-to-nearest-even and saturation.  An all-zero block stores scale 0
// and zero codes.
// (append_load and append_store are its halves, for callers with several rows
// in flight; append_row_at takes new row `b` into pool row r, wherever the
// caller's layout puts it.)
struct AppendPiece {
  uint2 kv;   // the thread's four latent values
  uint4 pe;   // t < 8: sixteen bytes of the rotary key
};
__device__ __forceinline__ AppendPiece append_load(const AppendRows& p, size_t b, int t) {
  AppendPiece x;
  x.kv = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.kv_new) + b * kDc + t * 4);
  x.pe = make_uint4(0, 0, 0, 0);
  if (t < 8)   // rotary key: 64 bf16 = 8 x 16 bytes
    x.pe = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.pe_new) + b * kDr)[t];
  return x;
}
__device__ __forceinline__ void append_store(const AppendRows& p, size_t r, int t, const AppendPiece& x) {
  const int blk = t >> 5, lane = t & 31;
  const int col = blk * kBlk + lane * 4;
  const uint2 raw = x.kv;
  if (p.fmt == 0) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.kv) + r * kDc + col) = raw;
  } else {
    const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&raw);
    const float2 x01 = __bfloat1622float2(h2[0]);
    const float2 x23 = __bfloat1622float2(h2[1]);
    float scale;
    const uint32_t packed = quantize4(x01, x23, p.fmt, &scale);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.kv) + r * kDc + col) = packed;
    if (lane == 0) p.kv_scale[r * kNblk + blk] = scale;
  }
  if (t < 8) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.pe) + r * kDr)[t] = x.pe;
}
__device__ __forceinline__ void append_row_at(const AppendRows& p, size_t b, size_t r, int t) {
  append_store(p, r, t, append_load(p, b, t));
}
__device__ __forceinline__ void append_row(const AppendRows& p, int b, int row, int t) {
  append_row_at(p, (size_t)b, (size_t)b * p.max_seq_len + row, t);
}

// The new row of sequence b of a paged call at position pos, by 128 threads
// that form four whole warps; `owner` also starts the row's weight.  Raises
// bits in *flags (shared memory) where it has to leave the row out.
__device__ __forceinline__ void append_paged_row(const AppendRows& ap, const PagedTable& pt, float* weight, int b, int pos,
                                                 int t, bool owner, uint32_t* flags) {
  const int row = pt.row(b, pos);
  if (row >= 0) {
    append_row_at(ap, b, row, t);
    if (t == 0 && owner && weight) weight[row] = 0.f;
  } else if (t == 0) {
    atomicOr(flags, kDevAppendSkipped);
  }
}

// A row is appended by a dense call only where the decode reads it: end_pos
// in [1, max_end_pos] (then row end_pos - 1 < max_seq_len).
__device__ __forceinline__ bool append_row_valid(int end, int max_end_pos) {
  return end >= 1 && end <= max_end_pos;
}

}  // namespace mla
