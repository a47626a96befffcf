// mla_api.cu -- the C ABI declared in include/mla.h: argument checks, the
// workspace carve-up and the launch sequence of each call.  Every check that
// the host can make happens before the first launch.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/mla.h"
#include "common.cuh"

namespace {

thread_local char g_last_error[256] = "";

mla_status cuda_fail(cudaError_t e, const char* where) {
  snprintf(g_last_error, sizeof(g_last_error), "%s: %s", where, cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

// Per-thread trace of the main decode kernel (see mla_trace_begin).
struct Trace {
  bool on = false;
  int cap = 0, n = 0, launches = 0;
  cudaEvent_t* ev = nullptr;  // [2 * cap]: start, stop pairs
};
thread_local Trace g_trace;

void trace_launches(int k) {
  if (g_trace.on) g_trace.launches += k;
}

bool trace_start(cudaStream_t s) {
  if (!g_trace.on || g_trace.n >= g_trace.cap) return false;
  // External records become real event nodes when the stream is being captured
  // into a graph (a plain record would only mark a dependency); outside
  // capture they behave as ordinary records.
  return cudaEventRecordWithFlags(g_trace.ev[2 * g_trace.n], s, cudaEventRecordExternal) == cudaSuccess;
}

void trace_stop(cudaStream_t s, bool started) {
  if (!started) return;
  if (cudaEventRecordWithFlags(g_trace.ev[2 * g_trace.n + 1], s, cudaEventRecordExternal) == cudaSuccess)
    ++g_trace.n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// a stride of bf16 elements that keeps 16-byte alignment
bool bf16_stride(int64_t n, int64_t least) { return n >= least && (n & 7) == 0 && n < (int64_t(1) << 40); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// SM count of the current device, cached per device.
int num_sms(int* out) {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return -1;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return -1;
    }
    cache[dev] = n;
  }
  *out = cache[dev];
  return 0;
}

bool supported_heads(int H) { return H == 16 || H == 32 || H == 64 || H == 128; }

mla_status check_cache(const mla_cache* c) {
  if (!c || !c->kv || !c->pe) return MLA_ERR_INVALID_ARG;
  if (c->fmt != MLA_KV_BF16 && c->fmt != MLA_KV_FP8_E4M3_B128 && c->fmt != MLA_KV_FP8_E4M3_B128_POW2)
    return MLA_ERR_UNSUPPORTED;
  if (c->max_batch <= 0 || c->max_seq_len <= 0) return MLA_ERR_INVALID_ARG;
  if (!aligned16(c->kv) || !aligned16(c->pe)) return MLA_ERR_INVALID_ARG;
  if (c->fmt != MLA_KV_BF16 && (!c->kv_scale || !aligned16(c->kv_scale)))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

mla::AppendRows append_rows(const mla_cache* c, const void* kv_new, const void* pe_new) {
  mla::AppendRows r{};
  r.fmt = c->fmt;
  r.max_seq_len = c->max_seq_len;
  r.kv = c->kv;
  r.kv_scale = c->kv_scale;
  r.pe = c->pe;
  r.kv_new = kv_new;
  r.pe_new = pe_new;
  return r;
}

struct DecodeArgs {
  const mla_cache* cache;
  const void* q_latent;
  const void* q_pe;
  const int32_t* end_pos;
  int32_t max_end_pos, B, H;
  float softmax_scale;
  void* out;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int32_t mtp_s;   // new tokens per sequence; B counts B / mtp_s cache slots x mtp_s
};

mla_status check_decode(const DecodeArgs& a, int K, mla::Workspace* ws) {
  mla_status st = check_cache(a.cache);
  if (st != MLA_OK) return st;
  if (!supported_heads(a.H)) return MLA_ERR_UNSUPPORTED;
  if (a.B <= 0 || a.B / a.mtp_s > a.cache->max_batch) return MLA_ERR_INVALID_ARG;
  if (a.max_end_pos <= 0 || a.max_end_pos > a.cache->max_seq_len) return MLA_ERR_OUT_OF_RANGE;
  if (!a.q_latent || !a.q_pe || !a.end_pos || !a.out) return MLA_ERR_INVALID_ARG;
  if (!aligned16(a.q_latent) || !aligned16(a.q_pe) || !aligned16(a.out) || !aligned4(a.end_pos))
    return MLA_ERR_INVALID_ARG;
  if (a.lse && !aligned4(a.lse)) return MLA_ERR_INVALID_ARG;
  if (!(a.softmax_scale == a.softmax_scale)) return MLA_ERR_INVALID_ARG;  // NaN
  int sms = 0;
  if (num_sms(&sms) != 0) return MLA_ERR_UNSUPPORTED;
  mla::Workspace need = mla::carve_workspace(nullptr, a.B, a.H, K, sms);
  if (!a.workspace || !aligned16(a.workspace) || a.ws_bytes < need.bytes) return MLA_ERR_WORKSPACE;
  *ws = mla::carve_workspace(a.workspace, a.B, a.H, K, sms);
  return MLA_OK;
}

mla::DecodeParams make_params(const DecodeArgs& a, const mla::Workspace& ws, int K) {
  mla::DecodeParams p{};
  p.fmt = mla::decode_fmt(a.cache->fmt);
  p.max_seq_len = a.cache->max_seq_len;
  p.kv = a.cache->kv;
  p.kv_scale = a.cache->kv_scale;
  p.pe = a.cache->pe;
  p.q_latent = a.q_latent;
  p.q_pe = a.q_pe;
  p.B = a.B;
  p.H = a.H;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.out = a.out;
  p.lse = a.lse;
  p.ws = ws;
  p.K = K;
  p.mtp_s = a.mtp_s;
  p.spin_limit = 0;
  p.withhold_tile = -1;
  return p;
}

// Decode path: the tensor-memory kernel for H = 128 unless MLA_DECODE_PATH=mma
// (read once per process) selects the warp-MMA kernel.
bool use_tc_path(int H) {
  static int forced = -1;
  static std::once_flag once;
  std::call_once(once, [] {
    const char* v = getenv("MLA_DECODE_PATH");
    forced = (v && strcmp(v, "mma") == 0) ? 0 : 1;
  });
  return forced && mla::decode_tc_supported(H);
}

// schedule -> decode -> combine, after the lengths are known on the device.
// ap (dense, one token per slot): also write row end_pos[b] - 1 of every
// sequence from ap.kv_new / ap.pe_new -- inside the tensor-memory decode
// kernel, or by a kernel of its own ahead of the warp-MMA path.
mla_status run_decode(const DecodeArgs& a, const mla::Workspace& ws, int K, cudaStream_t s,
                      long long spin_limit = 0, int withhold_tile = -1,
                      const mla::AppendRows* ap = nullptr) {
  int sms = 0;
  num_sms(&sms);
  const bool tc = use_tc_path(a.H);
  cudaError_t e;
  if (ap && !tc) {
    e = mla::launch_append_end(*ap, a.end_pos, a.max_end_pos, a.B, s);
    if (e != cudaSuccess) return cuda_fail(e, "append");
    trace_launches(1);
  }
  const int target =
      tc ? mla::decode_tc_units(mla::decode_fmt(a.cache->fmt), K > 0, sms) : mla::target_units_mma(a.H, sms);
  const int granule = tc ? mla::decode_tc_granule(mla::decode_fmt(a.cache->fmt), K > 0) : mla::decode_mma_granule();
  // dense bf16 and sparse calls of up to kWarpScheduleMaxB sequences on the
  // tensor-memory kernel: every CTA pair works out its own unit (a sparse
  // call from the gather counts the prep kernel wrote), so no schedule kernel
  // sits between the call's start (or its prep) and the first loads.  (The
  // dense FP8 variant runs at its register limit, where the added code cost
  // more than it saved; long calls -- prefill chunks -- keep the schedule
  // kernel.)
  const bool fused_schedule =
      tc && a.B <= mla::kWarpScheduleMaxB && (K > 0 || mla::decode_fmt(a.cache->fmt) == 0);
  if (!fused_schedule) {
    e = mla::launch_schedule(K ? nullptr : a.end_pos, a.max_end_pos, ws, a.B, target, granule, tc, a.mtp_s,
                             ap != nullptr, s);
    if (e != cudaSuccess) return cuda_fail(e, "schedule");
    trace_launches(1);
  }
  const bool traced = trace_start(s);
  mla::DecodeParams p = make_params(a, ws, K);
  p.spin_limit = spin_limit;
  p.withhold_tile = withhold_tile;
  if (ap && tc) p.ap = *ap;
  if (fused_schedule && K == 0)
    p.sched = mla::DenseSchedule{a.end_pos, a.max_end_pos, a.B, target, granule, a.mtp_s, 1, ap != nullptr ? 1 : 0};
  else if (fused_schedule)
    p.sched = mla::DenseSchedule{nullptr, a.max_end_pos, a.B, target, granule, 1, 1, 0, ws.lengths, ws.seq_flags};
  e = tc ? mla::launch_decode_tc(p, s) : mla::launch_decode_mma(p, s);
  trace_stop(s, traced);
  if (e != cudaSuccess) return cuda_fail(e, "decode");
  e = mla::launch_combine(ws, a.B, a.H, a.out, a.lse, s);
  if (e != cudaSuccess) return cuda_fail(e, "combine");
  trace_launches(2);
  return MLA_OK;
}

mla_status check_paged(const mla_paged_cache* c, const int32_t* table, int32_t max_pages) {
  if (!c || !c->kv || !c->pe || !table) return MLA_ERR_INVALID_ARG;
  if (c->fmt != MLA_KV_BF16 && c->fmt != MLA_KV_FP8_E4M3_B128 && c->fmt != MLA_KV_FP8_E4M3_B128_POW2)
    return MLA_ERR_UNSUPPORTED;
  if (c->num_pages <= 0 || c->page_size <= 0 || max_pages <= 0) return MLA_ERR_INVALID_ARG;
  if (c->page_size % 16 || c->page_size > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  if (!aligned16(c->kv) || !aligned16(c->pe) || !aligned4(c->weight) || !aligned4(table)) return MLA_ERR_INVALID_ARG;
  if (c->fmt != MLA_KV_BF16 && (!c->kv_scale || !aligned16(c->kv_scale))) return MLA_ERR_INVALID_ARG;
  if ((int64_t)c->num_pages * c->page_size > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;   // row numbers are int32
  return MLA_OK;
}

// the bound on a paged call's lengths: what the table can name, and 2^30 (the
// kernels look up positions a few tiles past a sequence's end in 32 bits)
mla_status check_paged_end(const mla_paged_cache* c, int32_t max_pages, int32_t max_end_pos) {
  if (max_end_pos <= 0 || max_end_pos > mla::kMaxPagedEnd) return MLA_ERR_OUT_OF_RANGE;
  return max_end_pos > (int64_t)max_pages * c->page_size ? MLA_ERR_OUT_OF_RANGE : MLA_OK;
}

mla::PagedTable paged_table(const mla_paged_cache* c, const int32_t* table, int32_t max_pages) {
  return mla::make_paged_table(table, max_pages, c->page_size, c->num_pages);
}

mla::PagedAppend paged_append(const mla_paged_cache* c, const int32_t* table, int32_t max_pages,
                              const void* kv_new, const void* pe_new, const int32_t* end_pos, int32_t B,
                              int32_t s, uint32_t* status) {
  mla::PagedAppend p{};
  p.rows.fmt = c->fmt;
  p.rows.kv = c->kv;
  p.rows.kv_scale = c->kv_scale;
  p.rows.pe = c->pe;
  p.rows.kv_new = kv_new;
  p.rows.pe_new = pe_new;
  p.pt = paged_table(c, table, max_pages);
  p.weight = c->weight;
  p.end_pos = end_pos;
  p.B = B;
  p.s = s;
  p.max_pos = (long long)max_pages * c->page_size;
  p.status = status;
  return p;
}

// mla_paged_decode; withhold_tile >= 0: the self-test of its bounded waits
mla_status run_paged_decode(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                            const void* q_latent, const void* q_pe, const int32_t* end_pos,
                            int32_t max_end_pos, int32_t B, int32_t H, float softmax_scale,
                            const void* kv_new, const void* pe_new, void* out, float* lse,
                            void* workspace, size_t ws_bytes, void* stream, int withhold_tile) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!supported_heads(H)) return MLA_ERR_UNSUPPORTED;
  if (B <= 0 || B > mla::kMaxPagedB) return MLA_ERR_INVALID_ARG;
  if ((st = check_paged_end(cache, max_pages, max_end_pos)) != MLA_OK) return st;
  if (!q_latent || !q_pe || !end_pos || !out) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_latent) || !aligned16(q_pe) || !aligned16(out) || !aligned4(end_pos) || !aligned4(lse))
    return MLA_ERR_INVALID_ARG;
  if ((kv_new == nullptr) != (pe_new == nullptr) || !aligned16(kv_new) || !aligned16(pe_new))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale)) return MLA_ERR_INVALID_ARG;  // NaN
  int sms = 0;
  if (num_sms(&sms) != 0) return MLA_ERR_UNSUPPORTED;
  mla::Workspace ws = mla::carve_paged(workspace, B, H, sms);
  if (!workspace || !aligned16(workspace) || ws_bytes < ws.bytes) return MLA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int fmt = mla::decode_fmt(cache->fmt);
  // 128 heads: the CTA-pair kernel (decode_tc.cu); fewer: one CTA per unit
  // (paged_decode.cu)
  const bool pair = H == 128;
  if (pair && !mla::decode_tc_supported(H)) return MLA_ERR_UNSUPPORTED;
  const int target = pair ? mla::decode_tc_paged_units(fmt, sms) : sms;
  const int granule = pair ? mla::decode_tc_granule(fmt, false) : mla::kPagedGranule;
  mla::DecodeParams p{};
  p.fmt = fmt;
  p.max_seq_len = cache->page_size;
  p.kv = cache->kv;
  p.kv_scale = cache->kv_scale;
  p.pe = cache->pe;
  p.q_latent = q_latent;
  p.q_pe = q_pe;
  p.B = B;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.ws = ws;
  p.mtp_s = 1;
  p.withhold_tile = withhold_tile;
  p.spin_limit = withhold_tile < 0 ? 0 : 1LL << 16;   // (the pair kernel's waits)
  p.pt = paged_table(cache, table, max_pages);
  cudaError_t e;
  if (kv_new) {   // written by the unit that reads it
    p.ap = paged_append(cache, table, max_pages, kv_new, pe_new, end_pos, B, 1, nullptr).rows;
    p.ap_weight = cache->weight;
  }
  // up to kWarpScheduleMaxB sequences: every CTA works out its own unit (the
  // pair kernel's FP8 variant has no registers to spare for it: 4 x 131072
  // positions 208 us with a schedule kernel, 213 without)
  const bool fused_schedule = B <= mla::kWarpScheduleMaxB && (!pair || fmt == 0);
  // Short sequences are not split: what a split saves the combine kernel costs
  // again.  At 256 positions, split and whole: one sequence of 16 heads 9.5 and
  // 9.0 us, 8 of 64 14.4 and 12.3, 64 of 16 (FP8) 18.1 and 12.9, one of 64 (FP8)
  // 13.1 and 16.0; at 512: 9.3 and 13.0, 15.1 and 17.6, 21.0 and 19.7, 13.1 and
  // 23.5.  The length alone decides, which costs a single sequence of 64 heads in
  // FP8 3 us.
  const bool whole = !pair && fused_schedule && max_end_pos <= mla::kPagedWhole;
  const mla::DenseSchedule sched{end_pos, max_end_pos, B, target, granule, 1, 1, kv_new != nullptr ? 1 : 0};
  if (fused_schedule) {
    p.sched = sched;
  } else {
    e = B <= mla::kWarpScheduleMaxB
            ? mla::launch_paged_schedule(ws, sched, s)
            : mla::launch_schedule(end_pos, max_end_pos, ws, B, target, granule, true, 1, kv_new != nullptr, s);
    if (e != cudaSuccess) return cuda_fail(e, "schedule");
    trace_launches(1);
  }
  const bool traced = trace_start(s);
  e = pair ? mla::launch_decode_tc(p, s) : mla::launch_paged_decode(p, whole, s);
  trace_stop(s, traced);
  if (e != cudaSuccess) return cuda_fail(e, "paged_decode");
  trace_launches(1);
  if (whole) return MLA_OK;
  e = mla::launch_paged_combine(ws, B, H, out, lse, pair ? 2 : 1, s);
  if (e != cudaSuccess) return cuda_fail(e, "combine");
  trace_launches(1);
  return MLA_OK;
}

// Workspace of a windowed call of n tokens: as a paged decode's while tokens are
// split, else the status word and no more than the kernels' maps want.
mla::Workspace carve_window(void* base, int n, int H, int sms) {
  return n <= mla::kWarpScheduleMaxB ? mla::carve_paged(base, n, H, sms) : mla::carve_units(base, 1, H, 0, 1, true);
}
// its size (128 heads: or as twice the tokens of 64)
size_t window_bytes(int n, int H, int sms) {
  const size_t bytes = carve_window(nullptr, n, H, sms).bytes;
  return H == 128 ? std::max(bytes, carve_window(nullptr, 2 * n, 64, sms).bytes) : bytes;
}

// withhold_tile >= 0: the self-test of the kernels' bounded waits
mla_status run_paged_window(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages, const void* q_latent,
                            const void* q_pe, const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t s_new,
                            int32_t H, float softmax_scale, int32_t window, int32_t sinks, void* out, float* lse,
                            void* workspace, size_t ws_bytes, cudaStream_t s, int withhold_tile) {
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!supported_heads(H)) return MLA_ERR_UNSUPPORTED;
  if (B <= 0 || B > mla::kMaxPagedB || s_new < 1 || s_new > mla::kMaxMtp || B > (1 << 22) / s_new) return MLA_ERR_INVALID_ARG;
  if ((st = check_paged_end(cache, max_pages, max_end_pos)) != MLA_OK) return st;
  if (window < 1 || sinks < 0) return MLA_ERR_INVALID_ARG;
  if (!q_latent || !q_pe || !end_pos || !out) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_latent) || !aligned16(q_pe) || !aligned16(out) || !aligned4(end_pos) || !aligned4(lse))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale)) return MLA_ERR_INVALID_ARG;  // NaN
  int sms = 0;
  if (num_sms(&sms) != 0) return MLA_ERR_UNSUPPORTED;
  const int tokens = B * s_new;
  if (!workspace || !aligned16(workspace) || ws_bytes < window_bytes(tokens, H, sms)) return MLA_ERR_WORKSPACE;
  const int fmt = mla::decode_fmt(cache->fmt);
  if (H == 128 && !mla::decode_tc_supported(H)) return MLA_ERR_UNSUPPORTED;
  // numbers past what a sequence can have say no more than that
  window = window < max_end_pos ? window : max_end_pos;
  sinks = sinks < max_end_pos ? sinks : max_end_pos;
  const int64_t longest = (int64_t)window + sinks + 30, places = longest < max_end_pos ? longest : max_end_pos;
  const bool many = tokens > mla::kWarpScheduleMaxB, small = places <= mla::kPagedWhole;
  // By columns (paged_chunk.cu), where its units fill three quarters of the SMs, or
  // there are more tokens than SMs and than a warp schedules.  Otherwise and so
  // (us): 128 tokens of two sequences of 5000, windows of 512 and 4096, bf16, 32 heads
  // (64 units) 18.2 and 21.4, 100 and 97; 64 heads (128 units) 23.1 and 22.9, 119 and 97;
  // FP8, 128 heads (256), 58.0 and 47.3, 248 and 234.  One token of 64 sequences of
  // 4000 to 5000, 128 heads, windows of 226 and 4096: 16.7 and 16.8, 128 and 107 (FP8
  // 21.9 and 18.7, 135 and 128); of 112, 64 heads, 1024 and 4096: 40.1 and 40.9, 120
  // and 113 (FP8 48.8 and 45.3, 139 and 130), but 226 18.0 and 19.3, which
  // is why such short ones of up to 64 heads are left out.  FP8 from half the SMs on
  // too, for runs of up to 34 tiles (100 sequences of 64 heads, windows of 1024,
  // 2048 and 4096: 48.3 and 44.5, 79.2 and 73.2, 128 and 130; 52 of 128, 1024 and 2048:
  // 43.9 and 43.2, 80.1 and 71.8; bf16, 100 of 64 heads, 1024: 38.7 and 39.6), and for
  // short runs of 128 heads, where a pair takes longer than a CTA (32 tokens, 98 and 226:
  // 20.6 and 14.5, 22.2 and 18.7; 16, 98: 16.3 and 14.6; 8: 14.3 and 14.7).
  const int units = mla::chunk_units(B, s_new, H);
  const bool fills = units >= std::min(sms - sms / 4, mla::kWarpScheduleMaxB + 1);   // (128 heads: a warp schedules what is left)
  const bool half = 2 * units > sms && !small && places <= 34 * 64;
  const bool chunk = (int64_t)s_new * H >= 64 && (many    ? fills || tokens > sms
                                                  : fills ? s_new > 1 || H == 128 || !small
                                                          : fmt != 0 && (half || (H == 128 && small && tokens >= 16)));
  // Else 128 heads over bf16 rows are two CTAs' of 64 heads, each with its own run: a
  // row comes from memory once and from L2 once, and no scores go from CTA to CTA.
  // As pairs and so (us): one token, windows of 512 and 16000, 12.6 and 11.4, 24.6 and
  // 21.7; 8, 1024, 17.7 and 17.0; 32, 512 and 4096, 26.6 and 24.0, 67.3 and 63.3; 30 of 6
  // sequences, 512, 24.3 and 21.8.  FP8 rows would be converted twice (32, 4096: 68.9 and 78.4).
  const bool halves = H == 128 && fmt == 0 && !chunk, pair = H == 128 && !halves;
  const int n = halves ? 2 * tokens : tokens;   // (halves: at most what a warp schedules, else `fills` holds)
  if (halves) H = 64;
  const int target = pair ? mla::decode_tc_window_units(sms) : sms;
  const int granule = pair ? mla::decode_tc_granule(fmt, false) : mla::kPagedGranule;
  mla::Workspace ws = carve_window(workspace, n, H, sms);
  mla::DecodeParams p{};
  p.fmt = fmt;
  p.max_seq_len = cache->page_size;
  p.kv = cache->kv;
  p.kv_scale = cache->kv_scale;
  p.pe = cache->pe;
  p.q_latent = q_latent;
  p.q_pe = q_pe;
  p.B = n;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.ws = ws;
  p.mtp_s = s_new;
  p.withhold_tile = withhold_tile;
  p.spin_limit = withhold_tile < 0 ? 0 : 1LL << 16;   // (the pair kernel's waits)
  p.pt = paged_table(cache, table, max_pages);
  p.sched = mla::DenseSchedule{end_pos, max_end_pos, n, target, granule, s_new, 1, 0};
  p.sched.window = window;
  p.sched.sinks = sinks;
  p.sched.halves = halves ? 1 : 0;
  // A CTA takes a token whole: more tokens than a warp schedules, or a few with runs
  // of two tiles, which saves the combine (8 of 64 heads, window 98: 9.0 us, 9.6
  // with one; 128 tokens 17.6 and 13.1, since one warp looks at all their pages).
  const bool whole = !chunk && (many || (!pair && n <= 32 && places <= 128));
  // Else the tokens' runs are split over the GPU in as many equal parts a token as
  // there are places for, which a CTA finds from its own token's length, up to 34
  // tiles a part in bf16 and 20 in FP8 (balanced and so, us, bf16 and FP8, sequences of
  // 1k to 16k: 100 tokens of 16 heads, windows of 1024 and 2048, 43.7 and 30.8, 59.8 and
  // 50.3, FP8 48.0 and 40.5, 66.4 and 70.3; 64 of 64 heads, 2048 and 4096, 49.9 and 46.5, 71.8
  // and 70.9, FP8 54.8 and 52.7, 80.6 and 85.3).  Longer ones are balanced, which
  // evens out sequences that are shorter than the window.  A short run is not
  // split where the partial outputs, all tokens' of them, cost more than it takes
  // (split and not: 64 tokens of 64 heads, windows of 98, 350 and 720: 18.8 and 11.3, 23.0
  // and 17.7, 27.8 and 27.9; 32, 226 and 480: 15.9 and 13.7, 17.9 and 19.8; 48 of 16
  // heads, 162 and 350: 11.5 and 10.9, 12.4 and 13.2).
  if (!chunk && !whole && n <= target) {
    const int per = !pair && places <= (int64_t)n * (4 + H / 16) ? 1 : target / n;
    const int64_t share = ((places + per - 1) / per + granule - 1) / granule * granule;
    if (share <= (fmt == 0 ? 34 : 20) * 64) {
      p.sched.chunk = (int)share;
      p.sched.per_token = (int)((places + share - 1) / share);
    }
  }
  cudaError_t e;
  if (chunk || many) {
    p.status_cleared = true;
    e = cudaMemsetAsync(ws.status, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "status");
  } else if (pair && p.sched.chunk == 0) {   // (its kernel has no registers to spare for the schedule)
    e = mla::launch_paged_schedule(ws, p.sched, s);
    if (e != cudaSuccess) return cuda_fail(e, "schedule");
    trace_launches(1);
  }
  const bool traced = trace_start(s);
  e = chunk  ? mla::launch_paged_chunk(p, sms, s)
      : pair ? mla::launch_decode_tc(p, s)
             : mla::launch_paged_decode(p, whole, s);
  trace_stop(s, traced);
  if (e != cudaSuccess) return cuda_fail(e, "paged_decode_window");
  trace_launches(1);
  if (chunk || whole) return MLA_OK;
  e = mla::launch_paged_combine(ws, n, H, out, lse, pair ? 2 : 1, s);
  if (e != cudaSuccess) return cuda_fail(e, "combine");
  trace_launches(1);
  return MLA_OK;
}

// mla_paged_weights; withhold_tile >= 0: the self-test of its bounded waits
mla_status run_paged_weights(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                             const void* q_latent, const void* q_pe, const float* lse,
                             const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                             float softmax_scale, uint32_t* status, void* stream, int withhold_tile) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!supported_heads(H)) return MLA_ERR_UNSUPPORTED;
  if (B <= 0 || B > mla::kMaxPagedB) return MLA_ERR_INVALID_ARG;
  if ((st = check_paged_end(cache, max_pages, max_end_pos)) != MLA_OK) return st;
  if (!q_latent || !q_pe || !lse || !end_pos || !cache->weight) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_latent) || !aligned16(q_pe) || !aligned4(lse) || !aligned4(end_pos) || !aligned4(status))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale)) return MLA_ERR_INVALID_ARG;  // NaN
  int sms = 0;
  if (num_sms(&sms) != 0) return MLA_ERR_UNSUPPORTED;
  mla::WeightsParams p{};
  p.fmt = mla::decode_fmt(cache->fmt);
  p.kv = cache->kv;
  p.kv_scale = cache->kv_scale;
  p.pe = cache->pe;
  p.weight = cache->weight;
  p.pt = paged_table(cache, table, max_pages);
  p.q_latent = q_latent;
  p.q_pe = q_pe;
  p.lse = lse;
  p.end_pos = end_pos;
  p.max_end_pos = max_end_pos;
  p.B = B;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.status = status;
  p.withhold_tile = withhold_tile;
  cudaError_t e = mla::launch_paged_weights(p, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged_weights");
  trace_launches(1);
  return MLA_OK;
}

mla_status check_absorb(const void* x, const void* wkv_b, int32_t B, int32_t H, const void* y,
                        const uint32_t* status) {
  if (!x || !wkv_b || !y || !aligned16(x) || !aligned16(wkv_b) || !aligned16(y)) return MLA_ERR_INVALID_ARG;
  if (status && !aligned4(status)) return MLA_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || B > (1 << 22) || H > (1 << 16)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}
}  // namespace

extern "C" {

mla_status mla_cache_append(const mla_cache* cache, const void* kv_new, const void* pe_new,
                            const int32_t* start_pos, int32_t B, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_cache(cache);
  if (st != MLA_OK) return st;
  if (!kv_new || !pe_new || !start_pos) return MLA_ERR_INVALID_ARG;
  if (!aligned16(kv_new) || !aligned16(pe_new)) return MLA_ERR_INVALID_ARG;
  if (B <= 0 || B > cache->max_batch || B > mla::kMaxAppendB) return MLA_ERR_INVALID_ARG;
  for (int b = 0; b < B; ++b)
    if (start_pos[b] < 0 || start_pos[b] >= cache->max_seq_len) return MLA_ERR_OUT_OF_RANGE;
  mla::AppendParams p{};
  p.rows = append_rows(cache, kv_new, pe_new);
  p.B = B;
  memcpy(p.pos, start_pos, sizeof(int32_t) * (size_t)B);
  cudaError_t e = mla::launch_append_host_pos(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "append");
  trace_launches(1);
  return MLA_OK;
}

size_t mla_workspace_size(int32_t B, int32_t H, int32_t max_end_pos, int32_t topk) {
  (void)max_end_pos;
  if (B <= 0 || !supported_heads(H) || topk < 0 || topk > mla::kMaxTopK) return 0;
  int sms = 0;
  if (num_sms(&sms) != 0) return 0;
  return mla::carve_workspace(nullptr, B, H, topk, sms).bytes;
}

mla_status mla_decode(const mla_cache* cache, const void* q_latent, const void* q_pe,
                      const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                      float softmax_scale, void* out, float* lse, void* workspace,
                      size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, out, lse,
               workspace, ws_bytes, 1};
  mla::Workspace ws;
  mla_status st = check_decode(a, 0, &ws);
  if (st != MLA_OK) return st;
  // the call's first kernel (the schedule kernel, or a decode kernel that
  // computes its own schedule) writes the status word afresh
  return run_decode(a, ws, 0, static_cast<cudaStream_t>(stream));
}

mla_status mla_decode_append(const mla_cache* cache, const void* kv_new, const void* pe_new,
                             const void* q_latent, const void* q_pe, const int32_t* end_pos,
                             int32_t max_end_pos, int32_t B, int32_t H, float softmax_scale, void* out,
                             float* lse, void* workspace, size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  if (!kv_new || !pe_new || !aligned16(kv_new) || !aligned16(pe_new)) return MLA_ERR_INVALID_ARG;
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, out, lse,
               workspace, ws_bytes, 1};
  mla::Workspace ws;
  mla_status st = check_decode(a, 0, &ws);
  if (st != MLA_OK) return st;
  const mla::AppendRows ap = append_rows(cache, kv_new, pe_new);
  return run_decode(a, ws, 0, static_cast<cudaStream_t>(stream), 0, -1, &ap);
}

}  // extern "C"

namespace mla {

// The dense decode of mla_decode with a scratch region supplied by the library
// itself (mla_noalloc.cu) instead of a caller workspace: the same argument
// checks (a scratch smaller than this B and H need -> MLA_ERR_WORKSPACE), the
// same kernels and launch sequence, the same error reporting.
mla_status decode_in_scratch(const mla_cache* cache, const void* q_latent, const void* q_pe,
                             const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                             float softmax_scale, void* out, float* lse, void* scratch,
                             size_t scratch_bytes, void* stream) {
  g_last_error[0] = 0;
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, out, lse,
               scratch, scratch_bytes, 1};
  mla::Workspace ws;
  mla_status st = check_decode(a, 0, &ws);
  if (st != MLA_OK) return st;
  return run_decode(a, ws, 0, static_cast<cudaStream_t>(stream));
}

}  // namespace mla

extern "C" {

mla_status mla_topk_select(const float* scores, const int32_t* end_pos, int32_t B, int32_t max_end_pos,
                           int32_t K, int32_t* topk_idx, void* stream) {
  g_last_error[0] = 0;
  if (!scores || !end_pos || !topk_idx || !aligned4(scores) || !aligned4(end_pos) || !aligned4(topk_idx))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || max_end_pos < 1 || K < 1 || K > mla::kMaxTopK) return MLA_ERR_INVALID_ARG;
  cudaError_t e = mla::launch_topk_select(scores, end_pos, B, max_end_pos, K, topk_idx,
                                          static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "topk_select");
  trace_launches(1);
  return MLA_OK;
}

mla_status mla_selftest_decode_timeout(const mla_cache* cache, const void* q_latent, const void* q_pe,
                                       const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                                       float softmax_scale, void* out, float* lse, void* workspace,
                                       size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, out, lse,
               workspace, ws_bytes, 1};
  mla::Workspace ws;
  mla_status st = check_decode(a, 0, &ws);
  if (st != MLA_OK) return st;
  if (!use_tc_path(H)) return MLA_ERR_UNSUPPORTED;
  // the first unit's first tile is never loaded; every wait gives up after
  // 2^16 polls (milliseconds)
  return run_decode(a, ws, 0, static_cast<cudaStream_t>(stream), 1LL << 16, 0);
}

mla_status mla_decode_mtp(const mla_cache* cache, const void* q_latent, const void* q_pe,
                          const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t s,
                          int32_t H, float softmax_scale, void* out, float* lse, void* workspace,
                          size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  if (s < 1 || s > mla::kMaxMtp || B <= 0 || B > (1 << 30) / s) return MLA_ERR_INVALID_ARG;
  // B * s sequences; sequence b * s + j is token j of cache slot b
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B * s, H, softmax_scale, out, lse,
               workspace, ws_bytes, s};
  mla::Workspace ws;
  mla_status st = check_decode(a, 0, &ws);
  if (st != MLA_OK) return st;
  return run_decode(a, ws, 0, static_cast<cudaStream_t>(stream));
}

mla_status mla_decode_sparse(const mla_cache* cache, const void* q_latent, const void* q_pe,
                             const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                             float softmax_scale, const int32_t* topk_idx, int32_t K,
                             const void* kv_new, const void* pe_new, void* out, float* lse,
                             int32_t* gidx_out, int32_t* gcount_out, void* workspace,
                             size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  if (!topk_idx || K <= 0 || K > mla::kMaxTopK || !aligned4(topk_idx)) return MLA_ERR_INVALID_ARG;
  if (cache && B > 0 && (int64_t)B * cache->max_seq_len > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
  if ((kv_new == nullptr) != (pe_new == nullptr)) return MLA_ERR_INVALID_ARG;
  if (kv_new && (!aligned16(kv_new) || !aligned16(pe_new) || B > mla::kMaxAppendB))
    return MLA_ERR_INVALID_ARG;
  if ((gidx_out && !aligned4(gidx_out)) || (gcount_out && !aligned4(gcount_out)))
    return MLA_ERR_INVALID_ARG;
  DecodeArgs a{cache, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, out, lse,
               workspace, ws_bytes, 1};
  mla::Workspace ws;
  mla_status st = check_decode(a, K, &ws);
  if (st != MLA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the prep kernel also appends the new rows (kv_new may be NULL); the
  // schedule after it writes the status word, so no memset precedes them
  cudaError_t e = mla::launch_sparse_prep(topk_idx, K, end_pos, max_end_pos, ws, B, gidx_out,
                                          gcount_out, append_rows(cache, kv_new, pe_new), s);
  if (e != cudaSuccess) return cuda_fail(e, "sparse_prep");
  trace_launches(1);
  return run_decode(a, ws, K, s);
}

mla_status mla_workspace_status(const void* workspace, uint32_t* flags, void* stream) {
  if (!workspace || !flags) return MLA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(flags, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "status");
}

mla_status mla_absorb_q(const void* q_nope, const void* wkv_b, int32_t B, int32_t H, void* q_latent,
                        uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_absorb(q_nope, wkv_b, B, H, q_latent, status);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_absorb_q(q_nope, wkv_b, B, H, q_latent, status, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "absorb_q");
  trace_launches(1);
  return MLA_OK;
}

mla_status mla_project_out(const void* x, const void* wkv_b, int32_t B, int32_t H, void* o,
                           uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_absorb(x, wkv_b, B, H, o, status);
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_project_out(x, wkv_b, B, H, o, status, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "project_out");
  trace_launches(1);
  return MLA_OK;
}

mla_status mla_read_ceiling(const void* buf, size_t bytes, uint32_t* sink, void* stream) {
  g_last_error[0] = 0;
  if (!buf || !sink || bytes == 0 || (bytes & 15u) || !aligned16(buf) || !aligned4(sink))
    return MLA_ERR_INVALID_ARG;
  int sms = 0;
  if (num_sms(&sms) != 0) return MLA_ERR_UNSUPPORTED;
  cudaError_t e = mla::launch_read_ceiling(buf, bytes, sink, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "read_ceiling");
  trace_launches(1);
  return MLA_OK;
}

mla_status mla_paged_append(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                            const void* kv_new, const void* pe_new, const int32_t* end_pos, int32_t B,
                            int32_t s, uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!kv_new || !pe_new || !end_pos || !aligned16(kv_new) || !aligned16(pe_new) || !aligned4(end_pos))
    return MLA_ERR_INVALID_ARG;
  if (B <= 0 || s <= 0 || s > (1 << 30) / B || !aligned4(status)) return MLA_ERR_INVALID_ARG;
  cudaError_t e = mla::launch_paged_append(
      paged_append(cache, table, max_pages, kv_new, pe_new, end_pos, B, s, status), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged_append");
  trace_launches(1);
  return MLA_OK;
}

size_t mla_paged_workspace_size(int32_t B, int32_t H) {
  int sms = 0;
  if (B <= 0 || B > mla::kMaxPagedB || !supported_heads(H) || num_sms(&sms) != 0) return 0;
  return mla::carve_paged(nullptr, B, H, sms).bytes;
}

mla_status mla_paged_decode(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                            const void* q_latent, const void* q_pe, const int32_t* end_pos,
                            int32_t max_end_pos, int32_t B, int32_t H, float softmax_scale,
                            const void* kv_new, const void* pe_new, void* out, float* lse,
                            void* workspace, size_t ws_bytes, void* stream) {
  return run_paged_decode(cache, table, max_pages, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, kv_new,
                          pe_new, out, lse, workspace, ws_bytes, stream, -1);
}

mla_status mla_paged_weights(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                             const void* q_latent, const void* q_pe, const float* lse,
                             const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                             float softmax_scale, uint32_t* status, void* stream) {
  return run_paged_weights(cache, table, max_pages, q_latent, q_pe, lse, end_pos, max_end_pos, B, H, softmax_scale,
                           status, stream, -1);
}

mla_status mla_selftest_paged_decode_timeout(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                                             const void* q_latent, const void* q_pe, const int32_t* end_pos,
                                             int32_t max_end_pos, int32_t B, int32_t H, float softmax_scale,
                                             void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return run_paged_decode(cache, table, max_pages, q_latent, q_pe, end_pos, max_end_pos, B, H, softmax_scale, nullptr,
                          nullptr, out, lse, workspace, ws_bytes, stream, 0);
}

mla_status mla_selftest_paged_weights_timeout(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                                              const void* q_latent, const void* q_pe, const float* lse,
                                              const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t H,
                                              float softmax_scale, uint32_t* status, void* stream) {
  return run_paged_weights(cache, table, max_pages, q_latent, q_pe, lse, end_pos, max_end_pos, B, H, softmax_scale,
                           status, stream, 0);
}

mla_status mla_paged_evict(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                           const int32_t* end_pos, int32_t max_end_pos, int32_t B, int32_t keep,
                           int32_t sinks, int32_t recent, const int32_t* new_table,
                           int32_t new_max_pages, int32_t* kept, int32_t* new_end_pos,
                           uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (B <= 0 || B > mla::kMaxPagedB) return MLA_ERR_INVALID_ARG;
  if ((st = check_paged_end(cache, max_pages, max_end_pos)) != MLA_OK) return st;
  if (!end_pos || !new_table || !kept || !new_end_pos || !cache->weight || new_max_pages <= 0)
    return MLA_ERR_INVALID_ARG;
  if (!aligned4(end_pos) || !aligned4(new_table) || !aligned4(kept) || !aligned4(new_end_pos) || !aligned4(status))
    return MLA_ERR_INVALID_ARG;
  if (keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep) return MLA_ERR_INVALID_ARG;
  if (keep > mla::kMaxPagedEnd || keep > (int64_t)new_max_pages * cache->page_size) return MLA_ERR_OUT_OF_RANGE;
  if (new_table == table) return MLA_ERR_INVALID_ARG;   // rows would be overwritten before they are read
  mla::EvictParams p{};
  p.fmt = mla::decode_fmt(cache->fmt);
  p.kv = cache->kv;
  p.kv_scale = cache->kv_scale;
  p.pe = cache->pe;
  p.weight = cache->weight;
  p.pt = paged_table(cache, table, max_pages);
  p.to = paged_table(cache, new_table, new_max_pages);
  p.end_pos = end_pos;
  p.max_end_pos = max_end_pos;
  p.B = B;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.kept = kept;
  p.new_end = new_end_pos;
  p.status = status;
  cudaError_t e = mla::launch_paged_evict(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged_evict");
  trace_launches(2);
  return MLA_OK;
}

mla_status mla_rotary_turns(const double* freq, int32_t n, uint64_t* turns) {
  g_last_error[0] = 0;
  if (!freq || !turns || n < 1) return MLA_ERR_INVALID_ARG;
  // 1 / (2 pi) in two parts: freq / (2 pi) = p + e, p the rounded product with the
  // first, e what the rounding left and the product with the second
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(freq[i]);   // (a negative one's turns are the negative, modulo 2^64)
    if (!(f <= 1e6)) return MLA_ERR_INVALID_ARG;
    const double p = f * hi, e = std::fma(f, hi, -p) + f * lo;
    const double part = p - std::floor(p);   // in [0, 1), exact
    // 2^64 * part in two halves of 32 bits
    const double up = std::floor(part * 4294967296.0), low = part * 4294967296.0 - up;
    const uint64_t whole = ((uint64_t)up << 32) + (uint64_t)(low * 4294967296.0);
    const uint64_t turn = whole + (uint64_t)(int64_t)std::llrint(e * 18446744073709551616.0);
    turns[i] = freq[i] < 0.0 ? 0 - turn : turn;
  }
  return MLA_OK;
}

mla_status mla_paged_append_rotary(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                                   const void* kv_a, int64_t kv_stride_b, int64_t kv_stride_s,
                                   const void* norm_weight, int32_t norm_f32, float eps, const mla_rotary* rotary,
                                   const int32_t* pos, const int32_t* end_pos, int32_t B, int32_t s, const void* q,
                                   int64_t q_stride_b, int64_t q_stride_s, int64_t q_stride_h, int32_t H, void* q_nope,
                                   void* q_pe, uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!kv_a || !norm_weight || !rotary || !rotary->turns || !pos || !end_pos) return MLA_ERR_INVALID_ARG;
  if (!aligned16(kv_a) || !aligned16(norm_weight) || (reinterpret_cast<uintptr_t>(rotary->turns) & 7u) ||
      !aligned4(pos) || !aligned4(end_pos) || !aligned4(status))
    return MLA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps) || !std::isfinite(rotary->gain)) return MLA_ERR_INVALID_ARG;
  if (norm_f32 != 0 && norm_f32 != 1) return MLA_ERR_INVALID_ARG;
  if (rotary->halves != 0 && rotary->halves != 1) return MLA_ERR_INVALID_ARG;
  if (B <= 0 || s <= 0 || s > (1 << 30) / B) return MLA_ERR_INVALID_ARG;
  // (a dimension of one has a stride that is not used, and may be any number)
  if (B == 1) kv_stride_b = q_stride_b = 0;
  if (s == 1) kv_stride_s = q_stride_s = 0;
  if (!bf16_stride(kv_stride_b, 0) || !bf16_stride(kv_stride_s, 0)) return MLA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_nope == nullptr) || (q == nullptr) != (q_pe == nullptr)) return MLA_ERR_INVALID_ARG;
  mla::RotaryAppend p{};
  if (q) {
    if (!supported_heads(H)) return MLA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(q_nope) || !aligned16(q_pe) || !bf16_stride(q_stride_b, 0) ||
        !bf16_stride(q_stride_s, 0) || !bf16_stride(q_stride_h, 0) || (int64_t)B * s * H > (1 << 30))
      return MLA_ERR_INVALID_ARG;
    for (p.log_h = 4; (1 << p.log_h) < H; ++p.log_h) {}
  }
  const mla::PagedAppend a = paged_append(cache, table, max_pages, nullptr, nullptr, end_pos, B, s, status);
  p.rows = a.rows;
  p.pt = a.pt;
  p.weight = a.weight;
  p.end_pos = a.end_pos;
  p.B = B;
  p.s = s;
  p.max_pos = a.max_pos;
  p.status = status;
  p.kv_a = static_cast<const __nv_bfloat16*>(kv_a);
  p.kv_sb = kv_stride_b;
  p.kv_ss = kv_stride_s;
  p.norm = norm_weight;
  p.norm_f32 = norm_f32;
  p.eps = eps;
  p.turns = rotary->turns;
  p.gain = rotary->gain;
  p.halves = rotary->halves;
  p.pos = pos;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_sb = q_stride_b;
  p.q_ss = q_stride_s;
  p.q_sh = q_stride_h;
  p.q_nope = static_cast<__nv_bfloat16*>(q_nope);
  p.q_pe = static_cast<__nv_bfloat16*>(q_pe);
  cudaError_t e = mla::launch_append_rotary(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged_append_rotary");
  trace_launches(1);
  return MLA_OK;
}

mla_status mla_paged_read(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages, const int32_t* offsets,
                          const int32_t* first, int32_t B, int32_t total, void* kv, int64_t kv_stride, void* pe,
                          int64_t pe_stride, uint32_t* status, void* stream) {
  g_last_error[0] = 0;
  mla_status st = check_paged(cache, table, max_pages);
  if (st != MLA_OK) return st;
  if (!offsets || !aligned4(offsets) || !aligned4(first) || !aligned4(status)) return MLA_ERR_INVALID_ARG;
  if (B <= 0 || B > (1 << 30) || total < 0 || total > (1 << 30)) return MLA_ERR_INVALID_ARG;
  if (total == 1) {   // (its stride is not used, and may be any number)
    kv_stride = mla::kDc;
    pe_stride = mla::kDr;
  }
  if (!bf16_stride(kv_stride, mla::kDc) || !bf16_stride(pe_stride, mla::kDr)) return MLA_ERR_INVALID_ARG;
  if (total == 0) return MLA_OK;
  if (!kv || !pe || !aligned16(kv) || !aligned16(pe)) return MLA_ERR_INVALID_ARG;
  mla::PagedRead p{};
  p.fmt = mla::decode_fmt(cache->fmt);
  p.kv = cache->kv;
  p.kv_scale = cache->kv_scale;
  p.pe = cache->pe;
  p.pt = paged_table(cache, table, max_pages);
  p.max_pos = (long long)max_pages * cache->page_size;
  p.offsets = offsets;
  p.first = first;
  p.B = B;
  p.total = total;
  p.out_kv = static_cast<__nv_bfloat16*>(kv);
  p.out_pe = static_cast<__nv_bfloat16*>(pe);
  p.kv_stride = kv_stride;
  p.pe_stride = pe_stride;
  p.status = status;
  cudaError_t e = mla::launch_paged_read(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged_read");
  trace_launches(1);
  return MLA_OK;
}

size_t mla_paged_window_workspace_size(int32_t B, int32_t s, int32_t H) {
  int sms = 0;
  if (B <= 0 || B > mla::kMaxPagedB || s < 1 || s > mla::kMaxMtp || B > (1 << 22) / s || !supported_heads(H) || num_sms(&sms) != 0)
    return 0;
  return window_bytes(B * s, H, sms);
}

mla_status mla_paged_decode_window(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                                   const void* q_latent, const void* q_pe, const int32_t* end_pos, int32_t max_end_pos,
                                   int32_t B, int32_t s, int32_t H, float softmax_scale, int32_t window, int32_t sinks,
                                   void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  return run_paged_window(cache, table, max_pages, q_latent, q_pe, end_pos, max_end_pos, B, s, H, softmax_scale, window,
                          sinks, out, lse, workspace, ws_bytes, static_cast<cudaStream_t>(stream), -1);
}

mla_status mla_selftest_paged_window_timeout(const mla_paged_cache* cache, const int32_t* table, int32_t max_pages,
                                             const void* q_latent, const void* q_pe, const int32_t* end_pos,
                                             int32_t max_end_pos, int32_t B, int32_t s, int32_t H, float softmax_scale,
                                             int32_t window, int32_t sinks, void* out, float* lse, void* workspace,
                                             size_t ws_bytes, void* stream) {
  g_last_error[0] = 0;
  return run_paged_window(cache, table, max_pages, q_latent, q_pe, end_pos, max_end_pos, B, s, H, softmax_scale, window,
                          sinks, out, lse, workspace, ws_bytes, static_cast<cudaStream_t>(stream), 0);
}

const char* mla_status_string(mla_status status) {
  switch (status) {
    case MLA_OK: return "MLA_OK";
    case MLA_ERR_INVALID_ARG: return "MLA_ERR_INVALID_ARG";
    case MLA_ERR_OUT_OF_RANGE: return "MLA_ERR_OUT_OF_RANGE";
    case MLA_ERR_UNSUPPORTED: return "MLA_ERR_UNSUPPORTED";
    case MLA_ERR_WORKSPACE: return "MLA_ERR_WORKSPACE";
    case MLA_ERR_CUDA: return "MLA_ERR_CUDA";
  }
  return "MLA_ERR_UNKNOWN";
}

const char* mla_last_error(void) { return g_last_error; }

mla_status mla_trace_begin(int32_t max_records) {
  if (g_trace.on || max_records < 0 || max_records > (1 << 20)) return MLA_ERR_INVALID_ARG;
  Trace t;
  t.cap = max_records;
  if (max_records > 0) {
    t.ev = new (std::nothrow) cudaEvent_t[2 * (size_t)max_records];
    if (!t.ev) return MLA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 2 * max_records; ++i) {
    cudaError_t e = cudaEventCreate(&t.ev[i]);
    if (e != cudaSuccess) {
      for (int j = 0; j < i; ++j) cudaEventDestroy(t.ev[j]);
      delete[] t.ev;
      return cuda_fail(e, "trace_begin");
    }
  }
  t.on = true;
  g_trace = t;
  return MLA_OK;
}

mla_status mla_trace_end(float* main_kernel_ms, int32_t* timed_launches, int32_t* kernel_launches) {
  if (!g_trace.on) return MLA_ERR_INVALID_ARG;
  Trace t = g_trace;
  g_trace = Trace();
  mla_status st = MLA_OK;
  double total = 0.0;
  if (t.n > 0) {
    cudaError_t e = cudaEventSynchronize(t.ev[2 * t.n - 1]);
    for (int i = 0; e == cudaSuccess && i < t.n; ++i) {
      float ms = 0.f;
      e = cudaEventElapsedTime(&ms, t.ev[2 * i], t.ev[2 * i + 1]);
      total += ms;
    }
    if (e != cudaSuccess) st = cuda_fail(e, "trace_end");
  }
  for (int i = 0; i < 2 * t.cap; ++i) cudaEventDestroy(t.ev[i]);
  delete[] t.ev;   // null when only launches were counted
  if (main_kernel_ms) *main_kernel_ms = (float)total;
  if (timed_launches) *timed_launches = t.n;
  if (kernel_launches) *kernel_launches = t.launches;
  return st;
}

}  // extern "C"
