// What the kernels over a serving cache of grouped heads share.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace rf {

// Two floats -> fp16 pair, round to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Columns 4 lane .. + 3 of a 16-bit row, widened (by L2 alone: the kernel may not have waited)
template <bool F16>
__device__ __forceinline__ float4 load_row4(const uint8_t* row, int lane) {
  const uint2 u = __ldcg(reinterpret_cast<const uint2*>(row + lane * 8));
  if constexpr (F16) {
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  } else {
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  }
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ long long scan_warp(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

constexpr int kDecodeTile = 16;        // keys of one tile of the decode kernels

// Programmatic dependent launch: a kernel launched with launch_after begins when
// every CTA of the kernel before it on the stream has called
// allow_dependents() or ended, and may use that kernel's results (and those of
// everything before it) after wait_prerequisite().  So that this holds along a chain
//  * a call's first kernel waits before it reads anything and before it allows
//    dependents, whatever ran before it on the stream;
//  * a kernel ends only after its prerequisite has (at least one CTA waits);
//  * what an earlier kernel may have written is not read through the read-only path,
//    which may load ahead of the wait;
//  * a call's later kernel may read what was there before the call's first one without
//    a wait of its own (a decode beside the pair kernel that it follows: with the wait a
//    mixed batch takes 327 us instead of 315).  It begins after every CTA of the kernel
//    before it has waited and said so, when those writes have been performed; but it is a
//    wait that makes them visible past a kernel's own caches.  So paged_decode reads them
//    by L2 alone (__ldcg, cp.async.cg), at no cost.  cache_decode behind a prefix does so
//    with keys and values only: lengths and queries, 4 bytes at a time, it reads through
//    L1, and relies on L1 to hold no line from before its kernel began (by L2 alone a
//    step of 128 sequences takes 64.7 us instead of 64.2, of 38 sequences 19.4 and 18.4).
// Back to back, a single-token decode takes 6.0 us so and 8.2 us when its kernel is
// set up only after the one before has ended.
__device__ __forceinline__ void allow_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prerequisite() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... Params, typename... Args>
inline rf_status launch_after(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                              cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return RF_ERR_CUDA;
  }
  return launch_status();
}

// Keys of a piece of a row at least: one step of the CTA's four warps in a small
// call, enough to pay for a CTA's start and end in a large one.
constexpr int kFewKeys = 4 * kDecodeTile, kManyKeys = 768;

// Counts reach the largest int, where a + b - 1 would not fit one.
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Whether a call of `groups` row groups of up to `keys` visible keys is small: its
// pieces fit two CTAs on every SM, at most sixteen steps of 64 keys each (with a
// limit of four, 64 rows of 2048 keys took 17.4 us instead of 15.6, 8 rows of 32768
// 33.3 instead of 26.6; with 64, 192 ragged rows of 3000 39.8 instead of 36.0).
inline bool decode_is_few(long long groups, int keys, int sms) {
  return groups <= 2ll * sms && groups * ceil_div(keys, kFewKeys) <= 32ll * sms;
}

// Pieces of the longest row of a large call.  Rows of up to two pieces stay whole, to
// save the merge: 256 rows of 1536 keys take 32.7 us so and 37.7 us in two pieces,
// 1024 rows of 1024 keys 56.5 and 60.2 us; one row of 1536 among 255 of 192 keys takes
// 17.8 and 14.2 us.
inline int decode_many_pieces(int keys) {
  return keys <= 2 * kManyKeys ? 1 : (int)ceil_div(keys, kManyKeys);
}

// Pieces per row for such a call: a small one is divided as far as one wave of two
// CTAs per SM goes (a second one costs 3 us, a longer piece 0.6 us per step), a large
// one into the smallest pieces that are worth a CTA.
inline int decode_segments(int groups, int keys, int sms) {
  long long s;
  if (decode_is_few(groups, keys, sms)) {
    s = 2ll * sms / groups;
    const long long steps = ceil_div(keys, kFewKeys);
    if (s > steps) s = steps;
  } else {
    s = decode_many_pieces(keys);
  }
  return (int)(s > 4096 ? 4096 : s);
}

// Whether a shared prefix is read once per sequence, as keys before its own, instead
// of by the prefix kernel: a small call, in which that takes less than the second
// launch (4 sequences behind 1000 keys 7.4 us, 9.3 with it; 38 behind 300 keys 9.4 and
// 13.9; at 16 steps per SM, 30 sequences behind 500 keys, 12.9 and 10.8).
constexpr int kSharedSteps = 14;
static_assert(kSharedSteps <= 32, "such a call is small");
inline bool decode_prefix_is_few(long long groups, long long prefix, int cap, int sms) {
  const long long keys = prefix + cap;
  return groups <= 2ll * sms && groups * ceil_div(keys, kFewKeys) <= (long long)kSharedSteps * sms;
}

// Whether a windowed prefill is so small that a CTA per position and row group is
// faster than the pair kernel's 256 rows at a time (26 rows of 20 heads, 27 keys: 3.2
// us, 7.3 with the pair kernel; 32 rows of 32 heads, 132 keys: 5.4 and 8.4; 4 rows of
// 32 heads, 1004 keys: 11.8 and 13.2; 256 rows of 16 heads, at 6.7 steps per SM: 8.6
// and 7.6).
constexpr int kRowsSteps = 6, kRowsKeys = 1024;
inline bool prefill_is_few(long long groups, long long keys, int sms) {
  return groups <= 2ll * sms && keys <= kRowsKeys &&
         groups * ceil_div(keys, kFewKeys) <= (long long)kRowsSteps * sms;
}

// One call's arguments.  Segment states are scratch between kernels: seg_m
// holds log2 units, and a segment without keys has m = -inf, l = 0 and an
// accumulator that is neither written nor read.
struct CacheDecode {
  const uint8_t *q, *k, *v;      // [B, H, 128], [B, Hkv, cap, 128] of a 16-bit type
  const int32_t* lens;           // [B] or null (every sequence holds cap keys)
  int B, H, Hkv, cap;
  int window, sinks;             // window 0: every key is visible
  const uint8_t *kp, *vp;        // [Hkv, prefix, 128]: keys before every sequence's own, where
  int prefix;                    // decode_prefix_is_few (no window, no scores); else 0
  int S, S_total, seg0;          // this kernel's slots seg0 .. seg0 + S - 1 of S_total
  int positions;                 // launch_prefill_rows: rows per head, q and out [B, H, positions, 128]
  float scale_log2;
  float *seg_m, *seg_l, *seg_acc;   // [B * H, S_total (, 128)]
  int* counters;                 // [B * Hkv * mtiles], zero before and after the call
  void* out;                     // [B, H, 128]
  int out_dtype;
  float* lse;                    // [B, H] or null
  float* scores;                 // [B, H, cap] log2-unit scores, or null
  int G, mtiles, piece_keys;     // set by the launcher
};

// With seg0 > 0 the kernel before it on the stream writes the first seg0 slots.
rf_status launch_cache_decode(CacheDecode a, int dtype, cudaStream_t st);
// Attention of each of the last `positions` of cap positions, one CTA per position
// and row group: window and sinks as in prefill, no scratch.
rf_status launch_prefill_rows(CacheDecode a, int dtype, cudaStream_t st);
// weight may be null (zeros) or equal to total (in place)
rf_status launch_add_weights(const CacheDecode& a, const float* weight, float* total,
                             cudaStream_t st);
// window 0: none.  scale > 0.
rf_status launch_prefill_window(const void* q, const void* k, const void* v, int B, int H, int Hkv,
                                int N, int L, int window, int sinks, float scale, int dtype,
                                void* out, float* lse, cudaStream_t st);
// State slots that the prefix kernel would use per row on the current device
// (at least 2), 0 if it cannot run there.  B, H / Hkv <= 128 as checked.
int prefix_segments(int B, int H, int Hkv, int prefix);
// States of every row over the shared prefix, in slots 0 .. Sp - 1 of S_total
// (unused ones marked empty).  Sp >= 2, scale > 0.
rf_status launch_prefix_states(const void* q, const void* kp, const void* vp, int prefix, int B,
                               int H, int Hkv, int Sp, int S_total, float scale, int dtype,
                               float* seg_m, float* seg_l, float* seg_acc, cudaStream_t st);
rf_status launch_cache_evict(const void* k, const void* v, const float* weight,
                             const int32_t* lens, int B, int Hkv, int cap, int row_bytes, int keep,
                             int sinks, int recent, int cap_out, void* k_out, void* v_out,
                             float* weight_out, int32_t* lens_out, int32_t* kept,
                             cudaStream_t st);

// The step of a loop over a paged cache.
constexpr int kMaxTableRequests = 8192;    // of launch_page_tables
rf_status launch_page_tables(const int32_t* lens, const int32_t* news, int B, int32_t* table, int width,
                             int32_t* stack, int P, const int32_t* n_free, int page, int T,
                             int32_t* starts, int32_t* positions, int32_t* slots, int32_t* lens_out,
                             int32_t* n_free_out, cudaStream_t st);
// steps: elements from a token's row to the next; slots null: k to k_out [T, Hkv, D] and no v,
// else k and v to the pages k_out, v_out [P, Hkv, page, D].  w32: weights are fp32.
rf_status launch_qk_norm_rope(const void* q, long long q_step, const void* k, long long k_step,
                              const void* v, long long v_step, int T, int H, int Hkv, int D,
                              const void* qw, const void* kw, bool w32, float eps,
                              const int32_t* positions, int axes, const float* freq,
                              const int32_t* axis, int R, bool interleaved, int dtype,
                              const int32_t* slots, int P, int page, void* q_out, void* k_out,
                              void* v_out, cudaStream_t st);

}  // namespace rf
