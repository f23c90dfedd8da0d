// What the kernels over a serving cache of grouped heads share.
#pragma once

#include "common.cuh"

namespace rf {

// Two floats -> fp16 pair, round to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Keys of a segment when n keys are split into S: whole 16-key tiles, and at
// least 64 keys (one tile for each of a CTA's four warps), so that short
// sequences leave segments empty instead of warps idle.
__host__ __device__ __forceinline__ int segment_keys(int n, int S) {
  const int c = ((n + S - 1) / S + 15) & ~15;
  return c < 64 ? 64 : c;
}

// Segments for `groups` rows of CTAs of up to `keys` visible keys each: two
// resident CTAs on every SM, in segments of no more than 512 keys where there
// are more CTAs than that anyway (so that the last ones to run are short), and
// no segment below 64 keys.
inline int decode_segments(int groups, int keys, int sms) {
  const long long fill = (2ll * sms + groups - 1) / groups;
  const long long fine = groups >= sms / 4 ? (keys + 511) / 512 : 1;
  long long s = fill > fine ? fill : fine;
  const long long most = (keys + 63) / 64;
  if (s > most) s = most;
  if (s > 4096) s = 4096;
  return (int)(s < 1 ? 1 : s);
}

// One call's arguments.  Segment states are scratch between kernels: seg_m
// holds log2 units, and a segment without keys has m = -inf, l = 0 and an
// accumulator that is neither written nor read.
struct CacheDecode {
  const uint8_t *q, *k, *v;      // [B, H, 128], [B, Hkv, cap, 128] of a 16-bit type
  const int32_t* lens;           // [B] or null (every sequence holds cap keys)
  int B, H, Hkv, cap;
  int window, sinks;             // window 0: every key is visible
  int S, S_total, seg0;          // this kernel's segments seg0 .. seg0 + S - 1 of S_total
  float scale_log2;
  float *seg_m, *seg_l, *seg_acc;   // [B * H, S_total (, 128)]
  int* counters;                 // [B * Hkv * mtiles], zero before and after
  void* out;                     // [B, H, 128]
  int out_dtype;
  float* lse;                    // [B, H] or null
  float* scores;                 // [B, H, cap] log2-unit scores, or null
  int G, mtiles;                 // set by the launcher
};

rf_status launch_cache_decode(CacheDecode a, int dtype, cudaStream_t st);
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

}  // namespace rf
