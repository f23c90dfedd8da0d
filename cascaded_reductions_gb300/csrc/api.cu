// C ABI of librf.so: argument validation, then one launch per kernel.
// Every check happens on the host before anything is enqueued.

#include <math.h>

#include "paged.cuh"
#include "tc_common.cuh"

namespace {

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// The checks that the calls over a cache of grouped heads share.  Sizes first
// (RF_ERR_INVALID_ARG), then what is outside the supported set.
rf_status check_cache_shape(int B, int H, int Hkv, int cap, int D, float scale, int dtype) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || cap <= 0 || D <= 0) return RF_ERR_INVALID_ARG;
  if (H % Hkv != 0 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16 && dtype != RF_F16) return RF_ERR_INVALID_ARG;
  if (D != 128 || dtype == RF_F32 || cap > (1 << 30)) return RF_ERR_UNSUPPORTED;
  return RF_OK;
}

rf_status check_segments(int B, int H, int Hkv, int S, int dtype, int out_dtype) {
  if (S < 1) return RF_ERR_INVALID_ARG;
  if (out_dtype != RF_F32 && out_dtype != dtype) return RF_ERR_INVALID_ARG;
  if (S > 4096) return RF_ERR_UNSUPPORTED;
  const long long tiles = ((long long)H / Hkv + 15) / 16;
  const long long groups = (long long)B * Hkv;             // below 2^62
  if (groups > 0x7fffffffLL / tiles || groups * tiles > 0x7fffffffLL / S) return RF_ERR_UNSUPPORTED;
  return RF_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < na : x - y < nb;
}
// The same with `rows` rows of nb bytes, `step` bytes from one to the next: what lies
// between them is no part of them.
bool overlap_rows(const void* a, size_t na, const void* b, size_t rows, size_t nb, size_t step) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (x < y) return y - x < na;
  const uintptr_t d = x - y;
  if ((unsigned __int128)(rows - 1) * step + nb <= d) return false;   // behind the last row
  const uintptr_t i = d < nb ? 0 : (d - nb) / step + 1;               // the first row that ends behind x
  return i * step <= d || i * step - d < na;
}

// The sizes of a step over a paged cache.  A window that no request outgrows hides nothing.
rf::PagedShape paged_shape(int B, int T, int H, int Hkv, int max_new, int max_len, int window, int sinks) {
  if (window >= max_len) window = 0;
  if (window == 0 && sinks > 0) sinks = 0;
  rf::PagedShape s = {B, T, H, Hkv, max_new, max_len, window, sinks > max_len && max_len > 0 ? max_len : sinks,
                      rf::kPagedRows, 0};
  if (B > 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && max_new > 0 && max_len > 0) s.divide(rf::tc::sm_count());
  return s;
}

rf_status check_paged(const rf::PagedShape& s) {
  if (s.B <= 0 || s.T <= 0 || s.H <= 0 || s.Hkv <= 0 || s.max_new <= 0 || s.max_len <= 0 || s.window < 0 ||
      s.sinks < 0)
    return RF_ERR_INVALID_ARG;
  if (s.H % s.Hkv != 0 || s.max_new > s.T) return RF_ERR_INVALID_ARG;
  // row and unit numbers stay within an int
  if (s.max_len > (1 << 30) || (long long)s.T * s.H > 0x7fffffffLL || s.B > (1 << 20) || s.H > (1 << 16) ||
      (long long)s.B * s.Hkv * s.tiles() > 0x1fffffffLL)
    return RF_ERR_UNSUPPORTED;
  return RF_OK;
}

rf_status make_plan(const int32_t* starts, const int32_t* lens, const int32_t* slots, const rf::PagedShape& s,
                    void* plan, size_t bytes, void* stream) {
  if (!starts || !lens || !plan) return RF_ERR_INVALID_ARG;
  const rf_status st = check_paged(s);
  if (st != RF_OK) return st;
  if (reinterpret_cast<uintptr_t>(plan) % 256 != 0) return RF_ERR_MISALIGNED;
  rf::PagedLayout l;
  if (!rf::paged_layout(s, &l)) return RF_ERR_CUDA;
  if (bytes < l.bytes) return RF_ERR_INVALID_ARG;
  return rf::launch_paged_plan(starts, lens, slots, s, plan, as_stream(stream));
}

}  // namespace

extern "C" {

const char* rf_status_string(int status) {
  switch (status) {
    case RF_OK: return "RF_OK";
    case RF_ERR_INVALID_ARG: return "RF_ERR_INVALID_ARG";
    case RF_ERR_UNSUPPORTED: return "RF_ERR_UNSUPPORTED";
    case RF_ERR_MISALIGNED: return "RF_ERR_MISALIGNED";
    case RF_ERR_CUDA: return "RF_ERR_CUDA";
    case RF_ERR_TIMEOUT: return "RF_ERR_TIMEOUT";
    case RF_ERR_BOUNDS: return "RF_ERR_BOUNDS";
    default: return "RF_ERR_UNKNOWN";
  }
}

int rf_version(void) { return 10000; }

rf_status rf_attn_decode_split(const void* q, const void* k, const void* v, int R, int L, int D,
                               int S, float scale, int dtype, float* seg_m, float* seg_l,
                               float* seg_acc, void* stream) {
  if (!q || !k || !v || !seg_m || !seg_l || !seg_acc) return RF_ERR_INVALID_ARG;
  if (R <= 0 || L <= 0 || D <= 0 || S < 1 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16) return RF_ERR_INVALID_ARG;
  if (!((dtype == RF_F32 && D == 64) || (dtype == RF_BF16 && D == 128))) return RF_ERR_UNSUPPORTED;
  if ((long long)R * S > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(seg_acc))
    return RF_ERR_MISALIGNED;
  return rf::launch_decode_split(q, k, v, R, L, D, S, scale, dtype, seg_m, seg_l, seg_acc,
                                 as_stream(stream));
}

rf_status rf_attn_decode_fused(const void* q, const void* k, const void* v, int R, int L, int D,
                               int S, float scale, int dtype, float* seg_m, float* seg_l,
                               float* seg_acc, int* counters, void* out, int out_dtype,
                               float* lse, void* stream) {
  if (!q || !k || !v || !seg_m || !seg_l || !seg_acc || !counters || !out)
    return RF_ERR_INVALID_ARG;
  if (R <= 0 || L <= 0 || D <= 0 || S < 1 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16) return RF_ERR_INVALID_ARG;
  if (out_dtype != RF_F32 && out_dtype != RF_BF16) return RF_ERR_INVALID_ARG;
  if (!((dtype == RF_F32 && D == 64) || (dtype == RF_BF16 && D == 128))) return RF_ERR_UNSUPPORTED;
  if ((long long)R * S > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(seg_acc) ||
      !rf::aligned16(out) || !rf::aligned16(counters))
    return RF_ERR_MISALIGNED;
  return rf::launch_decode_fused(q, k, v, R, L, D, S, scale, dtype, seg_m, seg_l, seg_acc,
                                 counters, out, out_dtype, lse, as_stream(stream));
}

rf_status rf_attn_decode_split_twopass(const void* q, const void* k, const void* v, int R, int L,
                                       int D, int S, float scale, int dtype, float* seg_m,
                                       float* seg_l, float* seg_acc, void* stream) {
  if (!q || !k || !v || !seg_m || !seg_l || !seg_acc) return RF_ERR_INVALID_ARG;
  if (R <= 0 || L <= 0 || D <= 0 || S < 1 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16) return RF_ERR_INVALID_ARG;
  if (!((dtype == RF_F32 && D == 64) || (dtype == RF_BF16 && D == 128))) return RF_ERR_UNSUPPORTED;
  if ((long long)R * S > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(seg_acc))
    return RF_ERR_MISALIGNED;
  return rf::launch_decode_twopass(q, k, v, R, L, D, S, scale, dtype, seg_m, seg_l, seg_acc,
                                   as_stream(stream));
}

rf_status rf_state_merge(const float* seg_m, const float* seg_l, const float* seg_acc, int R,
                         int S, int D, void* out, int out_dtype, float* lse, void* stream) {
  if (!seg_m || !seg_l || !seg_acc || !out) return RF_ERR_INVALID_ARG;
  if (R <= 0 || S <= 0 || D <= 0) return RF_ERR_INVALID_ARG;
  if (out_dtype != RF_F32 && out_dtype != RF_BF16) return RF_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 512) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(seg_acc) || !rf::aligned16(out)) return RF_ERR_MISALIGNED;
  return rf::launch_state_merge(seg_m, seg_l, seg_acc, R, S, D, out, out_dtype, lse,
                                as_stream(stream));
}

rf_status rf_mla_decode_split(const void* q, const void* c, int B, int H, int L, int Dk,
                              int Dv, int S, float scale, float* seg_m, float* seg_l,
                              float* seg_acc, void* stream) {
  if (!q || !c || !seg_m || !seg_l || !seg_acc) return RF_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || L <= 0 || S < 1 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (Dk != 576 || Dv != 512 || H % 16 != 0) return RF_ERR_UNSUPPORTED;
  if ((long long)B * L >= (1ll << 31) || (long long)B * H >= (1ll << 31)) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(c) || !rf::aligned16(seg_acc)) return RF_ERR_MISALIGNED;
  return rf::launch_mla_decode(q, c, B, H, L, S, scale, seg_m, seg_l, seg_acc, as_stream(stream));
}

rf_status rf_attn_prefill(const void* q, const void* k, const void* v, int B, int H, int N, int D,
                          int causal, float scale, void* out, float* lse, void* stream) {
  if (!q || !k || !v || !out) return RF_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || N <= 0 || D <= 0 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (D != 128) return RF_ERR_UNSUPPORTED;
  if ((long long)B * H * N >= (1ll << 31)) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(out))
    return RF_ERR_MISALIGNED;
  return rf::launch_prefill(q, k, v, B, H, N, D, causal ? 1 : 0, scale, out, lse,
                            as_stream(stream));
}

rf_status rf_softmax_topk(const float* logits, int T, int E, int k, int renormalize, int32_t* idx,
                          float* w, void* stream) {
  if (!logits || !idx || !w) return RF_ERR_INVALID_ARG;
  if (T <= 0 || E <= 0 || k < 1 || k > E) return RF_ERR_INVALID_ARG;
  if (E > 1024 || k > 32) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(logits) || !rf::aligned16(idx) || !rf::aligned16(w)) return RF_ERR_MISALIGNED;
  return rf::launch_softmax_topk(logits, T, E, k, renormalize ? 1 : 0, idx, w, as_stream(stream));
}

rf_status rf_absmax_quant_e4m3(const void* x, int M, int K, uint8_t* xq, float* sx,
                               void* stream) {
  if (!x || !xq || !sx) return RF_ERR_INVALID_ARG;
  if (M <= 0 || K <= 0) return RF_ERR_INVALID_ARG;
  if (K % 8 != 0) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(x) || !rf::aligned16(xq)) return RF_ERR_MISALIGNED;
  return rf::launch_absmax_quant(x, M, K, xq, sx, as_stream(stream));
}

static rf_status check_gemm_shape(int M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0) return RF_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > 65536) return RF_ERR_UNSUPPORTED;
  return RF_OK;
}

rf_status rf_fp8_gemm_scaled(const uint8_t* xq, const float* sx, const uint8_t* wq,
                             const float* sw, int M, int N, int K, void* y, void* stream) {
  if (!xq || !sx || !wq || !sw || !y) return RF_ERR_INVALID_ARG;
  rf_status s = check_gemm_shape(M, N, K);
  if (s != RF_OK) return s;
  if (!rf::aligned16(xq) || !rf::aligned16(wq) || !rf::aligned16(y) || !rf::aligned16(sw))
    return RF_ERR_MISALIGNED;
  return rf::launch_fp8_gemm(xq, sx, wq, sw, M, N, K, y, as_stream(stream));
}

rf_status rf_absmax_quant_fp8_gemm(const void* x, int M, int K, const uint8_t* wq, const float* sw,
                                   int N, uint8_t* xq, float* sx, void* y, void* stream) {
  if (!x || !wq || !sw || !xq || !sx || !y) return RF_ERR_INVALID_ARG;
  rf_status s = check_gemm_shape(M, N, K);
  if (s != RF_OK) return s;
  if (!rf::aligned16(x) || !rf::aligned16(wq) || !rf::aligned16(xq) || !rf::aligned16(y) ||
      !rf::aligned16(sw))
    return RF_ERR_MISALIGNED;
  s = rf::launch_absmax_quant(x, M, K, xq, sx, as_stream(stream));
  if (s != RF_OK) return s;
  return rf::launch_fp8_gemm(xq, sx, wq, sw, M, N, K, y, as_stream(stream));
}

static rf_status check_row_args(int R, int n, int level) {
  if (R <= 0 || n <= 0) return RF_ERR_INVALID_ARG;
  if (level < RF_FUSE_NONE || level > RF_FUSE_BLOCK) return RF_ERR_INVALID_ARG;
  if (n % 4 != 0) return RF_ERR_UNSUPPORTED;
  return RF_OK;
}

rf_status rf_row_softmax(const float* x, int R, int n, float* y, int level, float* work,
                         void* stream) {
  if (!x || !y) return RF_ERR_INVALID_ARG;
  rf_status s = check_row_args(R, n, level);
  if (s != RF_OK) return s;
  if (level == RF_FUSE_NONE && !work) return RF_ERR_INVALID_ARG;
  if (level != RF_FUSE_NONE && n > 8192) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(x) || !rf::aligned16(y)) return RF_ERR_MISALIGNED;
  return rf::launch_row_softmax(x, R, n, y, level, work, as_stream(stream));
}

rf_status rf_row_variance(const float* x, int R, int n, float* mean, float* var, int level,
                          void* stream) {
  if (!x || !mean || !var) return RF_ERR_INVALID_ARG;
  rf_status s = check_row_args(R, n, level);
  if (s != RF_OK) return s;
  if (!rf::aligned16(x)) return RF_ERR_MISALIGNED;
  return rf::launch_row_variance(x, R, n, mean, var, level, as_stream(stream));
}

rf_status rf_moment_of_inertia(const float* mass, const float* pos, int R, int n, float* center,
                               float* inertia, int level, void* stream) {
  if (!mass || !pos || !center || !inertia) return RF_ERR_INVALID_ARG;
  rf_status s = check_row_args(R, n, level);
  if (s != RF_OK) return s;
  if (!rf::aligned16(mass) || !rf::aligned16(pos)) return RF_ERR_MISALIGNED;
  return rf::launch_moment_of_inertia(mass, pos, R, n, center, inertia, level, as_stream(stream));
}

rf_status rf_layer_norm(const float* x, const float* gamma, const float* beta, int R, int n,
                        float eps, float* y, int level, float* work, void* stream) {
  if (!x || !gamma || !beta || !y) return RF_ERR_INVALID_ARG;
  rf_status s = check_row_args(R, n, level);
  if (s != RF_OK) return s;
  if (!(eps >= 0.f) || !isfinite(eps)) return RF_ERR_INVALID_ARG;
  if (level == RF_FUSE_NONE && !work) return RF_ERR_INVALID_ARG;
  if (level != RF_FUSE_NONE && n > 8192) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(x) || !rf::aligned16(y) || !rf::aligned16(gamma) || !rf::aligned16(beta))
    return RF_ERR_MISALIGNED;
  return rf::launch_layer_norm(x, gamma, beta, R, n, eps, y, level, work, as_stream(stream));
}

rf_status rf_rms_norm(const float* x, const float* gamma, int R, int n, float eps, float* y,
                      int level, float* work, void* stream) {
  if (!x || !gamma || !y) return RF_ERR_INVALID_ARG;
  rf_status s = check_row_args(R, n, level);
  if (s != RF_OK) return s;
  if (!(eps >= 0.f) || !isfinite(eps)) return RF_ERR_INVALID_ARG;
  if (level == RF_FUSE_NONE && !work) return RF_ERR_INVALID_ARG;
  if (level != RF_FUSE_NONE && n > 8192) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(x) || !rf::aligned16(y) || !rf::aligned16(gamma)) return RF_ERR_MISALIGNED;
  return rf::launch_rms_norm(x, gamma, R, n, eps, y, level, work, as_stream(stream));
}

rf_status rf_incremental_quant_fp8_gemm(const void* x, int M, int K, const uint8_t* wq,
                                        const float* sw, int N, void* y, float* sx_final,
                                        void* stream) {
  if (!x || !wq || !sw || !y) return RF_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0) return RF_ERR_INVALID_ARG;
  if (M % 128 != 0 || N % 512 != 0 || K % 128 != 0) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(x) || !rf::aligned16(wq) || !rf::aligned16(y) || !rf::aligned16(sw))
    return RF_ERR_MISALIGNED;
  // clusters of 8 (or 4) CTAs share the quantisation where N allows it
  const rf_status s =
      rf::launch_fp8_incremental_cluster(x, wq, sw, M, N, K, y, sx_final, as_stream(stream));
  if (s != RF_ERR_UNSUPPORTED) return s;
  return rf::launch_fp8_incremental(x, wq, sw, M, N, K, y, sx_final, as_stream(stream));
}

int rf_decode_segments(int groups, int keys) {
  const int sms = rf::tc::sm_count();
  if (sms <= 0) return 0;
  if (groups < 1) groups = 1;
  if (keys < 1) keys = 1;
  return rf::decode_segments(groups, keys, sms);
}

rf_status rf_attn_decode_window(const void* q, const void* k, const void* v, const int32_t* lens,
                                int B, int H, int Hkv, int cap, int D, int window, int sinks,
                                int S, float scale, int dtype, float* seg_m, float* seg_l,
                                float* seg_acc, int* counters, void* out, int out_dtype,
                                float* lse, void* stream) {
  if (!q || !k || !v || !seg_m || !seg_l || !seg_acc || !counters || !out)
    return RF_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return RF_ERR_INVALID_ARG;
  rf_status s = check_cache_shape(B, H, Hkv, cap, D, scale, dtype);
  if (s != RF_OK) return s;
  s = check_segments(B, H, Hkv, S, dtype, out_dtype);
  if (s != RF_OK) return s;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(out) ||
      !rf::aligned16(seg_acc))
    return RF_ERR_MISALIGNED;
  rf::CacheDecode a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.lens = lens;
  a.B = B, a.H = H, a.Hkv = Hkv, a.cap = cap;
  a.window = window, a.sinks = sinks;
  a.S = a.S_total = S;
  a.scale_log2 = scale * rf::kLog2e;
  a.seg_m = seg_m, a.seg_l = seg_l, a.seg_acc = seg_acc;
  a.counters = counters;
  a.out = out, a.out_dtype = out_dtype, a.lse = lse;
  return rf::launch_cache_decode(a, dtype, as_stream(stream));
}

rf_status rf_attn_decode_weights(const void* q, const void* k, const void* v, const int32_t* lens,
                                 int B, int H, int Hkv, int cap, int D, int S, float scale,
                                 int dtype, float* seg_m, float* seg_l, float* seg_acc,
                                 int* counters, float* scores, void* out, int out_dtype,
                                 float* lse, const float* weight, float* weight_out,
                                 void* stream) {
  if (!q || !k || !v || !seg_m || !seg_l || !seg_acc || !counters || !scores || !out ||
      !weight_out)
    return RF_ERR_INVALID_ARG;
  rf_status s = check_cache_shape(B, H, Hkv, cap, D, scale, dtype);
  if (s != RF_OK) return s;
  s = check_segments(B, H, Hkv, S, dtype, out_dtype);
  if (s != RF_OK) return s;
  const size_t bytes = (size_t)B * Hkv * cap * sizeof(float);
  if (weight != weight_out && overlap(weight, bytes, weight_out, bytes)) return RF_ERR_INVALID_ARG;
  if ((long long)B * Hkv * ((cap + 255) / 256) > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(out) ||
      !rf::aligned16(seg_acc) || !rf::aligned16(scores))
    return RF_ERR_MISALIGNED;
  rf::CacheDecode a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.lens = lens;
  a.B = B, a.H = H, a.Hkv = Hkv, a.cap = cap;
  a.S = a.S_total = S;
  a.scale_log2 = scale * rf::kLog2e;
  a.seg_m = seg_m, a.seg_l = seg_l, a.seg_acc = seg_acc;
  a.counters = counters;
  a.out = out, a.out_dtype = out_dtype, a.lse = lse;
  a.scores = scores;
  s = rf::launch_cache_decode(a, dtype, as_stream(stream));
  if (s != RF_OK) return s;
  return rf::launch_add_weights(a, weight, weight_out, as_stream(stream));
}

rf_status rf_attn_prefill_window(const void* q, const void* k, const void* v, int B, int H,
                                 int Hkv, int N, int L, int D, int window, int sinks, float scale,
                                 int dtype, void* out, float* lse, void* stream) {
  if (!q || !k || !v || !out) return RF_ERR_INVALID_ARG;
  if (N <= 0 || N > L || window < 0 || sinks < 0) return RF_ERR_INVALID_ARG;
  const rf_status s = check_cache_shape(B, H, Hkv, L, D, scale, dtype);
  if (s != RF_OK) return s;
  if (!(scale > 0.f)) return RF_ERR_UNSUPPORTED;
  const long long heads = (long long)B * H;
  if (heads > 0x7fffffffLL || heads * N > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(out))
    return RF_ERR_MISALIGNED;
  const int sms = rf::tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  const long long keys = window > 0 && (long long)window + sinks < L ? (long long)window + sinks : L;
  const long long rows = (long long)B * Hkv * N;              // below 2^31
  if (rf::prefill_is_few(rows * ((H / Hkv + 15) / 16), keys, sms)) {
    rf::CacheDecode a = {};
    a.q = static_cast<const uint8_t*>(q);
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.B = B, a.H = H, a.Hkv = Hkv, a.cap = L;
    a.window = window, a.sinks = sinks;
    a.positions = N;
    a.scale_log2 = scale * rf::kLog2e;
    a.out = out, a.out_dtype = dtype, a.lse = lse;
    return rf::launch_prefill_rows(a, dtype, as_stream(stream));
  }
  return rf::launch_prefill_window(q, k, v, B, H, Hkv, N, L, window, sinks, scale, dtype, out, lse,
                                   as_stream(stream));
}

int rf_prefix_segments(int B, int H, int Hkv, int prefix) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || H / Hkv > 128 || prefix <= 0 ||
      prefix > (1 << 30) || (long long)B * Hkv > 0x7fffffffLL)
    return 0;
  return rf::prefix_segments(B, H, Hkv, prefix);
}

rf_status rf_attn_decode_shared(const void* q, const void* kp, const void* vp, int prefix,
                                const void* k, const void* v, const int32_t* lens, int B, int H,
                                int Hkv, int cap, int D, int Sp, int S, float scale, int dtype,
                                float* seg_m, float* seg_l, float* seg_acc, int* counters,
                                void* out, int out_dtype, float* lse, void* stream) {
  if (!q || !kp || !vp || !k || !v || !seg_m || !seg_l || !seg_acc || !counters || !out)
    return RF_ERR_INVALID_ARG;
  if (prefix <= 0 || Sp < 2) return RF_ERR_INVALID_ARG;
  rf_status s = check_cache_shape(B, H, Hkv, cap, D, scale, dtype);
  if (s != RF_OK) return s;
  s = check_segments(B, H, Hkv, S, dtype, out_dtype);
  if (s != RF_OK) return s;
  if (!(scale > 0.f) || Sp > 4096 || H / Hkv > 128 || prefix > (1 << 30)) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(kp) || !rf::aligned16(vp) || !rf::aligned16(k) ||
      !rf::aligned16(v) || !rf::aligned16(out) || !rf::aligned16(seg_acc))
    return RF_ERR_MISALIGNED;
  const int sms = rf::tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  const bool few = rf::decode_prefix_is_few((long long)B * Hkv * ((H / Hkv + 15) / 16), prefix, cap, sms);
  if (!few) {
    s = rf::launch_prefix_states(q, kp, vp, prefix, B, H, Hkv, Sp, Sp + S, scale, dtype, seg_m,
                                 seg_l, seg_acc, as_stream(stream));
    if (s != RF_OK) return s;
  }
  rf::CacheDecode a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.lens = lens;
  a.B = B, a.H = H, a.Hkv = Hkv, a.cap = cap;
  a.S_total = Sp + S;
  if (few) {
    a.kp = static_cast<const uint8_t*>(kp);
    a.vp = static_cast<const uint8_t*>(vp);
    a.prefix = prefix;
    a.S = rf::decode_segments((int)((long long)B * Hkv * ((H / Hkv + 15) / 16)), prefix + cap, sms);
    if (a.S > a.S_total) a.S = a.S_total;
  } else {
    a.S = S, a.seg0 = Sp;
  }
  a.scale_log2 = scale * rf::kLog2e;
  a.seg_m = seg_m, a.seg_l = seg_l, a.seg_acc = seg_acc;
  a.counters = counters;
  a.out = out, a.out_dtype = out_dtype, a.lse = lse;
  return rf::launch_cache_decode(a, dtype, as_stream(stream));
}

rf_status rf_cache_evict(const void* k, const void* v, const float* weight, const int32_t* lens,
                         int B, int Hkv, int cap, int D, int dtype, int keep, int sinks,
                         int recent, int cap_out, void* k_out, void* v_out, float* weight_out,
                         int32_t* lens_out, int32_t* kept, void* stream) {
  if (!k || !weight || !k_out || !weight_out || !lens_out || !kept || (v == nullptr) != (v_out == nullptr))
    return RF_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || cap <= 0 || D <= 0 || keep < 1 || keep > cap_out || sinks < 0 ||
      recent < 0 || (long long)sinks + recent > keep)
    return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16 && dtype != RF_F16) return RF_ERR_INVALID_ARG;
  const long long row_bytes = (long long)D * (dtype == RF_F32 ? 4 : 2);
  if (row_bytes % 16 != 0 || row_bytes > 65536 || cap > (1 << 30) || cap_out > (1 << 30) ||
      (long long)B * Hkv > 0x7fffffffLL)
    return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(k_out) || !rf::aligned16(v_out))
    return RF_ERR_MISALIGNED;
  const size_t groups = (size_t)B * Hkv;
  const struct { const void* p; size_t n; } in[] = {
      {k, groups * cap * row_bytes}, {v, groups * cap * row_bytes}, {weight, groups * cap * 4},
      {lens, (size_t)B * 4}};
  const struct { const void* p; size_t n; } out[] = {
      {k_out, groups * cap_out * row_bytes}, {v_out, groups * cap_out * row_bytes},
      {weight_out, groups * cap_out * 4}, {lens_out, (size_t)B * 4}, {kept, groups * keep * 4}};
  for (int i = 0; i < 5; ++i) {
    for (const auto& x : in)
      if (overlap(out[i].p, out[i].n, x.p, x.n)) return RF_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return RF_ERR_INVALID_ARG;
  }
  return rf::launch_cache_evict(k, v, weight, lens, B, Hkv, cap, (int)row_bytes, keep, sinks,
                                recent, cap_out, k_out, v_out, weight_out, lens_out, kept,
                                as_stream(stream));
}

rf_status rf_page_tables(const int32_t* lens, const int32_t* news, int B, int32_t* table, int width,
                         int32_t* stack, int pages, const int32_t* n_free, int page, int T,
                         int32_t* starts, int32_t* positions, int32_t* slots, int32_t* lens_out,
                         int32_t* n_free_out, void* stream) {
  if (!lens || !news || !table || !stack || !n_free || !starts || !positions || !slots || !lens_out ||
      !n_free_out)
    return RF_ERR_INVALID_ARG;
  if (B <= 0 || width <= 0 || pages <= 0 || page <= 0 || T <= 0) return RF_ERR_INVALID_ARG;
  if (B > rf::kMaxTableRequests || (long long)B * width > 0x7fffffffLL ||
      (long long)pages * page > 0x7fffffffLL || (long long)width * page > 0x7fffffffLL)
    return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(positions) || !rf::aligned16(slots)) return RF_ERR_MISALIGNED;
  // lens_out may be lens and n_free_out n_free; nothing else may overlap
  const struct { const void* p; size_t n; } buf[] = {
      {lens, (size_t)B * 4}, {n_free, 4}, {news, (size_t)B * 4}, {table, (size_t)B * width * 4},
      {stack, (size_t)pages * 4}, {starts, ((size_t)B + 1) * 4}, {positions, (size_t)T * 4},
      {slots, (size_t)T * 4}, {lens_out, (size_t)B * 4}, {n_free_out, 4}};
  for (int i = 3; i < 10; ++i)
    for (int j = 0; j < i; ++j) {
      if ((i == 8 && j == 0 && lens_out == lens) || (i == 9 && j == 1 && n_free_out == n_free)) continue;
      if (overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n)) return RF_ERR_INVALID_ARG;
    }
  return rf::launch_page_tables(lens, news, B, table, width, stack, pages, n_free, page, T, starts,
                                positions, slots, lens_out, n_free_out, as_stream(stream));
}

rf_status rf_qk_norm_rope(const void* q, long long q_step, const void* k, long long k_step,
                          const void* v, long long v_step, int T, int H, int Hkv, int D,
                          const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                          const int32_t* positions, int axes, const float* freq, const int32_t* axis,
                          int R, int interleaved, int dtype, const int32_t* slots, int pages, int page,
                          void* q_out, void* k_out, void* v_out, void* stream) {
  if (!q || !k || !positions || !freq || !q_out || !k_out) return RF_ERR_INVALID_ARG;
  if ((slots != nullptr) != (v != nullptr) || (v != nullptr) != (v_out != nullptr)) return RF_ERR_INVALID_ARG;
  if (T <= 0 || H <= 0 || Hkv <= 0 || D <= 0 || axes <= 0 || R <= 0 || R > D) return RF_ERR_INVALID_ARG;
  if (slots && (pages <= 0 || page <= 0)) return RF_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !isfinite(eps)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16 && dtype != RF_F16) return RF_ERR_INVALID_ARG;
  if (weight_dtype != RF_F32 && weight_dtype != dtype) return RF_ERR_INVALID_ARG;
  if (dtype == RF_F32 || (D != 64 && D != 128 && D != 256) || R % 16 != 0) return RF_ERR_UNSUPPORTED;
  if ((long long)H * D > 0x7fffffffLL || (long long)Hkv * D > 0x7fffffffLL ||
      (long long)H + 2ll * Hkv > 0x7fffffffLL || (long long)T * ((H + 2ll * Hkv + 7) / 8) > 0x7fffffffLL ||
      (slots && (long long)pages * page > 0x7fffffffLL))
    return RF_ERR_UNSUPPORTED;
  if (q_step < (long long)H * D || k_step < (long long)Hkv * D || (v && v_step < (long long)Hkv * D))
    return RF_ERR_INVALID_ARG;
  if (q_step > (1ll << 40) || k_step > (1ll << 40) || (v && v_step > (1ll << 40))) return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(k) || !rf::aligned16(v) || !rf::aligned16(q_out) ||
      !rf::aligned16(k_out) || !rf::aligned16(v_out) || q_step % 8 != 0 || k_step % 8 != 0 ||
      (v && v_step % 8 != 0))
    return RF_ERR_MISALIGNED;
  // q_out may be q and k_out k, row for row; nothing else may overlap
  const size_t rows = (size_t)T, q_row = (size_t)H * D * 2, k_row = (size_t)Hkv * D * 2;
  const size_t kv = slots ? (size_t)pages * page * k_row : rows * k_row, w = weight_dtype == RF_F32 ? 4 : 2;
  const struct { const void* p; size_t n; } out[] = {{q_out, rows * q_row}, {k_out, kv}, {v_out, kv}};
  const struct { const void* p; size_t row, step; } tokens[] = {
      {q, q_row, (size_t)q_step * 2}, {k, k_row, (size_t)k_step * 2}, {v, k_row, (size_t)v_step * 2}};
  const struct { const void* p; size_t n; } in[] = {
      {q_weight, D * w}, {k_weight, D * w}, {positions, (size_t)axes * T * 4}, {freq, (size_t)R * 2},
      {axis, (size_t)R * 2}, {slots, rows * 4}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j) {
      const auto& t = tokens[j];
      const bool in_place = i == j && out[i].p == t.p && (i == 0 || slots == nullptr) && (T == 1 || t.step == t.row);
      if (!in_place && overlap_rows(out[i].p, out[i].n, t.p, rows, t.row, t.step)) return RF_ERR_INVALID_ARG;
    }
    for (const auto& x : in)
      if (overlap(out[i].p, out[i].n, x.p, x.n)) return RF_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return RF_ERR_INVALID_ARG;
  }
  return rf::launch_qk_norm_rope(q, q_step, k, k_step, v, v_step, T, H, Hkv, D, q_weight, k_weight,
                                 weight_dtype == RF_F32, eps, positions, axes, freq, axis, R,
                                 interleaved != 0, dtype, slots, pages, page, q_out, k_out, v_out,
                                 as_stream(stream));
}

size_t rf_paged_plan_bytes(int B, int T, int H, int Hkv, int max_new, int max_len, int window, int sinks) {
  const rf::PagedShape s = paged_shape(B, T, H, Hkv, max_new, max_len, window, sinks);
  rf::PagedLayout l;
  return check_paged(s) == RF_OK && rf::paged_layout(s, &l) ? l.bytes : 0;
}

rf_status rf_paged_plan(const int32_t* starts, const int32_t* lens, int B, int T, int H, int Hkv,
                        int max_new, int max_len, int window, int sinks, void* plan, size_t bytes,
                        void* stream) {
  return make_plan(starts, lens, nullptr, paged_shape(B, T, H, Hkv, max_new, max_len, window, sinks), plan, bytes,
                   stream);
}

rf_status rf_paged_plan_slots(const int32_t* starts, const int32_t* lens, const int32_t* slots, int B, int T,
                              int H, int Hkv, int max_new, int max_len, int window, int sinks, void* plan,
                              size_t bytes, void* stream) {
  if (!slots) return RF_ERR_INVALID_ARG;
  return make_plan(starts, lens, slots, paged_shape(B, T, H, Hkv, max_new, max_len, window, sinks), plan, bytes,
                   stream);
}

rf_status rf_attn_paged(const void* q, const void* kp, const void* vp, int pages, int page,
                        const int32_t* table, int width, void* plan, size_t bytes, int B, int T, int H,
                        int Hkv, int D, int max_new, int max_len, int window, int sinks, float scale,
                        int dtype, void* out, float* lse, void* stream) {
  if (!q || !kp || !vp || !table || !plan || !out) return RF_ERR_INVALID_ARG;
  if (pages <= 0 || page <= 0 || width <= 0 || D <= 0 || !isfinite(scale)) return RF_ERR_INVALID_ARG;
  if (dtype != RF_F32 && dtype != RF_BF16 && dtype != RF_F16) return RF_ERR_INVALID_ARG;
  const rf::PagedShape s = paged_shape(B, T, H, Hkv, max_new, max_len, window, sinks);
  rf_status st = check_paged(s);
  if (st != RF_OK) return st;
  if ((long long)width * page < max_len) return RF_ERR_INVALID_ARG;
  if (D != 128 || dtype == RF_F32 || !(scale > 0.f)) return RF_ERR_UNSUPPORTED;
  int log2 = 4;
  while (log2 < 8 && (1 << log2) != page) ++log2;
  if ((1 << log2) != page || (long long)pages * Hkv > 0x3fffffffLL || (long long)B * width > 0x7fffffffLL)
    return RF_ERR_UNSUPPORTED;
  if (!rf::aligned16(q) || !rf::aligned16(kp) || !rf::aligned16(vp) || !rf::aligned16(out) ||
      reinterpret_cast<uintptr_t>(plan) % 256 != 0)
    return RF_ERR_MISALIGNED;
  rf::PagedLayout l;
  if (!rf::paged_layout(s, &l)) return RF_ERR_CUDA;
  if (bytes < l.bytes) return RF_ERR_INVALID_ARG;
  rf::PagedAttn a = {};
  a.v = rf::paged_view(s, l, plan);
  a.q = static_cast<const uint8_t*>(q);
  a.kp = static_cast<const uint8_t*>(kp);
  a.vp = static_cast<const uint8_t*>(vp);
  a.table = table;
  a.pages = pages, a.page_log2 = log2, a.width = width;
  a.scale_log2 = scale * rf::kLog2e;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  const bool pairs = s.some_pairs();
  if (pairs) {
    st = rf::launch_paged_prefill(a, dtype, as_stream(stream));
    if (st != RF_OK) return st;
  }
  st = rf::launch_paged_decode(a, dtype, as_stream(stream));
  if (st != RF_OK || s.few) return st;
  return rf::launch_paged_finish(a, dtype, as_stream(stream));
}

rf_status rf_device_error(int* status, void* stream) {
  if (!status) return RF_ERR_INVALID_ARG;
  return rf::read_device_error(status, as_stream(stream));
}

}  // extern "C"

rf_status rf_selftest_wait_timeout(int* waited_ms, void* stream) {
  if (!waited_ms) return RF_ERR_INVALID_ARG;
  return rf::launch_selftest_wait_timeout(waited_ms, as_stream(stream));
}

int rf_bounds_checked(void) {
#ifdef RF_CHECK_BOUNDS
  return 1;
#else
  return 0;
#endif
}

rf_status rf_selftest_bounds(void* stream) {
#ifdef RF_CHECK_BOUNDS
  return rf::launch_selftest_bounds(as_stream(stream));
#else
  (void)stream;
  return RF_ERR_UNSUPPORTED;
#endif
}
