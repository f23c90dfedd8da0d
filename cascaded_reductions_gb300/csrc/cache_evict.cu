// Eviction from a serving cache by accumulated attention weight: of each
// (sequence, key head)'s len rows keep the first `sinks`, the last `recent`
// and, of those between, the rows of largest weight up to `keep` in all; the
// kept rows move to a new cache in their old order.
//
// Cascade: a selection (the need-th largest weight of the row), then a
// compaction that depends on it, then the copy that depends on both.
//
// evict_select_kernel, one CTA per (sequence, key head): weights become
// 32-bit keys whose unsigned order is the weights' order (NaN lowest, -0 as
// +0), the need-th largest is found digit by digit (four histograms of 8
// bits), and the compaction needs two sweeps with warp votes: the number kept
// before a row is  above_before + min(equal_before, equal_needed),  so ties go
// to the lowest index without a second selection.  Weights are read from
// memory once and kept in shared memory (up to 48 Ki of them; longer rows are
// read again from L2).
//
// evict_copy_kernel, bound by HBM (each kept row is read and written once):
// 16-byte streaming copies, eight in flight per lane.

#include "cache_common.cuh"

namespace rf {
namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_KEYS = 48 * 1024;              // keys that fit in shared memory

// unsigned order = weight order; NaN ranks below every number
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Evict {
  const float* weight;
  const int32_t* lens;
  int B, Hkv, cap, keep, sinks, recent;
  int32_t* lens_out;
  int32_t* kept;
};

__global__ void __launch_bounds__(SEL_THREADS)
evict_select_kernel(const Evict a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int above[SEL_WARPS], equal[SEL_WARPS];

  allow_dependents();
  const int group = blockIdx.x;
  const int b = group / a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.cap;
  if (a.lens != nullptr && RF_IDX_OK(b, a.B)) len = min(max(a.lens[b], 0), a.cap);
  const int count = min(len, a.keep);
  if (group % a.Hkv == 0 && tid == 0 && RF_IDX_OK(b, a.B)) a.lens_out[b] = count;
  const size_t slot0 = (size_t)group * a.keep;
  const size_t slots = (size_t)a.B * a.Hkv * a.keep;
  (void)slots;                                   // read by the checked build only
  for (int i = count + tid; i < a.keep; i += SEL_THREADS)
    if (RF_IDX_OK(slot0 + i, slots)) a.kept[slot0 + i] = -1;
  if (len <= a.keep) {
    for (int i = tid; i < count; i += SEL_THREADS)
      if (RF_IDX_OK(slot0 + i, slots)) a.kept[slot0 + i] = i;
    return;
  }

  // candidates: rows first .. last - 1, more of them than `need`
  const int first = min(a.sinks, len);
  const int last = max(first, len - a.recent);
  int need = a.keep - first - (len - last);
  const int n = last - first;
  const size_t w0 = (size_t)group * a.cap + first;
  const bool in_smem = n <= SEL_KEYS;
  const size_t weights = (size_t)a.B * a.Hkv * a.cap;
  (void)weights;
  auto load = [&](int i) -> uint32_t {
    return RF_IDX_OK(w0 + i, weights) ? order_key(a.weight[w0 + i]) : 0u;
  };
  auto key = [&](int i) -> uint32_t { return in_smem ? keys[i] : load(i); };
  if (in_smem)
    for (int i = tid; i < n; i += SEL_THREADS) keys[i] = load(i);

  // the need-th largest key, eight bits at a time from the top
  uint32_t prefix = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < n; i0 += SEL_THREADS) {
        const int i = i0 + tid;
        bool in = i < n;
        uint32_t k = 0;
        if (in) k = key(i);
        if (shift < 24) in = in && (k >> (shift + 8)) == (prefix >> (shift + 8));
        const uint32_t digit = in ? (k >> shift) & 255u : 256u;
        // one add per distinct digit of the warp: weights share exponents
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(peers) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(peers));
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds bins 8 l .. 8 l + 7; find the bin where the count from
        // the top reaches need
        uint32_t mine = 0;
        for (int e = 0; e < 8; ++e) mine += hist[8 * lane + e];
        uint32_t from_top = mine;                // sum over lanes >= this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_down_sync(0xffffffffu, from_top, o);
          if (lane + o < 32) from_top += x;
        }
        uint32_t before = from_top - mine;
        if (before < (uint32_t)need && from_top >= (uint32_t)need) {
          for (int e = 7; e >= 0; --e) {
            const uint32_t h = hist[8 * lane + e];
            if (before + h >= (uint32_t)need) {
              sh_prefix = prefix | ((uint32_t)(8 * lane + e) << shift);
              sh_need = (uint32_t)need - before;
              break;
            }
            before += h;
          }
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      need = (int)sh_need;
      __syncthreads();
    }
  } else {
    prefix = 0xffffffffu;                        // no weight's key: none is kept
    need = 0;
  }
  __syncthreads();

  // rows above the threshold are kept, and the first `need` equal to it
  const int per = ((n + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
  const int i_begin = min(n, warp * per), i_end = min(n, i_begin + per);
  int ca = 0, ce = 0;
  for (int i0 = i_begin; i0 < i_end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < i_end ? key(i) : 0u;
    ca += __popc(__ballot_sync(0xffffffffu, i < i_end && k > prefix));
    ce += __popc(__ballot_sync(0xffffffffu, i < i_end && k == prefix));
  }
  if (lane == 0) {
    above[warp] = ca;
    equal[warp] = ce;
  }
  __syncthreads();
  int ba = 0, be = 0;
  for (int w = 0; w < warp; ++w) {
    ba += above[w];
    be += equal[w];
  }
  for (int i = tid; i < first; i += SEL_THREADS)
    if (RF_IDX_OK(slot0 + i, slots)) a.kept[slot0 + i] = i;
  for (int i0 = i_begin; i0 < i_end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < i_end ? key(i) : 0u;
    const uint32_t va = __ballot_sync(0xffffffffu, i < i_end && k > prefix);
    const uint32_t ve = __ballot_sync(0xffffffffu, i < i_end && k == prefix);
    const uint32_t below = (1u << lane) - 1u;
    const int eb = be + __popc(ve & below);
    const bool take = ((va >> lane) & 1u) || (((ve >> lane) & 1u) && eb < need);
    const int pos = first + ba + __popc(va & below) + min(eb, need);
    if (take && RF_IDX_OK(slot0 + pos, slots)) a.kept[slot0 + pos] = first + i;
    ba += __popc(va);
    be += __popc(ve);
  }
  const int tail = a.keep - (len - last);
  for (int i = tid; i < len - last; i += SEL_THREADS)
    if (RF_IDX_OK(slot0 + tail + i, slots)) a.kept[slot0 + tail + i] = last + i;
}

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNROLL = 8;

// One unit is a 16-byte chunk of a kept row of K (or V); a CTA copies
// COPY_THREADS * COPY_UNROLL consecutive units of one (sequence, key head).
__global__ void __launch_bounds__(COPY_THREADS)
evict_copy_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                  const float* __restrict__ weight, const int32_t* kept, int groups,
                  int cap, uint32_t chunks, int keep, int cap_out, int blocks, uint4* __restrict__ k_out,
                  uint4* __restrict__ v_out, float* __restrict__ weight_out) {
  const int part = blockIdx.x % 2;                 // 0: K and the weights, 1: V
  const int block = (int)(blockIdx.x / 2) % blocks;
  const int group = (int)(blockIdx.x / 2) / blocks;
  const uint4* src = part ? v : k;
  uint4* dst = part ? v_out : k_out;
  wait_prerequisite();                             // the kept rows' indices
  if (src == nullptr) return;
  const uint32_t u0 = (uint32_t)block * (COPY_THREADS * COPY_UNROLL) + threadIdx.x;
  const uint32_t units = (uint32_t)keep * (uint32_t)chunks;      // below 2^31
  const int32_t* idx = kept + (size_t)group * keep;
  const size_t slots = (size_t)groups * keep;
  (void)slots;
  uint4 x[COPY_UNROLL];
  int row[COPY_UNROLL];
#pragma unroll
  for (int e = 0; e < COPY_UNROLL; ++e) {
    const uint32_t u = u0 + e * COPY_THREADS;
    row[e] = -1;
    if (u < units) {
      const uint32_t i = u / chunks;
      if (RF_IDX_OK((size_t)group * keep + i, slots)) row[e] = __ldcg(idx + i);
    }
  }
#pragma unroll
  for (int e = 0; e < COPY_UNROLL; ++e) {
    const uint32_t u = u0 + e * COPY_THREADS;
    if (row[e] < 0) continue;
    const uint32_t c = u % chunks;
    const size_t at = ((size_t)group * cap + row[e]) * chunks + c;
    if (RF_IDX_OK(at, (size_t)groups * cap * chunks)) x[e] = ld_stream_v4(src + at);
  }
#pragma unroll
  for (int e = 0; e < COPY_UNROLL; ++e) {
    const uint32_t u = u0 + e * COPY_THREADS;
    if (row[e] < 0) continue;
    const uint32_t i = u / chunks, c = u - i * chunks;
    const size_t at = ((size_t)group * cap_out + i) * chunks + c;
    if (RF_IDX_OK(at, (size_t)groups * cap_out * chunks)) __stcs(dst + at, x[e]);
    if (part == 0 && c == 0 && RF_IDX_OK((size_t)group * cap_out + i, (size_t)groups * cap_out) &&
        RF_IDX_OK((size_t)group * cap + row[e], (size_t)groups * cap))
      weight_out[(size_t)group * cap_out + i] = weight[(size_t)group * cap + row[e]];
  }
}

}  // namespace

rf_status launch_cache_evict(const void* k, const void* v, const float* weight,
                             const int32_t* lens, int B, int Hkv, int cap, int row_bytes, int keep,
                             int sinks, int recent, int cap_out, void* k_out, void* v_out,
                             float* weight_out, int32_t* lens_out, int32_t* kept,
                             cudaStream_t st) {
  const int chunks = row_bytes / 16;
  const long long units = (long long)keep * chunks;
  const long long blocks = (units + COPY_THREADS * COPY_UNROLL - 1) / (COPY_THREADS * COPY_UNROLL);
  if (units > 0x7fffffffLL || blocks * 2 * B * Hkv > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  static std::atomic<uint64_t> done{0};
  if (smem_attr(evict_select_kernel, SEL_KEYS * sizeof(uint32_t), done) != RF_OK) return RF_ERR_CUDA;
  const int held = cap < SEL_KEYS ? cap : SEL_KEYS;
  evict_select_kernel<<<(unsigned)(B * Hkv), SEL_THREADS, (size_t)held * sizeof(uint32_t), st>>>(
      Evict{weight, lens, B, Hkv, cap, keep, sinks, recent, lens_out, kept});
  const rf_status s = launch_status();
  if (s != RF_OK) return s;
  return launch_after(evict_copy_kernel, (unsigned)(blocks * 2 * B * Hkv), COPY_THREADS, 0, st,
                      static_cast<const uint4*>(k), static_cast<const uint4*>(v), weight, kept,
                      B * Hkv, cap, (uint32_t)chunks, keep, cap_out, (int)blocks,
                      static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), weight_out);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
