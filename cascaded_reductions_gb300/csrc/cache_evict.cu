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
// +0).  The need-th largest is found digit by digit, 11, 11 and 10 bits: one
// histogram over all keys, then two over the few that share its threshold's
// first digit, which are gathered for it (all keys again if there are more
// than 4096; up to 128 of them are ranked by comparing each with each instead,
// which saves 1 of 6.3 us on rows of 97 keys, while 256 would cost 1 us).  The
// compaction needs two sweeps with warp votes: the number kept before a row is
// above_before + min(equal_before, equal_needed),  so ties go to the lowest index
// without a second selection.  Weights are read from memory once and kept in
// shared memory (up to 48 Ki of them; longer rows are read again from L2).  Four
// 8-bit histograms over all keys, one add per
// distinct digit of a warp, took 44 us for 256 rows of 16384, this takes 26 us.
//
// evict_copy_kernel, bound by HBM: each kept row is read and written once.

#include "cache_common.cuh"

namespace rf {
namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_KEYS = 48 * 1024;              // keys that fit in shared memory
constexpr int SEL_BINS = 2048;
constexpr int SEL_RANKED = 128;                  // of those, as many as are compared with each other
constexpr int SEL_LIST = 4096;                   // keys gathered for the second and third digit

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

template <bool IN_SMEM>            // whether every row's keys fit in shared memory
__global__ void __launch_bounds__(SEL_THREADS)
evict_select_kernel(const Evict a) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) uint32_t list[SEL_LIST];
  __shared__ uint32_t hist[SEL_BINS], warp_sum[SEL_WARPS];
  __shared__ uint32_t sh_digit, sh_need, sh_count, sh_listed;
  __shared__ int above[SEL_WARPS], equal[SEL_WARPS];

  wait_prerequisite();
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
  const size_t weights = (size_t)a.B * a.Hkv * a.cap;
  (void)weights;
  auto load = [&](int i) -> uint32_t {
    return RF_IDX_OK(w0 + i, weights) ? order_key(a.weight[w0 + i]) : 0u;
  };
  auto key = [&](int i) -> uint32_t { return IN_SMEM ? keys[i] : load(i); };

  // Adds up hist[] and finds the digit at which the count from the top reaches
  // `need`: what is still needed of that digit's keys, and how many there are.
  auto pick_digit = [&]() {
    __syncthreads();
    // thread t holds the bins 2047 - 2 t and 2046 - 2 t
    const uint32_t hi = hist[SEL_BINS - 1 - 2 * tid], lo = hist[SEL_BINS - 2 - 2 * tid];
    uint32_t upto = hi + lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    uint32_t before = lane < warp ? warp_sum[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    upto += before;
    before = upto - hi - lo;
    const uint32_t want = (uint32_t)need;
    if (before < want && upto >= want) {
      const bool first_bin = before + hi >= want;
      sh_digit = (uint32_t)(SEL_BINS - 1 - 2 * tid) - (first_bin ? 0u : 1u);
      sh_need = want - before - (first_bin ? 0u : hi);
      sh_count = first_bin ? hi : lo;
    }
    __syncthreads();
    need = (int)sh_need;
  };
  auto clear = [&]() {
    hist[tid] = 0;
    hist[tid + SEL_THREADS] = 0;
    __syncthreads();
  };
  static_assert(SEL_BINS == 2 * SEL_THREADS, "two bins per thread");

  uint32_t prefix = 0xffffffffu;                 // no weight's key: none is kept
  if (need > 0) {
    if (tid == 0) sh_listed = 0;
    clear();
    for (int i = tid; i < n; i += SEL_THREADS) {
      const uint32_t k = load(i);
      if (IN_SMEM) keys[i] = k;
      atomicAdd(&hist[k >> 21], 1u);
    }
    pick_digit();
    prefix = sh_digit << 21;
    const bool listed = sh_count <= SEL_LIST;
    if (listed) {
      for (int i = tid; i < n; i += SEL_THREADS) {
        const uint32_t k = key(i);
        if (k >> 21 == prefix >> 21) list[atomicAdd(&sh_listed, 1u)] = k;
      }
    }
    const int m = listed ? (int)sh_count : n;
    if (listed && m <= SEL_RANKED) {
      // few: the key with fewer than `need` greater ones and, with its equals, at least
      // so many; the list is filled up with the lowest key
      if (tid >= m && tid < ((m + 3) & ~3)) list[tid] = 0u;
      __syncthreads();
      if (tid < m) {
        const uint32_t k = list[tid];
        int above_k = 0, equal_k = 0;
#pragma unroll 4
        for (int i = 0; i < m; i += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(&list[i]);
          above_k += (x.x > k) + (x.y > k) + (x.z > k) + (x.w > k);
          equal_k += (x.x == k) + (x.y == k) + (x.z == k) + (x.w == k);
        }
        if (above_k < need && above_k + equal_k >= need) {   // the same for all its equals
          sh_digit = k;
          sh_need = (uint32_t)(need - above_k);
        }
      }
      __syncthreads();
      prefix = sh_digit;
      need = (int)sh_need;
    } else {
      for (int shift = 10; shift >= 0; shift -= 10) {
        const int bits = shift == 10 ? 11 : 10;    // 20 .. 10, then 9 .. 0
        clear();
        for (int i = tid; i < m; i += SEL_THREADS) {
          const uint32_t k = listed ? list[i] : key(i);
          if (k >> (shift + bits) == prefix >> (shift + bits))
            atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
        }
        pick_digit();
        prefix |= sh_digit << shift;
      }
    }
  } else if (IN_SMEM) {
    for (int i = tid; i < n; i += SEL_THREADS) keys[i] = load(i);
  }
  __syncthreads();

  // rows above the threshold are kept, and the first `need` equal to it
  const int per = ((n + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
  const int i_begin = min(n, warp * per), i_end = min(n, i_begin + per);
  int ca = 0, ce = 0;
#pragma unroll 4
  for (int i = i_begin + lane; i < i_end; i += 32) {
    const uint32_t k = key(i);
    ca += k > prefix;
    ce += k == prefix;
  }
  ca = __reduce_add_sync(0xffffffffu, ca);
  ce = __reduce_add_sync(0xffffffffu, ce);
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

constexpr int COPY_THREADS = 128;
constexpr int COPY_UNROLL = 4;

// A thread keeps one 16-byte column c of the rows (one division, at the start)
// and COPY_UNROLL rows in flight; a CTA copies `rows` * COPY_UNROLL consecutive
// kept rows of K or V of one (sequence, key head), rows = 128 / chunks, or 1.
// With the selection, 256 rows of 4096 kept out of up to 16384 (1.09 GB): 187 us;
// eight rows in flight cost occupancy (214 us), 256 threads 188 us, plain
// stores instead of streaming ones 204 us.
__global__ void __launch_bounds__(COPY_THREADS)
evict_copy_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                  const float* __restrict__ weight, const int32_t* kept, int groups,
                  int cap, int chunks, int rows, int keep, int cap_out, int blocks,
                  uint4* __restrict__ k_out, uint4* __restrict__ v_out,
                  float* __restrict__ weight_out) {
  const int part = blockIdx.x % 2;                 // 0: K and the weights, 1: V
  const int block = (int)(blockIdx.x / 2) % blocks;
  const int group = (int)(blockIdx.x / 2) / blocks;
  const uint4* src = part ? v : k;
  uint4* dst = part ? v_out : k_out;
  const int r = min((int)threadIdx.x / chunks, rows);
  const int i0 = block * rows * COPY_UNROLL + r;   // this thread's first kept row
  allow_dependents();
  wait_prerequisite();                             // the kept rows' indices
  if (src == nullptr || r == rows) return;
  const int32_t* idx = kept + (size_t)group * keep;
  int row[COPY_UNROLL];
#pragma unroll
  for (int e = 0; e < COPY_UNROLL; ++e) {
    const int i = i0 + e * rows;
    row[e] = i < keep && RF_IDX_OK((size_t)group * keep + i, (size_t)groups * keep) ? __ldcg(idx + i) : -1;
  }
  const size_t in0 = (size_t)group * cap, out0 = (size_t)group * cap_out;
  for (int c = threadIdx.x - r * chunks; c < chunks; c += COPY_THREADS) {
    uint4 x[COPY_UNROLL];
#pragma unroll
    for (int e = 0; e < COPY_UNROLL; ++e)
      if (row[e] >= 0 && RF_IDX_OK((in0 + row[e]) * chunks + c, (size_t)groups * cap * chunks))
        x[e] = ld_stream_v4(src + (in0 + row[e]) * chunks + c);
#pragma unroll
    for (int e = 0; e < COPY_UNROLL; ++e) {
      const size_t o = out0 + i0 + e * rows;
      if (row[e] >= 0 && RF_IDX_OK(o * chunks + c, (size_t)groups * cap_out * chunks))
        __stcs(dst + o * chunks + c, x[e]);
    }
  }
  if (part == 0 && (int)threadIdx.x == r * chunks) {
#pragma unroll
    for (int e = 0; e < COPY_UNROLL; ++e) {
      const size_t o = out0 + i0 + e * rows;
      if (row[e] >= 0 && RF_IDX_OK(o, (size_t)groups * cap_out) &&
          RF_IDX_OK(in0 + row[e], (size_t)groups * cap))
        weight_out[o] = weight[in0 + row[e]];
    }
  }
}

}  // namespace

rf_status launch_cache_evict(const void* k, const void* v, const float* weight,
                             const int32_t* lens, int B, int Hkv, int cap, int row_bytes, int keep,
                             int sinks, int recent, int cap_out, void* k_out, void* v_out,
                             float* weight_out, int32_t* lens_out, int32_t* kept,
                             cudaStream_t st) {
  const int chunks = row_bytes / 16;
  const int rows = chunks < COPY_THREADS ? COPY_THREADS / chunks : 1;
  const long long blocks = ((long long)keep + rows * COPY_UNROLL - 1) / (rows * COPY_UNROLL);
  if (blocks * 2 * B * Hkv > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  static std::atomic<uint64_t> done{0};
  const Evict e{weight, lens, B, Hkv, cap, keep, sinks, recent, lens_out, kept};
  const bool in_smem = cap <= SEL_KEYS;
  if (in_smem && smem_attr(evict_select_kernel<true>, SEL_KEYS * sizeof(uint32_t), done) != RF_OK)
    return RF_ERR_CUDA;
  const rf_status s = launch_after(in_smem ? evict_select_kernel<true> : evict_select_kernel<false>,
                                   (unsigned)(B * Hkv), SEL_THREADS,
                                   in_smem ? (size_t)cap * sizeof(uint32_t) : 0, st, e);
  if (s != RF_OK) return s;
  return launch_after(evict_copy_kernel, (unsigned)(blocks * 2 * B * Hkv), COPY_THREADS, 0, st,
                      static_cast<const uint4*>(k), static_cast<const uint4*>(v), weight, kept,
                      B * Hkv, cap, chunks, rows, keep, cap_out, (int)blocks,
                      static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), weight_out);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
