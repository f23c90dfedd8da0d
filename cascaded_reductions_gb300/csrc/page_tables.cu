// Pages for the new tokens of a ragged batch of requests, and where each token
// goes: one launch per step of a serving loop, from lengths on the device.
//
// Mathematics: three prefix sums over the requests (new tokens, pages that ended
// requests give back, pages that the others need).  Page x of those needed is the
// x-th from the top of the stack of free pages, on which the pages given back lie
// above the ones that were free before; a request gets its pages if those needed up
// to it are there.  Token t belongs to the last request whose first token is at or
// before t.
//
// What bounds it: latency.  A step moves kilobytes (256 requests, 25 prompt chunks:
// 0.9 MB), and what it waits for are the launch, one read of the lengths, the sums and
// one read of a page number.  So it is one cluster: each of its CTAs makes the prefix sums
// for itself in shared memory, and then pages and tokens are dealt out to all threads,
// each of which finds its request by bisection.  Nothing that one thread writes is read
// by another (a page just given back is read from the ended request's table row), but for
// what the call may overwrite in place: the lengths and the number of free pages, which are
// written after a barrier of the cluster behind every read.  Eight SMs are few for a hundred
// thousand tokens: from MANY_TOKENS on the cluster places each request's first token only,
// and a kernel on all SMs that begins beside its end the others (256 requests, 102400
// tokens: 9.7 us, by the cluster alone 18.9; 1 request 2.9 us).

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace rf {
namespace {

struct Tables {
  const int32_t *lens, *news;
  int32_t *table, *stack;
  const int32_t* n_free;
  int32_t *starts, *positions, *slots, *lens_out, *n_free_out;
  int B, width, P, page, T;
  int page_log2;                             // -1: the page is no power of two
  bool firsts;                               // only each request's first token is placed
};

constexpr int MANY_TOKENS = 16384;

// pos / page
__device__ __forceinline__ int page_index(const Tables& a, int pos) {
  return a.page_log2 >= 0 ? pos >> a.page_log2 : pos / a.page;
}

constexpr int WARPS_MAX = 32;

// inclusive prefix sums over the CTA of two values per thread, with their totals
struct Sums {
  long long a[WARPS_MAX + 1], b[WARPS_MAX + 1];
};

// last i of n ascending values with v[i] <= x (v[0] = 0 <= x)
__device__ __forceinline__ int find(const int* v, int n, int x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (v[lo + half] <= x) lo += half;
    n -= half;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) page_tables_kernel(const Tables a) {
  extern __shared__ int smem[];              // 16 bytes per request
  __shared__ Sums sums;
  __shared__ int took_all;
  const int B = a.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  int* start = smem;                         // first new token, per request
  int* need0 = smem + B;                     // pages needed before it
  int* give0 = smem + 2 * B;                 // pages given back before it
  int* len0 = smem + 3 * B;                  // its length, or -1 - length where it gets nothing
  wait_prerequisite();
  allow_dependents();
  if (tid == 0) took_all = 0;
  const int nfree = min(max(a.n_free[0], 0), a.P);
  const int held_most = a.width;

  long long tokens = 0, moved = 0;           // of the requests so far; moved: given << 32 | needed
  for (int b0 = 0; b0 < B; b0 += (int)blockDim.x) {
    const int b = b0 + tid;
    int len = 0, now = 0;
    if (b < B && RF_IDX_OK(b, a.B)) {
      len = max(a.lens[b], 0);
      now = a.news[b];
    }
    const int held = min((int)(((long long)len + a.page - 1) / a.page), held_most);
    const long long total = ((long long)len + max(now, 0) + a.page - 1) / a.page;
    const bool fits = total <= a.width && now >= 0;
    const long long give = now < 0 ? held : 0, need = fits ? total - held : 0;
    const long long x = max(now, 0), y = give << 32 | need;
    const long long sx = scan_warp(x, lane), sy = scan_warp(y, lane);
    if (lane == 31) {
      sums.a[warp] = sx;
      sums.b[warp] = sy;
    }
    __syncthreads();
    if (warp == 0) {
      const long long p = scan_warp(lane < warps ? sums.a[lane] : 0, lane);
      const long long q = scan_warp(lane < warps ? sums.b[lane] : 0, lane);
      __syncwarp();
      sums.a[lane + 1] = p;                  // [w + 1]: of warps 0 .. w
      sums.b[lane + 1] = q;
      if (lane == 0) sums.a[0] = sums.b[0] = 0;
    }
    __syncthreads();
    const long long ix = tokens + sums.a[warp] + sx - x, iy = moved + sums.b[warp] + sy - y;
    if (b < B) {
      start[b] = (int)min(ix, 0x7fffffffll);
      need0[b] = (int)(iy & 0xffffffffll);
      give0[b] = (int)(iy >> 32);
      // the pool's top is known after the last chunk: see below
      len0[b] = fits ? len : -1 - len;
    }
    tokens += sums.a[warps];
    moved += sums.b[warps];
    __syncthreads();
  }
  const int given = (int)(moved >> 32), needed = (int)(moved & 0xffffffffll);
  const int top = (int)min((long long)nfree + given, (long long)a.P);
  // requests whose pages are not all there get nothing; of those that get theirs the
  // last one's pages end the ones taken
  for (int b = tid; b < B; b += (int)blockDim.x) {
    const int upto = b + 1 < B ? need0[b + 1] : needed;
    if (upto > need0[b]) {
      if (upto > top)
        len0[b] = -1 - len0[b];
      else
        atomicMax(&took_all, upto);
    }
  }
  const uint32_t ctas = gridDim.x;           // one cluster
  if (ctas > 1)
    tc::cluster_sync();                      // every CTA has read what may be overwritten
  else
    __syncthreads();
  const int took = took_all;
  // counts reach the largest int, past which a step may go: unsigned
  const unsigned first = blockIdx.x * blockDim.x + threadIdx.x, step = ctas * blockDim.x;
  const size_t entries = (size_t)B * a.width;
  (void)entries;                             // read by the checked build only

  auto given_page = [&](int y) -> int {      // the y-th page given back
    const int b = find(give0, B, y);
    const size_t at = (size_t)b * a.width + (y - give0[b]);
    return RF_IDX_OK(at, entries) ? a.table[at] : -1;
  };
  auto page_of = [&](int x) -> int {         // the x-th page taken
    const int i = top - 1 - x;
    if (i >= nfree) return given_page(i - nfree);
    return RF_IDX_OK(i, a.P) ? a.stack[i] : -1;
  };
  auto held_of = [&](int len) { return min((int)(((long long)len + a.page - 1) / a.page), held_most); };

  for (int b = (int)first; b < B; b += (int)step) {
    const int len = len0[b] < 0 ? -1 - len0[b] : len0[b];
    const int end = b + 1 < B ? start[b + 1] : (int)min(tokens, 0x7fffffffll);
    // an ended request gives pages where it has some; it has none of the tokens either way
    const int gave = (b + 1 < B ? give0[b + 1] : given) - give0[b];
    int out = len0[b] < 0 ? len : len + (end - start[b]);
    if (gave > 0) out = 0;
    if (RF_IDX_OK(b, a.B)) a.lens_out[b] = out;
    if (RF_IDX_OK(b + 1, a.B + 1)) a.starts[b + 1] = end;
    if (b == 0) {
      a.starts[0] = 0;
      a.n_free_out[0] = top - took;
    }
  }
  for (unsigned y = first; y < (unsigned)given && y < (unsigned)(a.P - nfree); y += step)
    if (RF_IDX_OK(nfree + y, a.P)) a.stack[nfree + y] = given_page((int)y);
  for (unsigned i = first; i < (unsigned)took; i += step) {
    const int x = (int)i, b = find(need0, B, x);
    const size_t at = (size_t)b * a.width + held_of(len0[b]) + (x - need0[b]);
    if (RF_IDX_OK(at, entries)) a.table[at] = page_of(x);
  }
  if (a.firsts) {
    for (int b = (int)first; b < B; b += (int)step) {
      const int t = start[b], end = b + 1 < B ? start[b + 1] : (int)min(tokens, 0x7fffffffll);
      if (t == end || t >= a.T || !RF_IDX_OK(t, a.T)) continue;
      const int len = len0[b], pos = len < 0 ? -1 - len : len;
      int slot = -1;
      if (len >= 0) {
        const int i = page_index(a, pos), held = held_of(len);
        const size_t at = (size_t)b * a.width + i;
        slot = (i >= held ? page_of(need0[b] + i - held) : RF_IDX_OK(at, entries) ? a.table[at] : -1) * a.page +
               (pos - i * a.page);
      }
      a.positions[t] = pos;
      a.slots[t] = slot;
    }
    return;
  }
  // four tokens per thread, in 16-byte stores
  for (int t0 = 4 * (int)first; t0 < a.T; t0 += 4 * (int)step) {   // below MANY_TOKENS
    int pos[4], slot[4];
    int b = t0 < tokens ? find(start, B, t0) : 0;
    int seen = -1, entry = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + e;
      pos[e] = 0;
      slot[e] = -1;
      if (t >= tokens || t >= a.T) continue;
      while (b + 1 < B && start[b + 1] <= t) {
        ++b;
        seen = -1;
      }
      const int len = len0[b];
      pos[e] = (len < 0 ? -1 - len : len) + (t - start[b]);
      if (len < 0) continue;
      const int i = page_index(a, pos[e]);
      if (i != seen) {
        const int held = held_of(len);
        const size_t at = (size_t)b * a.width + i;
        seen = i;
        entry = i >= held ? page_of(need0[b] + i - held) : RF_IDX_OK(at, entries) ? a.table[at] : -1;
      }
      slot[e] = entry * a.page + (pos[e] - i * a.page);
    }
    if (t0 + 4 <= a.T) {
      if (!RF_SPAN_OK(t0, 4, a.T)) continue;
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (t0 + e >= a.T || !RF_IDX_OK(t0 + e, a.T)) continue;
        a.positions[t0 + e] = pos[e];
        a.slots[t0 + e] = slot[e];
      }
    }
  }
}

// All tokens but the requests' first ones, which are in place and say where the others go;
// behind the last one positions are 0 and slots -1.
__global__ void __launch_bounds__(256) page_slots_kernel(const Tables a) {
  extern __shared__ int start[];             // [B + 1]
  wait_prerequisite();
  allow_dependents();
  for (int b = threadIdx.x; b <= a.B; b += 256) start[b] = RF_IDX_OK(b, a.B + 1) ? a.starts[b] : 0;
  __syncthreads();
  const unsigned tokens = (unsigned)start[a.B], T = (unsigned)a.T;
  // unsigned: T reaches the largest int, past which a step may go
  for (unsigned t0 = 4 * (blockIdx.x * 256 + threadIdx.x); t0 < T; t0 += 4 * 256 * gridDim.x) {
    int b = t0 < tokens ? find(start, a.B, (int)t0) : 0, of = -1, first_pos = 0, seen = -1, entry = 0;
    bool fits = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (t0 + e >= T || !RF_IDX_OK(t0 + e, a.T)) break;
      const int t = (int)(t0 + e);
      int pos = 0, slot = -1;
      if (t0 + e < tokens) {
        while (start[b + 1] <= t) ++b;
        if (start[b] == t) continue;
        if (of != b) {
          of = b, seen = -1;
          first_pos = __ldcg(a.positions + start[b]);
          fits = __ldcg(a.slots + start[b]) >= 0;
        }
        pos = first_pos + (t - start[b]);
        if (fits) {
          const int i = page_index(a, pos);
          const size_t at = (size_t)b * a.width + i;
          if (i != seen) seen = i, entry = RF_IDX_OK(at, (size_t)a.B * a.width) ? a.table[at] : 0;
          slot = entry * a.page + (pos - i * a.page);
        }
      }
      a.positions[t] = pos;
      a.slots[t] = slot;
    }
  }
}

}  // namespace

rf_status launch_page_tables(const int32_t* lens, const int32_t* news, int B, int32_t* table, int width,
                             int32_t* stack, int P, const int32_t* n_free, int page, int T,
                             int32_t* starts, int32_t* positions, int32_t* slots, int32_t* lens_out,
                             int32_t* n_free_out, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const size_t smem = (size_t)B * 16;
  if (smem_attr(page_tables_kernel, (size_t)kMaxTableRequests * 16, done) != RF_OK) return RF_ERR_CUDA;
  Tables a = {lens, news, table, stack, n_free, starts, positions, slots, lens_out, n_free_out,
              B, width, P, page, T, -1, T >= MANY_TOKENS};
  for (int e = 0; e < 31; ++e)
    if ((1 << e) == page) a.page_log2 = e;
  const bool small = B <= 256 && T <= 1024;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = small ? 1 : 8;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(small ? 1 : 8);
  cfg.blockDim = dim3(small ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, page_tables_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return RF_ERR_CUDA;
  }
  if (!a.firsts) return launch_status();
  const int sms = tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  const long long ctas = ((long long)T + 1023) / 1024;
  return launch_after(page_slots_kernel, (unsigned)(ctas < 4ll * sms ? ctas : 4ll * sms), 256,
                      ((size_t)B + 1) * sizeof(int), st, a);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
