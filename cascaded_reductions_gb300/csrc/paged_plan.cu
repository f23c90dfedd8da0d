// The plan of a step over a paged cache: which CTA reads which keys, made on the
// device from the step's lengths, once for all layers.
//
// A table is made for the longest request that may come and the lengths are known to
// the device alone, so a grid of CTAs by the largest sizes would mostly be idle (64
// requests behind a table of 131072 keys: 87 000 CTAs).  One CTA sums up the work
// instead and deals it out:
//  * the streaming kernel's rows, in pieces of equal length: one wave of two CTAs per SM
//    where the call is small, of 6 to 24 steps of 64 keys, or longer ones, from a queue
//    where it is large (17 requests with 4 drafted tokens 67 us, 40 requests of 500 to
//    3930 keys 64; with pieces of 12 steps whatever the lengths 73 and 74);
//  * the pair kernel's blocks, counted in closed form per request, cut into ranges.
//    Tiles of one key head read the same keys, so ranges that run at the same time
//    should lie close together: with more keys than the L2 cache holds, the
//    blocks are dealt out in rounds (4 x 32 key heads of 8192 keys, 1705 -> 1605 us).  Ranges
//    of the rounds before the last end with a tile; each round gives a cluster what it
//    lacks to an equal share so far.

#include <limits.h>

#include "paged.cuh"
#include "tc_common.cuh"

namespace rf {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int MANY_LOW = 6, MANY_HIGH = 24;   // steps of a large call's pieces, as long as
constexpr int MANY_UNITS = 8;           // they are no more than these per CTA on average
constexpr int MAX_RANGES = 2048;
constexpr int WHOLE_BLOCKS = 3;         // of a tile that is never cut
constexpr int ROUND_BLOCKS = 32;        // of a range at least, where there are several rounds
constexpr long long ROUND_KEYS = 98304; // keys of all key heads (512 bytes each) of a round

struct Plan {
  PagedShape s;
  const int32_t *starts, *lens, *places;   // places: the rows' slots, null where every request has its own
  int* head;
  PagedSeq* seqs;
  long long* before;                    // [B + 1]: pair blocks of the requests before
  PagedRange* ranges;
  PagedJoin* joins;
  PagedUnit* units;
  int *merges, *counters;
  int unit_cap, state_cap, range_cap, merge_cap, clusters, slots;   // slots: CTAs of the streaming kernel at once
  uint32_t mark;
  int G, P_log2, groups;                // heads per key head; positions of a tile, head groups of the pair kernel
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// exclusive prefix sum over the CTA; *total gets the sum
__device__ __forceinline__ long long block_scan(long long x, long long* sm, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long s = scan_warp(x, lane);
  if (lane == 31) sm[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const long long p = scan_warp(sm[lane], lane);
    __syncwarp();
    sm[lane] = p;
  }
  __syncthreads();
  const long long r = s - x + (warp > 0 ? sm[warp - 1] : 0);
  *total = sm[WARPS - 1];
  __syncthreads();
  return r;
}

__device__ __forceinline__ int tiles_of(const Plan& a, const PagedSeq& q) {
  return q.pair ? 0 : (q.n * a.G + kPagedTileRows - 1) / kPagedTileRows;
}
__device__ __forceinline__ int steps_of(const PagedShape& s, const PagedSeq& q) {
  const int n = PagedTiles(q.n, q.len, s.window, s.sinks).steps();
  return n > 0 ? n : 1;                 // rows without keys need a CTA all the same
}
__device__ __forceinline__ int pieces_of(int steps, int piece) {
  return (int)(((unsigned)steps + piece - 1) / (unsigned)piece);
}

__global__ void __launch_bounds__(THREADS) plan_kernel(const Plan a) {
  __shared__ long long sm[WARPS], fit[WARPS];
  __shared__ int lengths[WARPS];
  __shared__ int n_joins, n_merges, top_blocks;
  __shared__ int2 cuts[THREADS];
  __shared__ long long firsts[THREADS], starts[MAX_RANGES + 1];
  const PagedShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = a.groups;
  if (tid == 0) top_blocks = 0;
  __syncthreads();
  wait_prerequisite();
  allow_dependents();
  long long steps = 0, blocks = 0, keys = 0;
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const int b = b0 + tid;
    PagedSeq q = {0, 0, 0, 0};
    if (b < s.B && RF_SPAN_OK(b, 2, s.B + 1)) {
      const int first = min(max(a.starts[b], 0), s.T), last = min(max(a.starts[b + 1], first), s.T);
      q.start = first;
      q.n = min(last - first, s.max_new);
      q.len = min(max(a.lens[b], 0), s.max_len);
      // a request that got no pages has its old length: none of its keys is for these rows
      if (a.places != nullptr && q.n > 0 && RF_IDX_OK(first, s.T) && a.places[first] < 0) q.len = 0;
      q.pair = (long long)q.n * a.G > s.limit;
    }
    long long mine = 0, total;
    if (q.pair) {
      const PagedBlocks k(q.n, q.len, a.P_log2, s.window, s.sinks);
      mine = k.before(k.tiles()) * groups;
      atomicMax(&top_blocks, k.blocks(k.tiles() - 1));
    }
    long long at = 0;
    if (a.clusters > 0) {
      at = block_scan(mine, sm, &total);
      if (b < s.B && RF_IDX_OK(b, s.B + 1)) a.before[b] = blocks + at;
      blocks += total;
    }
    if (b < s.B && RF_IDX_OK(b, s.B)) a.seqs[b] = q;
    int2 rows = make_int2(0, 0);        // 16-row tiles, steps
    if (q.n > 0 && !q.pair) rows = make_int2(tiles_of(a, q), steps_of(s, q));
    if (b0 == 0) cuts[tid] = rows;
    block_scan((long long)rows.x * rows.y, sm, &total);
    steps += total;
    if (a.clusters > 0) {
      block_scan(q.pair ? (long long)s.Hkv * min(q.len, s.window > 0 ? s.window + q.n : q.len) : 0, sm, &total);
      keys += total;
    }
  }
  __syncthreads();

  // The streaming kernel's pieces, of one candidate length per warp.  A small call takes
  // the shortest that fits one wave.  A large one takes its pieces from a queue, that of
  // fewest steps by waves times the longest piece; a step's time for each piece's ends.
  const long long ctas = steps * s.Hkv;
  long long piece = max(1ll, (ctas + a.slots - 1) / a.slots);
  const bool few = piece <= kPagedFewSteps;
  {
    const long long most = (long long)MANY_UNITS * a.slots;
    const int low = (int)(few ? piece : max((long long)MANY_LOW, (ctas + most - 1) / most));
    const int p = low + (few ? (low * warp + 15) / 16 : max(0, MANY_HIGH - low) * warp / (WARPS - 1));
    long long units = 0;
    int longest = 0;
    for (int b = lane; b < s.B; b += 32) {
      int2 rows = make_int2(0, 0);
      if (b < THREADS) {
        rows = cuts[b];
      } else {
        const PagedSeq q = a.seqs[b];
        if (q.n > 0 && !q.pair) rows = make_int2(tiles_of(a, q), steps_of(s, q));
      }
      if (rows.x == 0) continue;
      const int np = pieces_of(rows.y, p);
      units += (long long)rows.x * np;
      longest = max(longest, pieces_of(rows.y, np));
    }
    units = warp_sum(units) * s.Hkv;
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      long long cost = few ? p : (units + a.slots - 1) / a.slots * (longest + 1);
      if (few && units > a.slots) cost = LLONG_MAX >> 8;
      fit[warp] = cost << 5 | (WARPS - 1 - warp);     // equal ones: the longer
      lengths[warp] = p;
    }
    __syncthreads();
    long long best = fit[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
    piece = few && best >> 5 == LLONG_MAX >> 8 ? low : lengths[WARPS - 1 - (int)(best & 31)];
  }
  auto pieces = [&](int n) { return pieces_of(n, (int)piece); };
  if (tid == 0) n_joins = n_merges = 0;
  __syncthreads();
  long long counts = 0;                 // units so far << 32 | those with a state
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const int b = b0 + tid;
    PagedSeq q = {0, 0, 0, 1};
    if (b < s.B && RF_IDX_OK(b, s.B)) q = a.seqs[b];
    int nt = 0, ns = 0, np = 0;
    if (q.n > 0 && !q.pair) nt = tiles_of(a, q), ns = steps_of(s, q), np = pieces(ns);
    long long total;
    const long long mine = (long long)nt * np;
    const long long at = counts + block_scan(mine << 32 | (np > 1 ? mine : 0ll), sm, &total);
    // a warp per request writes its units
    cuts[tid] = make_int2(nt * np, np);
    if (nt * np > 0) firsts[tid] = at;
    __syncthreads();
    for (int w = warp; w < THREADS && b0 + w < s.B; w += WARPS) {
      const int count = cuts[w].x, n_p = cuts[w].y;
      if (count == 0) continue;
      const long long u0 = firsts[w] >> 32;
      const int s0 = (int)(firsts[w] & 0xffffffffll);
      const PagedSeq r = a.seqs[b0 + w];
      const int n_s = steps_of(s, r);
      for (int u = lane; u < count; u += 32) {
        const int tile = u / n_p, i = u - tile * n_p;
        if (u0 + u >= a.unit_cap || !RF_IDX_OK(u0 + u, a.unit_cap)) break;
        PagedUnit x;
        x.b = b0 + w;
        x.tile = tile;
        x.step0 = (int)((long long)n_s * i / n_p);
        x.step1 = (int)((long long)n_s * (i + 1) / n_p);
        x.first = (int)(u0 + tile * n_p);
        x.pieces = n_p;
        x.start = r.start, x.n = r.n, x.len = r.len;
        x.state = n_p > 1 ? min(s0 + u, a.state_cap - 1) : 0;
        x.pad[0] = x.pad[1] = 0;
        a.units[u0 + u] = x;
        if (i == 0 && n_p > 1) {
          const int m = atomicAdd(&n_merges, 1);
          if (m < a.merge_cap && RF_IDX_OK(m, a.merge_cap)) a.merges[m] = (int)(u0 + u);
        }
      }
    }
    __syncthreads();
    counts += total;
  }
  const int n_units = (int)min(counts >> 32, (long long)a.unit_cap);
  for (long long i = tid; i < (long long)n_units * s.Hkv; i += THREADS) a.counters[i] = 0;

  // the pair kernel's ranges
  int n_ranges = 0, active = 0, last0 = 0;
  if (blocks > 0 && a.clusters > 0) {
    active = (int)min((long long)a.clusters, blocks);
    // where block w of all lies: its tile's request, item, blocks, and its number in the tile
    auto locate = [&](long long w, PagedRange& r, int& mine) {
      int lo = 0, n = s.B;              // last request with before[b] <= w
      while (n > 1) {
        const int half = n >> 1;
        if (a.before[lo + half] <= w) lo += half;
        n -= half;
      }
      const PagedSeq q = a.seqs[lo];
      const PagedBlocks k(q.n, q.len, a.P_log2, s.window, s.sinks);
      const int tiles = k.tiles();
      const long long all = k.before(tiles);
      long long rel = w - a.before[lo];
      const int group = (int)(rel / all);
      rel -= group * all;               // blocks of the group's tiles before, the last tile first
      int t0 = 0, tn = tiles;           // the last count t of tiles with all - before(tiles - t) <= rel
      while (tn > 1) {
        const int half = tn >> 1;
        if (all - k.before(tiles - (t0 + half)) <= rel) t0 += half;
        tn -= half;
      }
      r.b = lo;
      r.item = group * tiles + t0;
      r.block = (int)(rel - (all - k.before(tiles - t0)));
      r.count = 0;
      mine = k.blocks(tiles - 1 - t0);
      return tiles * a.groups;          // the request's items
    };
    // Range i starts at block w; or, where its tile has at most `whole` blocks, at the end of
    // that tile that is nearer.
    auto start_range = [&](int i, long long w, int whole) {
      PagedRange r;
      int mine;
      const int items = locate(min(w, blocks - 1), r, mine);
      if (w >= blocks) {
        r.block = 0;                    // the range has no block
      } else if (mine <= whole && r.block > 0) {
        const bool up = 2 * r.block >= mine;
        w += up ? mine - r.block : -r.block;
        r.block = 0;
        if (up && ++r.item == items) {
          const int b = r.b;
          r.item = 0;
          while (++r.b < s.B && !a.seqs[r.b].pair) {
          }
          if (r.b == s.B) r.b = b;      // behind the last block
        }
      }
      starts[i] = w;
      if (RF_IDX_OK(i, a.range_cap)) a.ranges[i] = r;
    };
    // rounds of ranges that are long beside the longest tile, as they end with one
    const long long least = max(ROUND_BLOCKS, 2 * top_blocks);
    const long long rounds = max(1ll, min(min((keys + ROUND_KEYS - 1) / ROUND_KEYS, blocks / (active * least)),
                                          (long long)(a.range_cap / active)));
    n_ranges = (int)rounds * active;
    last0 = n_ranges - active;
    // A round gives a cluster what it lacks to its share of all rounds so far, so that what
    // one range has too many or too few by its tiles' ends the next one takes back.  The
    // share of a round is twice the longest tile, so no range lacks all of it.
    long long given = 0, first = 0, total;
    for (int k = 0; k < (int)rounds; ++k) {
      const long long goal = blocks / rounds * (k + 1) + blocks % rounds * (k + 1) / rounds;
      const long long lacks =
          tid < active ? max(0ll, goal * (tid + 1) / active - goal * tid / active - given) : 0;
      const long long at = block_scan(lacks, sm, &total);
      const bool last = k + 1 == (int)rounds;
      if (tid > 0 && tid < active)
        start_range(k * active + tid, first + (total > 0 ? (goal - first) * at / total : 0),
                    last ? WHOLE_BLOCKS : 0x7fffffff);
      if (tid == 0 && k == 0) start_range(0, 0, 0);
      if (tid == active && !last) start_range((k + 1) * active, goal, 0x7fffffff);
      __syncthreads();
      if (last) break;
      if (tid < active) given += starts[k * active + tid + 1] - starts[k * active + tid];
      first = starts[(k + 1) * active];
    }
    if (tid == 0) starts[n_ranges] = blocks;
    __syncthreads();
    for (int i = tid; i < n_ranges; i += THREADS)
      if (RF_IDX_OK(i, a.range_cap)) a.ranges[i].count = (int)(starts[i + 1] - starts[i]);
  }
  __syncthreads();
  // the tiles that a range's start cuts for the first time
  for (int i = last0 + 1 + tid; i < n_ranges; i += THREADS) {
    if (!RF_SPAN_OK(i - 1, 2, a.range_cap)) break;
    const PagedRange r = a.ranges[i], before = a.ranges[i - 1];
    const bool same = before.b == r.b && before.item == r.item;
    if (r.block == 0 || (same && before.block > 0)) continue;
    PagedJoin x = {};
    x.parts = 2;
    while (i + x.parts - 1 < n_ranges && RF_IDX_OK(i + x.parts - 1, a.range_cap)) {
      const PagedRange y = a.ranges[i + x.parts - 1];
      if (y.b != r.b || y.item != r.item || y.block == 0) break;
      ++x.parts;
    }
    const PagedSeq q = a.seqs[r.b];
    const int tiles = (q.n + (1 << a.P_log2) - 1) >> a.P_log2, group = r.item / tiles;
    x.b = r.b, x.start = q.start, x.rows = q.n, x.len = q.len;
    x.head = group * s.packed();
    x.kvh = x.head / a.G;
    x.row0 = (tiles - 1 - (r.item - group * tiles)) << a.P_log2;
    x.slot0 = 2 * (i - 1 - last0) + (same ? 0 : 1);
    x.rho = i - last0;
    const int at = atomicAdd(&n_joins, 1);
    if (RF_IDX_OK(at, a.range_cap)) a.joins[at] = x;
  }
  __syncthreads();
  if (tid < kPlanWords) {
    int x = 0;
    if (tid == kPlanJoins) x = n_joins;
    if (tid == kPlanMerges) x = min(n_merges, a.merge_cap);
    if (tid == kPlanMark) x = (int)a.mark;
    if (tid == kPlanUnits) x = n_units;
    if (tid == kPlanRanges) x = n_ranges;
    if (tid == kPlanClusters) x = active;
    if (tid == kPlanLast) x = last0;
    a.head[tid] = x;
  }
}

}  // namespace

bool paged_layout(const PagedShape& s, PagedLayout* l) {
  const int sms = tc::sm_count();
  if (sms <= 0) return false;
  const auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // units: a piece per tile, and what cutting adds (fewer than the pieces that the total makes)
  const long long tiles = (long long)s.B * s.tiles();
  const long long steps = ((long long)s.max_len + 4 * kDecodeTile - 1) / (4 * kDecodeTile) + 2;
  long long cut = (2ll * sms * MANY_UNITS + s.Hkv - 1) / s.Hkv;
  if (cut > tiles * (steps - 1)) cut = tiles * (steps - 1);
  l->unit_cap = (int)(tiles + cut);
  // states of the units of divided tiles alone: each of those tiles has one of the cuts at least
  l->state_cap = (int)(tiles < cut ? tiles + cut : 2 * cut);
  l->merge_cap = (int)tiles;
  l->range_cap = l->slot_cap = 0;
  if (s.some_pairs()) {
    // blocks at most, and the rounds that they make
    const long long groups = (long long)s.Hkv * (s.G() / s.packed());
    const long long pair_tiles = (long long)s.T / s.positions() + s.B;
    const long long blocks = groups * pair_tiles * ((long long)s.max_len / kPagedBlock + 2);
    const int pairs = sms / 2;
    long long rounds = blocks / ((long long)pairs * ROUND_BLOCKS);
    rounds = rounds < 1 ? 1 : rounds > kPagedRounds ? kPagedRounds : rounds;
    l->range_cap = (int)(rounds * pairs < MAX_RANGES ? rounds * pairs : MAX_RANGES);
    l->slot_cap = 2 * pairs;            // two parts of tiles per range of the last round
  }
  size_t at = align(kPlanWords * sizeof(int));
  const auto take = [&](size_t bytes) {
    const size_t p = at;
    at = align(at + bytes);
    return p;
  };
  const size_t rows = (size_t)l->state_cap * s.Hkv * s.unit_rows();
  l->seqs = take((size_t)s.B * sizeof(PagedSeq));
  l->before = take(((size_t)s.B + 1) * sizeof(long long));
  l->ranges = take((size_t)l->range_cap * sizeof(PagedRange));
  l->joins = take((size_t)l->range_cap * sizeof(PagedJoin));
  l->units = take((size_t)l->unit_cap * sizeof(PagedUnit));
  l->merges = take((size_t)l->merge_cap * sizeof(int));
  l->counters = take((size_t)l->unit_cap * s.Hkv * sizeof(int));
  l->unit_ml = take(rows * sizeof(float2));
  l->unit_acc = take(rows * 128 * sizeof(float));
  l->slots = take((size_t)l->slot_cap * kPagedSlotFloats * sizeof(float));
  l->bytes = at;
  uint32_t h = 0x9e3779b9u;             // FNV-like mixing of the sizes
  for (const int x : {s.B, s.T, s.H, s.Hkv, s.max_new, s.max_len, s.window, s.sinks, s.limit, sms})
    h = (h ^ (uint32_t)x) * 0x01000193u + 0x7f4a7c15u;
  l->mark = h;
  return true;
}

rf_status launch_paged_plan(const int32_t* starts, const int32_t* lens, const int32_t* slots, const PagedShape& s,
                            void* plan, cudaStream_t st) {
  PagedLayout l;
  const int sms = tc::sm_count();
  if (sms <= 0 || !paged_layout(s, &l)) return RF_ERR_CUDA;
  uint8_t* p = static_cast<uint8_t*>(plan);
  Plan a = {};
  a.s = s;
  a.starts = starts, a.lens = lens, a.places = slots;
  a.head = reinterpret_cast<int*>(p);
  a.seqs = reinterpret_cast<PagedSeq*>(p + l.seqs);
  a.before = reinterpret_cast<long long*>(p + l.before);
  a.ranges = reinterpret_cast<PagedRange*>(p + l.ranges);
  a.joins = reinterpret_cast<PagedJoin*>(p + l.joins);
  a.units = reinterpret_cast<PagedUnit*>(p + l.units);
  a.merges = reinterpret_cast<int*>(p + l.merges);
  a.counters = reinterpret_cast<int*>(p + l.counters);
  a.unit_cap = l.unit_cap, a.state_cap = l.state_cap, a.range_cap = l.range_cap, a.merge_cap = l.merge_cap;
  a.clusters = 0;
  if (s.some_pairs()) {
    a.clusters = paged_pairs();
    if (a.clusters <= 0) return RF_ERR_UNSUPPORTED;
    if (a.clusters > sms / 2) a.clusters = sms / 2;
  }
  a.slots = 2 * sms;
  a.G = s.G(), a.P_log2 = s.positions_log2(), a.groups = s.Hkv * (s.G() / s.packed());
  a.mark = l.mark;
  return launch_after(plan_kernel, 1, THREADS, 0, st, a);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
