// What the kernels of attention over a paged cache share: the plan of a step, and
// which blocks of keys a tile of query rows visits.
//
// Requests of few query rows per key head (new tokens times the heads that share it;
// PagedShape::limit) run on the streaming kernel (paged_decode.cu), 16 rows at a time;
// the others on CTA pairs (paged_prefill.cu), 256 rows at a time.  Both take their work
// from lists that paged_plan.cu makes once per step from the lengths on the device:
//   units    of the streaming kernel: 16 rows and a piece of their keys;
//   ranges   of the pair kernel: all 256-key blocks of all tiles, one after the other,
//            in a range per cluster and round; those of the last round are cut wherever an
//            equal share for all clusters falls, inside a tile too.
#pragma once

#include "cache_common.cuh"

namespace rf {

constexpr int kPagedRows = 64;          // query rows per key head of the streaming kernel at most
constexpr int kPagedManyRows = 32;      // and in a large call, for each tile of the pair kernel
constexpr int kPagedTileRows = 16;
constexpr int kPagedBlock = 256;        // keys of the pair kernel's blocks
constexpr int kPagedPairRows = 256;
constexpr int kPagedSlotFloats = kPagedPairRows * (128 + 2);   // a partial state: O, m, l
constexpr int kPagedRounds = 16;
constexpr int kPagedSinks = 64;         // keys of the pair kernel's copies at most
constexpr int kPagedFewSteps = 16;      // steps of 64 keys per CTA of a small call of the streaming kernel

// The sizes that a plan and the calls over it share.
struct PagedShape {
  int B, T, H, Hkv, max_new, max_len, window, sinks;
  int limit, few;                       // set by divide()
  __host__ __device__ int G() const { return H / Hkv; }
  // query heads of a tile, and positions of it
  __host__ __device__ int packed() const {
    const int g = G();
    return g % 8 == 0 ? 8 : g % 4 == 0 ? 4 : g % 2 == 0 ? 2 : 1;
  }
  __host__ __device__ int positions() const { return kPagedPairRows / packed(); }
  __host__ __device__ int positions_log2() const {
    const int p = packed();
    return p == 8 ? 5 : p == 4 ? 6 : p == 2 ? 7 : 8;
  }
  // Which kernels a call takes, by its sizes alone.  It is small (few) if its requests are
  // all of up to kPagedRows rows and the streaming kernel's units make about one wave, whatever
  // the lengths: that kernel alone then, a CTA per unit, in one launch.  A large call's
  // requests go to the pair kernel where that reads the keys less than half as often: 16 rows
  // a time here, there packed() heads and any of so few positions (24 requests of 8000 keys,
  // 32/8 heads, 40 rows: 162 us instead of 283, of 40 keys 20 instead of 18; 32 rows: 162
  // instead of 203 and 20 instead of 18, but 38 instead of 33 where 64 requests have 100 keys).
  __host__ __device__ void divide(int sms) {
    limit = kPagedRows;
    const long long units = (long long)B * tiles() * Hkv;
    const long long steps = units * (((long long)max_len + 4 * kDecodeTile - 1) / (4 * kDecodeTile));
    few = !some_pairs() && steps <= kPagedFewSteps * 2ll * sms;
    if (!few && kPagedManyRows * (G() / packed()) < kPagedRows) limit = kPagedManyRows * (G() / packed());
  }
  __host__ __device__ bool some_pairs() const { return (long long)max_new * G() > limit; }
  // of the streaming kernel: 16-row tiles per request at most
  __host__ __device__ int tiles() const {
    const long long rows = (long long)max_new * G();
    return (int)((rows < limit ? rows : limit) + kPagedTileRows - 1) / kPagedTileRows;
  }
  __host__ __device__ int unit_rows() const {
    const long long rows = (long long)max_new * G();
    return rows < kPagedTileRows ? (int)rows : kPagedTileRows;
  }
};

// Words of a plan's head.
enum { kPlanMark, kPlanUnits, kPlanRanges, kPlanClusters, kPlanLast, kPlanJoins, kPlanMerges, kPlanQueue, kPlanFlag, kPlanDone, kPlanWords = 64 };

// Where the parts of a plan lie, in bytes from its start.
struct PagedLayout {
  size_t seqs, before, ranges, joins, units, merges, counters, unit_ml, unit_acc, slots, bytes;
  int unit_cap, state_cap, range_cap, merge_cap, slot_cap;
  uint32_t mark;                        // of the sizes: a plan of others is refused on the device
};

// One request as the plan found it.
struct PagedSeq {
  int start, n, len, pair;              // first row, rows, keys with the new ones, on the pair kernel
};
struct PagedUnit {
  int b, tile, step0, step1;            // request, 16-row tile, steps of 64 keys
  int first, pieces;                    // unit of the tile's first piece, pieces
  int start, n, len;                    // the request, as in PagedSeq
  int state;                            // place of its state, with several pieces
  int pad[2];
};
struct PagedRange {
  int b, item, block, count;            // the first block's request, item and number in it; blocks
};
// A tile that cuts divide: its first part is the state slot0, the others are slots
// 2 rho, 2 rho + 2 .. (rho: the range of the second part, of the last round's)
struct PagedJoin {
  int b, start, rows, len;              // the request
  int head, kvh, row0;                  // first query head, key head, first new token of the tile
  int parts, slot0, rho;
  int pad[6];
};

struct PagedView {
  PagedShape s;
  int* head;
  const PagedSeq* seqs;
  const PagedRange* ranges;
  const PagedJoin* joins;
  const PagedUnit* units;
  const int* merges;                    // first units of the 16-row tiles in several pieces
  int* counters;                        // pieces of a small call's tiles that are done
  float2* unit_ml;                      // [state][Hkv][unit_rows]
  float* unit_acc;                      // [state][Hkv][unit_rows][128]
  float* slots;
  int unit_cap, state_cap, range_cap, merge_cap, slot_cap;
  uint32_t mark;
  int G, packed, P_log2, groups, key_groups;   // heads per key head and per tile; positions of a
                                        // tile; head groups in all and per key head
};

// The visible keys of a request's rows as tiles of 16: sinks' tiles first, then those
// from the window's first key on.
struct PagedTiles {
  int sink_tiles, lo_tile, tiles;       // key tile of t: t < sink_tiles ? t : t - sink_tiles + lo_tile
  __host__ __device__ PagedTiles(int n, int len, int window, int sinks) {
    const int lo = window > 0 ? (len - n - window + 1 > 0 ? len - n - window + 1 : 0) : 0;
    lo_tile = lo / kDecodeTile;
    const int ns = sinks < lo_tile * kDecodeTile ? sinks : lo_tile * kDecodeTile;
    sink_tiles = (ns + kDecodeTile - 1) / kDecodeTile;
    tiles = sink_tiles + (len + kDecodeTile - 1) / kDecodeTile - lo_tile;
  }
  __host__ __device__ int steps() const { return (tiles + 3) / 4; }
};

// The tiles of one head group of a request on the pair kernel: tile i holds positions
// p0 + i P .. , P = 256 / heads; it visits the window's blocks [lb, hb) and up to SB
// blocks of sinks below them.  Where the lowest window block begins with as many keys that
// no row of the tile sees as the sinks take (in 64s), the sinks go in their place: 4 sinks
// would else cost a block of their own.
struct PagedBlocks {
  int n, p0, log2, window, SB, S64;     // P = 2^log2
  __host__ __device__ PagedBlocks(int n_, int len, int log2_, int window_, int sinks)
      : n(n_), p0(len - n_), log2(log2_), window(window_),
        SB(window_ > 0 ? (int)(((long long)sinks + kPagedBlock - 1) / kPagedBlock) : 0),
        S64(window_ > 0 ? (sinks + kPagedSinks - 1) / kPagedSinks * kPagedSinks : 0) {}
  __host__ __device__ int tiles() const { return (n + (1 << log2) - 1) >> log2; }
  __host__ __device__ int end(int i) const { return (i + 1) << log2 < n ? (i + 1) << log2 : n; }
  __host__ __device__ int hb(int i) const {
    const int x = p0 + end(i);
    return x <= kPagedBlock ? 1 : (x + kPagedBlock - 1) / kPagedBlock;
  }
  __host__ __device__ int lo(int i) const { return p0 + (i << log2) - window + 1; }
  __host__ __device__ int lb(int i) const { return window > 0 && lo(i) > 0 ? lo(i) / kPagedBlock : 0; }
  __host__ __device__ bool folds(int i) const {
    return S64 > 0 && lo(i) >= kPagedBlock && lo(i) % kPagedBlock >= S64;
  }
  __host__ __device__ int sink_blocks(int i) const {
    const int l = lb(i);
    return folds(i) ? 0 : SB < l ? SB : l;
  }
  __host__ __device__ int blocks(int i) const { return hb(i) - lb(i) + sink_blocks(i); }

  // blocks of tiles 0 .. m - 1
  __host__ __device__ long long before(int m) const {
    if (m <= 0) return 0;
    long long sum = 0;
    if (m == tiles()) {                 // the last one may hold fewer positions
      --m;
      sum = blocks(m);
    }
    const long long P = 1ll << log2;
    const int r = 8 - log2;             // 256 / P = 2^r tiles to a block
    static_assert(kPagedBlock == 256, "as in r");
    // ends at or below 0 count one block; then ceil((p0 + (i + 1) P) / 256)
    long long s = p0 < 0 ? -(long long)p0 >> log2 : 0;
    if (s > m) s = m;
    const long long first = p0 + (s << log2);                   // above -P
    const long long u0 = first > 0 ? (first + P - 1) >> log2 : 0;
    sum += s + up(u0 + (m - s), r) - up(u0, r);
    if (window > 0) {                   // less the blocks below the window that no sink keeps
      long long c = (long long)p0 - window + 1 - (long long)kPagedBlock * SB;
      const long long k = c < 0 ? (-c + P - 1) >> log2 : 0;
      if (k < m) {
        c = (c + (k << log2)) >> log2;
        sum -= down(c + (m - k), r) - down(c, r);
      }
      if (S64 > 0 && S64 < kPagedBlock) {   // and a block for each tile that folds its sinks in
        const long long c1 = (long long)p0 - window + 1;
        const long long k1 = c1 < kPagedBlock ? (kPagedBlock - c1 + P - 1) >> log2 : 0;
        if (k1 < m) {
          const long long turns = (m - k1) >> r, rest = (m - k1) & ((1 << r) - 1);
          int all = 0, some = 0;
          for (int j = 0; j < 1 << r; ++j) {
            const bool is = ((c1 + ((k1 + j) << log2)) & (kPagedBlock - 1)) >= S64;
            all += is;
            some += is && j < rest;
          }
          sum -= turns * all + some;
        }
      }
    }
    return sum;
  }
  // sum of ceil(k / 2^r) for k = 1 .. x, of floor(k / 2^r) for k = 0 .. x - 1
  static __host__ __device__ long long up(long long x, int r) {
    const long long q = x >> r;
    return (q * (q + 1) << r) / 2 + (x - (q << r)) * (q + 1);
  }
  static __host__ __device__ long long down(long long x, int r) {
    const long long q = x >> r;
    return (q * (q - 1) << r) / 2 + (x - (q << r)) * q;
  }
};

// false where the device cannot be queried
bool paged_layout(const PagedShape& s, PagedLayout* l);
inline PagedView paged_view(const PagedShape& s, const PagedLayout& l, void* plan) {
  uint8_t* p = static_cast<uint8_t*>(plan);
  PagedView v;
  v.s = s;
  v.head = reinterpret_cast<int*>(p);
  v.seqs = reinterpret_cast<const PagedSeq*>(p + l.seqs);
  v.ranges = reinterpret_cast<const PagedRange*>(p + l.ranges);
  v.joins = reinterpret_cast<const PagedJoin*>(p + l.joins);
  v.units = reinterpret_cast<const PagedUnit*>(p + l.units);
  v.counters = reinterpret_cast<int*>(p + l.counters);
  v.unit_ml = reinterpret_cast<float2*>(p + l.unit_ml);
  v.unit_acc = reinterpret_cast<float*>(p + l.unit_acc);
  v.slots = reinterpret_cast<float*>(p + l.slots);
  v.merges = reinterpret_cast<const int*>(p + l.merges);
  v.unit_cap = l.unit_cap, v.state_cap = l.state_cap, v.range_cap = l.range_cap, v.merge_cap = l.merge_cap, v.slot_cap = l.slot_cap;
  v.mark = l.mark;
  v.G = s.G(), v.packed = s.packed(), v.P_log2 = s.positions_log2();
  v.key_groups = v.G / v.packed, v.groups = s.Hkv * v.key_groups;
  return v;
}

// The arguments of attention over a plan.
struct PagedAttn {
  PagedView v;
  const uint8_t *q, *kp, *vp;           // [T, H, 128], [pages, Hkv, page, 128] of a 16-bit type
  const int32_t* table;                 // [B, width]
  int pages, page_log2, width;
  float scale_log2;
  uint8_t* out;                         // [T, H, 128]
  float* lse;                           // [T, H] or null
};

// slots: of the new tokens, or null where every request has its place
rf_status launch_paged_plan(const int32_t* starts, const int32_t* lens, const int32_t* slots, const PagedShape& s,
                            void* plan, cudaStream_t st);
rf_status launch_paged_decode(const PagedAttn& a, int dtype, cudaStream_t st);
rf_status launch_paged_prefill(const PagedAttn& a, int dtype, cudaStream_t st);
rf_status launch_paged_finish(const PagedAttn& a, int dtype, cudaStream_t st);
int paged_pairs();                      // clusters of the pair kernel on the current device; 0: none

}  // namespace rf
