// Attention of many new tokens per request over a paged cache: chunks of prompts and
// whole ones, on CTA pairs (the kernel's body is in attn_pair.cuh).
//
// Mathematics: the windowed prefill's cascade, for packed rows of requests that each have
// a length and a number of new tokens of their own, over keys that lie in pages.
//
// What bounds it: the tensor pipe, 4 D flops per pair of row and key.  A tile is 256 query
// rows on one key head: up to 8 of the query heads that share it and 256 / heads adjacent
// positions.  It visits the 256-key blocks that its rows see, last block first.
//
// Pages: a block's pages are copied one by one, a lane of the copying warp each, from a
// map of [pages * Hkv][page][128] whose boxes are a page, or 64 rows of one, by 64
// columns.  Rows behind a request's end must not be read, NaN among them would reach
// every row (0 * NaN); a box has no shorter form, but one that starts above its page
// fills what lies outside with zeros.  So the last page is copied from row m - page on for the m rows in use,
// they end up at the end of the page's place in the block, and the mask counts from
// there.  Pages behind the last, and numbers outside the cache, are copied from
// outside the map: zeros.
//
// Balance: requests differ in length by orders, and a tile's work with its position.
// All blocks of all tiles form one line, cut into ranges of equal sums per cluster
// (paged_plan.cu).  A tile that a cut divides leaves a state per part (O, m and l of 256
// rows, 130 KiB), and paged_finish_kernel joins them; the others are written as they are.
// A warp that copies nothing steps through the items and hands the others their records,
// visible keys of a tile are worked out ahead as bits, and only blocks at an edge look at
// them (4 prompts of up to 8192 tokens 1226 -> 939 us).
//
// Measured: 4 x 32/8 heads of 8192 tokens 1580 us, 1.39 PFLOP/s (the dense cache's
// windowed kernel 1551); 512 tokens behind 32 256 keys 202 us (that kernel 228), 4864
// behind 27 904 1600 us (1627); tensor pipe 55 % on two prompts of up to 4096 tokens,
// the softmax between the two products is what it waits for.
//
// Values that are not finite: as in the windowed prefill a weight of 0 times NaN reaches
// rows that do not see the value.  Rows whose output is not finite are noted, and
// paged_finish_kernel computes their NaN columns again from the visible keys alone.
// Rows of huge scores (pair::huge) come out as NaN and are computed again in the same way.

#include <cuda_fp16.h>

#include "attn_pair.cuh"
#include "paged.cuh"

namespace rf {
namespace {

using pair::BM;
using pair::BN;
using pair::HALF_BYTES;
using pair::HD;
using pair::huge;
static_assert(2 * BM == kPagedPairRows && BN == kPagedBlock && HD == 128, "the plan's sizes");

// The items of a range, one after the other: tiles, or what of a tile the range holds.
struct RangeItem {
  int rho, left;       // range, and its blocks behind this item
  int b, group;        // request, head group
  int j0, n, next;     // first block of the tile, blocks, the block after them (0: no more)
  int slot;            // of the partial state, -1 for a whole tile
  int start, rows, len;           // the request
  int head, kvh, row0;            // first query head, key head, first new token of the tile
  int hb, nw;          // window blocks hb - 1, hb - 2 .. (nw of them), then those of the sinks from 0 on;
                       // with FOLDS the sinks are in the last window block's first places
  static constexpr int FOLDS = 1 << 30;
  __device__ __forceinline__ int windows() const { return nw & ~FOLDS; }
};

// the item from block j on of the tile at row0
__device__ __forceinline__ void place_item(const PagedView& v, bool first, int j, RangeItem& it) {
  const PagedBlocks k(it.rows, it.len, v.P_log2, v.s.window, v.s.sinks);
  const int i = it.row0 >> v.P_log2;
  it.hb = k.hb(i);
  it.nw = it.hb - k.lb(i);
  const int all = it.nw + k.sink_blocks(i);
  if (k.folds(i)) it.nw |= RangeItem::FOLDS;
  it.j0 = j;
  it.n = min(all - j, it.left);
  it.left -= it.n;
  it.next = j + it.n == all ? 0 : j + it.n;
  it.slot = it.n == all ? -1 : 2 * (it.rho - v.head[kPlanLast]) + (first ? 0 : 1);
}
__device__ __forceinline__ void place_group(const PagedView& v, int group, RangeItem& it) {
  it.group = group;
  it.head = group * v.packed;
  it.kvh = group / v.key_groups;
}
__device__ __forceinline__ PagedSeq load_seq(const PagedView& v, int b) {
  PagedSeq q = {0, 0, 0, 1};
  if (RF_IDX_OK(b, v.s.B)) *reinterpret_cast<int4*>(&q) = *reinterpret_cast<const int4*>(v.seqs + b);
  return q;
}
__device__ __forceinline__ void first_item(const PagedView& v, int rho, RangeItem& it) {
  PagedRange r = {0, 0, 0, 0};
  if (RF_IDX_OK(rho, v.range_cap)) *reinterpret_cast<int4*>(&r) = *reinterpret_cast<const int4*>(v.ranges + rho);
  const PagedSeq q = load_seq(v, r.b);
  it.rho = rho, it.left = r.count, it.b = r.b;
  it.start = q.start, it.rows = q.n, it.len = q.len;
  const int tiles = max(1, (q.n + (1 << v.P_log2) - 1) >> v.P_log2), group = r.item / tiles;
  place_group(v, group, it);
  it.row0 = (tiles - 1 - (r.item - group * tiles)) << v.P_log2;      // the last tile first
  place_item(v, true, r.block, it);
}
// the next item of the same range (left > 0)
__device__ __forceinline__ void step_item(const PagedView& v, RangeItem& it) {
  if (it.next == 0) {
    it.row0 -= 1 << v.P_log2;
    if (it.row0 < 0) {
      int group = it.group + 1;
      if (group == v.groups) {
        PagedSeq q;
        do {
          q = load_seq(v, ++it.b);
        } while (!q.pair);
        group = 0;
        it.start = q.start, it.rows = q.n, it.len = q.len;
      }
      place_group(v, group, it);
      it.row0 = (it.rows - 1) >> v.P_log2 << v.P_log2;
    }
  }
  place_item(v, false, it.next, it);
}

template <bool F16_>
struct PagedPrefill {
  static constexpr bool F16 = F16_;
  static constexpr bool CHAINED = true, STAGED = true, ROUNDS = false, REDOES = true;
  static constexpr float M_START = pair::LOWEST;
  using Item = RangeItem;
  struct Pages {
    int kkey, vkey;               // first keys of the lane's copies
    int kid, vid;                 // and their pages' entries, not looked at before the copies
  };
  struct Pending {
    int row, head;
    bool in, full;                // the row is one of the tile's, all 32 of the warp are
  };

  PagedAttn a;
  float scale_log2;

  __device__ __forceinline__ bool item(int t, int cluster, Item& it) const {
    if (t > 0 && it.left > 0) {
      step_item(a.v, it);
      return true;
    }
    if (a.v.head[kPlanMark] != (int)a.v.mark) return false;
    const int clusters = a.v.head[kPlanClusters], ranges = min(a.v.head[kPlanRanges], a.v.range_cap);
    if (cluster >= clusters) return false;
    for (int rho = t == 0 ? cluster : it.rho + clusters; rho < ranges; rho += clusters) {
      first_item(a.v, rho, it);
      if (it.n > 0) return true;                        // a range may have lost its few blocks
    }
    return false;
  }
  // the block of keys that is the item's j-th
  __device__ __forceinline__ int block_of(const Item& it, int j) const {
    const int J = it.j0 + j, nw = it.windows();
    return J < nw ? it.hb - 1 - J : J - nw;
  }
  // keys of the block's first places that are sinks instead
  __device__ __forceinline__ int folded(const Item& it, int j) const {
    return it.nw & Item::FOLDS && it.j0 + j == it.windows() - 1
               ? (a.v.s.sinks + kPagedSinks - 1) / kPagedSinks * kPagedSinks
               : 0;
  }
  __device__ __forceinline__ int page() const { return 1 << a.page_log2; }
  // rows that the last page lacks, and whether the block holds that page
  __device__ __forceinline__ int lacking(const Item& it) const { return -it.len & (page() - 1); }
  __device__ __forceinline__ bool holds_last(const Item& it, int block) const {
    return it.len > 0 && (it.len - 1) / BN == block;
  }
  __device__ __forceinline__ int head_of(int rank, int r) const { return (rank * BM + r) >> a.v.P_log2; }
  __device__ __forceinline__ int row_of(int rank, int r) const {
    return (rank * BM + r) & ((1 << a.v.P_log2) - 1);
  }

  __device__ __forceinline__ uint32_t q_bytes() const { return pair::TILE_BYTES; }
  __device__ __forceinline__ void load_q(uint8_t* dst, const CUtensorMap* map, uint32_t bar, const Item& it,
                                         int rank) const {
    const int row = it.start + it.row0 + row_of(rank, 0), head = it.head + head_of(rank, 0);
    tc::tma_load_3d_pair(dst, map, bar, 0, row, head);
    tc::tma_load_3d_pair(dst + HALF_BYTES, map, bar, 64, row, head);
  }
  // Keys are copied a page at a time, or 64 of a larger page: a half of K is 128 keys in
  // boxes of 64 columns, two of them each, V all 256 in one.
  __device__ __forceinline__ int box_log2() const { return min(a.page_log2, 6); }
  __device__ __forceinline__ int entry(const Item& it, int key) const {
    const int i = key >> a.page_log2;
    const size_t at = (size_t)it.b * a.width + i;
    return i < a.width && RF_IDX_OK(at, (size_t)a.v.s.B * a.width) ? a.table[at] : -1;
  }
  __device__ __forceinline__ Pages pages_of(const Item& it, int j, int rank, int lane) const {
    const int base = block_of(it, j) * BN, fold = folded(it, j), nk = BM >> box_log2();
    Pages p = {0, 0, -1, -1};
    if (lane < 2 * nk) {
      const int at = (rank * nk + (lane >= nk ? lane - nk : lane)) << box_log2();
      p.kkey = at < fold ? at : base + at;
      p.kid = entry(it, p.kkey);
    }
    if (lane < 2 * nk) {
      const int at = lane << box_log2();
      p.vkey = at < fold ? at : base + at;
      p.vid = entry(it, p.vkey);
    }
    return p;
  }
  // coordinates (y, z) of a key with that entry; zeros come from behind the map
  __device__ __forceinline__ void place(const Item& it, int key, int id, int& y, int& z) const {
    const int i = key >> a.page_log2, used = (it.len + page() - 1) >> a.page_log2;
    z = i < used && (unsigned)id < (unsigned)a.pages ? id * a.v.s.Hkv + it.kvh : a.pages * a.v.s.Hkv;
    y = (key & (page() - 1)) - (i == used - 1 ? lacking(it) : 0);
  }
  __device__ __forceinline__ void load_k(uint8_t* dst, const CUtensorMap* map, uint32_t bar, const Item& it,
                                         const Pages& p, int, int lane) const {
    const int nk = BM >> box_log2(), col = lane >= nk, i = lane - col * nk;
    if (lane >= 2 * nk) return;
    int y, z;
    place(it, p.kkey, p.kid, y, z);
    tc::tma_load_3d_pair(dst + col * HALF_BYTES + (i << box_log2()) * 128, map, bar, 64 * col, y, z);
  }
  __device__ __forceinline__ void load_v(uint8_t* dst, const CUtensorMap* map, uint32_t bar, const Item& it,
                                         const Pages& p, int rank, int lane) const {
    if (lane >= BN >> box_log2()) return;
    int y, z;
    place(it, p.vkey, p.vid, y, z);
    tc::tma_load_3d_pair(dst + (lane << box_log2()) * 128, map, bar, rank * 64, y, z);
  }
  __device__ __forceinline__ int keys(const Item&, int) const { return BN; }

  static __device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  }
  // Of a softmax thread: the item's blocks first .. end - 1 hide nothing from its warp, all
  // but those at the tile's own positions, at the window's edge, of the sinks, and one
  // whose last page has moved.
  struct Row {
    int first, end;
    __device__ __forceinline__ bool all(int j) const { return j >= first && j < end; }
  };
  __device__ __forceinline__ int position(const Item& it, int rank, int r) const {
    return it.len - it.rows + it.row0 + row_of(rank, r);
  }
  __device__ __forceinline__ Row row_of_item(const Item& it, int rank, int r, int kh) const {
    const int low = position(it, rank, r & ~31), window = a.v.s.window;
    const int top = (it.hb - 1) * BN + kh * BM;       // first key of the half in the tile's block 0
    int first = max(0, (top + BM - 1 - low + BN - 1) >> 8), end = it.windows();
    static_assert(BN == 256, "the shifts");
    if (lacking(it) != 0 && holds_last(it, it.hb - 1)) first = max(first, 1);
    if (window > 0) end = min(end, ((top - (low + 31 - window + 1)) >> 8) + 1);
    return {first - it.j0, end - it.j0};
  }
  __device__ __forceinline__ void visible(const Item& it, int j, int rank, int r, int kh, uint4& bits) const {
    const int block = block_of(it, j), base = block * BN + kh * BM;
    const int p = position(it, rank, r), window = a.v.s.window;
    const bool moved = holds_last(it, block) && lacking(it) != 0;
    // seen are keys up to hi, from lo on or below cs, counted from base; where the last
    // page moved by d, slots c0 + d .. of its place are keys c - d
    const int hi = min(p, it.len - 1) - base, lo = window > 0 ? p - window + 1 - base : -2 * BN;
    const int cs = a.v.s.sinks - base;
    const int d = moved ? lacking(it) : 0;
    const int c0 = moved ? ((it.len - 1) & ~(page() - 1)) - base : BN;
    // the sinks' places and those of them that hold sinks
    const int fold = folded(it, j) - kh * BM, sunk = a.v.s.sinks - kh * BM;
    uint32_t vis[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t plain = below(hi + 1 - 32 * q) & (~below(lo - 32 * q) | below(cs - 32 * q));
      const uint32_t behind = below(hi + d + 1 - 32 * q) & (~below(lo + d - 32 * q) | below(cs + d - 32 * q));
      vis[q] = (plain & below(c0 - 32 * q)) | (behind & ~below(c0 + d - 32 * q));
      vis[q] = (vis[q] & ~below(fold - 32 * q)) | (below(sunk - 32 * q) & below(fold - 32 * q));
    }
    bits = make_uint4(vis[0], vis[1], vis[2], vis[3]);
  }

  __device__ __forceinline__ bool partial(const Item& it) const { return it.slot >= 0; }
  __device__ __forceinline__ void keep(const Item& it, int rank, int r, int col, const uint32_t (&v)[32],
                                       float m, float lt) const {
    if (!RF_IDX_OK(it.slot, a.v.slot_cap)) return;
    float* slot = a.v.slots + (size_t)it.slot * kPagedSlotFloats;
    const int row = rank * BM + r;
#pragma unroll
    for (int c = 0; c < 32; c += 8) pair::st_global_v8(slot + row * HD + col + c, v + c);
    if (col == 0) {
      slot[kPagedPairRows * HD + row] = m;
      slot[kPagedPairRows * (HD + 1) + row] = lt;
    }
  }
  __device__ __forceinline__ Pending pending(const Item& it, int rank, int r) const {
    const int i = it.row0 + row_of(rank, r);
    return {it.start + i, it.head + head_of(rank, r), i < it.rows, (i | 31) < it.rows};
  }
  __device__ __forceinline__ bool boxed(const Pending& pend) const { return pend.full; }
  __device__ __forceinline__ bool pack(const Pending& pend, int col, const uint32_t (&v)[32], float m, float lt,
                                       uint32_t (&w)[16]) const {
    const float inv = lt == 0.f ? 0.f : 1.f / lt;       // 0: a row that sees nothing
    const uint64_t inv2 = pair::pack_f32x2(inv, inv);
    uint64_t probe = 0ull;                              // NaN if a value is not finite
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint64_t x = pair::mul_f32x2(
          pair::pack_f32x2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), inv2);
      probe = pair::fma_f32x2(x, 0ull, probe);
      float x0, x1;
      pair::unpack_f32x2(x, x0, x1);
      w[c] = pair::pack_16x2<F16>(x0, x1);
    }
    const size_t row = (size_t)pend.row * a.v.s.H + pend.head;
    if (pend.in && RF_IDX_OK(row, (size_t)a.v.s.T * a.v.s.H)) {
      if (a.lse != nullptr && col == 0) a.lse[row] = (m + log2f(lt)) * kLn2;
      if (!pend.full) pair::st_row32(a.out + (row * HD + col) * 2, w, false);
    }
    float p0, p1;
    pair::unpack_f32x2(probe, p0, p1);
    return pend.in && !(p0 == 0.f && p1 == 0.f);
  }
  // called by the warp's first lane, whose row is the boxes' first
  __device__ __forceinline__ void send(const CUtensorMap* map, const uint8_t* box, const Pending& pend) const {
    tc::tma_store_3d(map, box, 0, pend.row, pend.head);
    tc::tma_store_3d(map, box + HALF_BYTES, 64, pend.row, pend.head);
  }
  __device__ __forceinline__ void after(bool any, int, int, int, int) const {
    if (any) atomicOr(a.v.head + kPlanFlag, 1);
  }
};

template <class P>
__global__ void __launch_bounds__(pair::THREADS, 1)
paged_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                  const __grid_constant__ P p) {
  pair::attn_pair_body(tmQ, tmK, tmV, tmV, tmO, p);
}

// ------------------------------------------------------------------ finish --

constexpr int FIN_WARPS = 8, FIN_ROWS = 32, FIN_PARTS = kPagedPairRows / FIN_ROWS;

// Columns of a row that are NaN (bits of `todo`, four per lane), once more from the keys
// that the row sees.  Ends once they are all NaN again; with `whole` only if the sum is NaN too, so
// that *lse2 gets the row's sum and maximum (in log2 units).
template <bool F16>
__device__ __noinline__ float4 redo_row(const PagedAttn& a, const PagedJoin it, int i, int head, uint32_t todo,
                                        bool whole, float4 y, float* lse2, int lane) {
  constexpr int U = 8;                                // keys in flight
  const int p = it.len - it.rows + i, window = a.v.s.window, page = 1 << a.page_log2;
  const int last = min(p, it.len - 1);
  const int lo = window > 0 ? max(0, p - window + 1) : 0, ns = min(a.v.s.sinks, lo);
  const int n = last < 0 ? 0 : min(ns, last + 1) + max(0, last - lo + 1);
  const size_t row = (size_t)(it.start + i) * a.v.s.H + head;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (RF_IDX_OK(row, (size_t)a.v.s.T * a.v.s.H)) x = load_row4<F16>(a.q + row * HD * 2, lane);
  float m = -INFINITY, l = 0.f;
  float4 R = make_float4(0.f, 0.f, 0.f, 0.f);
  bool gone = false;
  for (int t0 = 0; !gone && t0 < n; t0 += U) {
    float s[U], mn = m;
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(t0 + u, n - 1), key = t < ns ? t : t - ns + lo, pi = key >> a.page_log2;
      const size_t e = (size_t)it.b * a.width + pi;
      const int id = pi < a.width && RF_IDX_OK(e, (size_t)a.v.s.B * a.width) ? a.table[e] : -1;
      float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
      v[u] = k;
      if ((unsigned)id < (unsigned)a.pages) {
        const size_t at = (((size_t)id * a.v.s.Hkv + it.kvh) << a.page_log2) + (key & (page - 1));
        if (RF_IDX_OK(at, ((size_t)a.pages * a.v.s.Hkv) << a.page_log2)) {
          k = load_row4<F16>(a.kp + at * HD * 2, lane);
          v[u] = load_row4<F16>(a.vp + at * HD * 2, lane);
        }
      }
      s[u] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, x.w * k.w)));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = t0 + u < n ? group_sum<32>(s[u]) * a.scale_log2 : -INFINITY;
      mn = fmaxf(mn, s[u]);
    }
    const float ref = ref_of(mn), corr = exp2f(m - ref);
    m = mn;
    l *= corr;
    R.x *= corr, R.y *= corr, R.z *= corr, R.w *= corr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u >= n) break;
      const float w = exp2f(s[u] - ref);
      l += w;
      R.x = fmaf(w, v[u].x, R.x);
      R.y = fmaf(w, v[u].y, R.y);
      R.z = fmaf(w, v[u].z, R.z);
      R.w = fmaf(w, v[u].w, R.w);
    }
    const uint32_t now = (R.x != R.x) | (R.y != R.y) << 1 | (R.z != R.z) << 2 | (R.w != R.w) << 3;
    gone = !__any_sync(0xffffffffu, (todo & ~now) != 0 || (whole && l == l));
  }
  if (whole) *lse2 = m + log2f(l);
  if (gone) return y;
  const float inv = l == 0.f ? 0.f : 1.f / l;         // 0: every visible score is -inf
  if (l == 0.f) R = make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(todo & 1u ? R.x * inv : y.x, todo & 2u ? R.y * inv : y.y, todo & 4u ? R.z * inv : y.z,
                     todo & 8u ? R.w * inv : y.w);
}

__device__ __forceinline__ uint32_t nan_of(const float4& y) {
  return (y.x != y.x) | (y.y != y.y) << 1 | (y.z != y.z) << 2 | (y.w != y.w) << 3;
}

// A row of the streaming kernel's tile, whose first piece is u, from the states of its pieces,
// in order; one warp, four columns per lane.
template <bool F16>
__device__ __forceinline__ void merge_row(const PagedAttn& a, const PagedUnit& u, int hk, int r, int lane) {
  constexpr int U = 16;                               // states in flight
  const PagedView& v = a.v;
  const size_t step = (size_t)v.s.Hkv * v.s.unit_rows(), base = u.state * step + (size_t)hk * v.s.unit_rows() + r;
  const size_t states = (size_t)v.state_cap * step;
  (void)states;                                       // read by the checked build only
  float M = -INFINITY, L = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < u.pieces; s0 += U) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < U && s0 + lane < u.pieces && RF_IDX_OK(base + (s0 + lane) * step, states))
      ml = __ldcg(v.unit_ml + base + (s0 + lane) * step);
    float4 o[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const size_t at = base + (s0 + j) * step;
      o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + j < u.pieces && RF_IDX_OK(at, states))
        o[j] = __ldcg(reinterpret_cast<const float4*>(v.unit_acc + at * HD) + lane);
    }
    const float top = fmaxf(M, group_max<32>(ml.x)), c = exp2f(M - ref_of(top));
    M = top;
    L *= c;
    A.x *= c, A.y *= c, A.z *= c, A.w *= c;
    float f = -1.f;                                   // a piece without keys: its accumulator is not read
    if (ml.x != -INFINITY) {
      f = exp2f(ml.x - ref_of(top));
      L = fmaf(f, ml.y, L);
    } else {
      L += ml.y;                                      // 0, or NaN where every score was NaN
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float fj = __shfl_sync(0xffffffffu, f, j);
      if (fj == -1.f) continue;
      A.x = fmaf(fj, o[j].x, A.x);
      A.y = fmaf(fj, o[j].y, A.y);
      A.z = fmaf(fj, o[j].z, A.z);
      A.w = fmaf(fj, o[j].w, A.w);
    }
    // every lane's share of L was rescaled alike; they are added up at the end
  }
  L = group_sum<32>(L);
  const int i = (u.tile * kPagedTileRows + r) / v.G, head = hk * v.G + u.tile * kPagedTileRows + r - i * v.G;
  const size_t row = (size_t)(u.start + i) * v.s.H + head;
  if (!RF_IDX_OK(row, (size_t)v.s.T * v.s.H)) return;
  const float4 y = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(A.x / L, A.y / L, A.z / L, A.w / L);
  *reinterpret_cast<uint2*>(a.out + row * HD * 2 + lane * 8) =
      make_uint2(pair::pack_16x2<F16>(y.x, y.y), pair::pack_16x2<F16>(y.z, y.w));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = (M + log2f(L)) * kLn2;
}

// What the kernels before it left in parts.  Rows of the streaming kernel in several pieces,
// a warp each; then the pair kernel's tiles, a CTA per 32 of a tile's 256 rows, eight to a
// tile: the first ones join the parts of a tile that cuts divide, and where that kernel
// noted a value that is not finite, a range's eight look at its whole tiles.
template <bool F16>
__global__ void __launch_bounds__(FIN_WARPS * 32)
paged_finish_kernel(const __grid_constant__ PagedAttn a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int join = (int)(blockIdx.x / FIN_PARTS), part = (int)(blockIdx.x % FIN_PARTS);
  wait_prerequisite();
  allow_dependents();
  const PagedView& v = a.v;
  const size_t all_rows = (size_t)v.s.T * v.s.H;
  (void)all_rows;                                     // read by the checked build only
  PagedJoin it = {};
  if (join < v.range_cap) {                           // asked for before it is known whether it is one
    const int4* at = reinterpret_cast<const int4*>(v.joins + join);
    int4* to = reinterpret_cast<int4*>(&it);
#pragma unroll
    for (int e = 0; e < 3; ++e) to[e] = at[e];
  }
  if (v.head[kPlanMark] != (int)v.mark) return;
  const int ranges = min(v.head[kPlanRanges], v.range_cap), flag = v.head[kPlanFlag];
  const int P = 1 << v.P_log2;
  {
    const int per = v.s.Hkv * v.s.unit_rows();        // rows of a tile, over the key heads
    const long long rows = (long long)min(v.head[kPlanMerges], v.merge_cap) * per;
    for (long long i = (long long)blockIdx.x * FIN_WARPS + warp; i < rows; i += (long long)gridDim.x * FIN_WARPS) {
      const int m = (int)(i / per), hk = (int)(i - (long long)m * per) / v.s.unit_rows();
      const int r = (int)(i - (long long)m * per) - hk * v.s.unit_rows();
      const int first = RF_IDX_OK(m, v.merge_cap) ? v.merges[m] : 0;
      if (!RF_IDX_OK(first, v.unit_cap)) continue;
      const PagedUnit u = v.units[first];
      if (r < u.n * v.G - u.tile * kPagedTileRows) merge_row<F16>(a, u, hk, r, lane);
    }
  }
  if (join < min(v.head[kPlanJoins], v.range_cap)) {
    constexpr int R = FIN_ROWS / FIN_WARPS;           // rows of a warp
    const int row0 = part * FIN_ROWS + warp * R;      // of the tile
    float M[R], L[R];
    float4 A[R];
    uint32_t again = 0;                               // a bit per row of huge scores
#pragma unroll
    for (int q = 0; q < R; ++q) M[q] = -INFINITY, L[q] = 0.f, A[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < it.parts; x0 += 2) {        // two parts in flight
      float4 o[2][R];
      float m[2][R], l[2][R];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int slot = x0 + x == 0 ? it.slot0 : 2 * (it.rho + x0 + x - 1);
        const bool in = x0 + x < it.parts && RF_IDX_OK(slot, v.slot_cap);
        const float* at = v.slots + (size_t)(in ? slot : 0) * kPagedSlotFloats;
#pragma unroll
        for (int q = 0; q < R; ++q) {
          o[x][q] = __ldcg(reinterpret_cast<const float4*>(at + (row0 + q) * HD) + lane);
          m[x][q] = __ldcg(at + kPagedPairRows * HD + row0 + q);
          l[x][q] = in ? __ldcg(at + kPagedPairRows * (HD + 1) + row0 + q) : 0.f;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int q = 0; q < R; ++q) {
          if (x0 + x < it.parts && huge<F16>(m[x][q])) again |= 1u << q;
          if (l[x][q] == 0.f) continue;               // the part holds nothing that the row sees
          const float top = fmaxf(M[q], m[x][q]), c = exp2f(M[q] - top), f = exp2f(m[x][q] - top);
          M[q] = top;
          L[q] = L[q] * c + l[x][q] * f;
          A[q].x = A[q].x * c + o[x][q].x * f;
          A[q].y = A[q].y * c + o[x][q].y * f;
          A[q].z = A[q].z * c + o[x][q].z * f;
          A[q].w = A[q].w * c + o[x][q].w * f;
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = it.row0 + ((row0 + q) & (P - 1)), head = it.head + ((row0 + q) >> v.P_log2);
      const size_t row = (size_t)(it.start + i) * v.s.H + head;
      if (i >= it.rows || !RF_IDX_OK(row, all_rows)) continue;
      const float inv = L[q] == 0.f ? 0.f : 1.f / L[q];
      float4 y = make_float4(A[q].x * inv, A[q].y * inv, A[q].z * inv, A[q].w * inv);
      float lse2 = M[q] + log2f(L[q]);
      const uint32_t todo = again >> q & 1u ? 15u : nan_of(y);
      if (__any_sync(0xffffffffu, todo != 0)) {
        const bool whole = (again >> q & 1u) != 0 || !(L[q] > 0.f && L[q] < INFINITY);
        y = redo_row<F16>(a, it, i, head, todo, whole, y, &lse2, lane);
      }
      *reinterpret_cast<uint2*>(a.out + row * HD * 2 + lane * 8) =
          make_uint2(pair::pack_16x2<F16>(y.x, y.y), pair::pack_16x2<F16>(y.z, y.w));
      if (lane == 0 && a.lse != nullptr) a.lse[row] = lse2 * kLn2;
    }
  }
  if (flag == 0) return;
  for (int rho = join; rho < ranges; rho += (int)(gridDim.x / FIN_PARTS)) {
    RangeItem whole;
    first_item(v, rho, whole);
    for (;;) {
      it.b = whole.b, it.start = whole.start, it.rows = whole.rows, it.len = whole.len;
      it.head = whole.head, it.kvh = whole.kvh, it.row0 = whole.row0;
      for (int q = warp; whole.slot < 0 && whole.n > 0 && q < FIN_ROWS; q += FIN_WARPS) {
        const int t = part * FIN_ROWS + q, i = it.row0 + (t & (P - 1)), head = it.head + (t >> v.P_log2);
        const size_t row = (size_t)(it.start + i) * v.s.H + head;
        if (i >= it.rows || !RF_IDX_OK(row, all_rows)) continue;
        const float4 y = load_row4<F16>(a.out + row * HD * 2, lane);
        const uint32_t todo = nan_of(y);
        if (!__any_sync(0xffffffffu, todo != 0)) continue;
        // masked scores never entered the lse in place; it is not finite where the sum said nothing
        float lse2 = NAN;
        const bool whole = a.lse != nullptr && !(fabsf(a.lse[row]) < INFINITY);
        const float4 z = redo_row<F16>(a, it, i, head, todo, whole, y, &lse2, lane);
        *reinterpret_cast<uint2*>(a.out + row * HD * 2 + lane * 8) =
            make_uint2(pair::pack_16x2<F16>(z.x, z.y), pair::pack_16x2<F16>(z.z, z.w));
        if (lane == 0 && whole) a.lse[row] = lse2 * kLn2;
      }
      if (whole.left == 0) break;
      step_item(v, whole);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // the last CTA that has looked takes the note away
    if (atomicInc(reinterpret_cast<unsigned*>(v.head) + kPlanDone, gridDim.x - 1) == gridDim.x - 1)
      atomicExch(v.head + kPlanFlag, 0);
  }
}

// a map of [outer][mid][128] 16-bit values with strides in bytes
bool make_map(CUtensorMap* map, bool f16, const void* base, uint64_t mid, uint64_t outer, uint64_t mid_step,
              uint64_t outer_step, uint32_t box_mid, uint32_t box_outer) {
  return tc::make_tmap_3d_16_strided(map, f16, base, HD, mid, outer, mid_step, outer_step, 64, box_mid, box_outer,
                                     CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool F16>
rf_status launch_pairs(const PagedAttn& a, cudaStream_t st) {
  using P = PagedPrefill<F16>;
  auto* kernel = paged_pair_kernel<P>;
  const int pairs = pair::resident_pairs_of<P>(kernel);
  if (pairs <= 0) return RF_ERR_UNSUPPORTED;
  const PagedShape& s = a.v.s;
  const uint64_t row = (uint64_t)HD * 2, page = 1ull << a.page_log2;
  const uint32_t box = s.positions() < BM ? s.positions() : BM;
  const uint32_t rows = (uint32_t)(page < 64 ? page : 64);
  CUtensorMap tq, tk, tv, to;
  if (!make_map(&tq, F16, a.q, s.T, s.H, row * s.H, row, box, BM / box) ||
      !make_map(&tk, F16, a.kp, page, (uint64_t)a.pages * s.Hkv, row, row * page,
                rows, 1) ||
      !make_map(&tv, F16, a.vp, page, (uint64_t)a.pages * s.Hkv, row, row * page, rows, 1) ||
      !make_map(&to, F16, a.out, s.T, s.H, row * s.H, row, 32, 1))
    return RF_ERR_CUDA;
  P p = {};
  p.a = a;
  p.scale_log2 = a.scale_log2;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair::pair_config(attr, 2u * (unsigned)pairs, st);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, to, p) != cudaSuccess) {
    cudaGetLastError();
    return RF_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

int paged_pairs() {
  // both types have the same registers and shared memory; each launch checks its own
  return pair::resident_pairs_of<PagedPrefill<false>>(paged_pair_kernel<PagedPrefill<false>>);
}

rf_status launch_paged_prefill(const PagedAttn& a, int dtype, cudaStream_t st) {
  return dtype == RF_F16 ? launch_pairs<true>(a, st) : launch_pairs<false>(a, st);
}

rf_status launch_paged_finish(const PagedAttn& a, int dtype, cudaStream_t st) {
  const int sms = tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  // eight CTAs per tile that may be cut, enough for all rows in pieces up to four CTAs per SM
  const PagedShape& s = a.v.s;
  const long long rows = ((long long)a.v.merge_cap * s.Hkv * s.unit_rows() + FIN_WARPS - 1) / FIN_WARPS;
  const long long pairs = (long long)a.v.slot_cap / 2 * FIN_PARTS, most = rows < 4ll * sms ? rows : 4ll * sms;
  const unsigned grid = (unsigned)((pairs > most ? pairs : most) + FIN_PARTS - 1) / FIN_PARTS * FIN_PARTS;
  return launch_after(dtype == RF_F16 ? paged_finish_kernel<true> : paged_finish_kernel<false>, grid,
                      FIN_WARPS * 32, 0, st, a);
}

RF_TIMEOUT_WORD_OF_THIS_FILE

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
