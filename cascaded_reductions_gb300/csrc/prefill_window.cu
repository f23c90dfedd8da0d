// Prefill of the last N of L positions with a sliding window and a few first
// tokens that stay visible, grouped heads, on CTA pairs (the kernel is in
// attn_pair.cuh).  A few rows of few heads go to the decode kernel instead
// (prefill_is_few).
//
// Mathematics: the causal prefill's cascade over the visible keys only,
//   visible(p) = { j <= p : j > p - window or j < sinks }.
//
// What bounds it: the tensor pipe, 4 D flops per pair of row and key.  An item
// is 256 query rows on one key head: up to 8 of the query heads that share it,
// and 256 / heads adjacent positions (256 rows of one head would need the keys
// of 256 positions; 64 positions of four heads need 192 fewer).  It visits the
// 256-key blocks that cover the keys any of its rows sees, last block first, a
// remainder of up to 64 keys as a narrow block, and then the sinks below that
// cover, narrow too where 64 keys are enough; a remainder and up to 64 sinks
// share one block (a block costs its chain of waits whatever its width).  Only
// the blocks at the two edges are masked, only by the warps that an edge crosses,
// a 32-key word at a time.
//
// A row that sees nothing of a block must not be disturbed by it: its
// reference starts at a finite value below every score, so such a block gives
// weights of exactly 0.  The products still multiply those zeros with V, and
// 0 * NaN is NaN: a value row that is not finite would reach rows that do not
// see it.  A row with NaN in its output is therefore looked at again after the
// last item: columns that are NaN by right (a value that the warp's 32 rows all see,
// found in one pass over their keys) stay, the others are computed from the
// row's visible keys alone.

#include <cuda_fp16.h>

#include "attn_pair.cuh"

namespace rf {
namespace {

using pair::BM;
using pair::BN;
using pair::HALF_BYTES;
using pair::HD;

template <bool F16_>
struct WindowPrefill {
  static constexpr bool F16 = F16_;
  static constexpr bool CHAINED = true, PARTIAL = true, STAGED = true;
  static constexpr float M_START = -1e30f;
  struct Item {
    int bh, kvh;     // first query head and key head, of the batch
    int row0;        // first position's row
    int lo;          // first key that a row sees beside the sinks
    int rem;         // keys of the narrow window block at lo, or 0
    int nb;          // full window blocks; block j < nb starts at lo + rem + 256 (nb - 1 - j)
    int nw;          // window blocks; block nb, if it is one, is the narrow one
    int limit;       // sinks below lo; block j >= nw starts at 256 (j - nw)
    bool mixed;      // block nb holds the remainder in keys 0-63 and the sinks in 64-127
    int n;
  };
  struct Pending {
    int bh, row;
    bool in;
  };

  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  int N, L, G, window, sinks;      // window and sinks at most L
  int heads;                       // B * H
  int packed, positions;           // query heads per item, 256 / packed positions
  int pairs;                       // items per `packed` heads
  float scale_log2;

  // items head-major (query heads of a key head together), last rows first, in
  // snake order as the causal prefill's
  __device__ __forceinline__ bool item(int t, int cluster, int nclusters, Item& it) const {
    const long long turn =
        (long long)t * nclusters + ((t & 1) ? nclusters - 1 - cluster : cluster);
    if (turn >= (long long)(heads / packed) * pairs) return false;
    const int i = (int)turn;                            // below B * H * N < 2^31
    it.bh = i / pairs * packed;
    it.kvh = it.bh / G;
    it.row0 = (pairs - 1 - i % pairs) * positions;
    const int p0 = L - N + it.row0;                     // the first position
    const int hi = min(p0 + positions, L) - 1;          // last key of the last one
    it.lo = max(0, p0 - window + 1);
    const int span = hi - it.lo + 1;
    it.nb = span / BN;
    it.rem = span - it.nb * BN;
    if (it.rem > pair::NARROW || it.nb == 0) {
      ++it.nb;
      it.rem = 0;
    }
    it.nw = it.nb + (it.rem > 0);
    it.limit = min(sinks, it.lo);
    it.mixed = it.rem > 0 && it.limit > 0 && it.limit <= pair::NARROW;
    it.n = it.mixed ? it.nw : it.nw + (it.limit + BN - 1) / BN;
    return true;
  }
  __device__ __forceinline__ int key0(const Item& it, int j) const {
    return j < it.nb ? it.lo + it.rem + (it.nb - 1 - j) * BN : j < it.nw ? it.lo : (j - it.nw) * BN;
  }
  // row r of CTA `rank`: head bh + head_of, position row0 + row_of
  __device__ __forceinline__ int head_of(int rank, int r) const { return (rank * BM + r) / positions; }
  __device__ __forceinline__ int row_of(int rank, int r) const {
    return (rank * BM + r) & (positions - 1);
  }
  __device__ __forceinline__ uint32_t q_bytes() const { return pair::TILE_BYTES; }
  __device__ __forceinline__ void load_q(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int rank) const {
    const int row = it.row0 + row_of(rank, 0), head = it.bh + head_of(rank, 0);
    tc::tma_load_3d_pair(dst, map, bar, 0, row, head);
    tc::tma_load_3d_pair(dst + HALF_BYTES, map, bar, 64, row, head);
  }
  __device__ __forceinline__ void load_k(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int j, int rank) const {
    // of a mixed block the second CTA's half are the sinks
    const int key = it.mixed && j == it.nb ? (rank == 0 ? it.lo : 0) : key0(it, j) + rank * (keys(it, j) / 2);
    tc::tma_load_3d_pair(dst, map, bar, 0, key, it.kvh);
    tc::tma_load_3d_pair(dst + HALF_BYTES, map, bar, 64, key, it.kvh);
  }
  __device__ __forceinline__ uint32_t v_bytes(const Item& it, int j) const {
    return it.mixed && j == it.nb ? 2 * pair::NARROW * 128 : pair::TILE_BYTES;
  }
  // `narrow`: the map whose boxes are 64 keys high
  __device__ __forceinline__ void load_v(uint8_t* dst, const CUtensorMap* map, const CUtensorMap* narrow,
                                         uint32_t bar, const Item& it, int j, int rank) const {
    if (it.mixed && j == it.nb) {
      tc::tma_load_3d_pair(dst, narrow, bar, rank * 64, it.lo, it.kvh);
      tc::tma_load_3d_pair(dst + pair::NARROW * 128, narrow, bar, rank * 64, 0, it.kvh);
    } else {
      tc::tma_load_3d_pair(dst, map, bar, rank * 64, key0(it, j), it.kvh);
    }
  }
  __device__ __forceinline__ int keys(const Item& it, int j) const {
    return j < it.nb ? BN
           : it.mixed ? pair::MIXED
           : j < it.nw || it.limit <= pair::NARROW ? pair::NARROW : BN;
  }
  // bits below n of a word
  static __device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  }
  // A warp whose rows see none of its keys of a block (half of those at the two
  // edges) skips its scores.
  __device__ __forceinline__ bool sees(const Item& it, int j, int rank, int r, int kh) const {
    if (j >= it.nb) return kh == 0 || keys(it, j) == BN;
    const int base = key0(it, j) + kh * 128;
    const int first = L - N + it.row0 + row_of(rank, r & ~31), last = first + 31;
    return j == 0 || (last >= base && (first - window + 1 < base + 128 || sinks > base));
  }
  // A word of visible keys per row and 32 of them; an edge crosses a warp's 32
  // rows within one or two words.
  __device__ __forceinline__ void mask(const Item& it, int j, int rank, int r, int kh,
                                       float (&s)[128]) const {
    const int base = key0(it, j) + kh * 128;
    const int p = L - N + it.row0 + row_of(rank, r);    // this row's position
    const int first = p - (r & 31), last = first + 31;   // the warp's positions
    // keys [lo, hi] and below cs, counted from base
    int hi = p - base, lo = p - window + 1 - base, cs = sinks - base;
    if (j < it.nb) {
      if (first - base >= 127 && last - window + 1 <= base) return;
    } else if (j < it.nw) {
      hi = min(hi, it.rem - 1);                         // the rest is the next block's
      if (it.mixed) {                                   // (and kh is 0)
        mask_words<0, 2>(hi, lo, cs, s);
        mask_words<2, 4>(pair::NARROW + it.limit - 1, 0, 0, s);
        return;
      }
    } else {
      hi = 127, lo = 128, cs = it.limit - base;
      if (cs >= 128) return;
    }
    mask_words<0, 4>(hi, lo, cs, s);
  }
  // words Q0 .. Q1 - 1 of s: visible are keys [lo, hi], and of those up to hi the
  // ones below cs
  template <int Q0, int Q1>
  static __device__ __forceinline__ void mask_words(int hi, int lo, int cs, float (&s)[128]) {
#pragma unroll
    for (int q = Q0; q < Q1; ++q) {
      const uint32_t vis = below(hi + 1 - 32 * q) & (~below(lo - 32 * q) | below(cs - 32 * q));
      if (!__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!(vis & (1u << c))) s[32 * q + c] = -INFINITY;
      }
    }
  }
  __device__ __forceinline__ Pending pending(const Item& it, int rank, int r) const {
    const int row = it.row0 + row_of(rank, r);
    return {it.bh + head_of(rank, r), row, row < N};
  }
  __device__ __forceinline__ bool pack(const Pending& pend, int col, const uint32_t (&v)[32], float m,
                                       float lt, uint32_t (&w)[16]) const {
    const float inv = 1.f / lt;
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
    const size_t row = (size_t)pend.bh * N + pend.row;
    if (lse != nullptr && col == 0 && pend.in && RF_IDX_OK(row, (size_t)heads * N))
      lse[row] = (m + log2f(lt)) * kLn2;
    float p0, p1;
    pair::unpack_f32x2(probe, p0, p1);
    return pend.in && !(p0 == 0.f && p1 == 0.f);
  }
  // called by the warp's first lane, whose row is the boxes' first; rows past N
  // lie past the map's extent and are not written
  __device__ __forceinline__ void send(const CUtensorMap* map, const uint8_t* box,
                                       const Pending& pend) const {
    if (!pend.in) return;
    tc::tma_store_3d(map, box, 0, pend.row, pend.bh);
    tc::tma_store_3d(map, box + HALF_BYTES, 64, pend.row, pend.bh);
  }

  static __device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
  static __device__ __forceinline__ void widen4(const uint2& u, float (&f)[4]) {
    const float2 a = widen2(u.x), b = widen2(u.y);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  }
  // elements [i, i + 4) of a tensor of n elements
  static __device__ __forceinline__ uint2 load4(const uint16_t* t, size_t i, size_t n) {
    (void)n;                                            // read by the checked build only
    return RF_SPAN_OK(i, 4, n) ? *reinterpret_cast<const uint2*>(t + i) : make_uint2(0, 0);
  }
  // bits 0 and 1: whether the 32-bit word's two values are NaN
  static __device__ __forceinline__ uint32_t nan_bits(uint32_t w) {
    const uint32_t inf = F16 ? 0x7c00u : 0x7f80u;
    return ((w & 0x7fffu) > inf) | (((w >> 16) & 0x7fffu) > inf) << 1;
  }
  static __device__ __forceinline__ uint32_t nan_bits(const uint2& u) {
    return nan_bits(u.x) | nan_bits(u.y) << 2;
  }
  size_t __device__ __forceinline__ q_elems() const { return (size_t)heads * N * HD; }
  size_t __device__ __forceinline__ kv_elems() const { return (size_t)(heads / G) * L * HD; }

  // Of this lane's four columns (bits), those that are NaN by right in all of rows
  // first .. last: one of the values that all of them see is NaN, or one of the keys.
  // `want`: the columns to look at.
  __device__ __forceinline__ uint32_t nan_for_all(int bh, int first, int last, uint32_t want, int lane) const {
    constexpr int U = 8;                                // keys in flight
    const int p0 = L - N + first, lo = max(0, L - N + last - window + 1);
    const int ns = min(min(sinks, lo), p0 + 1), n = ns + max(0, p0 - lo + 1);
    const size_t kv0 = (size_t)(bh / G) * L;
    uint32_t got = 0;
    for (int t0 = 0; t0 < n; t0 += U) {
      uint2 kk[U], vv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(t0 + u, n - 1), key = t < ns ? t : t - ns + lo;
        kk[u] = load4(k, (kv0 + key) * HD + lane * 4, kv_elems());
        vv[u] = load4(v, (kv0 + key) * HD + lane * 4, kv_elems());
      }
      uint32_t bad_key = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        bad_key |= nan_bits(kk[u]);
        got |= nan_bits(vv[u]);
      }
      if (__any_sync(0xffffffffu, bad_key != 0)) return 15u;
      if (!__any_sync(0xffffffffu, (want & ~got) != 0)) break;
    }
    return got;
  }

  // The NaN columns of one output row, but for those that are NaN by `right`, once
  // more from the keys that the row sees; four columns per lane.  Ends once they are
  // all NaN again.  The lse in place stands (no masked score entered it), unless
  // the weights all vanished against the reference that the row started from.
  // A row costs about 0.2 us per key.  The form of the loops here was chosen by the time
  // of calls that never reach them, whose code lies beside it: other widths and
  // orders cost the long windowed prefill 501 to 538 us instead of 499.
  __device__ __forceinline__ void redo(int bh, int row, uint32_t right, int lane) const {
    const size_t q0 = ((size_t)bh * N + row) * HD, o = q0 + lane * 4;
    uint2 word = RF_SPAN_OK(o, 4, q_elems()) ? *reinterpret_cast<const uint2*>(out + o) : make_uint2(0, 0);
    const uint32_t todo = nan_bits(word) & ~right;
    if (!__any_sync(0xffffffffu, todo != 0)) return;
    const int p = L - N + row;
    const int lo = max(0, p - window + 1), ns = min(sinks, lo), n = ns + p - lo + 1;
    const size_t kv0 = (size_t)(bh / G) * L;
    float qf[4];
    widen4(load4(q, q0 + lane * 4, q_elems()), qf);
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool gone = false;
    constexpr int U = 4;                                // keys in flight
#pragma unroll 1
    for (int t0 = 0; !gone && t0 < n; t0 += U) {
      uint2 kk[U], vv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(t0 + u, n - 1), key = t < ns ? t : t - ns + lo;
        kk[u] = load4(k, (kv0 + key) * HD + lane * 4, kv_elems());
        vv[u] = load4(v, (kv0 + key) * HD + lane * 4, kv_elems());
      }
      float s[U], mn = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float kf[4];
        widen4(kk[u], kf);
        s[u] = fmaf(qf[0], kf[0], fmaf(qf[1], kf[1], fmaf(qf[2], kf[2], qf[3] * kf[3])));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = t0 + u < n ? group_sum<32>(s[u]) * scale_log2 : -INFINITY;
        mn = fmaxf(mn, s[u]);
      }
      const float ref = ref_of(mn), corr = exp2f(m - ref);
      m = mn;
      l *= corr;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= corr;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u >= n) break;
        float vf[4];
        widen4(vv[u], vf);
        const float w = exp2f(s[u] - ref);
        l += w;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, vf[e], acc[e]);
      }
      uint32_t now = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) now |= (uint32_t)(acc[e] != acc[e]) << e;
      gone = !__any_sync(0xffffffffu, (todo & ~now) != 0);
    }
    if (gone) return;
    float y[4];                                         // l = 0: every visible score is -inf
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = l == 0.f ? 0.f : acc[e] / l;
    const uint32_t y01 = pair::pack_16x2<F16>(y[0], y[1]), y23 = pair::pack_16x2<F16>(y[2], y[3]);
    const uint32_t m01 = (todo & 1u ? 0xffffu : 0u) | (todo & 2u ? 0xffff0000u : 0u);
    const uint32_t m23 = (todo & 4u ? 0xffffu : 0u) | (todo & 8u ? 0xffff0000u : 0u);
    word.x = (word.x & ~m01) | (y01 & m01);
    word.y = (word.y & ~m23) | (y23 & m23);
    if (RF_SPAN_OK(o, 4, q_elems())) *reinterpret_cast<uint2*>(out + o) = word;
    const size_t i = (size_t)bh * N + row;
    if (lse != nullptr && lane == 0 && RF_IDX_OK(i, (size_t)heads * N) && lse[i] == -INFINITY)
      lse[i] = (m + log2f(l)) * kLn2;
  }

  // Rows of this thread whose stored values hold a NaN are looked at again, a
  // warp's 32 adjacent positions of a head together.
  __device__ __forceinline__ void repair(int cluster, int nclusters, int rank, int r) const {
    Item it;
    const int lane = r & 31;
    for (int t = 0; item(t, cluster, nclusters, it); ++t) {
      const int row = it.row0 + row_of(rank, r), head = it.bh + head_of(rank, r);
      bool nan = false;
      if (row < N) {
        const size_t o = ((size_t)head * N + row) * HD;
        for (int c = 0; c < 16; ++c) {
          if (!RF_SPAN_OK(o + c * 8, 8, q_elems())) continue;
          const uint4 u = *(reinterpret_cast<const uint4*>(out + o) + c);
          nan |= (nan_bits(u.x) | nan_bits(u.y) | nan_bits(u.z) | nan_bits(u.w)) != 0;
        }
      }
      const uint32_t rows = __ballot_sync(0xffffffffu, nan);
      if (rows == 0) continue;
      const int row0 = row - lane, last = min(row0 + 31, N - 1);
      uint32_t want = 0;                                // of this lane's columns, in any of the rows
      for (uint32_t left = rows; left; left &= left - 1) {
        const size_t o = ((size_t)head * N + row0 + __ffs(left) - 1) * HD + lane * 4;
        if (RF_SPAN_OK(o, 4, q_elems())) want |= nan_bits(*reinterpret_cast<const uint2*>(out + o));
      }
      const uint32_t right = nan_for_all(head, row0, last, want, lane);
      for (uint32_t left = rows; left; left &= left - 1) redo(head, row0 + __ffs(left) - 1, right, lane);
    }
  }
  __device__ __forceinline__ void after(bool any, int cluster, int nclusters, int rank, int r) const {
    if (!__any_sync(0xffffffffu, any)) return;
    // the outputs were written by bulk copies; they are read as memory now
    asm volatile("fence.proxy.async;" ::: "memory");
    repair(cluster, nclusters, rank, r);
  }
};

template <bool F16>
rf_status launch_t(const void* q, const void* k, const void* v, int B, int H, int Hkv, int N, int L,
                   int window, int sinks, float scale, void* out, float* lse, cudaStream_t st) {
  using P = WindowPrefill<F16>;
  const int pairs = pair::resident_pairs<P>();
  if (pairs <= 0) return RF_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv, tw, to;
  const uint64_t qh = (uint64_t)B * H, kh = (uint64_t)B * Hkv;
  const int G = H / Hkv;
  const int packed = G % 8 == 0 ? 8 : G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1;
  const int positions = 2 * BM / packed, box = positions < BM ? positions : BM;
  if (!tc::make_tmap_3d_16(&tq, F16, q, HD, N, qh, 64, box, BM / box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&tk, F16, k, HD, L, kh, 64, BN / 2, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&tv, F16, v, HD, L, kh, 64, BN, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&tw, F16, v, HD, L, kh, 64, pair::NARROW, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&to, F16, out, HD, N, qh, 64, 32, 1, CU_TENSOR_MAP_SWIZZLE_128B))
    return RF_ERR_CUDA;
  P p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.N = N, p.L = L, p.G = G;
  p.window = window == 0 || window > L ? L : window;
  p.sinks = sinks > L ? L : sinks;
  p.heads = B * H;
  p.packed = packed, p.positions = positions;
  p.pairs = (N + positions - 1) / positions;
  p.scale_log2 = scale * kLog2e;
  const long long items = (long long)(p.heads / packed) * p.pairs;
  return pair::launch_pair(tq, tk, tv, tw, to, p, (int)(pairs < items ? pairs : items), st);
}

}  // namespace

rf_status launch_prefill_window(const void* q, const void* k, const void* v, int B, int H, int Hkv,
                                int N, int L, int window, int sinks, float scale, int dtype,
                                void* out, float* lse, cudaStream_t st) {
  return dtype == RF_F16
             ? launch_t<true>(q, k, v, B, H, Hkv, N, L, window, sinks, scale, out, lse, st)
             : launch_t<false>(q, k, v, B, H, Hkv, N, L, window, sinks, scale, out, lse, st);
}

RF_TIMEOUT_WORD_OF_THIS_FILE

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
