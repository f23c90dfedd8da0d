// The prefix half of single-token decode for a batch whose sequences all begin
// with the same keys: every query row of a key head (B sequences x G heads)
// meets the one prefix, so each of its keys is read once for up to 256 rows
// instead of once per sequence (the kernel, on CTA pairs, is in attn_pair.cuh).
// Small calls do without it (decode_prefix_is_few).
//
// Mathematics: segment states (m, l, acc) of the split-KV decode, one per row
// and piece of the prefix; the decode over the sequences' own keys merges them
// with its own (cache_decode.cu).
//
// What bounds it: a block of 256 prefix keys (128 KiB of K and V) takes the
// tensor pipe about as long as its bytes take HBM when the item's 256 rows are
// full; with fewer rows the kernel still computes 256 and stays near the HBM
// bound, and with more rows the prefix comes from L2 after the first item.
//
// Split: the blocks of all items (key head, 256 rows) are numbered through and
// every cluster takes an equal, contiguous share, so clusters finish
// together and a row has one state per cluster that touched its item (about
// clusters / items + 1) rather than one per fixed-size segment.  The cluster
// that ends an item marks the item's unused state slots empty.
//
// A cluster whose share crosses from one item into the next pays for a second
// start and end, about as long as five blocks (16 items of 128 blocks without own
// keys: 67 us on 64 clusters, which stay within their item, and 69 us on all 76).
// So where the largest multiple of the items costs at most kSwitchBlocks blocks
// more, only so many clusters run: the idle SMs begin with the sequences' own keys
// (128 sequences of up to 512: 88.5 -> 86 us) and the merge has fewer states.

#include "attn_pair.cuh"

namespace rf {
namespace {

using pair::BM;
using pair::BN;
using pair::HALF_BYTES;
using pair::HD;

constexpr int kSwitchBlocks = 6;

struct Split {
  int blocks;          // key blocks of the prefix
  int tiles;           // items: Hkv * tiles_per_head
  int clusters;
  long long total;     // tiles * blocks
  // first block of cluster c's share
  __host__ __device__ long long begin(long long c) const { return c * total / clusters; }
  // the cluster whose share holds block x: the largest c with begin(c) <= x
  __host__ __device__ int owner(long long x) const {
    return (int)(((x + 1) * clusters + total - 1) / total) - 1;
  }
};

template <bool F16_>
struct PrefixStates {
  static constexpr bool F16 = F16_;
  static constexpr bool CHAINED = true, PARTIAL = false, STAGED = false;
  static constexpr float M_START = -1e30f;
  struct Item {
    int hk, seq0;            // key head; first sequence of the pair of tiles
    int block0, n;           // this cluster's blocks of the item
    int slot, end;           // state slot; 1: the item's last block is here
  };
  struct Pending {
    size_t row;              // b * H + query head
    int slot, end;
    bool in;
  };

  float *seg_m, *seg_l, *seg_acc;
  int B, H, G, P;            // P: prefix length
  int nb;                    // sequences per tile of 128 rows: 128 / G
  int tiles_per_head;
  int S_total, prefix_slots;
  Split split;
  float scale_log2;

  __device__ __forceinline__ bool item(int t, int cluster, int nclusters, Item& it) const {
    (void)nclusters;
    const long long u0 = split.begin(cluster), u1 = split.begin(cluster + 1);
    const int i = (int)(u0 / split.blocks) + t;
    const long long first = (long long)i * split.blocks;
    const long long a = first > u0 ? first : u0;
    const long long b = first + split.blocks < u1 ? first + split.blocks : u1;
    if (a >= b) return false;
    it.hk = i / tiles_per_head;
    it.seq0 = (i - it.hk * tiles_per_head) * 2 * nb;
    it.block0 = (int)(a - first);
    it.n = (int)(b - a);
    it.slot = cluster - split.owner(first);
    it.end = b == first + split.blocks;
    return true;
  }
  __device__ __forceinline__ uint32_t q_bytes() const { return (uint32_t)(nb * G) * HD * 2; }
  __device__ __forceinline__ void load_q(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int rank) const {
    const int b = it.seq0 + rank * nb;
    tc::tma_load_3d_pair(dst, map, bar, 0, it.hk * G, b);
    tc::tma_load_3d_pair(dst + HALF_BYTES, map, bar, 64, it.hk * G, b);
  }
  __device__ __forceinline__ void load_k(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int j, int rank) const {
    const int key = (it.block0 + j) * BN + rank * (BN / 2);
    tc::tma_load_3d_pair(dst, map, bar, 0, key, it.hk);
    tc::tma_load_3d_pair(dst + HALF_BYTES, map, bar, 64, key, it.hk);
  }
  __device__ __forceinline__ uint32_t v_bytes(const Item&, int) const { return pair::TILE_BYTES; }
  __device__ __forceinline__ void load_v(uint8_t* dst, const CUtensorMap* map, const CUtensorMap*,
                                         uint32_t bar, const Item& it, int j, int rank) const {
    tc::tma_load_3d_pair(dst, map, bar, rank * 64, (it.block0 + j) * BN, it.hk);
  }
  __device__ __forceinline__ int keys(const Item&, int) const { return BN; }
  __device__ __forceinline__ void mask(const Item& it, int j, int rank, int r, int kh,
                                       float (&s)[128]) const {
    (void)rank;
    (void)r;
    const int lim = P - (it.block0 + j) * BN - kh * 128;
    if (lim < 128) {
#pragma unroll
      for (int c = 0; c < 128; ++c)
        if (c >= lim) s[c] = -INFINITY;
    }
  }
  __device__ __forceinline__ Pending pending(const Item& it, int rank, int r) const {
    // row r of the tile: sequence r / G, query head r % G of the group
    const int b = it.seq0 + rank * nb + r / G, g = r - (r / G) * G;
    return {(size_t)b * H + (size_t)it.hk * G + g, it.slot, it.end, r < nb * G && b < B};
  }
  __device__ __forceinline__ void store(const Pending& pend, int col, const uint32_t (&v)[32],
                                        float m, float lt) const {
    if (!pend.in) return;
    const size_t slot = pend.row * S_total + pend.slot;
    const size_t states = (size_t)B * H * S_total;
    (void)states;                                 // read by the checked build only
    if (RF_SPAN_OK(slot * HD + col, 32, states * HD)) {
      uint4* dst = reinterpret_cast<uint4*>(seg_acc + slot * HD + col);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        dst[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
    if (col == 0 && RF_IDX_OK(slot, states)) {
      seg_m[slot] = m;
      seg_l[slot] = lt;
      if (pend.end)
        for (int s = pend.slot + 1; s < prefix_slots; ++s)
          if (RF_IDX_OK(pend.row * S_total + s, states)) {
            seg_m[pend.row * S_total + s] = -INFINITY;
            seg_l[pend.row * S_total + s] = 0.f;
          }
    }
  }
  __device__ __forceinline__ void after(bool, int, int, int, int) const {}
};

// The split for B sequences of G heads on Hkv key heads, at most `slots` states
// per row; clusters 0 if the device cannot run the kernel.
Split make_split(int B, int H, int Hkv, int prefix, int slots, int pairs) {
  const int G = H / Hkv, nb = 128 / G;
  Split s = {};
  s.blocks = (int)ceil_div(prefix, BN);
  s.tiles = Hkv * (int)ceil_div(B, 2 * nb);
  s.total = (long long)s.tiles * s.blocks;
  long long c = pairs < s.total ? pairs : s.total;
  // an item is touched by at most ceil(clusters / tiles) + 1 clusters
  const long long most = (long long)(slots - 1) * s.tiles;
  if (c > most) c = most;
  const long long even = c - c % s.tiles;       // whole clusters per item
  if (even > 0 && (s.total + even - 1) / even <= s.total / c + kSwitchBlocks) c = even;
  s.clusters = (int)c;
  return s;
}

template <bool F16>
rf_status launch_t(const void* q, const void* kp, const void* vp, int prefix, int B, int H, int Hkv,
                   int Sp, int S_total, float scale, float* seg_m, float* seg_l, float* seg_acc,
                   cudaStream_t st) {
  using P = PrefixStates<F16>;
  const int pairs = pair::resident_pairs<P>();
  if (pairs <= 0) return RF_ERR_UNSUPPORTED;
  P p = {};
  p.seg_m = seg_m, p.seg_l = seg_l, p.seg_acc = seg_acc;
  p.B = B, p.H = H, p.G = H / Hkv, p.P = prefix;
  p.nb = 128 / p.G;
  p.tiles_per_head = (int)ceil_div(B, 2 * p.nb);
  p.S_total = S_total;
  p.prefix_slots = Sp;
  p.split = make_split(B, H, Hkv, prefix, Sp, pairs);
  p.scale_log2 = scale * kLog2e;
  CUtensorMap tq, tk, tv;
  if (!tc::make_tmap_3d_16(&tq, F16, q, HD, H, B, 64, p.G, p.nb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&tk, F16, kp, HD, prefix, Hkv, 64, BN / 2, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_3d_16(&tv, F16, vp, HD, prefix, Hkv, 64, BN, 1, CU_TENSOR_MAP_SWIZZLE_128B))
    return RF_ERR_CUDA;
  return pair::launch_pair(tq, tk, tv, tv, tq, p, p.split.clusters, st);
}

}  // namespace

int prefix_segments(int B, int H, int Hkv, int prefix) {
  const int pairs = pair::resident_pairs<PrefixStates<false>>();
  if (pairs <= 0) return 0;
  const Split s = make_split(B, H, Hkv, prefix, 1 << 20, pairs);
  const int n = (s.clusters + s.tiles - 1) / s.tiles + 1;
  // or the decode kernel's pieces, where the call may be small enough for it
  const long long groups = (long long)B * Hkv * ((H / Hkv + 15) / 16);
  const int sms = tc::sm_count();
  const int few = sms > 0 && decode_prefix_is_few(groups, prefix, 1, sms)
                      ? decode_segments((int)groups, prefix, sms) : 0;
  return n > few ? (n < 2 ? 2 : n) : (few < 2 ? 2 : few);
}

rf_status launch_prefix_states(const void* q, const void* kp, const void* vp, int prefix, int B,
                               int H, int Hkv, int Sp, int S_total, float scale, int dtype,
                               float* seg_m, float* seg_l, float* seg_acc, cudaStream_t st) {
  return dtype == RF_F16 ? launch_t<true>(q, kp, vp, prefix, B, H, Hkv, Sp, S_total, scale, seg_m,
                                          seg_l, seg_acc, st)
                         : launch_t<false>(q, kp, vp, prefix, B, H, Hkv, Sp, S_total, scale, seg_m,
                                           seg_l, seg_acc, st);
}

RF_TIMEOUT_WORD_OF_THIS_FILE

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
