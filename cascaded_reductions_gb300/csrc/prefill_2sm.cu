// Causal prefill attention on CTA pairs (the kernel is in attn_pair.cuh).
//
// The cascade (RedFuser episode transcript, cue 9): S = Q K^T, then the row
// max, the exp-sum and the weighted sum with V.  Fused form (cues 15-19, 31):
// each 128-row query tile streams its key blocks once and keeps the running
// state per row; the state lives at the block level of the reduction tree.
//
// A work item is 256 adjacent query rows of one head: CTA r of the cluster
// takes the 128-row tile 2 p + r.  Items are numbered head-major, heaviest
// first within a head, and taken in snake order.

#include "attn_pair.cuh"

namespace rf {
namespace {

using pair::BM;
using pair::BN;
using pair::HALF_BYTES;
using pair::HD;

struct CausalPrefill {
  static constexpr bool F16 = false;
  static constexpr bool CHAINED = false, PARTIAL = false, STAGED = false;
  static constexpr float M_START = -INFINITY;
  // A work item: 256 query rows (two 128-row tiles) of one head.
  struct Item {
    int key0;     // first row of the head in Q, K, V and out
    int pair;     // tiles 2 pair and 2 pair + 1 of the head
    int n;        // key blocks (the same for both CTAs)
  };
  struct Pending {
    int row;
    bool in;
  };

  __nv_bfloat16* out;
  float* lse;
  int N, causal, num_items;
  float scale_log2;

  // Cluster c takes the item c of every even round of nclusters items and
  // item nclusters - 1 - c of every odd round: with items weighted p + 1 under
  // the causal mask, the snake evens out the clusters' totals (plain
  // round-robin leaves some clusters a tenth more work than the mean).
  __device__ __forceinline__ bool item(int t, int cluster, int nclusters, Item& it) const {
    const int i = t * nclusters + ((t & 1) ? nclusters - 1 - cluster : cluster);
    if (i >= num_items) return false;
    const int NB = (N + BM - 1) / BM;                   // 128-row query tiles per head
    const int NP = (NB + 1) / 2;                        // pairs of tiles per head
    it.key0 = (i / NP) * N;
    it.pair = NP - 1 - i % NP;
    it.n = causal ? it.pair + 1 : (N + BN - 1) / BN;
    return true;
  }
  __device__ __forceinline__ uint32_t q_bytes() const { return pair::TILE_BYTES; }
  __device__ __forceinline__ void load_q(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int rank) const {
    const int row = it.key0 + (2 * it.pair + rank) * BM;
    tc::tma_load_2d_pair(dst, map, bar, 0, row);
    tc::tma_load_2d_pair(dst + HALF_BYTES, map, bar, 64, row);
  }
  __device__ __forceinline__ void load_k(uint8_t* dst, const CUtensorMap* map, uint32_t bar,
                                         const Item& it, int j, int rank) const {
    const int row = it.key0 + j * BN + rank * (BN / 2);
    tc::tma_load_2d_pair(dst, map, bar, 0, row);
    tc::tma_load_2d_pair(dst + HALF_BYTES, map, bar, 64, row);
  }
  __device__ __forceinline__ uint32_t v_bytes(const Item&, int) const { return pair::TILE_BYTES; }
  __device__ __forceinline__ void load_v(uint8_t* dst, const CUtensorMap* map, const CUtensorMap*,
                                         uint32_t bar, const Item& it, int j, int rank) const {
    tc::tma_load_2d_pair(dst, map, bar, rank * 64, it.key0 + j * BN);
  }
  __device__ __forceinline__ int keys(const Item&, int) const { return BN; }
  __device__ __forceinline__ void mask(const Item& it, int j, int rank, int r, int kh,
                                       float (&s)[128]) const {
    const int NKB = (N + BN - 1) / BN;
    if (causal && j == it.n - 1) {
      const int lim = BM * rank + r - kh * 128;
#pragma unroll
      for (int c = 0; c < 128; ++c)
        if (c > lim) s[c] = -INFINITY;
    } else if (!causal && j == NKB - 1 && N % BN != 0) {
      const int kmax = N - j * BN - kh * 128;
#pragma unroll
      for (int c = 0; c < 128; ++c)
        if (c >= kmax) s[c] = -INFINITY;
    }
  }
  __device__ __forceinline__ Pending pending(const Item& it, int rank, int r) const {
    const int m_tile = 2 * it.pair + rank;
    return {it.key0 + m_tile * BM + r, m_tile * BM + r < N};
  }
  __device__ __forceinline__ void store(const Pending& pend, int col, const uint32_t (&v)[32],
                                        float m, float lt) const {
    const long long heads = (long long)num_items / ((((N + BM - 1) / BM) + 1) / 2);
    (void)heads;                                    // read by the checked build only
    const bool out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    const float inv = 1.f / lt;
    uint32_t pkd[16];
#pragma unroll
    for (int c = 0; c < 16; ++c)
      pkd[c] = pack_bf16x2(__uint_as_float(v[2 * c]) * inv, __uint_as_float(v[2 * c + 1]) * inv);
    if (pend.in && RF_SPAN_OK((size_t)pend.row * HD + col, 32, heads * N * HD))
      pair::st_row32(out + (size_t)pend.row * HD + col, pkd, out32);
    if (lse != nullptr && col == 0 && pend.in && RF_IDX_OK(pend.row, heads * N))
      lse[pend.row] = (m + log2f(lt)) * kLn2;
  }
  __device__ __forceinline__ void after(bool, int, int, int, int) const {}
};

}  // namespace

// RF_ERR_UNSUPPORTED when a cluster of two of these CTAs cannot be resident
// on the device (or the item count overflows an int).
rf_status launch_prefill(const void* q, const void* k, const void* v, int B, int H, int N, int D,
                         int causal, float scale, void* out, float* lse, cudaStream_t st) {
  (void)D;                                      // 128, checked by the caller
  const int pairs = pair::resident_pairs<CausalPrefill>();
  if (pairs <= 0) return RF_ERR_UNSUPPORTED;
  const uint64_t rows = (uint64_t)B * H * N;
  CUtensorMap tq, tk, tv;
  const uint64_t stride = HD * 2;
  if (!tc::make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, HD, rows, stride, 64, BM,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, k, HD, rows, stride, 64, BN / 2,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, v, HD, rows, stride, 64, BN,
                        CU_TENSOR_MAP_SWIZZLE_128B))
    return RF_ERR_CUDA;
  const int NB = (N + BM - 1) / BM;
  const long long items = (long long)B * H * ((NB + 1) / 2);
  if (items > INT32_MAX) return RF_ERR_UNSUPPORTED;
  const int clusters = (int)(pairs < items ? pairs : items);
  const CausalPrefill p{static_cast<__nv_bfloat16*>(out), lse, N, causal, (int)items, scale * kLog2e};
  return pair::launch_pair(tq, tk, tv, tv, tq, p, clusters, st);
}

RF_TIMEOUT_WORD_OF_THIS_FILE

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
