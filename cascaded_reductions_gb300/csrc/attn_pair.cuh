// Attention on CTA pairs: GEMM -> online softmax -> GEMM with every MMA issued
// across the two SMs of a cluster (tcgen05 cta_group::2).  The kernel is shared
// by the calls that run it; a policy says which query rows and key blocks a
// work item has, which scores its mask removes and where its result goes.
//
// A work item is 256 query rows that share their keys: CTA r of the cluster
// takes rows 128 r .. 128 r + 127.  Key blocks are 256 keys wide.  Per block j:
//   S(j)  = Q K_j^T, one M = 256, N = 256 MMA per 16 columns of the head
//           dimension: CTA r supplies its Q tile (A) and keys [128 r, 128 r +
//           128) of the block (its half of B); each CTA's TMEM receives its
//           own 128 rows x 256 keys;
//   P(j)  = exp2(S scale log2(e) - m) in 16 bits, written by the softmax warps
//           into TMEM columns of its own (not over S);
//   O    += P(j) V_j, M = 256, N = 128 MMAs with A = P read from each CTA's
//           TMEM and B = V_j split by columns: CTA r holds head-dimension
//           columns [64 r, 64 r + 64) of all 256 keys.
// Because P does not overwrite S, S(j + 1) is issued as soon as the softmax
// has read S(j) into registers, and runs on the tensor pipe while the
// softmax of block j is still exponentiating: the pipe order is
// S(0) S(1) PV(0) S(2) PV(1) ...  The kernel is persistent (one cluster per
// pair of SMs), and the numbering of blocks runs on across items: the next
// item's first S is computed during the current item's last softmax, and its
// first softmax while the output warps still write the current item's rows.
//
// TMEM (512 columns, allocated for the pair): S 0-255, P 256-383 (bf16 pairs,
// key pair (2c, 2c + 1) in column c), O 384-511.
// Shared memory per CTA: Q tiles (two buffers), K halves and V halves in
// 2-stage rings, 32 KiB each, all 128-byte swizzled.
// Roles, both CTAs:
//   warp 8      TMA: this CTA's Q tile, then its halves of K_j and V_j; the
//               copies of both CTAs complete on CTA 0's barriers;
//   warp 9      TMEM allocation; in CTA 0 one thread issues every MMA and
//               commits to both CTAs' barriers;
//   warps 0-7   softmax of this CTA's 128 rows: warp w reads TMEM lanes
//               32 (w % 4) .. + 31 (thread = row) and keys 128 (w / 4) .. + 127
//               of the block into registers; the two warps of a row exchange
//               their partial maxima through shared memory;
//   warps 12-15 output of an item's rows: O from TMEM once its last P V is done,
//               while the softmax warps are in the next item's first block.
// Two softmax warps per SM sub-partition (not four) leave the MMA-issuing
// thread, which shares a sub-partition with two of them, enough issue slots
// for the 64-cycle P V MMAs.  Their threads hold 128 scores each, so the
// registers are divided unevenly between the warpgroups.  Output by the softmax
// warps themselves took 1300 to 1900 cycles of an item's first block (code that
// runs once per item comes cold from the instruction cache): 569 us instead of
// 536 for 4 x 32 heads of 8192 with a window of 1024.
// Rescaling is lazy: the reference max m_ref of a row moves (and O and l are
// multiplied by exp2(m_ref_old - m_ref_new)) only when the block max exceeds
// it by more than 8, so p <= 2^8.  An fp16 p has 11 bits down to 2^-14 and ends at
// 2^-24, so it is taken 2^7 times as large (at most 2^15, of 65504): weights down
// to 2^-21 of exp2(m_ref) keep their bits and only those below 2^-32 vanish from the
// product (which l, summed unrounded, counts).  Without the factor 32768 keys
// at 2^-26 of a first key's weight were lost altogether.
//
// The softmax warps tell CTA 0's MMA thread that S was read, that P was
// written and that O was read with relaxed arrivals: each follows the
// tcgen05.wait that completes those TMEM accesses, so it needs no release
// (a release at cluster scope costs the arriving warp about 1000 cycles).
// For the same reason the MMA thread waits at CTA scope: what it orders
// after a wait are MMAs, whose operands were completed by the TMA
// transaction count or by the softmax warps' tcgen05.wait (an acquire at
// cluster scope idles the tensor pipe about 160 cycles per wait).
// Every barrier wait is bounded (see tc_common.cuh); the two CTAs meet at a
// cluster barrier before either exits.
//
// A policy P holds the call's arguments and has
//   F16                        operands are fp16 (else bf16)
//   M_START                    a row's reference before its first block: -inf
//                              where the first block always holds a visible
//                              key, else a finite value below every score, for
//                              which a block without visible keys gives p = 0
//   CHAINED                    the kernel is set up beside the end of the one before
//                              it on the stream, and lets the next one begin so
//   Item, Pending              a work item; what its output still needs
//   item(t, c, nc, it)         cluster c's t-th item of nc clusters; it.n key
//                              blocks, at least one; false past the last
//   q_bytes()                  bytes of one CTA's Q tile that load_q copies
//   load_q / load_k / load_v   the TMA copies of one CTA, into its halves
//   keys(it, j)                256, or 128 or 64 where no row sees the block's
//                              other keys: its products stop there
//   v_bytes(it, j)             bytes that load_v copies (with one map or both)
//   PARTIAL, sees(it, j, rank, row, kh)  with PARTIAL, whether the warp's rows
//                              see any of its 128 keys (128 kh ..) of block j;
//                              true for block 0
//   mask(it, j, rank, row, kh, s)  sets their hidden scores to -inf
//   pending(it, rank, row)     what an output row needs beside its values, and
//   store(pend, col, v, m, l)  its columns col .. + 31 from O, with the row's
//                              reference m (log2 units) and sum l
//   STAGED                     instead of store():  pack(pend, col, v, m, l, w)
//                              gives the columns in 16 bits (true: call
//                              after(true, ...)), and  send(map, box, pend)
//                              starts the copies of a warp's two 32 x 64 boxes,
//                              HALF_BYTES apart in shared memory
//   after(any, c, nc, rank, row)  once everything of the row's items is stored
#pragma once

#include <cuda_bf16.h>

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace rf {
namespace pair {

constexpr int BM = 128;                      // query rows per CTA (256 per pair)
constexpr int BN = 256;                      // keys per block
constexpr int NARROW = 64, MIXED = 128;      // keys of a narrow block, and of two in one
constexpr int HD = 128;                      // head dim
constexpr int STAGES = 2;
constexpr int TILE_BYTES = 32768;            // Q tile, K half or V half
constexpr int HALF_BYTES = 16384;            // one 64-column swizzled box of a 128-row tile
constexpr int SM_WARPS = 8;                // softmax warps: two per TMEM lane quarter
constexpr int TMA_WARP = 8, MMA_WARP = 9;
constexpr int OUT_WARP = 12, OUT_WARPS = 4;  // output warps, one per TMEM lane quarter
constexpr int THREADS = 16 * 32;             // four warpgroups (10 and 11 only fill theirs)
// Registers per thread: at launch, then softmax warps and the others.
constexpr int REGS = 128, REGS_SOFTMAX = 176, REGS_OTHER = 80;
static_assert(256 * REGS_SOFTMAX + 256 * REGS_OTHER == THREADS * REGS,
              "the shares of the four warpgroups add up to what the CTA is launched with");
constexpr int TMEM_COLS = 512;
constexpr uint32_t S_COL = 0, P_COL = 256, O_COL = 384;
constexpr float RESCALE_THRESHOLD = 8.0f;    // log2 units
constexpr float P_SHIFT = 7.0f;              // log2 of the factor that an fp16 p is taken with,
constexpr float P_SHIFT_LIMIT = 1048576.0f;  // for references up to 2^20: there m - 7 is off by at most
                                             // 2^-4, while from 2^24 on it may be m - 8 or less, and p 2^16

struct Shared {
  uint64_t q_full[2];           // CTA 0: both Q tiles of a buffer
  uint64_t q_empty[2];          // each CTA: the item's S MMAs are done with the buffer (and, with
                                // STAGED, the output warps' copies have read it)
  uint64_t k_full[STAGES];      // CTA 0: both K halves of a stage
  uint64_t v_full[STAGES];      // CTA 0: both V halves of a stage
  uint64_t k_empty[STAGES];     // each CTA: S of that block done
  uint64_t v_empty[STAGES];     // each CTA: P V of that block done
  uint64_t s_full;              // each CTA: S(g) complete
  uint64_t pv_done;             // each CTA: P V(g) complete
  uint64_t s_free;              // CTA 0: both CTAs' softmax warps have read S(g) (32 warps)
  uint64_t p_ready;             // CTA 0: both CTAs' P(g) and O rescale written (32 warps)
  uint64_t o_full;              // each CTA: the item's last P V complete
  uint64_t o_free;              // CTA 0: both CTAs' output warps have read O (8 warps)
  uint64_t l_ready[2];          // each CTA: an item's row sums and references are in part_l, row_m
  uint64_t red_bar[4];          // each CTA, per lane quarter: its two warps' maxima
  float red[2][2][BM];          // [exchange & 1][key half][row]: partial row maxima
  float part_l[2][2][BM];       // [item & 1][key half][row]: partial row sums of an item
  float row_m[2][BM];           // [item & 1][row]: its reference maxima
  uint32_t tmem_base;
  int abort;
};

// layout: Q[2] | K[STAGES] | V[STAGES] | Shared
constexpr size_t SMEM_BYTES = (size_t)(2 + 2 * STAGES) * TILE_BYTES + sizeof(Shared) + 1024;
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KiB of shared memory a CTA may use");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// fp32 pairs in one 64-bit register for the packed FMA / add of sm_100+
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// one 32-byte global store (sm_100+); `dst` 32-byte aligned
__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 16-bit values (64 bytes) of an output row; `wide` if rows are 32-byte aligned
__device__ __forceinline__ void st_row32(void* dst, const uint32_t (&w)[16], bool wide) {
  if (wide) {
    st_global_v8(dst, w);
    st_global_v8(static_cast<uint8_t*>(dst) + 32, w + 8);
  } else {
    uint4* d4 = static_cast<uint4*>(dst);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d4[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

template <int N>
struct Words {
  static constexpr int value = N;
};

// arrival on a barrier of CTA 0 without release semantics (see the file
// comment for why none is needed)
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// instruction descriptor of kind::f16 with both operands fp16 (format 0) or bf16 (1)
template <bool F16>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool b_mn_major) {
  return F16 ? tc::idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10))
             : tc::idesc_bf16_f32(M, N, b_mn_major);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi) {
  if constexpr (F16) return pack_f16x2(lo, hi);
  return pack_bf16x2(lo, hi);
}

template <class P>
__global__ void __launch_bounds__(THREADS, 1)
attn_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmO, const __grid_constant__ P p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                 // two buffers
  uint8_t* sK = smem + 2 * TILE_BYTES;
  uint8_t* sV = sK + STAGES * TILE_BYTES;
  Shared* sh = reinterpret_cast<Shared*>(sV + STAGES * TILE_BYTES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();        // 0 or 1
  const int cluster = (int)(blockIdx.x >> 1), nclusters = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&sh->q_full[b], 1);
      tc::mbar_init(&sh->q_empty[b], P::STAGED ? 1 + OUT_WARPS : 1);
      tc::mbar_init(&sh->l_ready[b], SM_WARPS);
    }
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&sh->k_full[s], 1);
      tc::mbar_init(&sh->v_full[s], 1);
      tc::mbar_init(&sh->k_empty[s], 1);
      tc::mbar_init(&sh->v_empty[s], 1);
    }
    tc::mbar_init(&sh->s_full, 1);
    tc::mbar_init(&sh->pv_done, 1);
    tc::mbar_init(&sh->s_free, 2 * SM_WARPS);
    tc::mbar_init(&sh->p_ready, 2 * SM_WARPS);
    tc::mbar_init(&sh->o_full, 1);
    tc::mbar_init(&sh->o_free, 2 * OUT_WARPS);
    for (int q = 0; q < 4; ++q) tc::mbar_init(&sh->red_bar[q], 2);
    sh->abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == MMA_WARP) tc::tmem_alloc_pair(&sh->tmem_base, TMEM_COLS);
  tc::fence_before_sync();
  // both CTAs' barriers are initialised before any copy, commit or arrival
  // reaches them
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort = &sh->abort;
  if constexpr (P::CHAINED) {
    wait_prerequisite();              // what lies above ran beside the kernel before
    allow_dependents();
  }

  // Each warpgroup takes its share of the registers, all its warps alike.
  if (warp < SM_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // --------------------------------------------------- softmax ----
    const int quarter = warp & 3;                   // TMEM lanes 32 quarter .. + 31
    const int kh = warp >> 2;                       // keys 128 kh .. + 127 of each block
    const int r = quarter * 32 + lane;              // this thread's row of the tile
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_free0 = tc::mapa(tc::smem_u32(&sh->s_free), 0);
    const uint32_t p_ready0 = tc::mapa(tc::smem_u32(&sh->p_ready), 0);
    const float scale_log2 = p.scale_log2;
    const uint64_t sl2 = pack_f32x2(scale_log2, scale_log2);
    uint32_t g = 0, x = 0;                          // blocks and red_bar exchanges so far
    bool ok = true;
    typename P::Item it;
    for (int t = 0; ok; ++t) {
      if (!p.item(t, cluster, nclusters, it)) break;
      float m_ref = P::M_START, l = 0.f;
      // One block, of which this warp's rows see some of its 128 keys (NW = 4
      // 32-key words) or none (NW = 0); false if a wait gave up.
      auto block = [&](auto words, int j) -> bool {
        constexpr int NW = decltype(words)::value;
        if (!tc::mbar_wait(&sh->s_full, g & 1u, abort)) return false;
        tc::fence_after_sync();
        float s[NW > 0 ? 32 * NW : 1];              // s[c] = key 128 kh + c of block j
        if constexpr (NW > 0) {
#pragma unroll
          for (int q = 0; q < NW; ++q) {
            uint32_t (&v)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]);
            tc::tmem_ld_32x32b_x32(lanes + S_COL + (uint32_t)(kh * 128 + 32 * q), v);
          }
          tc::tmem_ld_wait();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_cluster_relaxed(s_free0);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if constexpr (NW > 0) {
          p.mask(it, j, rank, r, kh, s);
#pragma unroll
          for (int c = 0; c < 32 * NW; c += 2)
            mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], s[c], s[c + 1]);
        }
        float* red = &sh->red[x & 1u][0][0];
        red[kh * BM + r] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh->red_bar[quarter]);
        if (!tc::mbar_wait(&sh->red_bar[quarter], x & 1u, abort)) return false;
        ++x;
        const float pm = fmaxf(red[r], red[BM + r]);
        const float mt = pm * scale_log2;
        // an fp16 reference lies P_SHIFT below the maximum that it was taken from
        const bool low = P::F16 && fabsf(m_ref) < P_SHIFT_LIMIT;
        const bool move = mt > m_ref + (low ? RESCALE_THRESHOLD + P_SHIFT : RESCALE_THRESHOLD);
        const float m_top = P::F16 && fabsf(mt) < P_SHIFT_LIMIT ? mt - P_SHIFT : mt;
        const float m_new = move ? m_top : m_ref;
        const float alpha = ex2(m_ref - m_new);
        l *= alpha;
        m_ref = m_new;
        uint32_t w[NW > 0 ? 16 * NW : 1];
        if constexpr (NW > 0) {
          const uint64_t nm2 = pack_f32x2(-m_new, -m_new);
          uint64_t sum2 = 0ull;
#pragma unroll
          for (int c = 0; c < 16 * NW; ++c) {
            float a0, a1;
            unpack_f32x2(fma_f32x2(pack_f32x2(s[2 * c], s[2 * c + 1]), sl2, nm2), a0, a1);
            const float p0 = ex2(a0), p1 = ex2(a1);
            sum2 = add_f32x2(sum2, pack_f32x2(p0, p1));
            w[c] = pack_16x2<P::F16>(p0, p1);
          }
          float s0, s1;
          unpack_f32x2(sum2, s0, s1);
          l += s0 + s1;
        }
        // the last block's P V is done: P may be overwritten, and O rescaled
        if (g > 0) {
          if (!tc::mbar_wait(&sh->pv_done, (g - 1) & 1u, abort)) return false;
          tc::fence_after_sync();
          if (j > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t oc = lanes + O_COL + (uint32_t)(kh * 64 + hh * 32);
              uint32_t v[32];
              tc::tmem_ld_32x32b_x32(oc, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
              tc::tmem_st_32x32b_x32(oc, v);
            }
          }
        }
        // P: the words in hand; a full block's products read the others as zeros
        if constexpr (NW >= 2) {
#pragma unroll
          for (int h = 0; h < NW / 2; ++h) {
            uint32_t (&wh)[32] = *reinterpret_cast<uint32_t(*)[32]>(&w[32 * h]);
            tc::tmem_st_32x32b_x32(lanes + P_COL + (uint32_t)(kh * 64 + 32 * h), wh);
          }
        } else if (p.keys(it, j) == BN) {
          uint32_t z[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) z[c] = 0u;
          tc::tmem_st_32x32b_x32(lanes + P_COL + (uint32_t)(kh * 64), z);
          tc::tmem_st_32x32b_x32(lanes + P_COL + (uint32_t)(kh * 64 + 32), z);
        }
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_cluster_relaxed(p_ready0);
        return true;
      };
      for (int j = 0; ok && j < it.n; ++j, ++g) {
        if constexpr (P::PARTIAL) {
          const bool some = p.sees(it, j, rank, r, kh);
          ok = some ? block(Words<4>{}, j) : block(Words<0>{}, j);
        } else {
          ok = block(Words<4>{}, j);
        }
      }
      if (!ok) break;
      // The output warps have read what was here two items ago: this block waited
      // for a P V that was issued after they had read that item's O.
      sh->part_l[t & 1][kh][r] = l;
      if (kh == 0) sh->row_m[t & 1][r] = m_ref;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh->l_ready[t & 1]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == TMA_WARP) {
      // ------------------------------------------------------ TMA ----
      if (lane == 0) {
        tc::prefetch_tmap(&tmQ);
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
        uint32_t g = 0;                                 // key blocks loaded so far
        bool ok = true;
        typename P::Item it;
        for (int t = 0; ok; ++t) {
          if (!p.item(t, cluster, nclusters, it)) break;
          const int qb = t & 1;
          if (!(ok = tc::mbar_wait(&sh->q_empty[qb], ((uint32_t)(t >> 1) & 1u) ^ 1u, abort))) break;
          if (rank == 0) tc::mbar_arrive_expect_tx(&sh->q_full[qb], 2 * p.q_bytes());
          p.load_q(sQ + qb * TILE_BYTES, &tmQ, tc::mapa(tc::smem_u32(&sh->q_full[qb]), 0), it, rank);
          for (int j = 0; j < it.n; ++j, ++g) {
            const int s = (int)(g & 1u);
            const uint32_t ph = (g >> 1) & 1u;
            if (!(ok = tc::mbar_wait(&sh->k_empty[s], ph ^ 1u, abort))) break;
            if (rank == 0) tc::mbar_arrive_expect_tx(&sh->k_full[s], 2 * TILE_BYTES);
            p.load_k(sK + s * TILE_BYTES, &tmK, tc::mapa(tc::smem_u32(&sh->k_full[s]), 0), it, j, rank);
            if (!(ok = tc::mbar_wait(&sh->v_empty[s], ph ^ 1u, abort))) break;
            if (rank == 0) tc::mbar_arrive_expect_tx(&sh->v_full[s], 2 * p.v_bytes(it, j));
            p.load_v(sV + s * TILE_BYTES, &tmV, &tmW, tc::mapa(tc::smem_u32(&sh->v_full[s]), 0), it, j,
                   rank);
          }
        }
      }
    } else if (warp == MMA_WARP) {
      // ------------------------------------------------------ MMA ----
      if (lane == 0 && rank == 0) {
        constexpr uint32_t idesc_s = idesc_16<P::F16>(2 * BM, BN, false);
        constexpr uint32_t idesc_s_narrow = idesc_16<P::F16>(2 * BM, NARROW, false);
        constexpr uint32_t idesc_s_mixed = idesc_16<P::F16>(2 * BM, MIXED, false);
        constexpr uint32_t idesc_pv = idesc_16<P::F16>(2 * BM, HD, true);
        // first K-step descriptors; a K-step adds its byte offset >> 4
        const uint64_t q_desc0 = tc::sdesc_sw128(tc::smem_u32(sQ), 16, 1024);
        const uint64_t q_desc1 = tc::sdesc_sw128(tc::smem_u32(sQ + TILE_BYTES), 16, 1024);
        static_assert(STAGES == 2, "one descriptor per stage, picked by g & 1");
        const uint64_t k_desc0 = tc::sdesc_sw128(tc::smem_u32(sK), 16, 1024);
        const uint64_t k_desc1 = tc::sdesc_sw128(tc::smem_u32(sK + TILE_BYTES), 16, 1024);
        // V halves are MN-major: 128-byte rows of 64 head-dimension columns,
        // 8-key groups 1 KiB apart (one swizzle atom wide, so the leading
        // offset is not used)
        const uint64_t v_desc0 = tc::sdesc_sw128(tc::smem_u32(sV), TILE_BYTES, 1024);
        const uint64_t v_desc1 = tc::sdesc_sw128(tc::smem_u32(sV + TILE_BYTES), TILE_BYTES, 1024);
        // S(g) = Q K^T from Q buffer qb: eight K-steps of 16 head-dimension
        // columns; the second 64 columns sit in the second swizzled box.  The
        // item's last S also releases its Q buffer.
        auto issue_s = [&](uint32_t g, int qb, int keys, bool last_of_item) -> bool {
          const int s = (int)(g & 1u);
          if (!tc::mbar_wait(&sh->k_full[s], (g >> 1) & 1u, abort)) return false;
          tc::fence_after_sync();
          const uint64_t kd = s ? k_desc1 : k_desc0;
          const uint64_t qd = qb ? q_desc1 : q_desc0;
          const uint32_t idesc = keys == BN ? idesc_s : keys == MIXED ? idesc_s_mixed : idesc_s_narrow;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * HALF_BYTES + (kk & 3) * 32) >> 4);
            tc::mma_pair_f16_ss(tmem + S_COL, qd + off, kd + off, idesc, kk != 0);
          }
          tc::commit_pair_both(&sh->s_full);
          tc::commit_pair_both(&sh->k_empty[s]);
          if (last_of_item) tc::commit_pair_both(&sh->q_empty[qb]);
          return true;
        };
        // O [+]= P V(g): sixteen K-steps of 16 keys (8 TMEM columns of P, 2 KiB of V)
        auto issue_pv = [&](uint32_t g, int keys, bool accumulate, bool last_of_item) -> bool {
          const int s = (int)(g & 1u);
          if (!tc::mbar_wait(&sh->v_full[s], (g >> 1) & 1u, abort)) return false;
          tc::fence_after_sync();
          const uint64_t vd = s ? v_desc1 : v_desc0;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            if ((kk == NARROW / 16 || kk == MIXED / 16) && kk * 16 >= keys) break;
            tc::mma_pair_f16_ts(tmem + O_COL, tmem + P_COL + (uint32_t)(kk * 8),
                                vd + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                                (accumulate || kk > 0) ? 1u : 0u);
          }
          tc::commit_pair_both(&sh->pv_done);
          tc::commit_pair_both(&sh->v_empty[s]);
          if (last_of_item) tc::commit_pair_both(&sh->o_full);
          return true;
        };
        // the first item's first S; then per block g: S(g + 1) (of this item or
        // the next) as soon as S(g) has been read, then P V(g) once P(g) is in
        typename P::Item it, next;
        bool ok = p.item(0, cluster, nclusters, it);
        if (ok) ok = tc::mbar_wait(&sh->q_full[0], 0, abort) && issue_s(0, 0, p.keys(it, 0), it.n == 1);
        uint32_t g = 0;
        for (int t = 0; ok; ++t) {
          const bool has_next = p.item(t + 1, cluster, nclusters, next);
          for (int j = 0; ok && j < it.n; ++j, ++g) {
            if (j + 1 < it.n || has_next) {
              // S(g + 1) overwrites S(g): both CTAs' softmax warps have read it
              if (!(ok = tc::mbar_wait(&sh->s_free, g & 1u, abort))) break;
              if (j + 1 < it.n) {
                ok = issue_s(g + 1, t & 1, p.keys(it, j + 1), j + 2 == it.n);
              } else {
                const int qb = (t + 1) & 1;
                ok = tc::mbar_wait(&sh->q_full[qb], ((uint32_t)(t + 1) >> 1) & 1u, abort) &&
                     issue_s(g + 1, qb, p.keys(next, 0), next.n == 1);
              }
              if (!ok) break;
            }
            if (!(ok = tc::mbar_wait(&sh->p_ready, g & 1u, abort))) break;
            // the item's first P V overwrites O: the last item's O has been read
            if (j == 0 && t > 0 && !(ok = tc::mbar_wait(&sh->o_free, (uint32_t)(t - 1) & 1u, abort)))
              break;
            ok = issue_pv(g, p.keys(it, j), j > 0, j + 1 == it.n);
          }
          if (!has_next) break;
          it = next;
        }
      }
    } else if (warp >= OUT_WARP) {
      // ---------------------------------------------------- output ----
      const int quarter = warp - OUT_WARP;            // TMEM lanes 32 quarter .. + 31
      const int r = quarter * 32 + lane;              // this thread's row of the tile
      const uint32_t o_cols = tmem + ((uint32_t)(quarter * 32) << 16) + O_COL;
      const uint32_t o_free0 = tc::mapa(tc::smem_u32(&sh->o_free), 0);
      bool ok = true, repair = false;
      typename P::Item it;
      for (int t = 0; ok; ++t) {
        if (!p.item(t, cluster, nclusters, it)) break;
        const int b = t & 1;
        // a whole item may pass meanwhile: 20 us more for each of its blocks (one takes 2)
        const unsigned long long limit = tc::kWaitLimitNs + (unsigned long long)it.n * 20000ull;
        ok = tc::mbar_wait(&sh->l_ready[b], (uint32_t)(t >> 1) & 1u, abort, limit) &&
             tc::mbar_wait(&sh->o_full, (uint32_t)t & 1u, abort);
        if (!ok) break;
        tc::fence_after_sync();
        const float lt = sh->part_l[b][0][r] + sh->part_l[b][1][r], m = sh->row_m[b][r];
        const typename P::Pending pending = p.pending(it, rank, r);
        // with STAGED, the warp's 32 rows x 64 columns twice, swizzled as the
        // map's box, over the item's own Q tile, whose products are long done
        uint8_t* box = sQ + b * TILE_BYTES + quarter * 4096;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t v[32];
          tc::tmem_ld_32x32b_x32(o_cols + (uint32_t)(32 * c), v);
          tc::tmem_ld_wait();
          if (c == HD / 32 - 1) {                     // all of O is in registers or out
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_cluster_relaxed(o_free0);
          }
          if constexpr (P::STAGED) {
            uint32_t w[16];
            repair |= p.pack(pending, 32 * c, v, m, lt, w);
            uint8_t* row = box + (c >> 1) * HALF_BYTES + lane * 128;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(row + ((((c & 1) * 4 + e) ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          } else {
            p.store(pending, 32 * c, v, m, lt);
          }
        }
        if constexpr (P::STAGED) {
          tc::fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) {
            p.send(&tmO, box, pending);
            tc::bulk_commit();
            tc::bulk_wait_read();                     // the Q buffer may be filled again
            tc::mbar_arrive(&sh->q_empty[b]);
          }
          __syncwarp();
        }
      }
      // no output is read from shared memory after the CTA is gone
      if (P::STAGED && lane == 0) tc::bulk_wait();
      __syncwarp();
      if (ok) p.after(repair, cluster, nclusters, rank, r);
    }
  }

  tc::fence_before_sync();
  __syncwarp();
  // neither CTA leaves while the other may still copy, commit or arrive into it
  tc::cluster_sync();
  if (warp == MMA_WARP) {
    if (*abort) {
      const unsigned long long t0 = tc::globaltimer_ns();
      while (tc::globaltimer_ns() - t0 < 200000ull) {
      }
    }
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

inline cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, unsigned grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// clusters of two of these CTAs that are resident at once on the current
// device (cached per device); 0 when none fits
template <class P>
int resident_pairs() {
  static std::atomic<int> count[64];
  static std::atomic<uint64_t> attr_done{0}, known{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const uint64_t bit = 1ull << dev;
  if (known.load(std::memory_order_acquire) & bit) return count[dev].load();
  int n = 0;
  // launched with fewer registers than the warpgroups' shares add up to, the
  // softmax warps would wait for them for ever
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, attn_pair_kernel<P>) == cudaSuccess && fa.numRegs == REGS &&
      smem_attr(attn_pair_kernel<P>, SMEM_BYTES, attr_done) == RF_OK) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pair_config(attr, 2u, 0);
    if (cudaOccupancyMaxActiveClusters(&n, attn_pair_kernel<P>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  count[dev].store(n);
  known.fetch_or(bit, std::memory_order_release);
  return n;
}

template <class P>
rf_status launch_pair(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      const CUtensorMap& w, const CUtensorMap& o, const P& p, int clusters,
                      cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config(attr, 2u * (unsigned)clusters, st);
  if (P::CHAINED) {
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  if (cudaLaunchKernelEx(&cfg, attn_pair_kernel<P>, q, k, v, w, o, p) != cudaSuccess) {
    cudaGetLastError();
    return RF_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace pair
}  // namespace rf
