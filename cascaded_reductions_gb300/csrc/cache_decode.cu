// Single-token decode over a cache of grouped heads: H query heads share Hkv
// key/value heads (head h reads key head h / G, G = H / Hkv), every sequence
// has its own length, and a mask may leave only the last `window` keys and the
// first `sinks` visible.  The same kernels, with their states numbered after
// those of the prefix kernel, are the suffix half of the shared-prefix decode (and
// all of it in a small call, with the prefix as every sequence's first keys),
// with their scores kept they feed the running total of each key's weight, and
// with a group per position they are the windowed prefill of a few rows.
//
// Mathematics: per row the cascade of the split-KV decode (running m, l, acc,
// rescale by exp2(m_old - m_new), states merged by the same rescale).
//
// What bounds it: HBM.  A key of a key head costs 512 bytes (K and V) and
// 4 G D = 512 G flops; on the FP32 pipes G = 4 heads would already need as
// long as the bytes, so both products run on the warp-level matrix
// instruction m16n8k16: the G query heads are its 16 rows (G < 16 leaves rows
// idle, which costs nothing here: 16 keys need 48 instructions while their
// 8 KiB take an SM about 350 cycles).
//
// Only visible keys are read: positions are numbered over the visible keys and
// mapped to cache rows, in tiles of 16 per warp; a warp fills a ring of its own
// (3 stages of 8 KiB) by 16-byte asynchronous copies.  Rows past a group's end
// are zero-filled, never read.
//
// P in two terms: the weights enter the second product as hi + lo, two 16-bit
// terms, so that they carry 16 (bf16) or 22 (fp16) bits and the output is
// rounded once; the 16 extra matrix instructions per tile are free here.  fp16
// ends at 2^-24, so its weights are taken 2^15 times as large (at most 2^15, of
// 65504): 22 bits down to 2^-18 of the warp's largest, and no more than 2^-40 of it lost.
// An infinite value times lo = 0, or times a lo below 0, makes its column NaN, so a
// piece's columns that are NaN are computed again with whole weights (redo_columns).
//
// Split: a row group (sequence, key head, 16-row tile of query heads) is divided
// into pieces by its own length, one CTA of four warps each; a step of the CTA
// is 64 keys, a tile per warp.  Warps merge through shared memory, a row per warp
// and four columns per lane (1216 rows of 128 keys: 21.9 us; 26.6 us when one warp
// took over the others' fragments, idle rows and all), pieces
// through state slots in memory: in small calls by the last CTA of the group to
// arrive (no second launch), in large ones by merge_kernel, launched to begin
// beside the last CTAs, because the fence and the count hold up the end of a
// CTA (a shared-prefix step of 128 sequences: 115 us with them, 103 us without).
// Both merge in order: the same lengths give the same bits.
//
// Measured (64 sequences, 8 key heads, 4100 visible keys each, 1.07 GB): 158 us,
// 6.8 TB/s, the card's copy rate, with pieces of 768 keys or more; 170 us with
// 512, where a CTA's start and end weigh more.  Pure streaming by the same
// copies takes 153 us.  Also built: equal contiguous shares of all tiles per
// warp, 173 us, or per CTA, 166 us (SMs stream at rates up to 10 % apart, which
// equal shares wait for), and per-warp shares with smaller units taken later
// from a queue, 188 us (a warp holds an eighth of an SM's bandwidth, so even a
// unit of six tiles takes 10 us).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace rf {
namespace {

constexpr int HD = 128;                 // head dimension
constexpr int ROW_BYTES = HD * 2;
constexpr int TK = kDecodeTile;         // keys per warp tile
static_assert(TK == 16, "two n8 tiles of scores, one k16 step of weights");
constexpr int WARPS = 4;
constexpr int STAGES = 3;
constexpr int STAGE_BYTES = 2 * TK * ROW_BYTES;   // K tile, V tile
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int MROWS = 16;               // query heads per row group
constexpr size_t SMEM_BYTES = (size_t)WARPS * RING_BYTES;
// floats per row of the merge buffer: 8 more than a row has, so that the eight
// rows of a fragment's store lie 8 banks apart
constexpr int MERGE_PITCH = HD + 8;
static_assert((size_t)WARPS * MROWS * MERGE_PITCH * 4 <= SMEM_BYTES, "the warps' accumulators reuse the rings");

// 16 bytes (or, for bytes = 0, zeros) with an L2 eviction policy
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes,
                                           uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(bytes), "l"(policy)
               : "memory");
}
__device__ __forceinline__ uint64_t l2_policy(bool evict_first) {
  uint64_t p;
  if (evict_first)
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// p0, p1 as hi + lo in the 16-bit type, packed for the A operand
template <bool F16>
__device__ __forceinline__ void split16(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  if constexpr (F16) {
    hi = pack_f16x2(p0, p1);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16x2(p0 - h.x, p1 - h.y);
  } else {
    hi = pack_bf16x2(p0, p1);
    lo = pack_bf16x2(p0 - bf16_lo(hi), p1 - bf16_hi(hi));
  }
}

// elements i and i + 1 (i even) of the output
__device__ __forceinline__ void store_out2(void* out, size_t i, float x, float y, int dtype) {
  if (dtype == RF_F32)
    *reinterpret_cast<float2*>(static_cast<float*>(out) + i) = make_float2(x, y);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + i) =
        dtype == RF_F16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
}

// acc / l, and 0 where the row has no weight at all (no visible key); a NaN
// sum stays NaN
__device__ __forceinline__ float normalised(float acc, float l) { return l == 0.f ? 0.f : acc / l; }

// A row group's keys: the visible ones of its sequence.
struct Group {
  int n, lo, ns;         // visible keys; key t is cache row t (t < ns) or t - ns + lo
  size_t kv0;            // first cache row of its key head
  size_t prefix0;        // with a prefix, key t < ns is its row prefix0 + t instead
};

__device__ __forceinline__ int visible_keys(const CacheDecode& a, int b, int& lo, int& ns) {
  int len = a.cap;
  if (a.lens != nullptr && RF_IDX_OK(b, a.B)) len = min(max(a.lens[b], 0), a.cap);
  lo = a.window > 0 ? max(0, len - a.window) : 0;
  ns = a.prefix > 0 ? a.prefix : min(a.sinks, lo);
  return ns + len - lo;
}

// tiles of n keys; at least one, so that a group without keys has an owner
__device__ __forceinline__ int tiles_of(int n) { return n > TK ? (n + TK - 1) / TK : 1; }

// group g = (b Hkv + key head) mtiles + tile of query heads; with POSITIONS, b is
// (sequence, position) and the position sees what lies before it
template <bool POSITIONS = false>
__device__ __forceinline__ Group group_of(const CacheDecode& a, int g) {
  Group r;
  const int head = g / a.mtiles;
  if constexpr (POSITIONS) {
    const int bp = head / a.Hkv, b = bp / a.positions, len = a.cap - a.positions + (bp - b * a.positions) + 1;
    r.lo = a.window > 0 ? max(0, len - a.window) : 0;
    r.ns = min(a.sinks, r.lo);
    r.n = r.ns + len - r.lo;
    r.kv0 = ((size_t)b * a.Hkv + (head - bp * a.Hkv)) * a.cap;
    r.prefix0 = 0;
    return r;
  }
  r.n = visible_keys(a, head / a.Hkv, r.lo, r.ns);
  r.kv0 = (size_t)head * a.cap;
  r.prefix0 = (size_t)(head % a.Hkv) * a.prefix;
  return r;
}

struct Rows {
  size_t row0, step;     // first query row, distance of one head's to the next
  int n;                 // 1 .. 16
};
template <bool POSITIONS = false>
__device__ __forceinline__ Rows rows_of(const CacheDecode& a, int g) {
  const int head = g / a.mtiles, mt = g - head * a.mtiles;
  const int b = head / a.Hkv, hk = head - b * a.Hkv;
  const int first = hk * a.G + mt * MROWS, n = min(MROWS, a.G - mt * MROWS);
  if constexpr (POSITIONS) {
    const int seq = b / a.positions;
    return {((size_t)seq * a.H + first) * a.positions + (b - seq * a.positions), (size_t)a.positions, n};
  }
  return {(size_t)b * a.H + first, 1, n};
}
// query rows of the call (for the checked build)
[[maybe_unused]] __device__ __forceinline__ size_t rows_in(const CacheDecode& a) {
  return (size_t)a.B * a.H * (a.positions > 0 ? a.positions : 1);
}

// The warp's copies of keys t0 .. t0 + 15 of a group into one stage: K rows,
// then V rows, 16-byte chunks permuted by row % 8 so that ldmatrix meets all
// banks; two rows per instruction.
template <bool PREFIX>
__device__ __forceinline__ void copy_tile(const CacheDecode& a, const Group& q, int t0, uint32_t stage,
                                          uint64_t policy, int lane) {
#pragma unroll
  for (int u = 0; u < TK / 2; ++u) {
    const int r = 2 * u + (lane >> 4), c = lane & 15;
    const int t = t0 + r;
    const int key = t < q.ns ? t : t - q.ns + q.lo;
    const bool shared = PREFIX && t < q.ns;
    const size_t row = (shared ? q.prefix0 : q.kv0) + key;
    (void)row;                                    // read by the checked build only
    const bool in = t < q.n && RF_IDX_OK(row, (size_t)a.Hkv * (shared ? (size_t)a.prefix : (size_t)a.B * a.cap));
    const size_t off = ((shared ? q.prefix0 : q.kv0) + (in ? key : 0)) * ROW_BYTES + c * 16;
    const uint32_t dst = stage + r * ROW_BYTES + ((c ^ (r & 7)) << 4);
    cp_async16(dst, (shared ? a.kp : a.k) + off, in ? 16u : 0u, policy);
    cp_async16(dst + TK * ROW_BYTES, (shared ? a.vp : a.v) + off, in ? 16u : 0u, policy);
  }
}

// One warp's running state of a row group: rows lane / 4 (index 0) and + 8
// (index 1); acc[d] holds columns 8 d + 2 (lane % 4) and + 1 of both.
template <bool F16, bool SCORES, bool POSITIONS>
struct State {
  // The weights' reference for the maximum m; the state given away has it for its m.
  // From 2^24 on m - 15 may round to m - 16 or less, and a weight to 2^16: m itself then.
  static __device__ __forceinline__ float below(float m) {
    if constexpr (!F16) return m;
    const float f = m - 15.f;
    return m - f > 15.5f ? m : f;
  }
  uint32_t qf[HD / 16][4];
  float acc[HD / 8][4];
  float m0, m1, l0, l1;

  __device__ __forceinline__ void start(const CacheDecode& a, const Rows& w, int lane) {
    // Q fragments: columns 16 kk + 2 (lane % 4) (+ 8) of the two rows
    const int r = lane >> 2;
    const size_t step = POSITIONS ? w.step : 1;
    const bool in0 = r < w.n && RF_IDX_OK(w.row0 + r * step, rows_in(a));
    const bool in1 = r + 8 < w.n && RF_IDX_OK(w.row0 + (r + 8) * step, rows_in(a));
    const uint8_t* q0 = a.q + (w.row0 + r * step) * ROW_BYTES + (lane & 3) * 4;
    const uint8_t* q1 = q0 + 8 * step * ROW_BYTES;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      qf[kk][0] = in0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32) : 0u;
      qf[kk][1] = in1 ? *reinterpret_cast<const uint32_t*>(q1 + kk * 32) : 0u;
      qf[kk][2] = in0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32 + 16) : 0u;
      qf[kk][3] = in1 ? *reinterpret_cast<const uint32_t*>(q1 + kk * 32 + 16) : 0u;
    }
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }

  // folds in keys t0 .. min(t0 + 15, n - 1), whose copies are in `st`
  __device__ __forceinline__ void tile(const CacheDecode& a, const Rows& w, uint32_t st, int t0, int n,
                                       int lane) {
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  {
    const int r = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const int c = 2 * kk + ((lane >> 3) & 1);
      uint32_t kb[4];
      ldmatrix_x4(st + r * ROW_BYTES + ((c ^ (r & 7)) << 4), kb);
      mma16816<F16>(s[0], qf[kk], kb[0], kb[1]);
      mma16816<F16>(s[1], qf[kk], kb[2], kb[3]);
    }
  }
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = t0 + nt * 8 + 2 * (lane & 3) + e;
      const bool in = t < n;
      s[nt][e] = in ? s[nt][e] * a.scale_log2 : -INFINITY;
      s[nt][2 + e] = in ? s[nt][2 + e] * a.scale_log2 : -INFINITY;
      mx0 = fmaxf(mx0, s[nt][e]);
      mx1 = fmaxf(mx1, s[nt][2 + e]);
    }
  if constexpr (SCORES) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int t = t0 + nt * 8 + 2 * (lane & 3);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = (lane >> 2) + 8 * half;
        if (r >= w.n || t >= n) continue;
        float* at = a.scores + (w.row0 + r) * a.cap + t;
        const size_t i = (w.row0 + r) * a.cap + t, all = (size_t)a.B * a.H * a.cap;
        (void)i, (void)all;                       // read by the checked build only
        if (t + 1 < n && a.cap % 2 == 0) {        // t is even, and so the pair is aligned
          if (RF_SPAN_OK(i, 2, all))
            *reinterpret_cast<float2*>(at) = make_float2(s[nt][2 * half], s[nt][2 * half + 1]);
        } else {
          if (RF_IDX_OK(i, all)) at[0] = s[nt][2 * half];
          if (t + 1 < n && RF_IDX_OK(i + 1, all)) at[1] = s[nt][2 * half + 1];
        }
      }
    }
  }
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
  mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
  mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
  const bool grew = mx0 > m0 || mx1 > m1;
  if (__any_sync(0xffffffffu, grew)) {
    const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
    // differences of the rounded references themselves
    const float c0 = exp2f(below(m0) - below(ref_of(n0))), c1 = exp2f(below(m1) - below(ref_of(n1)));
    m0 = n0;
    m1 = n1;
    l0 *= c0;
    l1 *= c1;
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) {
      acc[d][0] *= c0;
      acc[d][1] *= c0;
      acc[d][2] *= c1;
      acc[d][3] *= c1;
    }
  }
  const float f0 = below(ref_of(m0)), f1 = below(ref_of(m1));
  uint32_t hi[4], lw[4];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const float p00 = exp2f(s[nt][0] - f0), p01 = exp2f(s[nt][1] - f0);
    const float p10 = exp2f(s[nt][2] - f1), p11 = exp2f(s[nt][3] - f1);
    l0 += p00 + p01;
    l1 += p10 + p11;
    split16<F16>(p00, p01, hi[2 * nt], lw[2 * nt]);
    split16<F16>(p10, p11, hi[2 * nt + 1], lw[2 * nt + 1]);
  }
  {
    const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      const int c = 2 * d + (lane >> 4);
      uint32_t vb[4];
      ldmatrix_x4_trans(st + TK * ROW_BYTES + r * ROW_BYTES + ((c ^ (r & 7)) << 4), vb);
      mma16816<F16>(acc[2 * d], hi, vb[0], vb[1]);
      mma16816<F16>(acc[2 * d + 1], hi, vb[2], vb[3]);
      mma16816<F16>(acc[2 * d], lw, vb[0], vb[1]);
      mma16816<F16>(acc[2 * d + 1], lw, vb[2], vb[3]);
    }
  }
  }

  // the row sums over the four lanes that share a row; once, before the state is used
  __device__ __forceinline__ void close() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  }

  // the warp's rows into its part of the merge buffer
  __device__ __forceinline__ void give(float* acc_buf, float2* ml_buf, const Rows& w, int lane) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = (lane >> 2) + 8 * half;
      if (r >= w.n) continue;
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
        *reinterpret_cast<float2*>(acc_buf + r * MERGE_PITCH + d * 8 + 2 * (lane & 3)) =
            make_float2(acc[d][2 * half], acc[d][2 * half + 1]);
      if ((lane & 3) == 0) ml_buf[r] = half ? make_float2(below(m1), l1) : make_float2(below(m0), l0);
    }
  }
};

__device__ __forceinline__ bool any_nan(const float4& x) {
  return x.x != x.x || x.y != x.y || x.z != x.z || x.w != x.w;
}

// Columns 4 lane .. + 3 of a 16-bit row, widened
template <bool F16>
__device__ __forceinline__ float4 load_row4(const uint8_t* row, int lane) {
  const uint2 u = *reinterpret_cast<const uint2*>(row + lane * 8);
  if constexpr (F16) {
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  } else {
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  }
}

// A row's accumulator A over keys t0 .. t1 - 1, weights relative to `ref`, with the
// columns that are NaN computed again key by key: a visible value of +-inf gives that
// infinity.  Ends once they are all NaN again (a NaN value, or both infinities), which
// they stay.  A call, so that the code of it lies out of the kernels' way: in line it
// cost the single-token decode 0.2 of 5.6 us, although it does not run.
struct Redo {
  const uint8_t *q, *k, *v, *kp, *vp;    // the row; the group's keys and, before them, the prefix's
  int ns, lo;                            // as in Group
  int prefix, rows;                      // of kp and of k
  int t0, t1;
  float ref, scale_log2;
};
template <bool F16, bool PREFIX>
__device__ __noinline__ float4 redo_columns(const Redo d, float4 A, int lane) {
  constexpr int U = 8;                            // keys in flight
  const float4 x = load_row4<F16>(d.q, lane);
  float4 R = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t = d.t0; t < d.t1; t += U) {
    float s[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool shared = PREFIX && t + u < d.ns;
      const int key = t + u < d.ns ? t + u : t + u - d.ns + d.lo;
      float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
      v[u] = k;
      if (t + u < d.t1 && RF_IDX_OK(key, shared ? d.prefix : d.rows)) {
        k = load_row4<F16>((shared ? d.kp : d.k) + (size_t)key * ROW_BYTES, lane);
        v[u] = load_row4<F16>((shared ? d.vp : d.v) + (size_t)key * ROW_BYTES, lane);
      }
      s[u] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, x.w * k.w)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = t + u < d.t1 ? exp2f(__fmul_rn(s[u], d.scale_log2) - d.ref) : 0.f;
      R.x = fmaf(w, v[u].x, R.x);
      R.y = fmaf(w, v[u].y, R.y);
      R.z = fmaf(w, v[u].z, R.z);
      R.w = fmaf(w, v[u].w, R.w);
    }
    const bool again = (A.x != A.x && R.x == R.x) || (A.y != A.y && R.y == R.y) ||
                       (A.z != A.z && R.z == R.z) || (A.w != A.w && R.w == R.w);
    if (!__any_sync(0xffffffffu, again)) break;
  }
  return make_float4(A.x != A.x ? R.x : A.x, A.y != A.y ? R.y : A.y, A.z != A.z ? R.z : A.z,
                     A.w != A.w ? R.w : A.w);
}

// Row r of the CTA's warps merged by one warp, four columns per lane, into out
// and lse (`direct`: this was the whole group) or into the row's state `slot`.
// The CTA's keys are t0 .. t1 - 1 of group q.
template <bool F16, bool SCORES, bool PREFIX>
__device__ __forceinline__ void merge_warps(const CacheDecode& a, const float* acc_buf,
                                            const float2 (*ml_buf)[MROWS], size_t row, int r,
                                            bool direct, int slot, const Group& q, int t0, int t1,
                                            int lane) {
  if (!RF_IDX_OK(row, rows_in(a))) return;
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) M = fmaxf(M, ml_buf[i][r].x);
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const float2 ml = ml_buf[i][r];
    const float f = exp2f(ml.x - ref_of(M));
    const float4 v = *reinterpret_cast<const float4*>(acc_buf + (i * MROWS + r) * MERGE_PITCH + lane * 4);
    L = fmaf(f, ml.y, L);
    A.x = fmaf(f, v.x, A.x);
    A.y = fmaf(f, v.y, A.y);
    A.z = fmaf(f, v.z, A.z);
    A.w = fmaf(f, v.w, A.w);
  }
  if (__any_sync(0xffffffffu, L > 0.f && any_nan(A))) {
    const size_t own = q.kv0 * ROW_BYTES, pre = PREFIX ? q.prefix0 * ROW_BYTES : 0;
    A = redo_columns<F16, PREFIX>({a.q + row * ROW_BYTES, a.k + own, a.v + own, a.kp + pre, a.vp + pre, q.ns, q.lo,
                                   a.prefix, a.cap, t0, t1, ref_of(M), a.scale_log2},
                                  A, lane);
  }
  const size_t states = (size_t)a.B * a.H * a.S_total;
  (void)states;                                   // read by the checked build only
  if (direct) {
    const size_t o = row * HD + lane * 4;
    store_out2(a.out, o, normalised(A.x, L), normalised(A.y, L), a.out_dtype);
    store_out2(a.out, o + 2, normalised(A.z, L), normalised(A.w, L), a.out_dtype);
    if (lane == 0) {
      const float lse2 = M + log2f(L);
      if (a.lse != nullptr) a.lse[row] = lse2 * kLn2;
      if (SCORES && RF_IDX_OK(row * a.S_total, states)) a.seg_m[row * a.S_total] = lse2;
    }
  } else {
    const size_t s = row * a.S_total + slot;
    if (!RF_IDX_OK(s, states)) return;
    *(reinterpret_cast<float4*>(a.seg_acc + s * HD) + lane) = A;
    if (lane == 0) {
      a.seg_m[s] = M;
      a.seg_l[s] = L;
    }
  }
}

// Merges a group's rows, their states in order: the prefix's slots
// 0 .. seg0 - 1 and this kernel's seg0 .. seg0 + pieces - 1.  One warp, four
// columns per lane; RB rows and 32 / RB states are in flight at a time.
template <int RB, bool SCORES>
__device__ void merge_rows(const CacheDecode& a, size_t row0, int rows, int pieces, int lane) {
  const size_t states = (size_t)a.B * a.H * a.S_total;
  (void)states;                                   // read by the checked build only
  constexpr int SB = 32 / RB;                     // states in flight: 32 loads per lane
  const int n = a.seg0 + pieces;
  for (int r0 = 0; r0 < rows; r0 += RB) {
    const int nr = min(RB, rows - r0);
    float M[RB], L[RB];
    float4 A[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      M[r] = -INFINITY;
      L[r] = 0.f;
      A[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int cnt = min(32, n - s0);
      // lane j holds state s0 + j's maximum and sum, then its weight; -1 marks one
      // without keys.  The accumulators are asked for before the weights are known:
      // one wait for memory instead of three (1 sequence of 1028 visible keys:
      // 6.8 -> 5.7 us).
      float ms[RB], ls[RB], f[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        ms[r] = -INFINITY;
        ls[r] = 0.f;
        const size_t at = (row0 + r0 + r) * a.S_total + s0 + lane;
        if (r < nr && lane < cnt && RF_IDX_OK(at, states)) {
          ms[r] = __ldcg(a.seg_m + at);
          ls[r] = __ldcg(a.seg_l + at);
        }
      }
      for (int j0 = 0; j0 < cnt; j0 += SB) {
        float4 v[RB][SB];
#pragma unroll
        for (int j = 0; j < SB; ++j)
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            const size_t at = (row0 + r0 + r) * a.S_total + s0 + j0 + j;
            v[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nr && j0 + j < cnt && RF_SPAN_OK(at * HD + lane * 4, 4, states * HD))
              v[r][j] = __ldcg(reinterpret_cast<const float4*>(a.seg_acc + at * HD) + lane);
          }
        if (j0 == 0) {
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            const float top = fmaxf(M[r], group_max<32>(ms[r])), c = exp2f(M[r] - ref_of(top));
            M[r] = top;
            L[r] *= c;
            A[r].x *= c;
            A[r].y *= c;
            A[r].z *= c;
            A[r].w *= c;
            f[r] = -1.f;
            if (ms[r] != -INFINITY) {
              f[r] = exp2f(ms[r] - ref_of(top));
              L[r] = fmaf(f[r], ls[r], L[r]);
            } else {
              L[r] += ls[r];                      // 0, or NaN where every score was NaN
            }
          }
        }
#pragma unroll
        for (int j = 0; j < SB; ++j)
#pragma unroll
          for (int r = 0; r < RB; ++r) {
            const float fj = __shfl_sync(0xffffffffu, f[r], (j0 + j) & 31);
            if (j0 + j >= cnt || fj == -1.f) continue;
            A[r].x = fmaf(fj, v[r][j].x, A[r].x);
            A[r].y = fmaf(fj, v[r][j].y, A[r].y);
            A[r].z = fmaf(fj, v[r][j].z, A[r].z);
            A[r].w = fmaf(fj, v[r][j].w, A[r].w);
          }
      }
    }
    __syncwarp();                                 // every lane has read the rows' seg_m
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      L[r] = group_sum<32>(L[r]);
      const size_t row = row0 + r0 + r;
      if (r >= nr || !RF_IDX_OK(row, (size_t)a.B * a.H)) continue;
      const size_t o = row * HD + lane * 4;
      store_out2(a.out, o, normalised(A[r].x, L[r]), normalised(A[r].y, L[r]), a.out_dtype);
      store_out2(a.out, o + 2, normalised(A[r].z, L[r]), normalised(A[r].w, L[r]), a.out_dtype);
      if (lane == 0) {
        const float lse2 = M[r] + log2f(L[r]);
        if (a.lse != nullptr) a.lse[row] = lse2 * kLn2;
        if (SCORES && RF_IDX_OK(row * a.S_total, states)) a.seg_m[row * a.S_total] = lse2;
      }
    }
  }
}

// Pieces of a group of n keys: none below piece_keys, at most S.
__device__ __forceinline__ int pieces_of(const CacheDecode& a, int n) {
  return max(1, min(a.S, (n + a.piece_keys - 1) / a.piece_keys));
}

// One CTA per (group, piece); pieces that a group does not have return at once.
// PREFIX: keys of a shared prefix come before every sequence's own.  POSITIONS: a
// group for each of a prompt's last positions, whole (S = 1).
template <bool F16, bool SCORES, bool FUSED, bool PREFIX, bool POSITIONS>
__global__ void __launch_bounds__(WARPS * 32, 2)
cache_decode_kernel(const CacheDecode a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 sm_ml[WARPS][MROWS];
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = (int)(blockIdx.x / a.S), piece = (int)(blockIdx.x - (unsigned)g * a.S);
  if (a.seg0 == 0) wait_prerequisite();   // the prefix kernel has done so for its successor
  allow_dependents();
  const Group q = group_of<POSITIONS>(a, g);
  const int pieces = pieces_of(a, q.n);
  // Done means that the prefix is done too.  Where a kernel of its own merges, one
  // CTA's wait says so for all, and the others leave their SM to the rows that
  // follow, so that SMs without a prefix cluster work on own keys all along.
  const bool waits = FUSED || blockIdx.x == 0;
  if (piece >= pieces) {
    if (waits) wait_prerequisite();
    return;
  }
  const Rows w = rows_of<POSITIONS>(a, g);
  const int steps = (tiles_of(q.n) + WARPS - 1) / WARPS;
  const int k0 = (int)((long long)steps * piece / pieces);
  const int k1 = (int)((long long)steps * (piece + 1) / pieces);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * RING_BYTES;

  // a large call's cache is loaded evict-first, so that what it leaves in L2 for the
  // next kernel (states, scores) stays; with more than 16 query heads per key head
  // each tile of them reads the same keys
  const uint64_t policy = l2_policy(!FUSED);
  int in = 0;                           // the stage that the next copies go to
  auto issue = [&](int k) {
    const int t0 = (k * WARPS + warp) * TK;
    if (k < k1 && t0 < q.n) copy_tile<PREFIX>(a, q, t0, ring + (uint32_t)in * STAGE_BYTES, policy, lane);
    cp_async_commit();
    in = in + 1 == STAGES ? 0 : in + 1;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(k0 + i);
  State<F16, SCORES, POSITIONS> st;
  st.start(a, w, lane);
  int slot = 0;
  for (int k = k0; k < k1; ++k) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();                       // every lane's copies of this step landed, the last is read
    issue(k + STAGES - 1);
    const int t0 = (k * WARPS + warp) * TK;
    if (t0 < q.n) st.tile(a, w, ring + (uint32_t)slot * STAGE_BYTES, t0, q.n, lane);
    slot = slot + 1 == STAGES ? 0 : slot + 1;
  }
  cp_async_wait<0>();
  st.close();
  __syncthreads();                      // the rings are free

  float* acc_buf = reinterpret_cast<float*>(smem);
  st.give(acc_buf + warp * MROWS * MERGE_PITCH, sm_ml[warp], w, lane);
  __syncthreads();
  const bool direct = pieces == 1 && a.seg0 == 0;   // the output itself
  const int key0 = k0 * WARPS * TK, key1 = min(q.n, k1 * WARPS * TK);
  for (int r = warp; r < w.n; r += WARPS)
    merge_warps<F16, SCORES, PREFIX>(a, acc_buf, sm_ml, w.row0 + r * (POSITIONS ? w.step : 1), r, direct,
                                     a.seg0 + piece, q, key0, key1, lane);
  if constexpr (POSITIONS) return;
  if (waits) wait_prerequisite();       // the prefix's states, where there are some
  if constexpr (FUSED) {
    if (direct) return;
    // the last piece to arrive merges the group's rows, a row per warp at a time;
    // thread 0's fences stand for the CTA, which its barriers join
    __syncthreads();
    if (threadIdx.x == 0) {
      int seen = 0;
      if (pieces > 1) {
        __threadfence();
        seen = RF_IDX_OK(g, (size_t)a.B * a.Hkv * a.mtiles) ? atomicAdd(a.counters + g, 1) : -1;
        __threadfence();
      }
      last = seen == pieces - 1;
    }
    __syncthreads();
    if (!last) return;
    // a warp's rows all at once (33 sequences of 111 visible keys, 16 heads per
    // group: 7.9 us, row by row 9.2)
    const int share = (w.n + WARPS - 1) / WARPS, r = warp * share, nr = min(share, w.n - r);
    if (nr > 0) {
      if (share == 1)
        merge_rows<1, SCORES>(a, w.row0 + r, nr, pieces, lane);
      else if (share == 2)
        merge_rows<2, SCORES>(a, w.row0 + r, nr, pieces, lane);
      else
        merge_rows<4, SCORES>(a, w.row0 + r, nr, pieces, lane);
    }
    if (threadIdx.x == 0 && pieces > 1 && RF_IDX_OK(g, (size_t)a.B * a.Hkv * a.mtiles))
      a.counters[g] = 0;
  }
}

// Merges the rows of divided groups: with few states per row a warp per group,
// four rows at a time (4096 rows of 7 states: 94 us of a whole shared-prefix
// step, 99 us with a warp per row), with many a warp per row (1024 rows of 22:
// 225 us of a weight-totalling step, 232 us with a warp per group).
template <bool SCORES, bool BY_ROW>
__global__ void __launch_bounds__(WARPS * 32)
merge_kernel(const CacheDecode a) {
  const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const bool in = unit < (BY_ROW ? (long long)a.B * a.H : (long long)a.B * a.Hkv * a.mtiles);
  allow_dependents();
  Rows w = {0, 1, 0};
  int pieces = 1;
  if (in) {
    int g = (int)unit;
    if (BY_ROW) {
      const int b = (int)(unit / a.H), h = (int)(unit - (long long)b * a.H);
      g = (b * a.Hkv + h / a.G) * a.mtiles;
    }
    pieces = pieces_of(a, group_of(a, g).n);
    w = BY_ROW ? Rows{(size_t)unit, 1, 1} : rows_of(a, g);
  }
  wait_prerequisite();
  if (!in || (pieces == 1 && a.seg0 == 0)) return;   // written by its CTA
  merge_rows<BY_ROW ? 1 : 4, SCORES>(a, w.row0, w.n, pieces, lane);
}

// total[j] = weight[j] + sum over the group's heads of exp2(score - lse2):
// the weights of the row's softmax, each below 1, summed in fp32 head by head
// in order, HEADS of them in flight at a time.  KEYS adjacent keys per thread (4:
// 16-byte accesses, for rows that stay aligned); reads 4 (G + 1) bytes and writes 4 per key.
template <int KEYS, int HEADS>
__global__ void __launch_bounds__(256)
add_weights_kernel(const float* scores, const float* seg_m, const int32_t* __restrict__ lens,
                   const float* weight, float* total, int B, int Hkv, int G, int cap, int S,
                   int blocks) {
  const int group = blockIdx.x / blocks;
  const int j = ((blockIdx.x - group * blocks) * 256 + threadIdx.x) * KEYS;
  const int b = group / Hkv;
  const size_t row0 = (size_t)group * G;                          // b * H + key head * G
  allow_dependents();
  int len = cap;
  if (lens != nullptr && RF_IDX_OK(b, B)) len = min(max(lens[b], 0), cap);
  wait_prerequisite();
  if (j >= cap) return;
  const size_t i = (size_t)group * cap + j;
  if (!RF_SPAN_OK(i, KEYS, (size_t)B * Hkv * cap)) return;
  if (j >= len && weight == total) return;        // behind the end: left as it was
  float w[KEYS] = {};
  if (weight != nullptr) {
    if constexpr (KEYS == 4)
      *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(weight + i);
    else
      w[0] = weight[i];
  }
  if (j < len) {
    for (int g0 = 0; g0 < G; g0 += HEADS) {
      float z[HEADS], x[HEADS][KEYS];
#pragma unroll
      for (int u = 0; u < HEADS; ++u) {
        const size_t at = (row0 + g0 + u) * cap + j;
        z[u] = -INFINITY;                         // a row without weight adds none
        if (g0 + u >= G || !RF_SPAN_OK(at, KEYS, (size_t)B * Hkv * G * cap)) continue;
        z[u] = __ldcg(seg_m + (row0 + g0 + u) * S);
        if constexpr (KEYS == 4)
          *reinterpret_cast<float4*>(x[u]) = __ldcs(reinterpret_cast<const float4*>(scores + at));
        else
          x[u][0] = __ldcs(scores + at);
      }
#pragma unroll
      for (int u = 0; u < HEADS; ++u) {
        if (z[u] == -INFINITY) continue;
#pragma unroll
        for (int e = 0; e < KEYS; ++e)
          if (j + e < len) w[e] += exp2f(x[u][e] - z[u]);
      }
    }
  }
  if constexpr (KEYS == 4)
    *reinterpret_cast<float4*>(total + i) = *reinterpret_cast<const float4*>(w);
  else
    total[i] = w[0];
}

template <bool F16, bool SCORES>
rf_status launch_t(const CacheDecode& a, bool few, cudaStream_t st) {
  static std::atomic<uint64_t> done_few{0}, done_many{0};
  const unsigned groups = (unsigned)(a.B * a.Hkv * a.mtiles);
  auto* kernel = few ? cache_decode_kernel<F16, SCORES, true, false, false>
                     : cache_decode_kernel<F16, SCORES, false, false, false>;
  std::atomic<uint64_t>* done = few ? &done_few : &done_many;
  if constexpr (!SCORES) {
    static std::atomic<uint64_t> done_prefix{0};
    if (a.prefix > 0) {                 // always a small call
      kernel = cache_decode_kernel<F16, false, true, true, false>;
      done = &done_prefix;
    }
  }
  if (smem_attr(kernel, SMEM_BYTES, *done) != RF_OK) return RF_ERR_CUDA;
  const rf_status s = launch_after(kernel, groups * a.S, WARPS * 32, SMEM_BYTES, st, a);
  if (s != RF_OK || few || (a.S == 1 && a.seg0 == 0)) return s;
  if (a.seg0 + a.S <= 8)
    return launch_after(merge_kernel<SCORES, false>, (groups + WARPS - 1) / WARPS, WARPS * 32, 0, st, a);
  const unsigned rows = (unsigned)(((long long)a.B * a.H + WARPS - 1) / WARPS);
  return launch_after(merge_kernel<SCORES, true>, rows, WARPS * 32, 0, st, a);
}

}  // namespace

rf_status launch_cache_decode(CacheDecode a, int dtype, cudaStream_t st) {
  a.G = a.H / a.Hkv;
  a.mtiles = (a.G + MROWS - 1) / MROWS;
  const int sms = tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  const int keys = a.window > 0 && a.window < a.cap - a.sinks ? a.window + a.sinks : a.prefix + a.cap;
  const bool few = decode_is_few((long long)a.B * a.Hkv * a.mtiles, keys, sms);
  a.piece_keys = few ? kFewKeys : kManyKeys;
  // no more pieces than the longest possible row has
  const int most = few ? (keys + kFewKeys - 1) / kFewKeys : decode_many_pieces(keys);
  if (a.S > most) a.S = most;
  if (dtype == RF_F16)
    return a.scores ? launch_t<true, true>(a, few, st) : launch_t<true, false>(a, few, st);
  return a.scores ? launch_t<false, true>(a, few, st) : launch_t<false, false>(a, few, st);
}

rf_status launch_prefill_rows(CacheDecode a, int dtype, cudaStream_t st) {
  static std::atomic<uint64_t> done[2];
  a.G = a.H / a.Hkv;
  a.mtiles = (a.G + MROWS - 1) / MROWS;
  a.S = a.S_total = 1;
  a.piece_keys = 1 << 30;
  auto* kernel = dtype == RF_F16 ? cache_decode_kernel<true, false, true, false, true>
                                 : cache_decode_kernel<false, false, true, false, true>;
  if (smem_attr(kernel, SMEM_BYTES, done[dtype == RF_F16]) != RF_OK) return RF_ERR_CUDA;
  const unsigned groups = (unsigned)(a.B * a.positions * a.Hkv * a.mtiles);
  return launch_after(kernel, groups, WARPS * 32, SMEM_BYTES, st, a);
}

rf_status launch_add_weights(const CacheDecode& a, const float* weight, float* total,
                             cudaStream_t st) {
  // four keys per thread only where that leaves threads enough: 16384 keys took
  // 5.8 us so, and 3.6 us with one
  const bool wide = (long long)a.B * a.Hkv * a.cap >= (1 << 19) && a.cap % 4 == 0 && aligned16(a.scores) &&
                    aligned16(weight) && aligned16(total);
  const int keys = wide ? 1024 : 256;             // of a CTA
  const int blocks = (a.cap + keys - 1) / keys;
  const long long grid = (long long)a.B * a.Hkv * blocks;
  if (grid > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  // eight heads in flight where there are more than four (2 x 16 heads of 595 keys:
  // 11.3 us with the decode, 12.1 with four; 4 heads: 8.4 us with four, 8.8 with eight)
  const int G = a.H / a.Hkv;
  return launch_after(wide    ? add_weights_kernel<4, 4>
                      : G > 4 ? add_weights_kernel<1, 8>
                              : add_weights_kernel<1, 4>,
                      (unsigned)grid, 256, 0, st,
                      a.scores, a.seg_m, a.lens, weight, total, a.B, a.Hkv, G, a.cap,
                      a.S_total, blocks);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
