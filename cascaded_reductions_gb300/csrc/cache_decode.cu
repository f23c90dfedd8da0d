// Single-token decode over a cache of grouped heads: H query heads share Hkv
// key/value heads (head h reads key head h / G, G = H / Hkv), every sequence
// has its own length, and a mask may leave only the last `window` keys and the
// first `sinks` visible.  The same kernel, with its segments numbered after
// those of the prefix kernel, is the suffix half of the shared-prefix decode,
// and with its scores kept it feeds the running total of each key's weight.
//
// Mathematics: per row the cascade of the split-KV decode (running m, l, acc,
// rescale by exp2(m_old - m_new), segment states merged by the same rescale).
//
// What bounds it: HBM.  A key of a key head costs 512 bytes (K and V) and
// 4 G D = 512 G flops; on the FP32 pipes G = 4 heads would already need as
// long as the bytes, so both products run on the warp-level matrix
// instruction m16n8k16: the G query heads are its 16 rows (G < 16 leaves rows
// idle, which costs nothing here: 16 keys need 48 instructions while their
// 8 KiB take an SM about 350 cycles).
//
// Split: one CTA per (sequence, key head, 16-row tile of query heads,
// segment); its four warps take turns over tiles of 16 keys, each warp with a
// ring of its own (3 stages of 8 KiB, filled by 16-byte asynchronous copies,
// so no block-wide barrier is needed until the end).  Only visible keys are
// read: positions are numbered over the visible keys and mapped to cache rows.
// Rows past a segment's end are zero-filled, never read.
//
// P in two terms: the weights enter the second product as hi + lo, two 16-bit
// terms, so that they carry 16 (bf16) or 22 (fp16) bits and the output is
// rounded once; the 16 extra matrix instructions per tile are free here.
//
// The CTA that completes a row group's count merges its segments in segment
// order (bitwise reproducible) and sets the count back to 0.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_common.cuh"

namespace rf {
namespace {

constexpr int HD = 128;                 // head dimension
constexpr int ROW_BYTES = HD * 2;
constexpr int TK = 16;                  // keys per warp tile
constexpr int WARPS = 4;
constexpr int STAGES = 3;
constexpr int STAGE_BYTES = 2 * TK * ROW_BYTES;   // K tile, V tile
constexpr int MROWS = 16;               // query heads per CTA
constexpr size_t SMEM_BYTES = (size_t)WARPS * STAGES * STAGE_BYTES;
static_assert(STAGE_BYTES >= MROWS * HD * 4, "a warp's state reuses its first stage");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
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

__device__ __forceinline__ void store_out(void* out, size_t i, float x, int dtype) {
  if (dtype == RF_F32)
    static_cast<float*>(out)[i] = x;
  else if (dtype == RF_F16)
    static_cast<__half*>(out)[i] = __float2half_rn(x);
  else
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
}

// acc / l, and 0 where the row has no weight at all (no visible key); a NaN
// sum stays NaN
__device__ __forceinline__ float normalised(float acc, float l) { return l == 0.f ? 0.f : acc / l; }

template <bool F16, bool SCORES>
__global__ void __launch_bounds__(WARPS * 32)
cache_decode_kernel(const CacheDecode a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[WARPS][MROWS], sm_l[WARPS][MROWS];
  __shared__ int last;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mt = blockIdx.x % a.mtiles;
  const int seg = (int)(blockIdx.x / a.mtiles) % a.S;
  const int group = (int)(blockIdx.x / a.mtiles) / a.S;            // b * Hkv + key head
  const int b = group / a.Hkv, hk = group - b * a.Hkv;
  const int rows = min(MROWS, a.G - mt * MROWS);
  const size_t row0 = (size_t)b * a.H + (size_t)hk * a.G + mt * MROWS;   // first query row

  // visible keys: t < ns are the sinks, the rest the last keys of the sequence
  int len = a.cap;
  if (a.lens != nullptr && RF_IDX_OK(b, a.B)) len = min(max(a.lens[b], 0), a.cap);
  const int lo = a.window > 0 ? max(0, len - a.window) : 0;
  const int ns = min(a.sinks, lo);
  const int n = ns + len - lo;
  const int chunk = segment_keys(n, a.S);
  const int t_begin = min(n, seg * chunk), t_end = min(n, t_begin + chunk);
  const int tiles = (t_end - t_begin + TK - 1) / TK;

  // Q fragments: rows lane / 4 and + 8, columns 16 kk + 2 (lane % 4) (+ 8)
  uint32_t qf[HD / 16][4];
  {
    const int r = lane >> 2;
    const bool in0 = r < rows, in1 = r + 8 < rows;
    const uint8_t* q0 = a.q + (row0 + r) * ROW_BYTES + (lane & 3) * 4;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const bool ok0 = in0 && RF_SPAN_OK((row0 + r) * ROW_BYTES + kk * 32, 32, (size_t)a.B * a.H * ROW_BYTES);
      const bool ok1 = in1 && RF_SPAN_OK((row0 + r + 8) * ROW_BYTES + kk * 32, 32, (size_t)a.B * a.H * ROW_BYTES);
      qf[kk][0] = ok0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32) : 0u;
      qf[kk][1] = ok1 ? *reinterpret_cast<const uint32_t*>(q0 + 8 * ROW_BYTES + kk * 32) : 0u;
      qf[kk][2] = ok0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32 + 16) : 0u;
      qf[kk][3] = ok1 ? *reinterpret_cast<const uint32_t*>(q0 + 8 * ROW_BYTES + kk * 32 + 16) : 0u;
    }
  }

  uint8_t* ring = smem + warp * STAGES * STAGE_BYTES;
  const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const size_t kv0 = (size_t)group * a.cap;                        // first cache row of the group

  // tile i of this warp: keys t_begin + (i WARPS + warp) TK ..
  auto issue = [&](int i) {
    const int t0 = t_begin + (i * WARPS + warp) * TK;
    if (t0 < t_end) {
      const uint32_t st = ring32 + (uint32_t)(i % STAGES) * STAGE_BYTES;
#pragma unroll
      for (int u = 0; u < TK / 2; ++u) {
        const int r = 2 * u + (lane >> 4), c = lane & 15;
        const int t = t0 + r;
        const int key = t < ns ? t : t - ns + lo;
        const bool in = t < t_end && RF_IDX_OK(kv0 + key, (size_t)a.B * a.Hkv * a.cap);
        const size_t off = (kv0 + (in ? key : 0)) * ROW_BYTES + c * 16;
        const uint32_t dst = st + r * ROW_BYTES + ((c ^ (r & 7)) << 4);
        cp_async16(dst, a.k + off, in ? 16u : 0u);
        cp_async16(dst + TK * ROW_BYTES, a.v + off, in ? 16u : 0u);
      }
    }
    cp_async_commit();
  };

  float acc[HD / 8][4];
#pragma unroll
  for (int d = 0; d < HD / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(i);
  for (int i = 0; i * WARPS + warp < tiles; ++i) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();                       // every lane's copies of tile i landed, tile i - 1 is read
    issue(i + STAGES - 1);
    const uint32_t st = ring32 + (uint32_t)(i % STAGES) * STAGE_BYTES;
    const int t0 = t_begin + (i * WARPS + warp) * TK;

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
        const bool in = t < t_end;
        s[nt][e] = in ? s[nt][e] * a.scale_log2 : -INFINITY;
        s[nt][2 + e] = in ? s[nt][2 + e] * a.scale_log2 : -INFINITY;
        mx0 = fmaxf(mx0, s[nt][e]);
        mx1 = fmaxf(mx1, s[nt][2 + e]);
        if constexpr (SCORES) {
          const int r = lane >> 2;
          if (in && r < rows && RF_IDX_OK((row0 + r) * a.cap + t, (size_t)a.B * a.H * a.cap))
            a.scores[(row0 + r) * a.cap + t] = s[nt][e];
          if (in && r + 8 < rows && RF_IDX_OK((row0 + r + 8) * a.cap + t, (size_t)a.B * a.H * a.cap))
            a.scores[(row0 + r + 8) * a.cap + t] = s[nt][2 + e];
        }
      }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    const bool grew = mx0 > m0 || mx1 > m1;
    if (__any_sync(0xffffffffu, grew)) {
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      const float c0 = exp2f(m0 - ref_of(n0)), c1 = exp2f(m1 - ref_of(n1));
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
    const float f0 = ref_of(m0), f1 = ref_of(m1);
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
  cp_async_wait<0>();
  __syncwarp();

  // warp states into shared memory (the warp's own first stage)
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  {
    const int r = lane >> 2;
    float* st = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) {
      const int col = d * 8 + 2 * (lane & 3);
      *reinterpret_cast<float2*>(st + r * HD + col) = make_float2(acc[d][0], acc[d][1]);
      *reinterpret_cast<float2*>(st + (r + 8) * HD + col) = make_float2(acc[d][2], acc[d][3]);
    }
    if ((lane & 3) == 0) {
      sm_m[warp][r] = m0;
      sm_m[warp][r + 8] = m1;
      sm_l[warp][r] = l0;
      sm_l[warp][r + 8] = l1;
    }
  }
  __syncthreads();
  const bool direct = a.S_total == 1;             // the only segment: the output itself
  const size_t states = (size_t)a.B * a.H * a.S_total;
  (void)states;                                   // read by the checked build only
  for (int r = 0; r < rows; ++r) {
    const int d = threadIdx.x;                    // WARPS * 32 == HD
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_m[w][r]);
    const float ref = ref_of(M);
    float A = 0.f, L = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2f(sm_m[w][r] - ref);
      A = fmaf(f, reinterpret_cast<const float*>(smem + (size_t)w * STAGES * STAGE_BYTES)[r * HD + d], A);
      L = fmaf(f, sm_l[w][r], L);
    }
    const size_t row = row0 + r;
    const size_t slot = row * a.S_total + a.seg0 + seg;
    if (direct) {
      if (RF_IDX_OK(row * HD + d, (size_t)a.B * a.H * HD))
        store_out(a.out, row * HD + d, normalised(A, L), a.out_dtype);
      if (d == 0) {
        const float lse2 = M + log2f(L);
        if (a.lse != nullptr && RF_IDX_OK(row, (size_t)a.B * a.H)) a.lse[row] = lse2 * kLn2;
        if (SCORES && RF_IDX_OK(slot, states)) a.seg_m[slot] = lse2;
      }
    } else {
      // a segment without keys leaves its accumulator unwritten: nobody reads it
      if (t_begin < t_end && RF_IDX_OK(slot * HD + d, states * HD)) a.seg_acc[slot * HD + d] = A;
      if (d == 0 && RF_IDX_OK(slot, states)) {
        a.seg_m[slot] = M;
        a.seg_l[slot] = L;
      }
    }
  }
  if (direct) return;

  // the last segment to arrive merges the rows
  __threadfence();
  __syncthreads();
  const int counter = group * a.mtiles + mt;
  if (threadIdx.x == 0) {
    const int seen = RF_IDX_OK(counter, (size_t)a.B * a.Hkv * a.mtiles)
                         ? atomicAdd(a.counters + counter, 1) : -1;
    last = seen == a.S - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int r = warp; r < rows; r += WARPS) {
    const size_t row = row0 + r;
    const float* sm = a.seg_m + row * a.S_total;
    const float* sl = a.seg_l + row * a.S_total;
    const float4* sa = reinterpret_cast<const float4*>(a.seg_acc + row * a.S_total * HD) + lane;
    float M = -INFINITY;
    for (int s = lane; s < a.S_total; s += 32)
      if (RF_IDX_OK(row * a.S_total + s, states)) M = fmaxf(M, __ldcg(sm + s));
    M = group_max<32>(M);
    const float ref = ref_of(M);
    float L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < a.S_total; s0 += 32) {
      // lane j holds segment s0 + j's weight; -1 marks one without keys
      float f = -1.f;
      const int s = s0 + lane;
      if (s < a.S_total && RF_IDX_OK(row * a.S_total + s, states)) {
        const float ms = __ldcg(sm + s);
        if (ms != -INFINITY) {
          f = exp2f(ms - ref);
          L = fmaf(f, __ldcg(sl + s), L);
        } else {
          L += __ldcg(sl + s);                    // 0, or NaN where every score was NaN
        }
      }
      const int cnt = min(32, a.S_total - s0);
#pragma unroll 4
      for (int j = 0; j < cnt; ++j) {
        const float fj = __shfl_sync(0xffffffffu, f, j);
        if (fj != -1.f && RF_SPAN_OK(((row * a.S_total + s0 + j) * HD + lane * 4), 4, states * HD)) {
          const float4 x = __ldcg(sa + (size_t)(s0 + j) * (HD / 4));
          A.x = fmaf(fj, x.x, A.x);
          A.y = fmaf(fj, x.y, A.y);
          A.z = fmaf(fj, x.z, A.z);
          A.w = fmaf(fj, x.w, A.w);
        }
      }
    }
    L = group_sum<32>(L);
    if (RF_SPAN_OK(row * HD + lane * 4, 4, (size_t)a.B * a.H * HD)) {
      const size_t o = row * HD + lane * 4;
      store_out(a.out, o, normalised(A.x, L), a.out_dtype);
      store_out(a.out, o + 1, normalised(A.y, L), a.out_dtype);
      store_out(a.out, o + 2, normalised(A.z, L), a.out_dtype);
      store_out(a.out, o + 3, normalised(A.w, L), a.out_dtype);
    }
    __syncwarp();                                 // every lane has read the states
    if (lane == 0) {
      const float lse2 = M + log2f(L);
      if (a.lse != nullptr && RF_IDX_OK(row, (size_t)a.B * a.H)) a.lse[row] = lse2 * kLn2;
      if (SCORES && RF_IDX_OK(row * a.S_total, states)) a.seg_m[row * a.S_total] = lse2;
    }
  }
  if (threadIdx.x == 0 && RF_IDX_OK(counter, (size_t)a.B * a.Hkv * a.mtiles)) a.counters[counter] = 0;
}

// total[j] = weight[j] + sum over the group's heads of exp2(score - lse2):
// the weights of the row's softmax, each below 1, summed in fp32 head by head
// in order.  One thread per key; reads 4 (G + 1) bytes and writes 4 per key.
__global__ void __launch_bounds__(256)
add_weights_kernel(const float* __restrict__ scores, const float* __restrict__ seg_m,
                   const int32_t* __restrict__ lens, const float* weight, float* total, int B,
                   int Hkv, int G, int cap, int S, int blocks) {
  const int group = blockIdx.x / blocks;
  const int j = (blockIdx.x - group * blocks) * 256 + threadIdx.x;
  const int b = group / Hkv;
  const size_t row0 = (size_t)group * G;                          // b * H + key head * G
  int len = cap;
  if (lens != nullptr && RF_IDX_OK(b, B)) len = min(max(lens[b], 0), cap);
  if (j >= cap) return;
  const size_t i = (size_t)group * cap + j;
  if (!RF_IDX_OK(i, (size_t)B * Hkv * cap)) return;
  float w = weight != nullptr ? weight[i] : 0.f;
  if (j < len) {
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
      if (!RF_IDX_OK((row0 + g) * cap + j, (size_t)B * Hkv * G * cap)) continue;
      const float z = __ldg(seg_m + (row0 + g) * S);
      const float x = __ldcs(scores + (row0 + g) * cap + j);
      w += z == -INFINITY ? 0.f : exp2f(x - z);   // a row without weight adds none
    }
  } else if (weight == total) {
    return;                                       // behind the end: left as it was
  }
  total[i] = w;
}

template <bool F16, bool SCORES>
rf_status launch_t(const CacheDecode& a, unsigned grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (smem_attr(cache_decode_kernel<F16, SCORES>, SMEM_BYTES, done) != RF_OK) return RF_ERR_CUDA;
  cache_decode_kernel<F16, SCORES><<<grid, WARPS * 32, SMEM_BYTES, st>>>(a);
  return launch_status();
}

}  // namespace

rf_status launch_cache_decode(CacheDecode a, int dtype, cudaStream_t st) {
  a.G = a.H / a.Hkv;
  a.mtiles = (a.G + MROWS - 1) / MROWS;
  const unsigned grid = (unsigned)((long long)a.B * a.Hkv * a.mtiles * a.S);
  if (dtype == RF_F16)
    return a.scores ? launch_t<true, true>(a, grid, st) : launch_t<true, false>(a, grid, st);
  return a.scores ? launch_t<false, true>(a, grid, st) : launch_t<false, false>(a, grid, st);
}

rf_status launch_add_weights(const CacheDecode& a, const float* weight, float* total,
                             cudaStream_t st) {
  const int blocks = (a.cap + 255) / 256;
  const long long grid = (long long)a.B * a.Hkv * blocks;
  if (grid > 0x7fffffffLL) return RF_ERR_UNSUPPORTED;
  add_weights_kernel<<<(unsigned)grid, 256, 0, st>>>(a.scores, a.seg_m, a.lens, weight, total, a.B,
                                                     a.Hkv, a.H / a.Hkv, a.cap, a.S_total, blocks);
  return launch_status();
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
