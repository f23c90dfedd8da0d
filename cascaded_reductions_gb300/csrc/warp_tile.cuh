// What the decode kernels over a cache of grouped heads are built from: rows of 128
// 16-bit values copied asynchronously into shared memory, and the warp-level matrix
// instruction m16n8k16 over tiles of 16 keys.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_common.cuh"

namespace rf {
namespace {

constexpr int HD = 128;                 // head dimension
constexpr int ROW_BYTES = HD * 2;

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

// One warp's running state of 16 rows: rows lane / 4 (index 0) and + 8 (index 1); acc[d]
// holds columns 8 d + 2 (lane % 4) and + 1 of both.
template <bool F16>
struct RowState {
  // The weights' reference for the maximum m: an fp16 weight is taken 2^15 times as large;
  // the state given away has it for its m.  From 2^24 on m - 15 may round to m - 16 or less,
  // and a weight to 2^16: m itself then.
  static __device__ __forceinline__ float below(float m) {
    if constexpr (!F16) return m;
    const float f = m - 15.f;
    return m - f > 15.5f ? m : f;
  }
  uint32_t qf[HD / 16][4];
  float acc[HD / 8][4];
  float m0, m1, l0, l1;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }

  // products of the rows with the 16 keys in `st`: s[n][e], key 8 n + 2 (lane % 4) + e % 2 of row e / 2
  __device__ __forceinline__ void products(uint32_t st, float (&s)[2][4], int lane) const {
    const int r = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const int c = 2 * kk + ((lane >> 3) & 1);
      uint32_t kb[4];
      ldmatrix_x4(st + r * ROW_BYTES + ((c ^ (r & 7)) << 4), kb);
      mma16816<F16>(s[0], qf[kk], kb[0], kb[1]);
      mma16816<F16>(s[1], qf[kk], kb[2], kb[3]);
    }
  }

  // folds in those keys, whose values follow them in `st`, by their scores in log2 units (-inf: hidden)
  __device__ __forceinline__ void fold(const float (&s)[2][4], uint32_t st, int lane) {
    float mx0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    float mx1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
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
    const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      const int c = 2 * d + (lane >> 4);
      uint32_t vb[4];
      ldmatrix_x4_trans(st + kDecodeTile * ROW_BYTES + r * ROW_BYTES + ((c ^ (r & 7)) << 4), vb);
      mma16816<F16>(acc[2 * d], hi, vb[0], vb[1]);
      mma16816<F16>(acc[2 * d + 1], hi, vb[2], vb[3]);
      mma16816<F16>(acc[2 * d], lw, vb[0], vb[1]);
      mma16816<F16>(acc[2 * d + 1], lw, vb[2], vb[3]);
    }
  }

  // the row sums over the four lanes that share a row; once, before the state is used
  __device__ __forceinline__ void close() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  }
};

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

__device__ __forceinline__ bool any_nan(const float4& x) {
  return x.x != x.x || x.y != x.y || x.z != x.z || x.w != x.w;
}

}  // namespace
}  // namespace rf
