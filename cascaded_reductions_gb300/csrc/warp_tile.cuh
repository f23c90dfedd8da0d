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

// Columns 4 lane .. + 3 of a 16-bit row, widened (by L2 alone: the kernel may not have waited)
template <bool F16>
__device__ __forceinline__ float4 load_row4(const uint8_t* row, int lane) {
  const uint2 u = __ldcg(reinterpret_cast<const uint2*>(row + lane * 8));
  if constexpr (F16) {
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  } else {
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  }
}

}  // namespace
}  // namespace rf
