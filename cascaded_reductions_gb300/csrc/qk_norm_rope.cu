// Norm of each query and key head, rotation by position, and the write of keys and
// values into a paged cache, from one read of a projection's rows.
//
// Mathematics, per head of D values:
//   y = x w / sqrt(mean x^2 + eps);  a pair (y_a, y_b) of the first R values turns by
//   t = pos f:  (y_a cos t - y_b sin t,  y_b cos t + y_a sin t);
// pairs are (i, i + R/2), or (2i, 2i + 1) interleaved, and pos is the token's position
// on the pair's axis (one for text; time, height and width for pictures).  All in
// fp32, rounded once.
//
// The angle: an fp32 product pos f is off by up to pos 2^-24, 0.06 rad at a million.
// A turn is taken as a 64-bit integer instead: f / 2 pi mod 1 in units of 2^-64 (from a
// product in fp64), times the position, is the angle mod a whole turn exactly as the
// integer wraps; its top 32 bits go through sincospi.  What is left of the error is
// pos max(1, |f|) 2^-52 rad from the rounding of f / 2 pi and half a step of fp32.
//
// What bounds it: HBM (a head is read once and written once), if little goes through
// shared memory.  A head takes D / 16 lanes, each with two 16-byte chunks that hold both
// halves of its pairs, so that only the sum of squares crosses lanes.  Angles cost some 40
// instructions a pair and are made once per token, for all heads.
//   Many tokens (norm_rope_kernel): a warp takes a share of all heads of all tokens, makes
// a token's angles, keeps them in registers and goes through its heads, the next group's rows
// in flight.
//   Few (norm_rope_few_kernel): the heads of a token are spread over the warps of one CTA or
// of several, each of which makes the token's angles for itself.
// [8192 tokens, 32 + 8 + 8 heads of 128, 201 MB]: 40 us, 5.0 TB/s, and 45 us by the second
// kernel, whose every item reads weights and angles from shared memory (85 % of its rate).
// The first issues an instruction in 61 % of the cycles; shares of whole tokens take 44 us (2.2
// per warp), two or more groups in flight 42, four CTAs per SM 45, two 44.

#include <cuda_fp16.h>

#include "cache_common.cuh"
#include "f32x2.cuh"
#include "tc_common.cuh"

namespace rf {
namespace {

constexpr int WARPS = 8;
constexpr int MANY = 8;                 // tokens per SM from which on a warp takes a share of all heads

struct NormRope {
  const uint16_t *q, *k, *v;
  long long q_step, k_step, v_step;     // elements from a token's row to the next
  const void *qw, *kw;                  // [D] or null
  const int32_t* positions;             // [axes, T]
  const float* freq;                    // [R / 2]
  const int32_t* axis;                  // [R / 2] or null
  const int32_t* slots;                 // [T] or null: k and v go to k_out, v is not taken
  uint16_t *q_out, *k_out, *v_out;      // k_out, v_out: the pages where slots is given
  long long n_slots;
  float eps;
  int T, H, Hkv, R, axes, page;
  bool w32;                             // weights are fp32
  int heads, slices;                    // per token with v; CTAs that share a token
};

template <bool F16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool F16>
__device__ __forceinline__ void widen8(const uint4& u, float* f) {
  const float2 a = widen<F16>(u.x), b = widen<F16>(u.y), c = widen<F16>(u.z), d = widen<F16>(u.w);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}
template <bool F16>
__device__ __forceinline__ uint4 round8(const float* f) {
  if constexpr (F16)
    return make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                      pack_f16x2(f[6], f[7]));
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
template <bool F16>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  const float2 f = widen<F16>(w);
  return pair::pack_f32x2(f.x, f.y);
}
template <bool F16>
__device__ __forceinline__ uint32_t round2(uint64_t x) {
  float a, b;
  pair::unpack_f32x2(x, a, b);
  if constexpr (F16) return pack_f16x2(a, b);
  return pack_bf16x2(a, b);
}
template <bool F16>
__device__ __forceinline__ float weight_of(const void* w, int i, bool w32) {
  if (w32) return static_cast<const float*>(w)[i];
  const uint32_t u = static_cast<const uint16_t*>(w)[i];
  return widen<F16>(u).x;
}

__device__ __forceinline__ uint4 ld16(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// a turn's 2^-64 th parts that position times makes of frequency f
__device__ __forceinline__ unsigned long long turn_unit(float freq) {
  double f = (double)freq * 0.15915494309189533577;           // 1 / (2 pi)
  f -= floor(f);
  return __double2ull_rn(f * 18446744073709551616.0);
}
__device__ __forceinline__ void turn_of(const NormRope& a, unsigned long long unit, int pair, size_t t, float* s,
                                        float* c) {
  int ax = a.axis && RF_IDX_OK(pair, a.R / 2) ? a.axis[pair] : 0;
  ax = min(max(ax, 0), a.axes - 1);
  const size_t at = (size_t)ax * a.T + t;
  const long long pos = RF_IDX_OK(at, (size_t)a.axes * a.T) ? a.positions[at] : 0;
  const unsigned long long frac = unit * (unsigned long long)pos + 0x80000000ull;
  // the top 32 bits as half turns in [-1, 1)
  sincospif((float)(int)(unsigned)(frac >> 32) * 4.656612873077393e-10f, s, c);
}

template <bool F16, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(WARPS * 32, 3)
norm_rope_kernel(const NormRope a) {
  constexpr int LANES = D / 16;                 // of a head
  constexpr int HEADS = 32 / LANES;             // of a warp
  extern __shared__ __align__(16) float smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = a.R / 2;
  // weights of q and k as the lanes take them, four floats each: [2][4][LANES][4]
  float* w_s = smem;
  unsigned long long* unit = reinterpret_cast<unsigned long long*>(smem + 2 * D);   // [R / 2]
  float* turn = reinterpret_cast<float*>(unit + half) + warp * a.R;                 // the warp's cos, sin
  wait_prerequisite();
  allow_dependents();
  const int hl = lane / LANES, j = lane % LANES;
  const int rc = a.R / 16;
  const int c0 = INTERLEAVED ? 2 * j : j < rc ? j : 2 * rc + 2 * (j - rc);
  const int c1 = INTERLEAVED ? 2 * j + 1 : j < rc ? j + rc : c0 + 1;
  // items of a token: groups of heads of q, then of k, then of v
  const int nq = (a.H + HEADS - 1) / HEADS, nk = (a.Hkv + HEADS - 1) / HEADS;
  const int items = nq + (a.slots ? 2 : 1) * nk;
  // the warp's share of all items, to the item: 8192 tokens for 3648 warps are 2.2 each
  const long long all = (long long)a.T * items, w0 = (long long)blockIdx.x * WARPS + warp;
  const long long ws = (long long)gridDim.x * WARPS;
  const long long first = all / ws * w0 + all % ws * w0 / ws, last = all / ws * (w0 + 1) + all % ws * (w0 + 1) / ws;
  // Walks over the items from item i of token t on: where the group's rows are, and the heads
  // from it to the end of its part.
  struct Walk {
    int t, part, heads;
  };
  auto open = [&](long long n) {
    Walk w;
    w.t = (int)(n / items);
    const int i = (int)(n - (long long)w.t * items);
    w.part = i < nq ? 0 : i < nq + nk ? 1 : 2;
    w.heads = (w.part ? a.Hkv : a.H) - HEADS * (i - (w.part == 0 ? 0 : w.part == 1 ? nq : nq + nk));
    return w;
  };
  // on to the next group; true in a new part
  auto step = [&](Walk& w) {
    w.heads -= HEADS;
    if (w.heads > 0) return false;
    if (++w.part == (a.slots ? 3 : 2)) w.part = 0, ++w.t;
    w.heads = w.part ? a.Hkv : a.H;
    return true;
  };
  const int o0 = hl * D + c0 * 8, o1 = hl * D + c1 * 8;
  auto from_of = [&](const Walk& w) {
    return w.part == 0   ? a.q + w.t * a.q_step + (a.H - w.heads) * D
           : w.part == 1 ? a.k + w.t * a.k_step + (a.Hkv - w.heads) * D
                         : a.v + w.t * a.v_step + (a.Hkv - w.heads) * D;
  };
  Walk in = open(first);
  const uint16_t* from = from_of(in);
  int to_load = (int)(last - first), to_do = to_load;
  struct Rows {
    uint4 x0, x1;
  };
  auto load = [&](Rows& r) {
    r.x0 = r.x1 = make_uint4(0, 0, 0, 0);
    if (to_load <= 0) return;
    if (hl < in.heads && RF_IDX_OK(in.t, a.T)) {
      r.x0 = ld16(from + o0);
      r.x1 = ld16(from + o1);
    }
    --to_load;
    from += HEADS * D;
    if (step(in)) from = from_of(in);
  };
  Walk at = in;
  Rows it, next;
  load(it);                                     // under way while the tables are made
  for (int e = tid; e < 2 * D; e += WARPS * 32) {
    const void* w = e < D ? a.qw : a.kw;
    const int f = e % D, k = f / (4 * LANES), l = f / 4 % LANES;          // part k of lane l
    const int lc0 = INTERLEAVED ? 2 * l : l < rc ? l : 2 * rc + 2 * (l - rc);
    const int lc1 = INTERLEAVED ? 2 * l + 1 : l < rc ? l + rc : lc0 + 1;
    w_s[e] = w ? weight_of<F16>(w, (k < 2 ? lc0 : lc1) * 8 + k % 2 * 4 + f % 4, a.w32) : 1.f;
  }
  for (int e = tid; e < half; e += WARPS * 32) unit[e] = turn_unit(RF_IDX_OK(e, half) ? a.freq[e] : 0.f);
  __syncthreads();

  while (to_do > 0) {
    const int t = at.t;
    __syncwarp();                               // the last token's angles have been read
    for (int e = lane; e < half; e += 32) turn_of(a, unit[e], e, t, &turn[half + e], &turn[e]);
    const int slot = a.slots && RF_IDX_OK(t, a.T) ? a.slots[t] : -1;
    const bool placed = slot >= 0 && slot < a.n_slots;
    const int page = placed ? slot / a.page : 0;
    // a key head's row of the token, and the distance to the next head's
    const size_t kv_row = a.slots ? (size_t)page * a.Hkv * a.page + (slot - page * a.page) : (size_t)t * a.Hkv;
    const size_t kv_step = a.slots ? a.page : 1;
    __syncwarp();
    uint64_t c[4], s[4], ns[4];
    if (j < rc) {
      const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(turn + 8 * j);
      const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(turn + half + 8 * j);
      c[0] = c2[0].x, c[1] = c2[0].y, c[2] = c2[1].x, c[3] = c2[1].y;
      s[0] = s2[0].x, s[1] = s2[0].y, s[2] = s2[1].x, s[3] = s2[1].y;
#pragma unroll
      for (int e = 0; e < 4; ++e) ns[e] = pair::mul_f32x2(s[e], pair::pack_f32x2(-1.f, -1.f));
    }
    while (to_do > 0 && at.t == t) {
      // the groups of one part
      const int part = at.part, all = part ? a.Hkv : a.H;
      const bool stored = part == 0 || a.slots == nullptr || placed, norms = part == 0 ? a.qw != nullptr : a.kw != nullptr;
      const size_t to_step = part == 0 ? D : kv_step * D;
      uint16_t* to = part == 0 ? a.q_out + ((size_t)t * a.H + all - at.heads) * D
                               : (part == 1 ? a.k_out : a.v_out) + (kv_row + (all - at.heads) * kv_step) * D;
      to += hl * to_step;
      const ulonglong2* w = reinterpret_cast<const ulonglong2*>(w_s + (part == 0 ? 0 : D)) + j;
      bool more = true;
      while (more && to_do > 0) {
        load(next);
        if (part < 2) {
          uint64_t x[8] = {widen2<F16>(it.x0.x), widen2<F16>(it.x0.y), widen2<F16>(it.x0.z), widen2<F16>(it.x0.w),
                           widen2<F16>(it.x1.x), widen2<F16>(it.x1.y), widen2<F16>(it.x1.z), widen2<F16>(it.x1.w)};
          if (norms) {
            uint64_t s2 = 0ull;
#pragma unroll
            for (int e = 0; e < 8; ++e) s2 = pair::fma_f32x2(x[e], x[e], s2);
            float s0, s1;
            pair::unpack_f32x2(s2, s0, s1);
            const float r = rsqrtf(group_sum<LANES>(s0 + s1) * (1.f / D) + a.eps);
            const uint64_t r2 = pair::pack_f32x2(r, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 w2 = w[e * LANES];
              x[2 * e] = pair::mul_f32x2(x[2 * e], pair::mul_f32x2(r2, w2.x));
              x[2 * e + 1] = pair::mul_f32x2(x[2 * e + 1], pair::mul_f32x2(r2, w2.y));
            }
          }
          if (j < rc) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // two pairs: their first values, their second ones
              uint64_t u = x[INTERLEAVED ? 2 * e : e], v = x[INTERLEAVED ? 2 * e + 1 : e + 4];
              float p0, p1, q0, q1;
              if constexpr (INTERLEAVED) {
                pair::unpack_f32x2(u, p0, p1);
                pair::unpack_f32x2(v, q0, q1);
                u = pair::pack_f32x2(p0, q0);
                v = pair::pack_f32x2(p1, q1);
              }
              uint64_t y = pair::fma_f32x2(u, c[e], pair::mul_f32x2(v, ns[e]));
              uint64_t z = pair::fma_f32x2(v, c[e], pair::mul_f32x2(u, s[e]));
              if constexpr (INTERLEAVED) {
                pair::unpack_f32x2(y, p0, q0);
                pair::unpack_f32x2(z, p1, q1);
                y = pair::pack_f32x2(p0, p1);
                z = pair::pack_f32x2(q0, q1);
              }
              x[INTERLEAVED ? 2 * e : e] = y;
              x[INTERLEAVED ? 2 * e + 1 : e + 4] = z;
            }
          }
          it.x0 = make_uint4(round2<F16>(x[0]), round2<F16>(x[1]), round2<F16>(x[2]), round2<F16>(x[3]));
          it.x1 = make_uint4(round2<F16>(x[4]), round2<F16>(x[5]), round2<F16>(x[6]), round2<F16>(x[7]));
        }
        if (stored && hl < at.heads) {
          *reinterpret_cast<uint4*>(to + c0 * 8) = it.x0;
          *reinterpret_cast<uint4*>(to + c1 * 8) = it.x1;
        }
        to += HEADS * to_step;
        --to_do;
        more = !step(at);
        it = next;
      }
    }
  }
}

// One CTA: a token's heads, or a slice of them.  Its warps take groups of 32 / (D / 16) heads
// at a time.
template <bool F16, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(WARPS * 32)
norm_rope_few_kernel(const NormRope a) {
  constexpr int LANES = D / 16;                 // of a head
  constexpr int HEADS = 32 / LANES;             // of a warp
  extern __shared__ __align__(16) float smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = a.R / 2;
  float* w_s = smem;                            // [2][D]: weights of q and k
  float2* turn = reinterpret_cast<float2*>(smem + 2 * D);   // [R / 2]: cos, sin
  const size_t t = blockIdx.x / a.slices;
  const int slice = (int)(blockIdx.x % a.slices);
  const int groups = (a.heads + HEADS - 1) / HEADS;
  wait_prerequisite();
  allow_dependents();

  // a lane's part of one head
  const int hl = lane / LANES, j = lane % LANES;
  // its chunks of 8 values: both halves of its pairs, or what lies behind R
  const int rc = a.R / 16;
  const int c0 = INTERLEAVED ? 2 * j : j < rc ? j : 2 * rc + 2 * (j - rc);
  const int c1 = INTERLEAVED ? 2 * j + 1 : j < rc ? j + rc : c0 + 1;
  struct Item {
    int h;                                      // head (q, then k, then v)
    uint4 x0, x1;
  };
  auto load = [&](int i, Item& it) {
    it.h = i * HEADS + hl;
    it.x0 = it.x1 = make_uint4(0, 0, 0, 0);
    if (i >= groups || it.h >= a.heads) return;
    const bool is_q = it.h < a.H, is_k = !is_q && it.h < a.H + a.Hkv;
    const int h = is_q ? it.h : is_k ? it.h - a.H : it.h - a.H - a.Hkv;
    const uint16_t* row = is_q ? a.q + t * a.q_step : is_k ? a.k + t * a.k_step : a.v + t * a.v_step;
    if (!RF_IDX_OK(t, a.T) || !RF_IDX_OK(h, is_q ? a.H : a.Hkv)) return;
    it.x0 = ld16(row + (size_t)h * D + c0 * 8);
    it.x1 = ld16(row + (size_t)h * D + c1 * 8);
  };
  const int stride = WARPS * a.slices;
  int i = slice * WARPS + warp;
  Item it;
  load(i, it);                                  // under way while the angles are made

  for (int e = tid; e < 2 * D; e += WARPS * 32) {
    const void* w = e < D ? a.qw : a.kw;
    w_s[e] = w ? weight_of<F16>(w, e < D ? e : e - D, a.w32) : 1.f;
  }
  for (int p = tid; p < half; p += WARPS * 32) {
    float s, c;
    turn_of(a, turn_unit(RF_IDX_OK(p, half) ? a.freq[p] : 0.f), p, t, &s, &c);
    turn[p] = make_float2(c, s);
  }
  __syncthreads();

  for (; i < groups; i += stride) {
    Item next;
    load(i + stride, next);
    const bool is_q = it.h < a.H, is_k = !is_q && it.h < a.H + a.Hkv;
    const bool in = it.h < a.heads;
    float x[16];
    widen8<F16>(it.x0, x);
    widen8<F16>(it.x1, x + 8);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (in && (is_q || is_k)) {
      if (is_q ? a.qw != nullptr : a.kw != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const float* w = w_s + (is_q ? 0 : D);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r * w[(e < 8 ? c0 * 8 : c1 * 8 - 8) + e];
      }
      if (j < rc) {
        const float2* cs = turn + 8 * j;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float2 z = cs[p];
          const int ia = INTERLEAVED ? 2 * p : p, ib = INTERLEAVED ? 2 * p + 1 : p + 8;
          const float xa = x[ia], xb = x[ib];
          x[ia] = fmaf(xa, z.x, -xb * z.y);
          x[ib] = fmaf(xb, z.x, xa * z.y);
        }
      }
      it.x0 = round8<F16>(x);
      it.x1 = round8<F16>(x + 8);
    }
    if (in) {
      uint16_t* dst = nullptr;
      if (is_q) {
        dst = a.q_out + (t * a.H + it.h) * D;
      } else {
        const int h = is_k ? it.h - a.H : it.h - a.H - a.Hkv;
        if (a.slots == nullptr) {
          dst = a.k_out + (t * a.Hkv + h) * D;
        } else {
          const int slot = RF_IDX_OK(t, a.T) ? a.slots[t] : -1;
          if (slot >= 0 && slot < a.n_slots) {
            const int p = slot / a.page;
            dst = (is_k ? a.k_out : a.v_out) + (((size_t)p * a.Hkv + h) * a.page + (slot - p * a.page)) * D;
          }
        }
      }
      if (dst) {
        *reinterpret_cast<uint4*>(dst + c0 * 8) = it.x0;
        *reinterpret_cast<uint4*>(dst + c1 * 8) = it.x1;
      }
    }
    it = next;
  }
}

template <bool F16, int D>
rf_status launch_d(NormRope a, bool interleaved, cudaStream_t st) {
  const int sms = tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  if (a.T >= MANY * sms) {
    const size_t smem = 2 * D * sizeof(float) + (a.R / 2) * sizeof(unsigned long long) + WARPS * a.R * sizeof(float);
    const long long ctas = ((long long)a.T + WARPS - 1) / WARPS, most = 3ll * sms;
    return launch_after(interleaved ? norm_rope_kernel<F16, D, true> : norm_rope_kernel<F16, D, false>,
                        (unsigned)(ctas < most ? ctas : most), WARPS * 32, smem, st, a);
  }
  const int heads_per_item = 32 / (D / 16);
  const long long groups = (a.heads + heads_per_item - 1) / heads_per_item;
  // where the tokens alone do not fill the device, several CTAs share one
  a.slices = 1;
  if (a.T < 4 * sms) {
    const long long most = (groups + WARPS - 1) / WARPS, want = 4ll * sms / a.T;
    a.slices = (int)(most < want ? most : want < 1 ? 1 : want);
  }
  const size_t smem = 2 * D * sizeof(float) + (size_t)(a.R / 2) * sizeof(float2);
  const long long grid = (long long)a.T * a.slices;
  auto* kernel = interleaved ? norm_rope_few_kernel<F16, D, true> : norm_rope_few_kernel<F16, D, false>;
  return launch_after(kernel, (unsigned)grid, WARPS * 32, smem, st, a);
}

}  // namespace

rf_status launch_qk_norm_rope(const void* q, long long q_step, const void* k, long long k_step,
                              const void* v, long long v_step, int T, int H, int Hkv, int D,
                              const void* qw, const void* kw, bool w32, float eps,
                              const int32_t* positions, int axes, const float* freq,
                              const int32_t* axis, int R, bool interleaved, int dtype,
                              const int32_t* slots, int P, int page, void* q_out, void* k_out,
                              void* v_out, cudaStream_t st) {
  NormRope a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_step = q_step, a.k_step = k_step, a.v_step = v_step;
  a.qw = qw, a.kw = kw, a.w32 = w32, a.eps = eps;
  a.positions = positions, a.axes = axes, a.freq = freq, a.axis = axis;
  a.slots = slots, a.page = page, a.n_slots = (long long)P * page;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.T = T, a.H = H, a.Hkv = Hkv, a.R = R;
  a.heads = H + (slots ? 2 : 1) * Hkv;
  if (dtype == RF_F16)
    return D == 64    ? launch_d<true, 64>(a, interleaved, st)
           : D == 128 ? launch_d<true, 128>(a, interleaved, st)
                      : launch_d<true, 256>(a, interleaved, st);
  return D == 64    ? launch_d<false, 64>(a, interleaved, st)
         : D == 128 ? launch_d<false, 128>(a, interleaved, st)
                    : launch_d<false, 256>(a, interleaved, st);
}

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
