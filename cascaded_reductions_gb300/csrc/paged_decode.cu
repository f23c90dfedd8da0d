// Attention of few new tokens per request over a paged cache: single tokens, drafted
// ones, short chunks.  The new tokens of a request times the query heads that share a
// key head are its rows; 16 of them share every key that is read.
//
// Mathematics: per row the cascade of the split-KV decode (running m, l, acc, rescale by
// exp2(m_old - m_new), states merged by the same rescale), over key <= position, in the
// window or below the sinks.
//
// What bounds it: HBM.  As in the dense cache's decode, both products run on the
// warp-level matrix instruction m16n8k16, four warps stream 16-key tiles of their own
// through three stages of asynchronous copies, and weights enter in two 16-bit terms.
// A tile of 16 keys lies in one page: a warp asks for the tile's page number one step
// before its keys.
//
// Work comes from the plan's units (16 rows of a request, a piece of their keys) times
// key heads.  Two kernels take it:
//  * paged_few_kernel where the call is small whatever the lengths: a CTA of four warps
//    per unit, the shortest way from launch to output; the CTA that ends a tile's last
//    piece merges them (1 request of 1028 keys, 32/8 heads: 7.0 us, by the other kernel
//    7.9; 16 000 keys 14.3 and 16.9).
//  * paged_decode_kernel otherwise: one CTA per SM, two teams of four streaming warps, a
//    unit each, the first by its number, the others from a queue.  A team's fifth warp
//    fetches the next unit, its page numbers and its query rows meanwhile, so that the
//    copies run on from unit to unit (64 requests of 4100 keys 160 us, 6.7 TB/s; without
//    169).  Pieces are left as states: paged_finish_kernel merges them, a warp per row
//    (17 requests with 4 drafted tokens 75 us; merged by the fifth warps 90).
// 64 requests of up to 16 384 keys run at the plain copy's rate, the 17 drafts at 82 % of
// it: 55 us of bytes stand beside a launch, the first page numbers and the merge.

#include <stddef.h>

#include "paged.cuh"
#include "tc_common.cuh"
#include "warp_tile.cuh"

namespace rf {
namespace {

constexpr int TK = kDecodeTile;
constexpr int TEAMS = 2;                // per CTA, one CTA per SM
constexpr int WARPS = 4;                // of a team that stream; one more closes
constexpr int CLOSE_WARP = TEAMS * WARPS;         // the first team's
constexpr int THREADS = (TEAMS * WARPS + 4) * 32;  // three warpgroups, two warps of the last idle
// Registers per thread: at launch, then streaming warps and the others.
constexpr int REGS = 168, REGS_STREAM = 200, REGS_CLOSE = 104;
static_assert(TEAMS * WARPS * 32 * REGS_STREAM + 128 * REGS_CLOSE == THREADS * REGS,
              "the shares of the warpgroups add up to what the CTA is launched with");
constexpr int STAGES = 3;
constexpr int STAGE_BYTES = 2 * TK * ROW_BYTES;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int MROWS = kPagedTileRows;
// A team's rings; its warps' accumulators of four rows at a time, rows 8 floats longer, so
// that those of a fragment's store lie 8 banks apart; its query rows
constexpr int MERGE_ROWS = WARPS, MERGE_PITCH = HD + 8;
constexpr int MERGE_BYTES = WARPS * MERGE_ROWS * MERGE_PITCH * 4;
constexpr int TEAM_BYTES = WARPS * RING_BYTES + MERGE_BYTES + MROWS * ROW_BYTES;
constexpr size_t SMEM_BYTES = (size_t)TEAMS * TEAM_BYTES;
static_assert(SMEM_BYTES + 4096 <= 232448, "exceeds the 227 KiB of shared memory a CTA may use");

// A team's barriers: its streaming warps; all five at a unit's end; its query rows have
// been read
enum { kBarStream = 1, kBarEnd, kBarRows, kBars = 3 };
template <int N>
__device__ __forceinline__ void named_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void named_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(N) : "memory");
}
constexpr int TEAM = (WARPS + 1) * 32;  // threads

// A unit's rows and keys, for one key head.
struct Work {
  int b, hk, start, n, len, row0, rows;  // rows row0 .. row0 + rows - 1 of n * G
  PagedTiles t;
  __device__ __forceinline__ Work(const PagedAttn& a, const PagedUnit& u, int hk_)
      : b(u.b), hk(hk_), start(u.start), n(u.n), len(u.len), row0(u.tile * MROWS),
        rows(min(MROWS, u.n * a.v.G - u.tile * MROWS)), t(u.n, u.len, a.v.s.window, a.v.s.sinks) {}
  // row r's query row in [T * H], and its position
  __device__ __forceinline__ size_t at(const PagedAttn& a, int r) const {
    const int G = a.v.G, i = (row0 + r) / G;
    return (size_t)(start + i) * a.v.s.H + hk * G + (row0 + r - i * G);
  }
  __device__ __forceinline__ int pos(const PagedAttn& a, int r) const {
    return len - n + (row0 + r) / a.v.G;
  }
  __device__ __forceinline__ int key_tile(int i) const {
    return i < t.sink_tiles ? i : i - t.sink_tiles + t.lo_tile;
  }
};

__device__ __forceinline__ int page_of(const PagedAttn& a, int b, int tile) {
  const int i = tile * TK >> a.page_log2;
  const size_t at = (size_t)b * a.width + i;
  return i < a.width && RF_IDX_OK(at, (size_t)a.v.s.B * a.width) ? __ldcg(a.table + at) : -1;
}
// cache rows in front of the tile's keys, where the page is one
__device__ __forceinline__ size_t row_of(const PagedAttn& a, int page, int hk, int tile) {
  return (((size_t)page * a.v.s.Hkv + hk) << a.page_log2) + (tile * TK & ((1 << a.page_log2) - 1));
}

// What a warp copies of a unit: every fourth tile of 16 keys, into a ring of stages.  Its
// lanes hold the page numbers of 32 tiles, and ask for the next 32 in time: behind a
// stream that takes all of the memory's rate such a load may take longer than a tile.
struct Stream {
  int b, hk, len, sink_tiles, lo_tile;
  int t, end, n;                        // next tile, the unit's last one, tiles so far
  int ids, ahead;                       // the lane's page numbers
  uint32_t ring;
  int in;                               // stage of the next tile

  __device__ __forceinline__ int key_tile(int i) const { return i < sink_tiles ? i : i - sink_tiles + lo_tile; }
  __device__ __forceinline__ int id_of(const PagedAttn& a, int i) const {
    return i < end ? page_of(a, b, key_tile(i)) : -1;
  }
  __device__ __forceinline__ void open(const PagedAttn& a, const PagedUnit& u, int head, int warp) {
    const PagedTiles k(u.n, u.len, a.v.s.window, a.v.s.sinks);
    b = u.b, hk = head, len = u.len;
    sink_tiles = k.sink_tiles, lo_tile = k.lo_tile;
    t = u.step0 * WARPS + warp;
    end = min(k.tiles, u.step1 * WARPS);
    n = 0;
  }
  // Keys of the next tile into the next stage: K rows, then V rows, 16-byte chunks permuted
  // by row % 8.  Rows past the request's end, and those of a page outside the cache, are zeros.
  __device__ __forceinline__ void copy(const PagedAttn& a, uint64_t policy, int lane) {
    const int tile = key_tile(t), now = __shfl_sync(0xffffffffu, ids, n & 31);
    ++n;
    if ((n & 31) == 8) ahead = id_of(a, t + (25 + lane) * WARPS);
    if ((n & 31) == 0) ids = ahead;
    const bool has = (unsigned)now < (unsigned)a.pages;
    const int rows = has ? min(len - tile * TK, TK) : 0, r0 = lane >> 4, c = lane & 15;
    const size_t first = row_of(a, has ? now : 0, hk, tile), at = first * ROW_BYTES + c * 16;
    const uint8_t *k = a.kp + at, *v = a.vp + at;
    const uint32_t stage = ring + (uint32_t)in * STAGE_BYTES;
#pragma unroll
    for (int u = 0; u < TK / 2; ++u) {
      const int r = 2 * u + r0;
      const bool on = r < rows && RF_IDX_OK(first + r, ((size_t)a.pages * a.v.s.Hkv) << a.page_log2);
      const int off = on ? r * ROW_BYTES : 0;
      const uint32_t dst = stage + r * ROW_BYTES + ((c ^ (r & 7)) << 4);
      cp_async16(dst, k + off, on ? 16u : 0u, policy);
      cp_async16(dst + TK * ROW_BYTES, v + off, on ? 16u : 0u, policy);
    }
    t += WARPS;
    in = in + 1 == STAGES ? 0 : in + 1;
  }
};

// One warp's running state, with the positions of its rows.
template <bool F16>
struct State : RowState<F16> {
  using RowState<F16>::qf;
  using RowState<F16>::acc;
  using RowState<F16>::m0;
  using RowState<F16>::m1;
  using RowState<F16>::l0;
  using RowState<F16>::l1;
  using RowState<F16>::below;
  int p0, p1, first, last;              // positions: the lane's rows', the tile's first and last

  // Q fragments: columns 16 kk + 2 (lane % 4) (+ 8) of the two rows, from rows in shared
  // memory or from the tensor
  __device__ __forceinline__ void load_rows(uint32_t sq, int lane) {
    const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
      ldmatrix_x4(sq + r * ROW_BYTES + (((2 * kk + (lane >> 4)) ^ (r & 7)) << 4), qf[kk]);
  }
  __device__ __forceinline__ void load_rows(const PagedAttn& a, const Work& w, int lane) {
    const int r = lane >> 2;
    const size_t rows = (size_t)a.v.s.T * a.v.s.H;
    (void)rows;                         // read by the checked build only
    const size_t a0 = w.at(a, r < w.rows ? r : 0), a1 = w.at(a, r + 8 < w.rows ? r + 8 : 0);
    const bool in0 = r < w.rows && RF_IDX_OK(a0, rows), in1 = r + 8 < w.rows && RF_IDX_OK(a1, rows);
    const uint8_t* q0 = a.q + a0 * ROW_BYTES + (lane & 3) * 4;
    const uint8_t* q1 = a.q + a1 * ROW_BYTES + (lane & 3) * 4;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      qf[kk][0] = in0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32) : 0u;
      qf[kk][1] = in1 ? *reinterpret_cast<const uint32_t*>(q1 + kk * 32) : 0u;
      qf[kk][2] = in0 ? *reinterpret_cast<const uint32_t*>(q0 + kk * 32 + 16) : 0u;
      qf[kk][3] = in1 ? *reinterpret_cast<const uint32_t*>(q1 + kk * 32 + 16) : 0u;
    }
  }

  __device__ __forceinline__ void start(const PagedAttn& a, const Work& w, int lane) {
    const int r = lane >> 2;
    this->clear();
    first = w.pos(a, 0);
    last = w.pos(a, w.rows - 1);
    p0 = w.pos(a, min(r, w.rows - 1));
    p1 = w.pos(a, min(r + 8, w.rows - 1));
  }

  // folds in keys key0 .. key0 + 15, whose copies are in `st`
  __device__ __forceinline__ void tile(const PagedAttn& a, uint32_t st, int key0, int lane) {
    float s[2][4];
    this->products(st, s, lane);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] *= a.scale_log2;
    const int window = a.v.s.window, sinks = a.v.s.sinks;
    const bool whole = key0 + TK - 1 <= first && (window == 0 || key0 > last - window || key0 + TK <= sinks);
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = key0 + nt * 8 + 2 * (lane & 3) + e;
          if (t > p0 || (window > 0 && t <= p0 - window && t >= sinks)) s[nt][e] = -INFINITY;
          if (t > p1 || (window > 0 && t <= p1 - window && t >= sinks)) s[nt][2 + e] = -INFINITY;
        }
    }
    this->fold(s, st, lane);
  }

  // the warp's rows r0 .. r0 + MERGE_ROWS - 1 into its part of the merge buffer
  __device__ __forceinline__ void give(float* acc_buf, float2* ml_buf, int r0, int rows, int lane) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = (lane >> 2) + 8 * half;
      if (r < r0 || r >= min(r0 + MERGE_ROWS, rows)) continue;
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
        *reinterpret_cast<float2*>(acc_buf + (r - r0) * MERGE_PITCH + d * 8 + 2 * (lane & 3)) =
            make_float2(acc[d][2 * half], acc[d][2 * half + 1]);
      if ((lane & 3) == 0) ml_buf[r - r0] = half ? make_float2(below(m1), l1) : make_float2(below(m0), l0);
    }
  }
};

// Row r's accumulator A over the keys of tiles t0 .. t1 - 1, weights relative to `ref`,
// with the columns that are NaN computed again key by key from the row's visible keys:
// an infinite value gives that infinity (its product with a weight's second term does
// not), and a value that another row of the tile sees does not reach this one.  Ends once
// the columns are all NaN again, which they stay.
template <bool F16>
__device__ __forceinline__ float4 redo_columns(const PagedAttn& a, const Work& w, int r, int t0, int t1, float ref,
                                               float4 A, int lane) {
  const int window = a.v.s.window, sinks = a.v.s.sinks, p = w.pos(a, r);
  const float4 x = load_row4<F16>(a.q + w.at(a, r) * ROW_BYTES, lane);
  float4 R = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t = t0; t < t1; ++t) {
    const int tile = w.key_tile(t), page = page_of(a, w.b, tile);
    const bool has = (unsigned)page < (unsigned)a.pages;
    const size_t row0 = row_of(a, has ? page : 0, w.hk, tile);
    for (int u0 = 0; u0 < TK; u0 += 8) {
      float s[8];
      float4 v[8];
      bool seen[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int key = tile * TK + u0 + u;
        seen[u] = key <= p && (window == 0 || key > p - window || key < sinks);
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
        v[u] = k;
        const size_t at = row0 + u0 + u;
        if (seen[u] && has && RF_IDX_OK(at, ((size_t)a.pages * a.v.s.Hkv) << a.page_log2)) {
          k = load_row4<F16>(a.kp + at * ROW_BYTES, lane);
          v[u] = load_row4<F16>(a.vp + at * ROW_BYTES, lane);
        }
        s[u] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, x.w * k.w)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < 8; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (!seen[u]) continue;
        const float e = exp2f(__fmul_rn(s[u], a.scale_log2) - ref);
        R.x = fmaf(e, v[u].x, R.x);
        R.y = fmaf(e, v[u].y, R.y);
        R.z = fmaf(e, v[u].z, R.z);
        R.w = fmaf(e, v[u].w, R.w);
      }
    }
    const bool again = (A.x != A.x && R.x == R.x) || (A.y != A.y && R.y == R.y) ||
                       (A.z != A.z && R.z == R.z) || (A.w != A.w && R.w == R.w);
    if (!__any_sync(0xffffffffu, again)) break;
  }
  return make_float4(A.x != A.x ? R.x : A.x, A.y != A.y ? R.y : A.y, A.z != A.z ? R.z : A.z,
                     A.w != A.w ? R.w : A.w);
}

// a finished row, four columns per lane
__device__ __forceinline__ void write_row(const PagedAttn& a, size_t row, float4 A, float M, float L, int lane,
                                          int dtype) {
  if (!RF_IDX_OK(row, (size_t)a.v.s.T * a.v.s.H)) return;
  const size_t o = row * HD + lane * 4;
  store_out2(a.out, o, normalised(A.x, L), normalised(A.y, L), dtype);
  store_out2(a.out, o + 2, normalised(A.z, L), normalised(A.w, L), dtype);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = (M + log2f(L)) * kLn2;
}

// Row r of the CTA's warps, in place `at` of the merge buffer, merged by one warp, four
// columns per lane, into the output or into the unit's state.
// Whether the row has NaN columns: *ml then gets its maximum and sum.
template <bool F16>
__device__ __forceinline__ bool merge_warps(const PagedAttn& a, const Work& w, const float* acc_buf,
                                            const float2 (*ml_buf)[MERGE_ROWS], int r, int at, bool direct,
                                            size_t state0, float2* ml_out, int lane) {
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) M = fmaxf(M, ml_buf[i][at].x);
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const float2 ml = ml_buf[i][at];
    const float f = exp2f(ml.x - ref_of(M));
    const float4 v = *reinterpret_cast<const float4*>(acc_buf + (i * MERGE_ROWS + at) * MERGE_PITCH + lane * 4);
    L = fmaf(f, ml.y, L);
    A.x = fmaf(f, v.x, A.x);
    A.y = fmaf(f, v.y, A.y);
    A.z = fmaf(f, v.z, A.z);
    A.w = fmaf(f, v.w, A.w);
  }
  if (direct) {
    write_row(a, w.at(a, r), A, M, L, lane, F16 ? RF_F16 : RF_BF16);
  } else {
    const size_t s = state0 + r;
    if (!RF_IDX_OK(s, (size_t)a.v.state_cap * a.v.s.Hkv * a.v.s.unit_rows())) return false;
    *(reinterpret_cast<float4*>(a.v.unit_acc + s * HD) + lane) = A;
    if (lane == 0) a.v.unit_ml[s] = make_float2(M, L);
  }
  const bool bad = __any_sync(0xffffffffu, L > 0.f && any_nan(A));
  if (bad && lane == 0) *ml_out = make_float2(M, L);
  return bad;
}

// The NaN columns of a row that merge_warps has written, once more.  A call, so that its
// code and its registers lie apart.
template <bool F16>
__device__ __noinline__ void redo_row(const PagedAttn& a, const Work w, int r, bool direct, size_t state0,
                                      float2 ml, int t0, int t1, int lane) {
  const size_t row = w.at(a, r), s = state0 + r;
  if (direct ? !RF_IDX_OK(row, (size_t)a.v.s.T * a.v.s.H)
             : !RF_IDX_OK(s, (size_t)a.v.state_cap * a.v.s.Hkv * a.v.s.unit_rows()))
    return;
  float4* state = reinterpret_cast<float4*>(a.v.unit_acc + s * HD) + lane;
  const float4 A = direct ? load_row4<F16>(a.out + row * ROW_BYTES, lane) : *state;
  float4 R = redo_columns<F16>(a, w, r, t0, t1, ref_of(ml.x), A, lane);
  if (direct) {                         // the other columns are normalised already
    R = make_float4(A.x != A.x ? R.x / ml.y : A.x, A.y != A.y ? R.y / ml.y : A.y, A.z != A.z ? R.z / ml.y : A.z,
                    A.w != A.w ? R.w / ml.y : A.w);
    const size_t o = row * HD + lane * 4;
    store_out2(a.out, o, R.x, R.y, F16 ? RF_F16 : RF_BF16);
    store_out2(a.out, o + 2, R.z, R.w, F16 ? RF_F16 : RF_BF16);
  } else {
    *state = R;
  }
}

// Rows r0 .. r0 + nr - 1 (at most RB) of a tile from the states of its pieces, in order;
// one warp, four columns per lane, LOADS / RB states in flight.
template <int RB, int LOADS>
__device__ __forceinline__ void merge_pieces(const PagedAttn& a, const Work& w, int first, int pieces, int r0,
                                             int nr, int dtype, int lane) {
  constexpr int SB = LOADS / RB;
  const size_t step = (size_t)a.v.s.Hkv * a.v.s.unit_rows();
  const size_t base = first * step + (size_t)w.hk * a.v.s.unit_rows() + r0;
  const size_t states = (size_t)a.v.state_cap * step;
  (void)states;                         // read by the checked build only
  float M[RB], L[RB];
  float4 A[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    M[r] = -INFINITY;
    L[r] = 0.f;
    A[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int s0 = 0; s0 < pieces; s0 += 32) {
    const int cnt = min(32, pieces - s0);
    // lane j holds piece s0 + j's maximum and sum, then its weight; the accumulators are
    // asked for before the weights are known
    float2 ml[RB];
    float f[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      ml[r] = make_float2(-INFINITY, 0.f);
      const size_t at = base + (s0 + lane) * step + r;
      if (r < nr && lane < cnt && RF_IDX_OK(at, states)) ml[r] = __ldcg(a.v.unit_ml + at);
    }
    for (int j0 = 0; j0 < cnt; j0 += SB) {
      float4 v[RB][SB];
#pragma unroll
      for (int j = 0; j < SB; ++j)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const size_t at = base + (s0 + j0 + j) * step + r;
          v[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < nr && j0 + j < cnt && RF_IDX_OK(at, states))
            v[r][j] = __ldcg(reinterpret_cast<const float4*>(a.v.unit_acc + at * HD) + lane);
        }
      if (j0 == 0) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float top = fmaxf(M[r], group_max<32>(ml[r].x)), c = exp2f(M[r] - ref_of(top));
          M[r] = top;
          L[r] *= c;
          A[r].x *= c;
          A[r].y *= c;
          A[r].z *= c;
          A[r].w *= c;
          f[r] = -1.f;                            // a piece without keys: its accumulator is not read
          if (ml[r].x != -INFINITY) {
            f[r] = exp2f(ml[r].x - ref_of(top));
            L[r] = fmaf(f[r], ml[r].y, L[r]);
          } else {
            L[r] += ml[r].y;                      // 0, or NaN where every score was NaN
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
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    L[r] = group_sum<32>(L[r]);
    if (r < nr) write_row(a, w.at(a, r0 + r), A[r], M[r], L[r], lane, dtype);
  }
}

// The small calls' kernel: a CTA per unit, of four warps that do everything, for the
// shortest way from launch to output.
template <bool F16>
__global__ void __launch_bounds__(WARPS * 32, 2)
paged_few_kernel(const __grid_constant__ PagedAttn a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 sm_ml[WARPS][MERGE_ROWS], sm_redo[MROWS];
  __shared__ int sm_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hkv = a.v.s.Hkv;
  float* acc_buf = reinterpret_cast<float*>(smem + WARPS * RING_BYTES);
  wait_prerequisite();
  allow_dependents();
  int total = 0x7fffffff;               // known with the first unit
  for (int i = blockIdx.x, turn = 0; i < total; i += (int)gridDim.x, ++turn) {
    const int unit = i / Hkv, hk = i - unit * Hkv;
    if (!RF_IDX_OK(unit, a.v.unit_cap)) break;
    PagedUnit u;
    {
      int4* to = reinterpret_cast<int4*>(&u);
      const int4* from = reinterpret_cast<const int4*>(a.v.units + unit);
      to[0] = from[0], to[1] = from[1], to[2] = from[2];
    }
    if (turn == 0) {
      total = a.v.head[kPlanMark] == (int)a.v.mark ? min(a.v.head[kPlanUnits], a.v.unit_cap) * Hkv : 0;
      if (i >= total) break;
    }
    const Work w(a, u, hk);
    Stream in;
    in.ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * RING_BYTES;
    in.in = 0;
    in.open(a, u, hk, warp);
    in.ids = in.id_of(a, in.t + lane * WARPS);
    const uint64_t policy = l2_policy(false);
    auto issue = [&]() {
      if (in.t < in.end) in.copy(a, policy, lane);
      cp_async_commit();
    };
    const int t0 = in.t;
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) issue();
    State<F16> st;
    st.start(a, w, lane);
    st.load_rows(a, w, lane);
    int slot = 0;
    for (int t = t0; t < in.end; t += WARPS) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();                     // every lane's copies of this tile landed, the last is read
      issue();
      st.tile(a, in.ring + (uint32_t)slot * STAGE_BYTES, in.key_tile(t) * TK, lane);
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    st.close();
    const size_t state0 = ((size_t)u.state * Hkv + hk) * a.v.s.unit_rows();
    uint32_t bad = 0;
    for (int r = 0; r < w.rows; r += MERGE_ROWS) {
      if (r > 0) __syncthreads();       // the last rows have been read
      st.give(acc_buf + warp * MERGE_ROWS * MERGE_PITCH, sm_ml[warp], r, w.rows, lane);
      __syncthreads();
      if (r + warp < w.rows &&
          merge_warps<F16>(a, w, acc_buf, sm_ml, r + warp, warp, u.pieces == 1, state0, &sm_redo[r + warp], lane))
        bad |= 1u << (r + warp);
    }
    __syncwarp();
    for (; bad != 0; bad &= bad - 1) {
      const int r = __ffs(bad) - 1;
      redo_row<F16>(a, w, r, u.pieces == 1, state0, sm_redo[r], u.step0 * WARPS, in.end, lane);
    }
    __syncthreads();                    // states stored, merge buffer free
    if (u.pieces == 1) continue;
    if (threadIdx.x == 0) {
      const size_t at = (size_t)u.first * Hkv + hk;
      int last = 0;
      if (RF_IDX_OK(at, (size_t)a.v.unit_cap * Hkv)) {
        __threadfence();                // stands for the CTA, which the barrier joined
        last = atomicAdd(a.v.counters + at, 1) == u.pieces - 1;
        __threadfence();
        if (last) a.v.counters[at] = 0;
      }
      sm_last = last;
    }
    __syncthreads();
    if (sm_last) {
      const int share = (w.rows + WARPS - 1) / WARPS, r = warp * share, nr = min(share, w.rows - r);
      const int first = u.state - (unit - u.first);          // the first piece's state
      constexpr int dtype = F16 ? RF_F16 : RF_BF16;
      if (nr > 0) {
        if (share == 1)
          merge_pieces<1, 32>(a, w, first, u.pieces, r, nr, dtype, lane);
        else if (share == 2)
          merge_pieces<2, 32>(a, w, first, u.pieces, r, nr, dtype, lane);
        else
          merge_pieces<4, 32>(a, w, first, u.pieces, r, nr, dtype, lane);
      }
    }
    __syncthreads();                    // sm_last may be written again
  }
}

// What a team's warps hand one another; units are copied 16 bytes at a time.
struct alignas(16) Team {
  PagedUnit unit[2];
  int pages[2][32 * WARPS];             // page numbers of a unit's first tiles
  float2 ml[WARPS][MERGE_ROWS], redo[MROWS];
  uint64_t ready;                       // a phase per unit: what comes behind it is known
  int next[2];
};

template <bool F16>
__global__ void __launch_bounds__(THREADS, 1)
paged_decode_kernel(const __grid_constant__ PagedAttn a, const bool behind_pairs) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Team teams[TEAMS];
  __shared__ int sm_abort;
  static_assert(sizeof(PagedUnit) == 48 && offsetof(Team, unit) == 0, "three 16-byte copies");
  static_assert(sizeof(Team) % 16 == 0, "in every team");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool closes = warp >= CLOSE_WARP;
  const int team = closes ? (warp - CLOSE_WARP) % TEAMS : warp / WARPS;
  Team& tm = teams[team];
  const int bars = team * kBars;
  uint8_t* base = smem + team * TEAM_BYTES;
  float* acc_buf = reinterpret_cast<float*>(base + WARPS * RING_BYTES);
  uint8_t* q_buf = base + WARPS * RING_BYTES + MERGE_BYTES;
  const int Hkv = a.v.s.Hkv;
  if (threadIdx.x < TEAMS) tc::mbar_init(&teams[threadIdx.x].ready, 1);
  if (threadIdx.x == 0) sm_abort = 0;
  // behind the pair kernel of the same call, which has waited: what was before that is read by L2 alone
  if (!behind_pairs) wait_prerequisite();
  allow_dependents();
  // by the closing warp
  auto fetch_unit = [&](int i, int to) {
    const int unit = i / Hkv;
    if (lane < 3 && RF_IDX_OK(unit, a.v.unit_cap))
      reinterpret_cast<int4*>(&tm.unit[to])[lane] = __ldcg(reinterpret_cast<const int4*>(a.v.units + unit) + lane);
    __syncwarp();
  };
  auto fetch_pages = [&](int at) {
    const PagedUnit& u = tm.unit[at];
    const PagedTiles k(u.n, u.len, a.v.s.window, a.v.s.sinks);
    const int t0 = u.step0 * WARPS, end = min(k.tiles, u.step1 * WARPS);
#pragma unroll
    for (int e = 0; e < WARPS; ++e) {
      const int t = t0 + e * 32 + lane;
      tm.pages[at][e * 32 + lane] =
          t < end ? page_of(a, u.b, t < k.sink_tiles ? t : t - k.sink_tiles + k.lo_tile) : -1;
    }
  };
  // two query rows per step of a loop; a row of none is zeros
  auto query_row = [&](const Work& w, int e) {
    const int r = 2 * e + (lane >> 4);
    const size_t row = r < w.rows ? w.at(a, r) : 0;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < w.rows && RF_IDX_OK(row, (size_t)a.v.s.T * a.v.s.H))
      x = __ldcg(reinterpret_cast<const uint4*>(a.q + row * ROW_BYTES) + (lane & 15));
    return x;
  };
  auto keep_row = [&](int e, const uint4& x) {
    const int r = 2 * e + (lane >> 4);
    *reinterpret_cast<uint4*>(q_buf + r * ROW_BYTES + (((lane & 15) ^ (r & 7)) << 4)) = x;
  };
  // every SM has a team at work before any has two
  int i = (int)(blockIdx.x + team * gridDim.x);
  const bool fits = i < a.v.unit_cap * Hkv;
  if (warp < CLOSE_WARP + TEAMS && closes && fits) fetch_unit(i, 0);   // before it is known whether it is one
  const bool planned = __ldcg(a.v.head + kPlanMark) == (int)a.v.mark;
  const int total = planned ? min(__ldcg(a.v.head + kPlanUnits), a.v.unit_cap) * Hkv : 0;
  const int at_once = (int)gridDim.x * TEAMS;
  const bool queued = total > at_once;
  if (warp < CLOSE_WARP + TEAMS && closes && i < total) fetch_pages(0);
  __syncthreads();

  if (!closes) {
    // ------------------------------------------------------ stream ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_STREAM));
    const int wt = warp % WARPS;        // of the team
    const uint32_t sq = static_cast<uint32_t>(__cvta_generic_to_shared(q_buf));
    // a large call's cache is read once and goes first; a small one's may be read again
    const uint64_t policy = l2_policy(queued);
    Stream in;
    in.ring = static_cast<uint32_t>(__cvta_generic_to_shared(base)) + wt * RING_BYTES;
    in.in = 0;
    // The copies run on from unit to unit: `turn` is the unit that is being computed, the
    // stream is in it (ahead = 0) or in the next.  calls counts issues, call0 and call1
    // are those of the first tile of the unit and the next: a tile has landed when all but
    // the last group of copies have, two issues after its own.
    int turn = 0, ahead = 0, calls = 0, call0 = 0, call1 = 0, slot = 0, next = total;
    bool known = true;                  // whether next is; the first unit's query rows come before it
    auto open = [&](int at, int head) {
      in.open(a, tm.unit[at], head, wt);
      in.ids = tm.pages[at][lane * WARPS + wt];
    };
    if (i < total) open(0, i - i / Hkv * Hkv);
    auto move_on = [&]() {              // the stream into the next unit, if there is one
      if (!known) {
        known = true;
        const bool there = tc::mbar_wait(&tm.ready, (uint32_t)turn & 1u, &sm_abort);
        __syncwarp();
        if (there) next = tm.next[turn & 1];
      }
      if (ahead == 0 && next < total) {
        ahead = 1;
        open((turn + 1) & 1, next - next / Hkv * Hkv);
      }
    };
    auto issue = [&]() {
      if (in.t >= in.end && ahead == 0) move_on();
      if (in.t < in.end) {
        if (in.n == 0) {
          call1 = ahead ? calls : call1;
          call0 = ahead ? call0 : calls;
        }
        in.copy(a, policy, lane);
      }
      cp_async_commit();
      ++calls;
    };
    while (i < total) {
      const PagedUnit& u = tm.unit[turn & 1];
      const int unit = i / Hkv, hk = i - unit * Hkv;
      const PagedTiles keys(u.n, u.len, a.v.s.window, a.v.s.sinks);
      const int t0 = u.step0 * WARPS, t1 = min(keys.tiles, u.step1 * WARPS);
      if (t0 + wt < t1) {
        if (ahead == 0 && in.n == 0) issue();
        while (calls - call0 < STAGES - 1) issue();
      }
      State<F16> st;
      st.start(a, Work(a, u, hk), lane);
      if (turn == 0) {                  // the first unit's query rows are in place
        named_sync<TEAM>(bars + kBarEnd);
        known = !queued;
      }
      st.load_rows(sq, lane);
      if (queued) named_arrive<TEAM>(bars + kBarRows);
      for (int t = t0 + wt; t < t1; t += WARPS) {
        cp_async_wait<STAGES - 2>();
        __syncwarp();                   // every lane's copies of this tile landed, the last is read
        issue();
        const int tile = t < keys.sink_tiles ? t : t - keys.sink_tiles + keys.lo_tile;
        st.tile(a, in.ring + (uint32_t)slot * STAGE_BYTES, tile * TK, lane);
        slot = slot + 1 == STAGES ? 0 : slot + 1;
      }
      st.close();
      const Work w(a, u, hk);
      const size_t state0 = ((size_t)u.state * Hkv + hk) * a.v.s.unit_rows();
      uint32_t bad = 0;
      for (int r = 0; r < w.rows; r += MERGE_ROWS) {
        if (r > 0) named_sync<WARPS * 32>(bars + kBarStream);   // the last rows have been read
        st.give(acc_buf + wt * MERGE_ROWS * MERGE_PITCH, tm.ml[wt], r, w.rows, lane);
        named_sync<WARPS * 32>(bars + kBarStream);
        if (r + wt < w.rows &&
            merge_warps<F16>(a, w, acc_buf, tm.ml, r + wt, wt, u.pieces == 1, state0, &tm.redo[r + wt], lane))
          bad |= 1u << (r + wt);
      }
      __syncwarp();
      for (; bad != 0; bad &= bad - 1) {
        const int r = __ffs(bad) - 1;
        redo_row<F16>(a, w, r, u.pieces == 1, state0, tm.redo[r], t0, t1, lane);
      }
      move_on();
      named_sync<TEAM>(bars + kBarEnd);  // states stored, merge buffer free, next query rows in place
      if (queued) {                     // as move_on has it, unless its wait gave up
        next = tm.next[turn & 1];
        known = true;
        move_on();
      }
      i = next;
      ++turn;
      ahead = 0;
      call0 = call1;
      next = total;
      known = false;
    }
    cp_async_wait<0>();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CLOSE));
    // ------------------------------------------------------- close ----
    if (warp >= CLOSE_WARP + TEAMS) i = total;    // fills its warpgroup
    if (i < total) {
      const Work w(a, tm.unit[0], i - i / Hkv * Hkv);
      for (int e = 0; e < MROWS / 2; ++e) keep_row(e, query_row(w, e));
      named_sync<TEAM>(bars + kBarEnd);
    }
    for (int turn = 0; i < total; ++turn) {
      int next = total;
      if (queued) {
        if (lane == 0) {
          const int got = atomicAdd(a.v.head + kPlanQueue, 1);
          next = at_once + got;
          // every unit fetches once, so this was the last fetch
          if (got == total - 1) atomicExch(a.v.head + kPlanQueue, 0);
        }
        next = __shfl_sync(0xffffffffu, next, 0);
        if (next < total) {
          fetch_unit(next, (turn + 1) & 1);
          fetch_pages((turn + 1) & 1);
        }
        __syncwarp();
        if (lane == 0) {
          tm.next[turn & 1] = next;
          tc::mbar_arrive(&tm.ready);
        }
        // this unit's rows have been read, the next one's take their place
        if (next < total) {
          const Work w(a, tm.unit[(turn + 1) & 1], next - next / Hkv * Hkv);
          uint4 x[MROWS / 2];
#pragma unroll
          for (int e = 0; e < MROWS / 2; ++e) x[e] = query_row(w, e);
          named_sync<TEAM>(bars + kBarRows);
#pragma unroll
          for (int e = 0; e < MROWS / 2; ++e) keep_row(e, x[e]);
        } else {
          named_sync<TEAM>(bars + kBarRows);
        }
      }
      named_sync<TEAM>(bars + kBarEnd);
      i = next;
    }
  }
  if (behind_pairs) wait_prerequisite();   // a kernel ends after the one before it
}

template <bool F16>
rf_status launch_few(const PagedAttn& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t bytes = (size_t)WARPS * RING_BYTES + MERGE_BYTES;
  if (smem_attr(paged_few_kernel<F16>, bytes, done) != RF_OK) return RF_ERR_CUDA;
  const long long most = (long long)a.v.unit_cap * a.v.s.Hkv;
  const unsigned grid = (unsigned)(most < 2ll * sms ? most : 2ll * sms);
  return launch_after(paged_few_kernel<F16>, grid, WARPS * 32, bytes, st, a);
}

template <bool F16>
rf_status launch_t(const PagedAttn& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const int sms = tc::sm_count();
  if (sms <= 0) return RF_ERR_CUDA;
  if (a.v.s.few) return launch_few<F16>(a, sms, st);
  auto* kernel = paged_decode_kernel<F16>;
  // launched with fewer registers than the warpgroups' shares add up to, the streaming
  // warps would wait for them for ever
  static const bool regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kernel) == cudaSuccess && fa.numRegs == REGS;
  }();
  if (!regs) return RF_ERR_UNSUPPORTED;
  if (smem_attr(kernel, SMEM_BYTES, done) != RF_OK) return RF_ERR_CUDA;
  const long long most = (long long)a.v.unit_cap * a.v.s.Hkv;
  const unsigned grid = (unsigned)(most < sms ? most : sms);
  return launch_after(kernel, grid, THREADS, SMEM_BYTES, st, a, a.v.s.some_pairs());
}

}  // namespace

rf_status launch_paged_decode(const PagedAttn& a, int dtype, cudaStream_t st) {
  return dtype == RF_F16 ? launch_t<true>(a, st) : launch_t<false>(a, st);
}

RF_TIMEOUT_WORD_OF_THIS_FILE

RF_BOUNDS_WORD_OF_THIS_FILE

}  // namespace rf
