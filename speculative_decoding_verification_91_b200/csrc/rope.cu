// Rotary positions on strided rows of heads (spec_rope): half or interleaved
// pairs over part of the head, any frequencies, forwards or back.
//
//   y0 = x0 c - x1 s,  y1 = x0 s + x1 c,   (c, s) = magnitude (cos, sin)(t f_j)
//
// Bound by memory: every element is read and written once.  Angles are formed once
// for a row and all heads (a thread's own for every pair would be 30 instructions an
// element).  Two forms:
//   direct  where 16-byte pieces hold whole pairs (interleaved) or lie opposite
//           each other (half: span / 2 a multiple of the piece): a thread keeps a
//           piece, or two opposite ones, of the head, forms their angles in
//           registers while the piece's loads of several heads are on their way,
//           turns them and goes on to its next row.  (Angles passed round a CTA in
//           shared memory: 61 us for the case below.)
//   staged  any other span or alignment: the heads pass through shared memory, in
//           16-byte pieces where rows and heads are aligned to them, else element
//           by element.
// 32,768 rows of 8 x 256 bf16, interleaved: 46.0 us, 5.8 TB/s (with 256 threads a CTA
// 51.5; four loads in flight instead of eight 48.0).  5 x 16 x 256: 2.5 us in a graph.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kRopeOpThreads = 256;     // staged
constexpr int kDirectThreads = 128;
constexpr int kRopeRows = 32;           // rows of a CTA
constexpr int kRopeTile = 16384;        // bytes of heads of a CTA

struct RopePlan {
  int rows, heads;                // direct: of a thread; staged: of a CTA
  int units;                      // pieces (or elements) of a head
  int groups, side, chunks;       // direct: of heads; rows side by side in a CTA; CTAs across a row's pieces
  int turning;                    // direct: pieces that turn, the first ones
  int head_blocks;                // staged: CTAs across the heads
  Div by_units, by_heads, by_pairs, by_n, by_turning, by_rest;   // by_n: a row's pieces and groups
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) { return f32_to_bf16(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }

template <typename T>
union Piece {
  uint4 v;
  T e[16 / sizeof(T)];
  uint32_t w[4];
};

// Two 16-bit elements of a word.
template <typename T>
__device__ __forceinline__ float2 two(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t word(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <typename T>
__device__ __forceinline__ void turn(T& a, T& b, float2 cs) {
  const float x0 = to_f<T>(a), x1 = to_f<T>(b);
  a = from_f<T>(x0 * cs.x - x1 * cs.y);
  b = from_f<T>(x0 * cs.y + x1 * cs.x);
}

// A whole piece's pairs (HALF: with the opposite piece b).  16-bit elements two at a time: taken out and rounded one by
// one they were a third of the kernel's instructions.
template <typename T, bool HALF>
__device__ __forceinline__ void turn_piece(Piece<T>& a, Piece<T>& b, const float2 (&c)[(HALF ? 16 : 8) / sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = two<T>(a.w[e]);
      if (HALF) {
        const float2 y = two<T>(b.w[e]), c0 = c[HALF ? 2 * e : 0], c1 = c[HALF ? 2 * e + 1 : 0];
        a.w[e] = word<T>(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
        b.w[e] = word<T>(x.x * c0.y + y.x * c0.x, x.y * c1.y + y.y * c1.x);
      } else {
        const float2 c0 = c[e];
        a.w[e] = word<T>(x.x * c0.x - x.y * c0.y, x.x * c0.y + x.y * c0.x);
      }
    }
  } else {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int e = 0; e < (HALF ? E : E / 2); ++e)
      turn(a.e[HALF ? e : 2 * e], HALF ? b.e[e] : a.e[2 * e + 1], c[e]);
  }
}

// The first `turning` pairs of a piece.
template <typename T, bool HALF>
__device__ __forceinline__ void turn_some(Piece<T>& a, Piece<T>& b, const float2 (&c)[(HALF ? 16 : 8) / sizeof(T)], int turning) {
  constexpr int PP = (HALF ? 16 : 8) / sizeof(T);
  if (turning == PP) {
    turn_piece<T, HALF>(a, b, c);
  } else {
#pragma unroll
    for (int e = 0; e < PP; ++e)
      if (e < turning) turn(a.e[HALF ? e : 2 * e], HALF ? b.e[HALF ? e : 0] : a.e[HALF ? 0 : 2 * e + 1], c[e]);
  }
}

// Positions and (c, s) of the CTA's rows; ends with a barrier.
__device__ __forceinline__ void angles(const RopeArgs& r, const RopeOpArgs& a, const RopePlan& p, int64_t row0,
                                       float2* cs, int* pos) {
  const int n = p.rows * r.n_rot;
  if (threadIdx.x < p.rows)
    pos[threadIdx.x] = row0 + threadIdx.x < a.n_rows ? a.positions[row0 + threadIdx.x] : -1;
  for (int i = threadIdx.x; i < n; i += kRopeOpThreads) {
    const int t = p.by_pairs(i), j = i - t * r.n_rot;
    const int at = row0 + t < a.n_rows ? a.positions[row0 + t] : -1;
    float c = 1.f, s = 0.f;
    if (at >= 0) rope_turn(at, r.step[j], static_cast<float>(r.magnitude), c, s);
    cs[i] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
}

// A thread keeps its piece (or two opposite ones) of a head, and with it the pairs'
// frequencies, and goes down the CTA's rows.
// ROWS: one head, so the loads of several rows are in flight instead of several heads'
// (the same call one row at a time: 132 us).
template <typename T, int LAYOUT, bool ROWS>
__global__ void __launch_bounds__(kDirectThreads) rope_direct_kernel(const __grid_constant__ RopeArgs r,
                                                                     const __grid_constant__ RopeOpArgs a,
                                                                     const __grid_constant__ RopePlan p) {
  constexpr int E = 16 / sizeof(T);
  constexpr bool HALF = LAYOUT == SPEC_ROPE_HALF;
  constexpr int B = HALF ? 4 : 8;          // heads in flight of a thread: eight 16-byte loads
  constexpr int PP = HALF ? E : E / 2;     // pairs of a piece
  pdl_trigger();
  pdl_wait();
  // (rows of the CTA, groups of heads, pieces): side by side on the threads
  const int block = blockIdx.x / p.chunks, n = p.groups * p.units;
  int i = (blockIdx.x - block * p.chunks) * kDirectThreads + threadIdx.x, t0 = 0;
  int grp = 0, u;
  if (p.chunks == 1 && p.groups == 1) {
    // the rows' turning pieces first, then the others: few warps form angles (262,144
    // rows of 1 x 192 bf16, 64 dims turned: 63 us, 99 with the pieces in order)
    const int m = p.side * p.turning;
    if (i < m) {
      t0 = p.by_turning(i);
      u = i - t0 * p.turning;
    } else {
      t0 = p.by_rest(i - m);
      u = p.turning + (i - m) - t0 * (n - p.turning);
    }
    if (i >= p.side * n) return;
  } else {
    if (p.chunks == 1) t0 = p.by_n(i), i -= t0 * n;
    if (i >= n || t0 >= p.side) return;
    grp = p.by_units(i);
    u = i - grp * p.units;
  }
  const int h0 = grp * p.heads, heads = min(p.heads, a.n_heads - h0);
  // half: pairs of pieces first, then the pieces that pass through
  const int pair_units = r.span / 2 / E;
  const bool pair = HALF && u < pair_units;
  const int d = HALF && !pair ? r.span + (u - pair_units) * E : u * E, j = HALF ? d : d / 2;
  const int turning = !HALF || pair ? min(PP, r.n_rot - j) : 0;   // pairs of the piece that turn
  uint64_t step[PP];
#pragma unroll
  for (int e = 0; e < PP; ++e) step[e] = e < turning ? r.step[j + e] : 0;
  const int64_t first = static_cast<int64_t>(block) * p.side * p.rows + t0, last = min(first + p.side * p.rows, static_cast<int64_t>(a.n_rows));
  const T* src0 = static_cast<const T*>(a.x) + h0 * a.x_head + d;
  T* dst0 = static_cast<T*>(a.out) + h0 * a.out_head + d;
  if (ROWS) {
    for (int64_t row = first; row < last; row += B * p.side) {
      Piece<T> x0[B], x1[HALF ? B : 1];
      int at[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int64_t rb = row + b * p.side;
        at[b] = -1;
        if (rb >= last) continue;
        at[b] = a.positions[rb];
        x0[b].v = __ldcs(reinterpret_cast<const uint4*>(src0 + rb * a.x_row));
        if (HALF && pair) x1[b].v = __ldcs(reinterpret_cast<const uint4*>(src0 + rb * a.x_row + r.span / 2));
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (at[b] < 0) continue;
        if (turning > 0) {
          float2 cs[PP];
#pragma unroll
          for (int e = 0; e < PP; ++e) {
            float c, s;
            rope_turn(at[b], step[e], static_cast<float>(r.magnitude), c, s);
            cs[e] = make_float2(c, a.inverse ? -s : s);
          }
          turn_some<T, HALF>(x0[b], x1[HALF ? b : 0], cs, turning);
        }
        T* dst = dst0 + (row + b * p.side) * a.out_row;
        *reinterpret_cast<uint4*>(dst) = x0[b].v;
        if (HALF && pair) *reinterpret_cast<uint4*>(dst + r.span / 2) = x1[b].v;
      }
    }
    return;
  }
  int pos = first < last ? a.positions[first] : -1;
  for (int64_t row = first; row < last; row += p.side) {
    const int at = pos;
    if (row + p.side < last) pos = a.positions[row + p.side];
    if (at < 0) continue;
    const T* src = src0 + row * a.x_row;
    T* dst = dst0 + row * a.out_row;
    Piece<T> x0[B], x1[HALF ? B : 1];
    auto load = [&](int h) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (h + b >= heads) break;
        x0[b].v = __ldcs(reinterpret_cast<const uint4*>(src + (h + b) * a.x_head));
        if (HALF && pair) x1[b].v = __ldcs(reinterpret_cast<const uint4*>(src + (h + b) * a.x_head + r.span / 2));
      }
    };
    load(0);
    float2 cs[PP];
#pragma unroll
    for (int e = 0; e < PP; ++e) {
      float c = 1.f, s = 0.f;
      if (turning > 0) rope_turn(at, step[e], static_cast<float>(r.magnitude), c, s);
      cs[e] = make_float2(c, a.inverse ? -s : s);
    }
    for (int h = 0; h < heads; h += B) {
      if (h > 0) load(h);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (h + b >= heads) break;
        turn_some<T, HALF>(x0[b], x1[HALF ? b : 0], cs, turning);
        *reinterpret_cast<uint4*>(dst + (h + b) * a.out_head) = x0[b].v;
        if (HALF && pair) *reinterpret_cast<uint4*>(dst + (h + b) * a.out_head + r.span / 2) = x1[b].v;
      }
    }
  }
}

// Staged form; PIECES: 16 bytes at a time.
template <typename T, bool PIECES>
__global__ void __launch_bounds__(kRopeOpThreads) rope_staged_kernel(const __grid_constant__ RopeArgs r,
                                                                     const __grid_constant__ RopeOpArgs a,
                                                                     const __grid_constant__ RopePlan p) {
  constexpr int E = PIECES ? 16 / sizeof(T) : 1;
  extern __shared__ float2 cs[];
  __shared__ int pos[kRopeRows];
  __shared__ __align__(16) uint8_t tile_raw[kRopeTile];
  T* tile = reinterpret_cast<T*>(tile_raw);
  pdl_trigger();
  pdl_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.head_blocks) * p.rows;
  const int h0 = (blockIdx.x % p.head_blocks) * p.heads, heads = min(p.heads, a.n_heads - h0);
  const int n = p.rows * p.heads * p.units;
  auto each = [&](auto&& f) {              // every piece of the CTA's heads
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kRopeOpThreads) {
      const int rh = p.by_units(i), u = i - rh * p.units, t = p.by_heads(rh), h = rh - t * p.heads;
      if (h < heads && row0 + t < a.n_rows) f(i, t, h, u * E);
    }
  };
  each([&](int i, int t, int h, int d) {
    const T* src = static_cast<const T*>(a.x) + (row0 + t) * a.x_row + (h0 + h) * a.x_head + d;
    if (PIECES) reinterpret_cast<uint4*>(tile)[i] = *reinterpret_cast<const uint4*>(src);
    else tile[i] = *src;
  });
  angles(r, a, p, row0, cs, pos);
  const bool half = r.layout == SPEC_ROPE_HALF;
  for (int i = threadIdx.x; i < p.rows * p.heads * r.n_rot; i += kRopeOpThreads) {
    const int rh = p.by_pairs(i), j = i - rh * r.n_rot, t = p.by_heads(rh);
    T* x = tile + rh * a.dim;
    turn(x[half ? j : 2 * j], x[half ? j + r.span / 2 : 2 * j + 1], cs[t * r.n_rot + j]);
  }
  __syncthreads();
  each([&](int i, int t, int h, int d) {
    if (pos[t] < 0) return;
    T* dst = static_cast<T*>(a.out) + (row0 + t) * a.out_row + (h0 + h) * a.out_head + d;
    if (PIECES) *reinterpret_cast<uint4*>(dst) = reinterpret_cast<uint4*>(tile)[i];
    else *dst = tile[i];
  });
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& r, const RopeOpArgs& a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const auto whole = [&](int64_t stride, int64_t count) { return count == 1 || stride % E == 0; };
  const bool pieces = a.dim % E == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && whole(a.x_row, a.n_rows) &&
                      whole(a.x_head, a.n_heads) && whole(a.out_row, a.n_rows) && whole(a.out_head, a.n_heads);
  const bool half = r.layout == SPEC_ROPE_HALF;
  const bool direct = pieces && (!half || (r.span / 2) % E == 0);
  RopePlan p{};
  p.units = !direct ? (pieces ? a.dim / E : a.dim) : half ? r.span / 2 / E + (a.dim - r.span) / E : a.dim / E;
  if (direct && a.x == a.out)               // in place: only what turns
    p.units = half ? (r.n_rot + E - 1) / E : (2 * r.n_rot + E - 1) / E;
  if (p.units < 1) return cudaSuccess;
  p.by_units = make_div(p.units);
  if (direct) {
    // few rows: the heads spread over threads, down to one; many: all heads to a
    // thread and up to 16 rows, so that angles and frequencies are formed and read
    // once (half as wide 47.1 us for the case above, twice as wide 48.9)
    const int64_t wide = 148 * 512, pieces_all = static_cast<int64_t>(a.n_rows) * a.n_heads * p.units;
    p.heads = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.n_heads, pieces_all / wide)));
    p.groups = (a.n_heads + p.heads - 1) / p.heads;
    const int n = p.groups * p.units;
    p.side = std::max(1, kDirectThreads / n);
    p.chunks = (n + kDirectThreads - 1) / kDirectThreads;
    p.rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, static_cast<int64_t>(a.n_rows) * n / (4 * wide))));
    p.by_n = make_div(n);
    p.turning = std::min(p.units, half ? (r.n_rot + E - 1) / E : (2 * r.n_rot + E - 1) / E);
    p.by_turning = make_div(std::max(p.turning, 1));
    p.by_rest = make_div(std::max(p.units - p.turning, 1));
    const int64_t per = static_cast<int64_t>(p.side) * p.rows, ctas = (a.n_rows + per - 1) / per * p.chunks;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(ctas)), block(kDirectThreads);
    if (a.n_heads == 1)
      return half ? launch_k(rope_direct_kernel<T, SPEC_ROPE_HALF, true>, grid, block, 0, st, r, a, p)
                  : launch_k(rope_direct_kernel<T, SPEC_ROPE_INTERLEAVED, true>, grid, block, 0, st, r, a, p);
    return half ? launch_k(rope_direct_kernel<T, SPEC_ROPE_HALF, false>, grid, block, 0, st, r, a, p)
                : launch_k(rope_direct_kernel<T, SPEC_ROPE_INTERLEAVED, false>, grid, block, 0, st, r, a, p);
  }
  // bytes of a CTA: enough in flight for many rows, spread over the SMs for few
  const int64_t head = static_cast<int64_t>(a.dim) * sizeof(T), total = head * a.n_heads * a.n_rows;
  int64_t bytes = total / (2 * 148);
  bytes = bytes < 4096 ? 4096 : bytes > kRopeTile ? kRopeTile : bytes;
  p.heads = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.n_heads, bytes / head)));
  p.rows = p.heads < a.n_heads ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kRopeRows, bytes / (head * a.n_heads))));
  p.head_blocks = (a.n_heads + p.heads - 1) / p.heads;
  p.by_heads = make_div(p.heads);
  p.by_pairs = make_div(std::max(r.n_rot, 1));
  const int64_t ctas = (static_cast<int64_t>(a.n_rows) + p.rows - 1) / p.rows * p.head_blocks;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  const size_t smem = static_cast<size_t>(p.rows) * r.n_rot * sizeof(float2);   // at most 32 KB
  // the staged form's tile comes on top
  auto kern = pieces ? rope_staged_kernel<T, true> : rope_staged_kernel<T, false>;
  static std::atomic<uint64_t> allowed[2] = {};
  const cudaError_t e = allow_smem(kern, kRopeRows * kMaxPairs * static_cast<int>(sizeof(float2)), allowed[pieces]);
  return e != cudaSuccess ? e : launch_k(kern, grid, dim3(kRopeOpThreads), smem, st, r, a, p);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& r, const RopeOpArgs& a, int dtype, cudaStream_t st) {
  if (dtype == SPEC_BF16) return launch_typed<uint16_t>(r, a, st);
  if (dtype == SPEC_FP16) return launch_typed<__half>(r, a, st);
  return launch_typed<float>(r, a, st);
}

}  // namespace sv
