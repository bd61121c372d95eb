// Rotary positions on strided rows of heads (spec_rope): half or interleaved
// pairs over part of the head, any frequencies, forwards or back.
//
//   y0 = x0 c - x1 s,  y1 = x0 s + x1 c,   (c, s) = magnitude (cos, sin)(t f_j)
//
// Bound by memory: every element is read and written once.  A CTA takes `rows`
// rows of `heads` heads; their cosines and sines are formed once in shared
// memory, while the first loads are on their way (a thread's own angles for every
// pair would be 30 instructions an element).  Two forms:
//   direct  where 16-byte pieces hold whole pairs (interleaved) or lie opposite
//           each other (half: span / 2 a multiple of the piece): a thread turns a
//           piece, or two opposite ones, in registers.
//   staged  any other span or alignment: the heads pass through shared memory, in
//           16-byte pieces where rows and heads are aligned to them, else element
//           by element.
// 32,768 rows of 8 x 256 bf16, interleaved: TUNED
#include <math.h>

#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kRopeOpThreads = 256;
constexpr int kRopeRows = 32;           // rows of a CTA
constexpr int kRopeTile = 16384;        // bytes of heads of a CTA

struct RopePlan {
  int rows, heads, head_blocks;   // of a CTA; CTAs across the heads
  int units;                      // pieces (direct) of a head
  int n_tab;                      // n_rot, to whole pieces (direct)
  Div by_units, by_heads, by_pairs, by_n;   // by_n: pieces of a row
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
};

template <typename T>
__device__ __forceinline__ void turn(T& a, T& b, float2 cs) {
  const float x0 = to_f<T>(a), x1 = to_f<T>(b);
  a = from_f<T>(x0 * cs.x - x1 * cs.y);
  b = from_f<T>(x0 * cs.y + x1 * cs.x);
}

// Positions and (c, s) of the CTA's rows; ends with a barrier.  PP pairs of a piece:
// pair j of a row at [j % PP][j / PP], so that the lanes of a warp, a piece each, read
// next to each other (in pair order the bank conflicts took half of the kernel's time).
template <int PP>
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
    cs[t * p.n_tab + (PP == 1 ? j : j % PP * (p.n_tab / PP) + j / PP)] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
}

// A thread keeps its piece (or two opposite ones) of a head and goes down the CTA's
// rows, so that what depends on the piece is formed once.
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeOpThreads) rope_direct_kernel(const __grid_constant__ RopeArgs r,
                                                                     const __grid_constant__ RopeOpArgs a,
                                                                     const __grid_constant__ RopePlan p) {
  constexpr int E = 16 / sizeof(T);
  constexpr bool HALF = LAYOUT == SPEC_ROPE_HALF;
  constexpr int B = HALF ? 2 : 4;          // rows in flight of a thread: four 16-byte loads
  constexpr int PP = HALF ? E : E / 2;     // pairs of a piece
  extern __shared__ float2 cs[];
  __shared__ int pos[kRopeRows];
  pdl_trigger();
  pdl_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.head_blocks) * p.rows;
  const int h0 = (blockIdx.x % p.head_blocks) * p.heads, heads = min(p.heads, a.n_heads - h0);
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), a.n_rows - row0));
  const int n = p.heads * p.units, pair_units = r.span / 2 / E;
  // threads side by side on a row's pieces, `side` rows at a time
  const int side = n < kRopeOpThreads ? p.by_n(kRopeOpThreads) : 1;
  const int t0 = n < kRopeOpThreads ? p.by_n(threadIdx.x) : 0;
  int i = threadIdx.x - t0 * n, t = t0, d = 0, j = 0;
  const T* src = nullptr;
  T* dst = nullptr;
  bool turns = false, pair = false;
  auto piece = [&]() -> bool {             // what depends on the piece; false: none left
    for (; i < n && t0 < side; i += kRopeOpThreads) {
      const int h = p.by_units(i), u = i - h * p.units;
      if (h >= heads) continue;
      // half: pairs of pieces first, then the pieces that pass through
      pair = HALF && u < pair_units;
      d = HALF && !pair ? r.span + (u - pair_units) * E : u * E;
      j = HALF ? d : d / 2;
      turns = (!HALF || pair) && j < r.n_rot;
      src = static_cast<const T*>(a.x) + (row0 + t0) * a.x_row + (h0 + h) * a.x_head + d;
      dst = static_cast<T*>(a.out) + (row0 + t0) * a.out_row + (h0 + h) * a.out_head + d;
      t = t0;
      return t < rows;
    }
    return false;
  };
  Piece<T> x0[B], x1[HALF ? B : 1];
  auto load = [&]() {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (t + b * side >= rows) break;
      x0[b].v = __ldcs(reinterpret_cast<const uint4*>(src + b * side * a.x_row));
      if (HALF && pair) x1[b].v = __ldcs(reinterpret_cast<const uint4*>(src + b * side * a.x_row + r.span / 2));
    }
  };
  bool some = piece();
  if (some) load();
  angles<PP>(r, a, p, row0, cs, pos);
  while (some) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int tb = t + b * side;
      if (tb >= rows) break;
      if (turns) {
        const float2* c = cs + tb * p.n_tab + j / PP;
        const int ce = p.n_tab / PP;       // from a piece's pair to its next
        if (j + PP <= r.n_rot) {
#pragma unroll
          for (int e = 0; e < PP; ++e) {
            if (HALF) turn(x0[b].e[e], x1[b].e[e], c[e * ce]);
            else turn(x0[b].e[2 * e], x0[b].e[2 * e + 1], c[e * ce]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < PP; ++e) {
            if (j + e >= r.n_rot) break;
            if (HALF) turn(x0[b].e[e], x1[b].e[e], c[e * ce]);
            else turn(x0[b].e[2 * e], x0[b].e[2 * e + 1], c[e * ce]);
          }
        }
      }
      if (pos[tb] < 0) continue;
      *reinterpret_cast<uint4*>(dst + b * side * a.out_row) = x0[b].v;
      if (HALF && pair) *reinterpret_cast<uint4*>(dst + b * side * a.out_row + r.span / 2) = x1[b].v;
    }
    t += B * side;
    src += B * side * a.x_row;
    dst += B * side * a.out_row;
    if (t >= rows) {
      i += kRopeOpThreads;
      some = piece();
    }
    if (some) load();
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
  angles<1>(r, a, p, row0, cs, pos);
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
  // bytes of a CTA: enough in flight for many rows, spread over the SMs for few
  const int64_t head = static_cast<int64_t>(a.dim) * sizeof(T), total = head * a.n_heads * a.n_rows;
  int64_t bytes = total / (2 * 148);
  const int64_t most = direct ? 2 * kRopeTile : kRopeTile;
  bytes = bytes < 4096 ? 4096 : bytes > most ? most : bytes;
  RopePlan p{};
  p.heads = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.n_heads, bytes / head)));
  p.rows = p.heads < a.n_heads ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kRopeRows, bytes / (head * a.n_heads))));
  p.head_blocks = (a.n_heads + p.heads - 1) / p.heads;
  p.units = !direct ? (pieces ? a.dim / E : a.dim) : half ? r.span / 2 / E + (a.dim - r.span) / E : a.dim / E;
  if (direct && a.x == a.out)               // in place: only what turns
    p.units = half ? (r.n_rot + E - 1) / E : (2 * r.n_rot + E - 1) / E;
  if (p.units < 1) return cudaSuccess;
  p.by_units = make_div(p.units);
  p.by_heads = make_div(p.heads);
  p.by_n = make_div(p.heads * p.units);
  p.by_pairs = make_div(std::max(r.n_rot, 1));
  const int64_t ctas = (static_cast<int64_t>(a.n_rows) + p.rows - 1) / p.rows * p.head_blocks;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kRopeOpThreads);
  const int pp = !direct ? 1 : half ? E : E / 2;
  p.n_tab = (r.n_rot + pp - 1) / pp * pp;
  const size_t smem = static_cast<size_t>(p.rows) * p.n_tab * sizeof(float2);   // at most 32 KB
  if (direct)
    return half ? launch_k(rope_direct_kernel<T, SPEC_ROPE_HALF>, grid, block, smem, st, r, a, p)
                : launch_k(rope_direct_kernel<T, SPEC_ROPE_INTERLEAVED>, grid, block, smem, st, r, a, p);
  // the staged form's tile comes on top
  auto kern = pieces ? rope_staged_kernel<T, true> : rope_staged_kernel<T, false>;
  static std::atomic<uint64_t> allowed[2] = {};
  const cudaError_t e = allow_smem(kern, kRopeRows * kMaxPairs * static_cast<int>(sizeof(float2)), allowed[pieces]);
  return e != cudaSuccess ? e : launch_k(kern, grid, block, smem, st, r, a, p);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& r, const RopeOpArgs& a, int dtype, cudaStream_t st) {
  if (dtype == SPEC_BF16) return launch_typed<uint16_t>(r, a, st);
  if (dtype == SPEC_FP16) return launch_typed<__half>(r, a, st);
  return launch_typed<float>(r, a, st);
}

}  // namespace sv
