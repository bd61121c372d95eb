// The 8-bit paged cache: the append that quantises (spec_qcache_write) and the
// queries' form for the attention over it (qattn.cu).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kPg = SPEC_PAGE_SIZE;
constexpr int kWriteThreads = 256;

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.4028234e38f; }

// A binary64 value as the binary32 one next to it towards zero, its last bit
// set when that was not exact (rounding to odd): rounding the result once more
// to few bits then gives what rounding the binary64 value at once gives.
__device__ __forceinline__ float to_odd(double y) {
  const float f = __double2float_rz(y);
  return static_cast<double>(f) == y ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Element d of a head of the row at p, turned by r at pos, rounded to odd.
__device__ __forceinline__ float turned(const RopeArgs& r, const uint16_t* p, int d, int pos) {
  const int half = r.span / 2;
  int j = -1, e = d;          // pair and partner dim
  bool second = false;
  if (r.layout == SPEC_ROPE_HALF) {
    if (d < r.n_rot) j = d, e = d + half;
    else if (d >= half && d < half + r.n_rot) j = d - half, e = j, second = true;
  } else if (d < 2 * r.n_rot) {
    j = d >> 1, e = d ^ 1, second = d & 1;
  }
  const double x = bf16_to_f32(p[d]);
  if (j < 0) return static_cast<float>(x);
  const double w = bf16_to_f32(p[e]);
  double c, s;
  rope_turn(pos, r.turns[j], c, s);
  c *= r.magnitude;
  s *= r.magnitude;
  return to_odd(second ? w * s + x * c : x * c - w * s);
}

// One CTA per (touched block of tokens, KV head, sequence), keys (z even) or
// values (z odd).
__global__ void __launch_bounds__(kWriteThreads) qcache_write_kernel(const __grid_constant__ RopeArgs r,
                                                                     const __grid_constant__ QWriteArgs a) {
  extern __shared__ float rows[];            // [block][dim]
  __shared__ float red[kWriteThreads / 32];
  pdl_trigger();
  pdl_wait();
  const QCacheArgs& c = a.c;
  const int b = blockIdx.z >> 1, is_v = blockIdx.z & 1, h = blockIdx.y;
  const int L = c.seq_lens[b];
  if (L < 0 || static_cast<int64_t>(L) + a.n > static_cast<int64_t>(c.max_pages) * kPg) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) flag_status(c.status, SPEC_DEV_BAD_LENGTH);
    return;
  }
  const int p0 = (L / c.block + static_cast<int>(blockIdx.x)) * c.block;   // first position of the block
  if (p0 >= L + a.n) return;
  const int page = c.block_table[static_cast<int64_t>(b) * c.max_pages + p0 / kPg];
  if (page < 0 || page >= c.num_pages) {
    if (threadIdx.x == 0) flag_status(c.status, SPEC_DEV_BAD_PAGE);
    return;
  }
  const int lo = max(p0, L), hi = min(p0 + c.block, L + a.n);   // new positions
  const int D = c.dim;
  const uint16_t* src = is_v ? a.v_new : a.k_new;
  const int64_t stride = is_v ? a.v_row : a.k_row;
  float amax = 0.f;
  bool bad = false;
  for (int i = threadIdx.x; i < (hi - lo) * D; i += kWriteThreads) {
    const int pos = lo + i / D, d = i % D;
    const uint16_t* p = src + (static_cast<int64_t>(b) * a.n + (pos - L)) * stride + static_cast<int64_t>(h) * D;
    const float y = is_v ? bf16_to_f32(p[d]) : turned(r, p, d, pos);
    rows[i] = y;
    if (finite_f(y)) amax = fmaxf(amax, fabsf(y));
    else bad = true;
  }
  if (bad) flag_status(c.status, SPEC_DEV_NONFINITE);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < kWriteThreads / 32; ++w) amax = fmaxf(amax, red[w]);

  const int64_t head = static_cast<int64_t>(page) * c.n_kv_heads + h;
  float* sc = (is_v ? c.vs : c.ks) + head * (kPg / c.block) + (p0 % kPg) / c.block;
  uint8_t* dst = (is_v ? c.v : c.k) + (head * kPg + p0 % kPg) * D;
  float now = pow2f(scale_exponent(amax));
  const float was = *sc;
  if (lo > p0) {
    now = fmaxf(now, was);
    if (now > was) {                         // rewrite the committed codes for the larger scale
      const float ratio = __fdiv_rn(was, now);
      for (int i = threadIdx.x; i < (lo - p0) * D / 2; i += kWriteThreads) {
        uint16_t* q = reinterpret_cast<uint16_t*>(dst) + i;
        const float2 v = e4m3_values(*q);
        *q = e4m3x2(v.x == v.x ? v.x * ratio : 0.f, v.y == v.y ? v.y * ratio : 0.f);
      }
    }
  }
  const float inv = __fdiv_rn(1.f, now);
  for (int i = threadIdx.x; i < (hi - lo) * D / 2; i += kWriteThreads) {
    float v[2] = {rows[2 * i], rows[2 * i + 1]};
#pragma unroll
    for (int e = 0; e < 2; ++e) v[e] = v[e] == v[e] ? v[e] * inv : 0.f;
    reinterpret_cast<uint16_t*>(dst + (lo - p0) * D)[i] = e4m3x2(v[0], v[1]);
  }
  __syncthreads();
  if (threadIdx.x == 0) *sc = now;
}

// Queries: one warp per head of a row.  q = q_scale * (code0 + code1): the
// first code keeps 4 significant bits, the second 4 of what is left, so the two
// hold a query to 2^-9 of itself (and 2^-19 of the row's largest), finer than
// bf16's 2^-9 on average, and both factors of the score product are e4m3.  A
// row with an infinity or NaN gets a NaN scale, which makes its result NaN.
// A CTA takes a row of a sequence and every blockIdx.y-th four of its heads, a warp a head (4 or
// 8 dims a lane): the row's angles once for all of them (each warp forming its own took 41 us
// instead of TUNED for 512 rows of 32 heads), the first head asked for before.
template <int D>
__global__ void __launch_bounds__(128) qcache_query_kernel(const __grid_constant__ RopeArgs r,
                                                           const __grid_constant__ QAttnArgs a) {
  constexpr int P = D / 32;
  __shared__ float2 cs[kMaxPairs];
  pdl_trigger();
  pdl_wait();
  const int H = a.c.n_kv_heads, n_heads = H * a.G, lane = threadIdx.x & 31;
  const int64_t bi = blockIdx.x;
  const int b = static_cast<int>(bi / a.n), i = static_cast<int>(bi % a.n);
  const int L = a.c.seq_lens[b];
  const int half = r.span / 2;
  int pair[P], partner[P];   // pair of the dim, -1: passes through; the second of its pair: + kMaxPairs
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const int d = lane * P + e;
    int j = -1, w = d;
    if (r.layout == SPEC_ROPE_HALF) {
      if (d < r.n_rot) j = d, w = d + half;
      else if (d >= half && d < half + r.n_rot) j = d - half + kMaxPairs, w = d - half;
    } else if (d < 2 * r.n_rot) {
      j = (d >> 1) + (d & 1) * kMaxPairs;
      w = d ^ 1;
    }
    pair[e] = j;
    partner[e] = w;
  }
  float own[P], with[P];
  auto load = [&](int hq) {
    const uint16_t* p = a.q + bi * a.q_row + static_cast<int64_t>(hq) * D;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      own[e] = bf16_to_f32(p[lane * P + e]);
      with[e] = bf16_to_f32(p[partner[e]]);
    }
  };
  int hq = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (hq < n_heads) load(hq);
  if (threadIdx.x < r.n_rot) {
    const int pos = min(max(L, 0), 1 << 30) + a.q_offset + i;
    float c, s;
    rope_turn(pos, r.turns[threadIdx.x], static_cast<float>(r.magnitude), c, s);
    cs[threadIdx.x] = make_float2(c, s);
  }
  __syncthreads();
  for (; hq < n_heads; hq += gridDim.y * 4) {
    if (hq >= static_cast<int>(gridDim.y) * 4) load(hq);
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (pair[e] >= 0) {
        const float2 t = cs[pair[e] & (kMaxPairs - 1)];
        own[e] = pair[e] >= kMaxPairs ? with[e] * t.y + own[e] * t.x : own[e] * t.x - with[e] * t.y;
      }
      if (finite_f(own[e])) amax = fmaxf(amax, fabsf(own[e]));
      else bad = true;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    bad = __any_sync(0xffffffffu, bad);
    const int e2 = scale_exponent(amax);
    const float inv = pow2f(-e2);
    const int h = hq / a.G, g = hq % a.G;
    const int64_t row = (static_cast<int64_t>(b) * H + h) * a.rows + static_cast<int64_t>(i) * a.G + g;
    const int64_t plane = static_cast<int64_t>(a.B) * H * a.rows * D;
    uint32_t c0[P / 4], c1[P / 4];
#pragma unroll
    for (int e = 0; e < P; e += 2) {
      const float u = bad ? 0.f : own[e] * inv, v = bad ? 0.f : own[e + 1] * inv;
      const uint32_t x = e4m3x2(u, v);
      const float2 f = e4m3_values(x);
      const uint32_t y = e4m3x2(u - f.x, v - f.y);
      c0[e / 4] = e % 4 ? c0[e / 4] | x << 16 : x;
      c1[e / 4] = e % 4 ? c1[e / 4] | y << 16 : y;
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.q_codes + row * D + lane * P);
    uint32_t* dst1 = reinterpret_cast<uint32_t*>(a.q_codes + plane + row * D + lane * P);
#pragma unroll
    for (int e = 0; e < P / 4; ++e) {
      dst[e] = c0[e];
      dst1[e] = c1[e];
    }
    if (lane == 0) a.q_scale[row] = bad ? __int_as_float(0x7fffffff) : pow2f(e2);
    // where results are written by the attention kernel itself, a sequence that
    // gives it no work gets its zeros here
    if (a.n_splits == 1 && seq_keys(a, L).blocks == 0) {
#pragma unroll
      for (int e = 0; e < P; e += 2) *reinterpret_cast<uint32_t*>(a.out + (bi * n_heads + hq) * D + lane * P + e) = 0u;
    }
  }
}

}  // namespace

cudaError_t launch_qcache_write(const RopeArgs& r, const QWriteArgs& a, cudaStream_t st) {
  const int blocks = (a.n + a.c.block - 2) / a.c.block + 1;   // that n tokens may touch
  const size_t smem = static_cast<size_t>(a.c.block) * a.c.dim * 4;
  cudaError_t e = cudaFuncSetAttribute(qcache_write_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       64 * 256 * 4);
  if (e != cudaSuccess) return e;
  return launch_k(qcache_write_kernel, dim3(blocks, a.c.n_kv_heads, 2 * a.B), dim3(kWriteThreads), smem, st,
                  r, a);
}

cudaError_t launch_qcache_queries(const RopeArgs& r, const QAttnArgs& a, cudaStream_t st) {
  // few rows: a warp for every head; many: the angles of a row formed once
  const int n_heads = a.c.n_kv_heads * a.G, rows = a.B * a.n;
  const dim3 grid(rows, rows >= 148 ? 1 : (n_heads + 3) / 4);
  return a.c.dim == 256 ? launch_k(qcache_query_kernel<256>, grid, dim3(128), 0, st, r, a)
                        : launch_k(qcache_query_kernel<128>, grid, dim3(128), 0, st, r, a);
}

int qcache_splits(int max_pages, int n, int window, int split) {
  const int64_t all = (static_cast<int64_t>(max_pages) * kPg + split - 1) / split;
  if (window == 0) return static_cast<int>(all);
  // keys of the rows span at most window + n - 1 positions
  const int64_t some = (static_cast<int64_t>(window) + n - 2) / split + 2;
  return static_cast<int>(some < all ? some : all);
}

}  // namespace sv
