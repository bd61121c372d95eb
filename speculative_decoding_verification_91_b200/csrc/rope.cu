// Rotary positions on strided rows of heads (spec_rope): half or interleaved
// pairs over part of the head, any frequencies, forwards or back.
#include <math.h>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kRopeOpThreads = 256;

template <typename T>
__device__ __forceinline__ float rope_load(const T* p);
template <>
__device__ __forceinline__ float rope_load<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }
template <>
__device__ __forceinline__ float rope_load<__half>(const __half* p) { return __half2float(*p); }
template <>
__device__ __forceinline__ float rope_load<float>(const float* p) { return *p; }
template <typename T>
__device__ __forceinline__ void rope_store(T* p, float v);
template <>
__device__ __forceinline__ void rope_store<uint16_t>(uint16_t* p, float v) { *p = f32_to_bf16(v); }
template <>
__device__ __forceinline__ void rope_store<__half>(__half* p, float v) { *p = __float2half_rn(v); }
template <>
__device__ __forceinline__ void rope_store<float>(float* p, float v) { *p = v; }

// One CTA per row: the row's cosines and sines once, then a thread per pair of
// any head, then the dims that pass through (nothing to do in place).
template <typename T>
__global__ void __launch_bounds__(kRopeOpThreads) rope_kernel(const __grid_constant__ RopeArgs r,
                                                              const __grid_constant__ RopeOpArgs a) {
  __shared__ float2 cs[kMaxPairs];
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int pos = a.positions[row];
  if (pos < 0) return;
  for (int j = threadIdx.x; j < r.n_rot; j += kRopeOpThreads) {
    double c, s;
    rope_turn(pos, r.turns[j], c, s);
    cs[j] = make_float2(static_cast<float>(c * r.magnitude),
                        static_cast<float>(s * (a.inverse ? -r.magnitude : r.magnitude)));
  }
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + row * a.x_row;
  T* out = static_cast<T*>(a.out) + row * a.out_row;
  for (int i = threadIdx.x; i < a.n_heads * r.n_rot; i += kRopeOpThreads) {
    const int h = i / r.n_rot, j = i % r.n_rot;
    const int d0 = r.layout == SPEC_ROPE_HALF ? j : 2 * j;
    const int d1 = r.layout == SPEC_ROPE_HALF ? j + r.span / 2 : 2 * j + 1;
    const float x0 = rope_load(x + h * a.x_head + d0), x1 = rope_load(x + h * a.x_head + d1);
    rope_store(out + h * a.out_head + d0, x0 * cs[j].x - x1 * cs[j].y);
    rope_store(out + h * a.out_head + d1, x0 * cs[j].y + x1 * cs[j].x);
  }
  if (a.x == a.out) return;
  for (int i = threadIdx.x; i < a.n_heads * a.dim; i += kRopeOpThreads) {
    const int h = i / a.dim, d = i % a.dim;
    const bool turned = r.layout == SPEC_ROPE_HALF
                            ? d < r.n_rot || (d >= r.span / 2 && d < r.span / 2 + r.n_rot)
                            : d < 2 * r.n_rot;
    if (!turned) out[h * a.out_head + d] = x[h * a.x_head + d];
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& r, const RopeOpArgs& a, int dtype, cudaStream_t st) {
  const dim3 grid(a.n_rows), block(kRopeOpThreads);
  if (dtype == SPEC_BF16) return launch_k(rope_kernel<uint16_t>, grid, block, 0, st, r, a);
  if (dtype == SPEC_FP16) return launch_k(rope_kernel<__half>, grid, block, 0, st, r, a);
  return launch_k(rope_kernel<float>, grid, block, 0, st, r, a);
}

}  // namespace sv
