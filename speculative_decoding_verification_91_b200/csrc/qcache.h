// Rotary positions and the 8-bit paged cache: arguments of the kernels and
// their launchers, shared by the C ABI (api_qcache.cu) and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace sv {

constexpr int kMaxPairs = SPEC_ROPE_MAX_DIM / 2;

// Raises a kernel's limit of dynamic shared memory, once per device (the driver
// call costs a microsecond or more of every launch otherwise).
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (f == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return f;
}

// i / d for i * d < 2^32: mul = floor(2^32 / d) + 1
struct Div {
  uint32_t d, mul;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return d == 1 ? i : __umulhi(i, mul); }
};
inline Div make_div(int d) { return Div{static_cast<uint32_t>(d), static_cast<uint32_t>((1ull << 32) / d) + 1}; }

// A rotary configuration as the kernels take it: step[j] is f_j / (2 pi) turns
// modulo 1, in units of 2^-64, so a position's fraction of a turn is a 64-bit product
// that wraps.
struct RopeArgs {
  int layout, span, n_rot;
  double magnitude;
  uint64_t step[kMaxPairs];
};

// (c, s) of pair j at a position, in binary64.
__device__ __forceinline__ void rope_turn(int pos, uint64_t step, double& c, double& s) {
  const int64_t f = static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(pos)) * step);   // -1/2 .. 1/2 turn
  sincospi(static_cast<double>(f) * 0x1p-63, &s, &c);
}

// magnitude * (cos, sin) in binary32: the fraction of a turn as a binary32 head of
// 23 bits and a tail that enters to first order, so the results are off by little
// more than half a step.  No binary64 and no conversions: those are at a fraction
// of the other instructions' rate, and formed half of spec_rope's time.
__device__ __forceinline__ void rope_turn(int pos, uint64_t step, float magnitude, float& c, float& s) {
  const uint64_t f = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * step + (1ull << 63);
  const uint32_t top = static_cast<uint32_t>(f >> 32), low = static_cast<uint32_t>(f >> 18);
  const float head = __uint_as_float(0x3f800000u | top >> 9) - 1.5f;                        // steps of 2^-23
  const float tail = (__uint_as_float(0x3f800000u | (low & 0x7fffffu)) - 1.f) * 0x1.921fb6p-21f;   // 2 pi 2^-23 of them
  float sh, ch;
  sincospif(2.f * head, &sh, &ch);
  c = (ch - sh * tail) * magnitude;
  s = (sh + ch * tail) * magnitude;
}

// ---------------------------------------------------------------- spec_rope
struct RopeOpArgs {
  const void* x;
  void* out;
  int64_t x_row, x_head, out_row, out_head;   // strides in elements
  const int32_t* positions;
  int n_rows, n_heads, dim, inverse;
};
cudaError_t launch_rope(const RopeArgs& r, const RopeOpArgs& a, int dtype, cudaStream_t st);

// ------------------------------------------------------------- 8-bit cache
struct QCacheArgs {
  int dim, n_kv_heads, num_pages, max_pages, block;   // block: tokens per scale
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* block_table;
  const int32_t* seq_lens;
  unsigned* status;
};

struct QWriteArgs {
  QCacheArgs c;
  int B, n;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t k_row, v_row;
};
cudaError_t launch_qcache_write(const RopeArgs& r, const QWriteArgs& a, cudaStream_t st);

// Queries of the attention: row r = i * G + g of (sequence, KV head) is query
// head h * G + g at position L + q_offset + i.
struct QAttnArgs {
  QCacheArgs c;
  int B, n, G, rows;            // rows = n * G per (sequence, KV head)
  int q_offset, kv_extra, window, split, n_splits;
  Div by_split, by_cost, by_G;  // of key blocks by those of a split, and by one more; of rows by G
  const uint16_t* q;
  int64_t q_row;
  float scale_log2;             // softmax scale * log2(e)
  uint8_t* q_codes;             // [2][B * Hkv * rows][dim]: q = (code0 + code1) * q_scale
  float* q_scale;               // [B * Hkv * rows]
  float* part_o;                // [B * Hkv][n_splits][rows][dim]
  float2* part_ml;              // [B * Hkv][n_splits][rows] (reference, sum of exponentials)
  uint16_t* out;
};
// Query rows of an item.  128 (prompt chunks) hold the weights in other codes, so calls
// whose rows' bits must not depend on n take 32 or 64.
inline int qattn_rows(int n, int64_t rows) { return rows <= 32 ? 32 : rows <= 64 || n <= SPEC_MAX_K + 1 ? 64 : 128; }
// Keys any row of a sequence may see, as whole blocks; none: blocks = 0.
constexpr int kQBlk = 128;   // keys of one MMA block
struct SeqKeys {
  int lo, hi, splits, blocks;
  // in halves of a key block's time; an item's start and end take about a block's
  __device__ int cost() const { return 2 * (blocks + splits); }
};
__device__ __forceinline__ SeqKeys seq_keys(const QAttnArgs& a, int L) {
  SeqKeys k{0, -1, 0, 0};
  if (L < 0 || static_cast<int64_t>(L) + a.kv_extra > static_cast<int64_t>(a.c.max_pages) * SPEC_PAGE_SIZE) return k;
  k.hi = min(L + a.kv_extra - 1, L + a.q_offset + a.n - 1);
  k.lo = a.window > 0 ? max(0, L + a.q_offset - a.window + 1) : 0;
  if (k.hi < k.lo) return k;
  k.splits = a.by_split(k.hi / kQBlk) - a.by_split(k.lo / kQBlk) + 1;
  k.blocks = k.hi / kQBlk - k.lo / kQBlk + 1;
  return k;
}

cudaError_t launch_qcache_queries(const RopeArgs& r, const QAttnArgs& a, cudaStream_t st);
cudaError_t launch_qcache_attn(const QAttnArgs& a, cudaStream_t st);

// Absolute splits that rows of a sequence can touch.
int qcache_splits(int max_pages, int n, int window, int split);

// ---------------------------------------------------------------- e4m3
// Two binary32 values to e4m3 codes (nearest, ties to even; beyond 448: 448;
// NaN: the NaN code); lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
  return d;
}
// Two codes to their values (exact).
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(codes)));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h2));
  return f;
}
// Least e in [-100, 100] with amax <= 448 * 2^e (448 = 1.75 * 2^8): amax =
// 1.m * 2^x needs e = x - 8, one more when 1.m > 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -100), 100);
}
__device__ __forceinline__ float pow2f(int e) {   // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace sv
