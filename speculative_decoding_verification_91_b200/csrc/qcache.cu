// The 8-bit paged cache: the append that quantises (spec_qcache_write) and the
// queries' form for the attention over it (qattn.cu).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kPg = SPEC_PAGE_SIZE;
constexpr int kWriteThreads = 256;
constexpr int kWriteWarps = kWriteThreads / 32;
constexpr int kWriteList = 1024;        // entries formed again in binary64 at the end of a CTA

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.4028234e38f; }

// A binary64 value as the binary32 one next to it towards zero, its last bit
// set when that was not exact (rounding to odd): rounding the result once more
// to few bits then gives what rounding the binary64 value at once gives.
__device__ __forceinline__ float to_odd(double y) {
  const float f = __double2float_rz(y);
  return static_cast<double>(f) == y ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Element d of a head of the row at p, turned by r at pos.
// (Out of line: needed for a few entries in 10^4.)
__device__ __noinline__ double turned(const RopeArgs& r, const uint16_t* p, int d, int pos) {
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
  if (j < 0) return x;
  const double w = bf16_to_f32(p[e]);
  double c, s;
  rope_turn(pos, r.step[j], c, s);
  c *= r.magnitude;
  s *= r.magnitude;
  return second ? w * s + x * c : x * c - w * s;
}

// The append.  A CTA takes one touched block of BT tokens of a sequence, keys (the
// first half of z) or values, for `heads` KV heads one after the other: its 8 warps
// hold the block's new rows in registers (a lane 8 dims, IT rows of each warp), find
// the largest magnitude, settle the scale and store the codes, the next head's rows
// on their way meanwhile; every row is read once.  The angles of the block's rows are
// formed once, in shared memory.  64 x 256 tokens of 8 heads (201 MB): 68.8 us, 2.9
// TB/s, bound by instruction issue with 16 warps an SM, which the rows in registers
// allow: the second set of codes costs 10 us of it, the angles 8.  One body for keys
// and values 74.8, one for both layouts of keys 70.6; 512 threads a CTA, or three CTAs
// an SM, spill (103 and 119 us).
//
// Codes are those of the exactly turned key.  Keys turn in binary32, off by less
// than kTurnErr (|x0| + |x1|) magnitude: cosine and sine 1.5 steps, the magnitude's own
// rounding to binary32 and that of its product with them, the product with the entry,
// the sum: 5.5 x 2^-24.  Where rounding that much
// lower and higher (by a lane's largest own and partner's magnitude) gives two codes
// (4 in 10^4) the entry is formed again in binary64, all of a CTA's together at its
// end.  Blocks with infinities or NaN, those that keep a scale that is no power of two
// and half pairs whose distance is no multiple of 8 take binary64 throughout.  (All
// of it in binary64, with each head its own angles, took 545 us for 64 x 256 tokens
// of 8 heads; entries formed again where they were found, 160-230; a warp a head that
// reads its rows twice, 135.)
constexpr float kTurnErr = 5.6f / 16777216.f;

__device__ __forceinline__ __nv_bfloat162 abs2(uint32_t w) {
  w &= 0x7fff7fffu;
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
// max that hands a NaN on
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

struct WriteShared {
  uint32_t red[2][kWriteWarps];
  int list_n;
  int2 list[kWriteList];                     // (head of the CTA, row, dim), the scale's inverse
};

// A CTA's block: of values (-1), or of keys whose pairs are laid out as LAYOUT (bodies
// of their own: values need neither angles nor a second set of codes).
template <int D, int BT, int LAYOUT>
__device__ __forceinline__ void write_block(const RopeArgs& r, const QWriteArgs& a, int heads, int n_tab, int b,
                                            float2* cs, WriteShared& s) {
  constexpr bool is_v = LAYOUT < 0, half = LAYOUT == SPEC_ROPE_HALF;
  constexpr int LR = D / 8;                  // lanes of a row
  constexpr int RI = 32 / LR;                // rows of a warp at a time
  constexpr int IT = BT / (kWriteWarps * RI) > 0 ? BT / (kWriteWarps * RI) : 1;
  const QCacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = c.seq_lens[b];
  if (L < 0 || static_cast<int64_t>(L) + a.n > static_cast<int64_t>(c.max_pages) * kPg) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) flag_status(c.status, SPEC_DEV_BAD_LENGTH);
    return;
  }
  const int p0 = (L / BT + static_cast<int>(blockIdx.x)) * BT;   // first position of the block
  if (p0 >= L + a.n) return;
  const int page = c.block_table[static_cast<int64_t>(b) * c.max_pages + p0 / kPg];
  const int lo = max(p0, L) - p0, hi = min(BT, L + a.n - p0);    // new rows of the block
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, c.n_kv_heads);
  const int64_t stride = is_v ? a.v_row : a.k_row;
  const int d0 = (lane % LR) * 8, t0 = warp * IT * RI + lane / LR;   // dims; rows t0, t0 + RI, ..
  const uint16_t* block0 = (is_v ? a.v_new : a.k_new) + (static_cast<int64_t>(b) * a.n + (p0 - L)) * stride;   // row 0
  uint32_t there = 0;                        // bit i: row t0 + i RI is new
#pragma unroll
  for (int i = 0; i < IT; ++i) there |= (t0 + i * RI >= lo && t0 + i * RI < hi) ? 1u << i : 0u;
  uint4 raw[IT];
  auto load = [&](int h) {
    const uint16_t* p = block0 + t0 * stride + h * D + d0;
#pragma unroll
    for (int i = 0; i < IT; ++i)
      raw[i] = there >> i & 1 ? __ldg(reinterpret_cast<const uint4*>(p + i * RI * stride)) : make_uint4(0, 0, 0, 0);
  };
  load(h0);
  if (page < 0 || page >= c.num_pages) {     // (looked up beside the first rows)
    if (threadIdx.x == 0) flag_status(c.status, SPEC_DEV_BAD_PAGE);
    return;
  }
  if (threadIdx.x == 0) s.list_n = 0;
  const bool turns_keys = !is_v && r.n_rot > 0;
  const int hs = r.span / 2;
  float2* none = cs + BT * n_tab;
  const int lanes = half ? n_tab / 8 : n_tab / 4;   // that share a row's turned pairs
  if (turns_keys) {
    const int j = threadIdx.x % n_tab, step = kWriteThreads / n_tab;   // a thread's pair stays, its row advances
    const uint64_t turn = j < r.n_rot ? r.step[j] : 0;
    const int at = half ? ((j % 8 / 2) * lanes + j / 8) * 2 + j % 2 : ((j % 4 / 2) * lanes + j / 4) * 2 + j % 2;
    if (threadIdx.x < 8) none[threadIdx.x] = make_float2(1.f, 0.f);
    for (int t = lo + threadIdx.x / n_tab; t < hi && threadIdx.x < step * n_tab; t += step) {
      float ca = 1.f, sa = 0.f;
      if (j < r.n_rot) rope_turn(p0 + t, turn, static_cast<float>(r.magnitude), ca, sa);
      cs[t * n_tab + at] = make_float2(ca, sa);
    }
  }
  // this lane's dims: pairs from j0 on (-1: they pass through); for half pairs the
  // partners lie `from` lanes away
  int j0 = -1, from = lane;
  uint32_t flip = 0x80008000u;               // signs of the partners' products
  if (turns_keys) {
    if (!half) {
      if (d0 / 2 < r.n_rot) j0 = d0 / 2;
    } else if (hs % 8 == 0 && d0 < r.span) {
      const bool second = d0 >= hs;
      const int j = second ? d0 - hs : d0;
      if (j < r.n_rot) {
        j0 = j;
        from = lane + (second ? -hs / 8 : hs / 8);
        if (second) flip = 0;
      }
    }
  }
  const bool plain = !(turns_keys && half && hs % 8 != 0);
  __syncthreads();
  auto block_max = [&](float x, int buf) {   // as bits (NaN above all)
    uint32_t m = __float_as_uint(x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) s.red[buf][warp] = m;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kWriteWarps; ++v) m = max(m, s.red[buf][v]);
    return m;
  };

  for (int h = h0; h < h1; ++h) {
    float y[IT][8], amax = 0.f, err = 0.f;
    __nv_bfloat162 top = abs2(0u), with = top;   // largest own and partner's magnitudes
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[i][2 * e] = __uint_as_float(w[e] << 16);
        y[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
      if (turns_keys) {
        // (dims that pass through turn by (1, 0), half pairs with themselves)
        const float4* ct = reinterpret_cast<const float4*>(j0 >= 0 && (there >> i & 1) ? cs + (t0 + i * RI) * n_tab + (half ? j0 / 8 : j0 / 4) * 2 : none);
        const int ce = j0 >= 0 && (there >> i & 1) ? lanes : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __hmax2(top, abs2(w[e]));
        if (half) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t o = __shfl_sync(0xffffffffu, w[e], from) ^ flip;
            const float4 q = ct[e * ce];
            with = __hmax2(with, abs2(o));
            y[i][2 * e] = fmaf(__uint_as_float(o << 16), q.y, y[i][2 * e] * q.x);
            y[i][2 * e + 1] = fmaf(__uint_as_float(o & 0xffff0000u), q.w, y[i][2 * e + 1] * q.z);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 q = ct[e * ce];
            const float x0 = y[i][4 * e], x1 = y[i][4 * e + 1], x2 = y[i][4 * e + 2], x3 = y[i][4 * e + 3];
            y[i][4 * e] = x0 * q.x - x1 * q.y;
            y[i][4 * e + 1] = x0 * q.y + x1 * q.x;
            y[i][4 * e + 2] = x2 * q.z - x3 * q.w;
            y[i][4 * e + 3] = x2 * q.w + x3 * q.z;
          }
        }
      }
      float m[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = max_nan(fabsf(y[i][2 * e]), fabsf(y[i][2 * e + 1]));
      amax = max_nan(amax, max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3])));
    }
    if (h + 1 < h1) load(h + 1);
    if (j0 >= 0) {
      if (!half) with = top;
      err = kTurnErr * static_cast<float>(r.magnitude) *
            (fmaxf(__low2float(top), __high2float(top)) + fmaxf(__low2float(with), __high2float(with)));
    }
    uint32_t m = block_max(plain ? amax : INFINITY, h & 1);
    const uint16_t* head0 = block0 + h * D;
    // the entries one by one, in binary64
    auto entries = [&](auto&& f) {
#pragma unroll 1
      for (int i = 0; i < IT; ++i) {
        if (!(there >> i & 1)) continue;
        const int t = t0 + i * RI;
#pragma unroll 1
        for (int e = 0; e < 8; ++e)
          f(t, e, is_v ? static_cast<double>(bf16_to_f32(head0[t * stride + d0 + e])) : turned(r, head0 + t * stride, d0 + e, p0 + t));
      }
    };
    const bool exact = m >= 0x7f800000u;     // (uniform in the CTA)
    // the scale turns at 1.75 x 2^x: a turned magnitude is within 2 kTurnErr of the
    // largest, 10 steps of binary32, of itself.  Next to that the largest is found in
    // binary64, among the entries that may be above (every block with one in a hundred
    // amaxes of bf16 comes here; all entries in binary64 took 40 us)
    if (turns_keys && !exact && abs(static_cast<int>(m & 0x7fffffu) - 0x600000) <= 16) {
      const uint32_t least = ((m & 0x7f800000u) | 0x600000u) - 16;
      uint64_t may = 0;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((__float_as_uint(y[i][e]) & 0x7fffffffu) >= least) may |= 1ull << (8 * i + e);
      float top = 0.f;
      for (; may; may &= may - 1) {
        const int k = __ffsll(static_cast<long long>(may)) - 1, t = t0 + k / 8 * RI;
        top = fmaxf(top, fabsf(to_odd(turned(r, head0 + t * stride, d0 + k % 8, p0 + t))));
      }
      __syncthreads();
      m = block_max(top, h & 1);
    }
    if (exact) {
      bool bad = false;
      amax = 0.f;
      entries([&](int, int, double y) {
        const float v = to_odd(y);
        if (finite_f(v)) amax = fmaxf(amax, fabsf(v));
        else bad = true;
      });
      if (bad) flag_status(c.status, SPEC_DEV_NONFINITE);
      __syncthreads();
      m = block_max(amax, h & 1);
    }
    amax = __uint_as_float(m);
    const int64_t head = static_cast<int64_t>(page) * c.n_kv_heads + h;
    float* sc = (is_v ? c.vs : c.ks) + head * (kPg / BT) + (p0 % kPg) / BT;
    uint8_t* dst = (is_v ? c.v : c.k) + (head * kPg + p0 % kPg) * D;
    const int e2 = scale_exponent(amax);
    float now = pow2f(e2), inv = pow2f(-e2);
    bool divide = false;                       // a scale that is no power of two: nothing of it is exact in binary32
    if (lo > 0) {                              // committed tokens share the block
      const float was = *sc;
      const bool odd = __float_as_uint(was) & 0x7fffffu;
      now = fmaxf(now, was);
      divide = odd && now == was;
      if (now == was && !odd) inv = __fdiv_rn(1.f, was);
      if (now > was) {                         // rewrite their codes for the larger scale
        const float ratio = __fdiv_rn(was, now);
        auto scaled = [&](float v) {           // (a code times the ratio: 28 bits where the ratio has 24)
          return v != v ? 0.f : odd ? to_odd(static_cast<double>(v) * ratio) : v * ratio;
        };
        for (int i = threadIdx.x; i < lo * D / 2; i += kWriteThreads) {
          uint16_t* q = reinterpret_cast<uint16_t*>(dst) + i;
          const float2 v = e4m3_values(*q);
          *q = e4m3x2(scaled(v.x), scaled(v.y));
        }
      }
    }
    if (exact || divide) {
      entries([&](int t, int e, double y) {
        const float v = to_odd(divide ? y / now : y * inv);
        dst[t * D + d0 + e] = static_cast<uint8_t>(e4m3x2(v == v ? v : 0.f, 0.f));
      });
    } else {
      err *= inv;                              // (0 where nothing turns, and for rows of zeros)
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        auto codes = [&](float add) {
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = e4m3x2(fmaf(y[i][2 * e], inv, add), fmaf(y[i][2 * e + 1], inv, add));
          return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        };
        const uint2 code = codes(-err);
        if (!(there >> i & 1)) continue;
        *reinterpret_cast<uint2*>(dst + (t0 + i * RI) * D + d0) = code;
        if (is_v) continue;
        const uint2 up = codes(err);
        uint32_t dx = code.x ^ up.x, dy = code.y ^ up.y;
        while (dx | dy) {
          const int e = (__ffs(dx ? dx : dy) - 1) >> 3, at = atomicAdd(&s.list_n, 1);
          if (at < kWriteList)
            s.list[at] = make_int2((h - h0) << 16 | (t0 + i * RI) << 8 | (d0 + e + (dx ? 0 : 4)), __float_as_int(inv));
          if (dx) dx &= ~(0xffu << (8 * e));
          else dy &= ~(0xffu << (8 * e));
        }
      }
    }
    __syncthreads();                           // everyone has read the old scale
    if (threadIdx.x == 0) *sc = now;
  }
  // ---- the entries next to a rounding border, over what was stored above (every one
  // of the CTA's, should they be more than the list holds)
  __syncthreads();
  const bool all = s.list_n > kWriteList;
  const int n = all ? (h1 - h0) * (hi - lo) * D : s.list_n;
  for (int i = threadIdx.x; i < n; i += kWriteThreads) {
    const int h = h0 + (all ? i / D / (hi - lo) : static_cast<uint32_t>(s.list[i].x) >> 16);
    const int t = all ? lo + i / D % (hi - lo) : s.list[i].x >> 8 & 0xff, d = all ? i % D : s.list[i].x & 0xff;
    const int64_t head = static_cast<int64_t>(page) * c.n_kv_heads + h;
    const double y = turned(r, block0 + t * stride + h * D, d, p0 + t);
    const float v = to_odd(all ? y / c.ks[head * (kPg / BT) + (p0 % kPg) / BT] : y * __int_as_float(s.list[i].y));
    c.k[(head * kPg + p0 % kPg + t) * D + d] = static_cast<uint8_t>(e4m3x2(v == v ? v : 0.f, 0.f));
  }
}

template <int D, int BT>
__global__ void __launch_bounds__(kWriteThreads, 2) qcache_write_kernel(const __grid_constant__ RopeArgs r,
                                                                        const __grid_constant__ QWriteArgs a, int heads,
                                                                        int n_tab) {
  // [BT][n_tab], (1, 0) past the turned pairs: two pairs next to each other, then those
  // of the next lane (in pair order the lanes' reads met in the same banks); 8 (1, 0)
  extern __shared__ __align__(16) float2 cs[];
  __shared__ WriteShared s;
  pdl_trigger();
  pdl_wait();
  const int B = gridDim.z / 2, z = blockIdx.z;     // keys first: their CTAs take longer
  if (z >= B)
    write_block<D, BT, -1>(r, a, heads, n_tab, z - B, cs, s);
  else if (r.layout == SPEC_ROPE_HALF)
    write_block<D, BT, SPEC_ROPE_HALF>(r, a, heads, n_tab, z, cs, s);
  else
    write_block<D, BT, SPEC_ROPE_INTERLEAVED>(r, a, heads, n_tab, z, cs, s);
}

// Queries: one warp per head of a row.  q = q_scale * (code0 + code1): the
// first code keeps 4 significant bits, the second 4 of what is left, so the two
// hold a query to 2^-9 of itself (and 2^-19 of the row's largest), finer than
// bf16's 2^-9 on average, and both factors of the score product are e4m3.  A
// row with an infinity, a NaN or a magnitude beyond the largest scale's codes gets a
// NaN scale, which makes its result NaN.
// A CTA takes a row of a sequence and every blockIdx.y-th four of its heads, a warp a head (4 or
// 8 dims a lane, one load): the row's angles once for all of them (each warp forming its own
// took 41 us for 512 rows of 32 heads, 12.5 now), the first head asked for before.  Few rows: 4.5
// us, most of it under the split kernel's start.
template <int D>
__global__ void __launch_bounds__(128) qcache_query_kernel(const __grid_constant__ RopeArgs r,
                                                           const __grid_constant__ QAttnArgs a) {
  constexpr int P = D / 32;
  __shared__ float2 cs[kMaxPairs];
  pdl_wait();
  pdl_trigger();   // after the wait: what ran before is done when the split kernel starts
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
  // the lane's own dims, and their partners: next to them, whole lanes away, or (half
  // pairs of an odd distance) anywhere
  const bool half_pairs = r.layout == SPEC_ROPE_HALF, far = half_pairs && half % P != 0;
  const int from = !half_pairs || far || lane * P >= r.span ? lane : lane * P < half ? lane + half / P : lane - half / P;
  uint32_t raw[P / 2];
  uint16_t other[P];
  auto load = [&](int hq) {
    const uint16_t* p = a.q + bi * a.q_row + static_cast<int64_t>(hq) * D;
    if (P == 8) {
      const uint4 z = *reinterpret_cast<const uint4*>(p + lane * P);
      raw[0] = z.x;
      raw[1] = z.y;
      raw[P / 2 - 2] = z.z;
      raw[P / 2 - 1] = z.w;
    } else {
      const uint2 z = *reinterpret_cast<const uint2*>(p + lane * P);
      raw[0] = z.x;
      raw[1] = z.y;
    }
    if (far) {
#pragma unroll
      for (int e = 0; e < P; ++e) other[e] = p[partner[e]];
    }
  };
  int hq = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (hq < n_heads) load(hq);
  if (threadIdx.x < r.n_rot) {
    const int pos = min(max(L, 0), 1 << 30) + a.q_offset + i;
    float c, s;
    rope_turn(pos, r.step[threadIdx.x], static_cast<float>(r.magnitude), c, s);
    cs[threadIdx.x] = make_float2(c, s);
  }
  __syncthreads();
  for (; hq < n_heads; hq += gridDim.y * 4) {
    if (hq >= static_cast<int>(gridDim.y) * 4) load(hq);
    float own[P], with[P], amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < P; e += 2) {
      const uint32_t o = __shfl_sync(0xffffffffu, raw[e / 2], from);
      own[e] = __uint_as_float(raw[e / 2] << 16);
      own[e + 1] = __uint_as_float(raw[e / 2] & 0xffff0000u);
      with[e] = far ? bf16_to_f32(other[e]) : half_pairs ? __uint_as_float(o << 16) : own[e + 1];
      with[e + 1] = far ? bf16_to_f32(other[e + 1]) : half_pairs ? __uint_as_float(o & 0xffff0000u) : own[e];
    }
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
    bad = __any_sync(0xffffffffu, bad) || amax > 448.f * 0x1p100f;   // (codes would saturate)
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
    uint8_t* dst = a.q_codes + row * D + lane * P;
    if (P == 8) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(c0[0], c0[P / 4 - 1]);
      *reinterpret_cast<uint2*>(dst + plane) = make_uint2(c1[0], c1[P / 4 - 1]);
    } else {
      *reinterpret_cast<uint32_t*>(dst) = c0[0];
      *reinterpret_cast<uint32_t*>(dst + plane) = c1[0];
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

template <int D, int BT>
cudaError_t launch_write(const RopeArgs& r, const QWriteArgs& a, cudaStream_t st) {
  const int blocks = (a.n + BT - 2) / BT + 1;                    // that n tokens may touch
  // one head a CTA until the GPU is full, then as many as share its angles
  const int64_t per_head = 2ll * blocks * a.B;
  const int heads = static_cast<int>(std::min<int64_t>(a.c.n_kv_heads, std::max<int64_t>(1, per_head * a.c.n_kv_heads / (8 * 148))));
  const int n_tab = (r.n_rot + 7) / 8 * 8;
  const size_t smem = (static_cast<size_t>(BT) * n_tab + 8) * sizeof(float2);
  auto kern = qcache_write_kernel<D, BT>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, (BT * kMaxPairs + 8) * static_cast<int>(sizeof(float2)), allowed);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(blocks, (a.c.n_kv_heads + heads - 1) / heads, 2 * a.B), dim3(kWriteThreads), smem, st,
                  r, a, heads, n_tab);
}

template <int D>
cudaError_t launch_write_dim(const RopeArgs& r, const QWriteArgs& a, cudaStream_t st) {
  return a.c.block == 64   ? launch_write<D, 64>(r, a, st)
         : a.c.block == 32 ? launch_write<D, 32>(r, a, st)
                           : launch_write<D, 16>(r, a, st);
}

cudaError_t launch_qcache_write(const RopeArgs& r, const QWriteArgs& a, cudaStream_t st) {
  return a.c.dim == 256 ? launch_write_dim<256>(r, a, st) : launch_write_dim<128>(r, a, st);
}

cudaError_t launch_qcache_queries(const RopeArgs& r, const QAttnArgs& a, cudaStream_t st) {
  // few rows: a warp for every head; many: up to eight CTAs an SM, so that the angles of
  // a row are formed once or twice (512 rows of 32 heads, the whole prompt chunk: 189 us
  // with one CTA a row, 182 with two, 187 with eight)
  const int n_heads = a.c.n_kv_heads * a.G, rows = a.B * a.n;
  const dim3 grid(rows, std::min((n_heads + 3) / 4, std::max(1, 8 * 148 / rows)));
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
