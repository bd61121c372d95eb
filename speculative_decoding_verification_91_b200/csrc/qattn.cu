// Split-KV attention over the 8-bit paged cache on the 5th-generation tensor
// cores (sm_100a), persistent, e4m3 in both products.
//
//   s_ij = q_scale_i k_scale_j scale (q_i . k_j)      p_ij = 2^(s_ij log2 e - m_i)
//   out_i = sum_j p_ij v_scale_j v_j / sum_j p_ij
//
// The cache is e4m3, so the products run in kind::f8f6f4 on the pages as TMA
// brought them, with no conversion of K or V.  The bf16 side of each product is
// held in two e4m3 codes whose sum keeps 8 bits: queries q = c0 + c1 (from the
// query kernel; in TMEM; two MMA passes into one accumulator) and weights p = w0 +
// w1 / 16 (w1 the rounding error of w0, stacked under w0 in the M dimension, so
// one pass gives both sums, in lanes r and 64 + r of the accumulator).
//
// Work item = (sequence, KV head, block of RP query rows, absolute split of
// split_tokens keys); items are ordered and every CTA (one per SM) takes those
// that start in an equal share of all key blocks.  11 warps:
//   warp 0     TMA producer: keys and values of 128-key blocks (two pages) into
//              a ring of kUnits units of 128 x dim bytes.
//   warp 1     allocates TMEM; one thread issues the MMAs: S[128][128 keys] = Q
//              K^T (A = Q from TMEM, B = K, K-major); O[rows][dim] += P V (A = P
//              in shared memory, K-major, B = V as stored, MN-major).  With Q in
//              shared memory too the two operands took all of its bandwidth.
//   warp 2     page ids -> the item's scales in shared memory, an item ahead.
//   warps 3-10 softmax: a thread takes one query row and RP / 2 of the block's
//              keys.  The queries sit 128 / RP times in the 128 lanes of Q, so
//              every TMEM lane quadrant, and with it every scheduler, takes an
//              equal part of the keys (one copy left all of the work to one or
//              two schedulers, at 4300 clocks a block).  A row's
//              reference m moves only when a block exceeds it by 2^kLazy (one
//              barrier vote per block); the v scale is folded into m and p
//              (p v_scale <= 2^kLazy), so blocks of any scale share one
//              accumulator; the sum of p is kept in binary32.
//
// Value rows of keys outside the item's range or on pages that were not loaded
// are zeroed in shared memory before P V, so stale slots (NaN codes among them)
// never reach it.  Key blocks start at absolute multiples of 128 and a row's
// weights depend on its own scores only, so a row's partial depends neither on n
// nor on the batch, its row slot or the CTA.  Every wait is bounded.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"
#include "tc_common.cuh"

namespace sv {

namespace {

constexpr int kBlk = 128;                  // keys per block
constexpr int kLgBlk = 7;
constexpr int kPg = SPEC_PAGE_SIZE;
constexpr int kSoftWarps = 8;
constexpr int kFirstSoft = 3;
constexpr int kThreads = (kFirstSoft + kSoftWarps) * 32;
constexpr uint32_t kSmemMax = 227u * 1024u;
constexpr uint32_t kTail = 8192;
constexpr uint32_t kPBytes = 128 * kBlk;   // w0 rows 0..63, w1 rows 64..127
constexpr int kMaxScales = 256;            // scales of one item: 4096 keys / 16
// p v_scale <= 2^kLazy; in code units times kUnit: at most 362 < 448.  A larger
// kLazy moves the reference less often, a larger kUnit keeps smaller weights
// (w1's least step is 2^-9 / (kUnit kLow) = 2^-18 of the reference).
constexpr float kLazy = 3.5f;
constexpr float kUnit = 32.f;
constexpr float kLow = 16.f;               // w1 is stored times 16
constexpr float kNoKey = -1e30f;           // reference of a row that has seen no key

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D (+)= A . B, e4m3 in, binary32 accumulation (K = 32 per instruction)
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in TMEM (lane = row, four K elements a column)
__device__ __forceinline__ void umma_e4m3_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: D binary32, A and B e4m3, M = 128, N = n,
// A K-major, B K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

template <int D>
struct Cfg {
  static constexpr uint32_t kUnitBytes = kBlk * D;              // one block's keys or values
  static constexpr int kPBufs = D == 128 ? 2 : 1;
  static constexpr int kUnits = D == 128 ? 11 : 6;
  static constexpr uint32_t kOffRing = kPBufs * kPBytes;
  static constexpr uint32_t kOffTail = kOffRing + kUnits * kUnitBytes;
  static constexpr uint32_t kSmem = 1024 + kOffTail + kTail;
  static_assert(kSmem <= kSmemMax, "shared memory");
  // TMEM columns: output, scores, both codes of the queries (4 dims a column)
  static constexpr int kSBufs = D == 128 ? 2 : 1;
  static constexpr uint32_t kColS = D;
  static constexpr uint32_t kColQ = kColS + kSBufs * kBlk;
  static_assert(kColQ + 2 * D / 4 <= 512, "tensor memory");
};

// Keys any row of a sequence may see, as whole blocks; none: blocks = 0.
struct SeqKeys {
  int lo, hi, splits, blocks;
};
__device__ __forceinline__ SeqKeys seq_keys(const QAttnArgs& a, int L) {
  SeqKeys k{0, -1, 0, 0};
  if (L < 0 || static_cast<int64_t>(L) + a.kv_extra > static_cast<int64_t>(a.c.max_pages) * kPg) return k;
  k.hi = min(L + a.kv_extra - 1, L + a.q_offset + a.n - 1);
  k.lo = a.window > 0 ? max(0, L + a.q_offset - a.window + 1) : 0;
  if (k.hi < k.lo) return k;
  k.splits = k.hi / a.split - k.lo / a.split + 1;
  k.blocks = k.hi / kBlk - k.lo / kBlk + 1;
  return k;
}

// Walks the items of one CTA; every role keeps its own.
struct Walker {
  const QAttnArgs* a;
  int RP, RB;              // rows of a block, row blocks
  int b, h, rb, sidx, L;
  int split0, p0, p1;      // the sequence's first split; positions of the row block's first and last row
  SeqKeys k;
  long base, end, pos;     // key blocks before (b, h, rb); where the CTA stops; this item's start
  int lo, hi, blk0, nb;    // this item's keys and blocks (nb = 0: none)
  bool fresh;              // the queries changed since the role last took them
  __device__ bool valid() const { return b < a->B && pos < end; }
  __device__ void load_seq() {
    L = a->c.seq_lens[b];
    k = seq_keys(*a, L);
    split0 = k.lo / a->split;
  }
  __device__ void load_rows() {
    const int r0 = rb * RP, r1 = min(a->rows, r0 + RP) - 1;
    p0 = L + a->q_offset + r0 / a->G;
    p1 = L + a->q_offset + r1 / a->G;
    fresh = true;
  }
  __device__ void derive() {
    const int s0 = (split0 + sidx) * a->split, start = max(s0, k.lo);
    pos = base + ((start >> kLgBlk) - (k.lo >> kLgBlk));
    lo = a->window > 0 ? max(start, p0 - a->window + 1) : start;
    hi = min(min(s0 + a->split - 1, k.hi), p1);
    blk0 = lo >> kLgBlk;
    nb = hi >= lo ? (hi >> kLgBlk) - blk0 + 1 : 0;
  }
  __device__ void next_rows() {   // the next (b, h, rb) that has keys, its first split
    sidx = 0;
    base += k.blocks;
    if (++rb == RB) {
      rb = 0;
      if (++h == a->c.n_kv_heads) {
        h = 0;
        do {
          if (++b >= a->B) return;
          load_seq();
        } while (k.blocks == 0);
      }
    }
    load_rows();
    derive();
  }
  __device__ void next() {
    if (++sidx < k.splits) derive();
    else next_rows();
  }
  __device__ void skip() {   // to the next item with keys
    while (valid() && nb == 0) next();
  }
  __device__ void start(const QAttnArgs* args, int rp, const int* at, long base0, long end0) {
    a = args;
    RP = rp;
    RB = (a->rows + RP - 1) / RP;
    b = at[0];
    end = end0;
    if (b >= a->B) return;
    load_seq();
    h = at[1] / RB;
    rb = at[1] % RB;
    sidx = at[2];
    base = base0 + static_cast<long>(at[1]) * k.blocks;
    load_rows();
    if (sidx < k.splits) derive();
    else next_rows();
  }
};

// Ring units of block g's keys and values: K0 K1 V0 K2 V1 K3 V2 ..
__device__ __forceinline__ int key_unit(int g) { return g == 0 ? 0 : 2 * g - 1; }
__device__ __forceinline__ int value_unit(int g) { return 2 * g + 2; }

__device__ __forceinline__ bool fwait(uint64_t* bar, uint32_t parity, unsigned* status, volatile int* fail) {
  if (*fail) return false;
  if (mbar_wait(bar, parity, status)) return true;
  *fail = 1;
  return false;
}

template <int D, int RP>
__global__ void __launch_bounds__(kThreads, 1) qattn_kernel(const __grid_constant__ CUtensorMap tk,
                                                            const __grid_constant__ CUtensorMap tv,
                                                            const __grid_constant__ QAttnArgs a) {
  using C = Cfg<D>;
  constexpr int NU = C::kUnits, PB = C::kPBufs, SB = C::kSBufs, ATOMS = D / 128;
  constexpr uint32_t kAtom = kBlk * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* pbuf = smem;
  uint8_t* ring = smem + C::kOffRing;
  uint8_t* tail = smem + C::kOffTail;
  uint64_t* u_full = reinterpret_cast<uint64_t*>(tail);   // [NU]
  uint64_t* u_empty = u_full + NU;                         // [NU]
  uint64_t* s_full = u_empty + NU;                         // [SB] by block
  uint64_t* s_free = s_full + 2;                           // [SB]
  uint64_t* q_ready = s_free + 2;
  uint64_t* p_full = q_ready + 1;                          // [2] by block parity
  uint64_t* pv_done = p_full + 2;                          // [2]
  uint64_t* sc_full = pv_done + 2;                         // [2] by item parity
  uint64_t* sc_empty = sc_full + 2;                        // [2]
  uint64_t* o_free = sc_empty + 2;
  uint64_t* mma_done = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* fail = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* at = reinterpret_cast<int*>(tmem_slot + 2);         // first item: b, (head, row block), split
  long* span = reinterpret_cast<long*>(tail + 512);        // key blocks before it, and where to stop
  float* red = reinterpret_cast<float*>(tail + 1024);      // [threads of a row][rows]
  float* ks_s = reinterpret_cast<float*>(tail + 4096);     // [2 items][kMaxScales]
  float* vs_s = ks_s + 2 * kMaxScales;                     // < 0: page not there
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NU; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], kSoftWarps);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&pv_done[i], 1);
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], kSoftWarps);
    }
    mbar_init(q_ready, kSoftWarps);
    mbar_init(o_free, kSoftWarps);
    mbar_init(mma_done, 1);
    *fail = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_trigger();
  pdl_wait();

  const int RB = (a.rows + RP - 1) / RP, per_b = a.c.n_kv_heads * RB;
  if (warp == 2) {
    // ---- this CTA's share [x0, x1) of all key blocks and its first item
    long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long n = 0;
      if (b0 + lane < a.B) {
        const int L = a.c.seq_lens[b0 + lane];
        n = seq_keys(a, L).blocks;
        if (blockIdx.x == 0 &&
            (L < 0 || static_cast<int64_t>(L) + a.kv_extra > static_cast<int64_t>(a.c.max_pages) * kPg))
          flag_status(a.c.status, SPEC_DEV_BAD_LENGTH);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
      total += n * per_b;
    }
    const long x0 = static_cast<long>(blockIdx.x) * total / gridDim.x;
    const long x1 = static_cast<long>(blockIdx.x + 1) * total / gridDim.x;
    long pre = 0;
    int found = a.B;
    long found_pre = 0;
    for (int b0 = 0; b0 < a.B && found == a.B && x1 > x0; b0 += 32) {
      long n = 0;
      if (b0 + lane < a.B) n = static_cast<long>(seq_keys(a, a.c.seq_lens[b0 + lane]).blocks) * per_b;
      long incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const long excl = pre + incl - n;
      const unsigned bal = __ballot_sync(0xffffffffu, n > 0 && x0 >= excl && x0 < excl + n);
      if (bal) {
        const int src = __ffs(bal) - 1;
        found = b0 + src;
        found_pre = __shfl_sync(0xffffffffu, excl, src);
      }
      pre += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      at[0] = found;
      at[1] = at[2] = 0;
      span[0] = found_pre;
      span[1] = x1;
      if (found < a.B) {
        const SeqKeys k = seq_keys(a, a.c.seq_lens[found]);
        const long rem = x0 - found_pre;
        at[1] = static_cast<int>(rem / k.blocks);
        const int r = static_cast<int>(rem % k.blocks), first = k.lo / kBlk, bps = a.split / kBlk;
        // the first split that starts at or after block r of the sequence
        at[2] = r == 0 ? 0 : (r + first + bps - 1) / bps - k.lo / a.split;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walker w;
  w.start(&a, RP, at, span[0], span[1]);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol = RB > 1 ? policy_evict_normal() : policy_evict_first();
      int last[NU];                       // unit last copied into each slot, -1: none
      for (int i = 0; i < NU; ++i) last[i] = -1;
      // block j of item x, keys or values, into ring unit u
      auto load = [&](const Walker& x, int j, int kv, int u) -> bool {
        const int32_t* bt = a.c.block_table + static_cast<int64_t>(x.b) * a.c.max_pages;
        int id[2];
        uint32_t bytes = 0;
        for (int p = 0; p < 2; ++p) {
          const int pg = (x.blk0 + j) * 2 + p;
          id[p] = -1;
          if (pg * kPg <= x.hi && pg * kPg + kPg - 1 >= x.lo) id[p] = bt[pg];
          if (id[p] < 0 || id[p] >= a.c.num_pages) id[p] = -1;
          else bytes += kPg * D;
        }
        const int s = u % NU;
        if (u >= NU && !fwait(&u_empty[s], ((u / NU) - 1) & 1, a.c.status, fail)) return false;
        mbar_arrive_expect_tx(&u_full[s], bytes);
        for (int p = 0; p < 2; ++p) {
          if (id[p] < 0) continue;
          const int y = (id[p] * a.c.n_kv_heads + x.h) * kPg;
#pragma unroll
          for (int t = 0; t < ATOMS; ++t)
            tma_load_2d(ring + s * C::kUnitBytes + t * kAtom + p * (kPg * 128), kv ? &tv : &tk, &u_full[s], t * 128,
                        y, pol);
        }
        last[s] = u;
        return true;
      };
      Walker wk = w;
      wk.skip();
      w.skip();
      int gk = 0, gv = 0, jk = 0, jv = 0;
      bool ok = true;
      // order of the copies: K0 K1 V0 K2 V1 ..: values are needed a softmax
      // later than their keys, and would hold a slot meanwhile
      while (ok && w.valid()) {
        while (ok && wk.valid() && gk < gv + 2) {
          ok = load(wk, jk, 0, key_unit(gk));
          ++gk;
          if (++jk >= wk.nb) {
            jk = 0;
            wk.next();
            wk.skip();
          }
        }
        ok = ok && load(w, jv, 1, value_unit(gv));
        ++gv;
        if (++jv >= w.nb) {
          jv = 0;
          w.next();
          w.skip();
        }
      }
      // every issued copy must land before the CTA may exit
      for (int i = 0; i < NU; ++i)
        if (last[i] >= 0) mbar_wait(&u_full[i], (last[i] / NU) & 1, a.c.status);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t id_qk = idesc_e4m3(kBlk, false), id_pv = idesc_e4m3(D, true);
      Walker wp = w;
      w.skip();
      wp.skip();
      int js = 0, jp = 0, ip = 0;         // block in item (scores, P V); items begun by P V
      int nqk = 0, npv = 0, nq = 0;       // blocks issued; query groups begun
      uint64_t t_last = 0;
      uint32_t polls = 0;
      while (wp.valid()) {
        bool progressed = false;
        if (npv < nqk) {                  // P V first: it frees a unit
          const int u = value_unit(npv);
          bool ready = mbar_test_wait(&p_full[npv & 1], (npv >> 1) & 1) &&
                       mbar_test_wait(&u_full[u % NU], (u / NU) & 1);
          if (jp == 0 && ip > 0) ready = ready && mbar_test_wait(o_free, (ip - 1) & 1);
          if (ready) {
            tc_fence_after();
            const uint32_t v_addr = smem_u32(ring + (u % NU) * C::kUnitBytes);
            const uint32_t p_addr = smem_u32(pbuf + (npv % PB) * kPBytes);
#pragma unroll
            for (int kk = 0; kk < kBlk / 32; ++kk)
              umma_e4m3(tmem, sw128_desc(p_addr + kk * 32), sw128_desc_mn(v_addr + kk * 4096, kAtom), id_pv,
                        (jp > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&pv_done[npv & 1]);
            umma_commit(&u_empty[u % NU]);
            ++npv;
            if (++jp >= wp.nb) {
              jp = 0;
              ++ip;
              wp.next();
              wp.skip();
            }
            progressed = true;
          }
        }
        if (w.valid()) {
          const int u = key_unit(nqk);
          bool ready = mbar_test_wait(&u_full[u % NU], (u / NU) & 1);
          if (nqk >= SB) ready = ready && mbar_test_wait(&s_free[nqk % SB], ((nqk / SB) - 1) & 1);
          if (w.fresh) ready = ready && mbar_test_wait(q_ready, nq & 1);
          if (ready) {
            if (w.fresh) ++nq;
            w.fresh = false;
            tc_fence_after();
            const uint32_t k_addr = smem_u32(ring + (u % NU) * C::kUnitBytes);
            const uint32_t t_s = tmem + C::kColS + (nqk % SB) * kBlk;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                umma_e4m3_ta(t_s, tmem + C::kColQ + c * (D / 4) + kk * 8,
                             sw128_desc(k_addr + (kk >> 2) * kAtom + (kk & 3) * 32), id_qk, (c > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&s_full[nqk % SB]);
            umma_commit(&u_empty[u % NU]);
            ++nqk;
            if (++js >= w.nb) {
              js = 0;
              w.next();
              w.skip();
            }
            progressed = true;
          }
        }
        if (progressed) {
          polls = 0;
        } else if ((++polls & 1023u) == 0) {
          const uint64_t now = globaltimer_ns();
          if (polls == 1024) t_last = now;
          else if (now - t_last > kWaitNs || *fail) {
            flag_status(a.c.status, SPEC_DEV_TIMEOUT);
            *fail = 1;
            break;
          }
        }
      }
      // nothing may be in flight when TMEM is freed
      umma_commit(mma_done);
      mbar_wait(mma_done, 0, a.c.status);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------- scales
    const int per_page = kPg / a.c.block;
    int i = 0;
    for (; w.valid(); w.next()) {
      if (w.nb == 0) continue;
      const int h = w.h;
      if (i >= 2) fwait(&sc_empty[i & 1], ((i >> 1) - 1) & 1, a.c.status, fail);
      const int32_t* bt = a.c.block_table + static_cast<int64_t>(w.b) * a.c.max_pages;
      const int count = w.nb * (kBlk / a.c.block);
      for (int e = lane; e < count; e += 32) {
        const int key = w.blk0 * kBlk + e * a.c.block, pg = key / kPg;
        float ks = 0.f, vs = -1.f;
        if (pg * kPg <= w.hi && pg * kPg + kPg - 1 >= w.lo) {
          const int id = bt[pg];
          if (id >= 0 && id < a.c.num_pages) {
            const int64_t sc = (static_cast<int64_t>(id) * a.c.n_kv_heads + h) * per_page + (key % kPg) / a.c.block;
            ks = a.c.ks[sc];
            vs = a.c.vs[sc];
          } else {
            flag_status(a.c.status, SPEC_DEV_BAD_PAGE);
          }
        }
        ks_s[(i & 1) * kMaxScales + e] = ks;
        vs_s[(i & 1) * kMaxScales + e] = vs;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[i & 1]);
      ++i;
    }
  } else {
    // ------------------------------------------------------------- softmax
    constexpr int KW = RP / 2;                 // keys of a block a thread takes
    constexpr int NG = kBlk / KW;              // threads of a row
    const int quad = warp & 3, cg = (warp - kFirstSoft) >> 2;     // TMEM lane quadrant; first or second half of its keys
    const int rh = RP == 64 ? quad & 1 : 0;                       // row half: rows 32 rh + lane
    const int grp = (RP == 64 ? quad >> 1 : quad) * 2 + cg;       // keys KW grp .. of the block
    const int row = rh * 32 + lane;
    const int st = (warp - kFirstSoft) * 32 + lane;               // 0..255
    const bool sums = RP == 64 || (quad & 1) == 0;                // lanes that hold sums of w0 (quadrants 0, 1) or w1
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int bar_rows = 1 + rh, bar_cg = 3 + rh * 2 + cg;
    constexpr int kRowThreads = RP == 64 ? 128 : 256;
    const int lg_bt = 31 - __clz(a.c.block);
    float* red_r = red + rh * (NG * 32);
    int g = 0, item = 0, p = 0;
    float qs = 0.f;
    // To the next item with keys (the partials of those without go out here);
    // where the queries change, this thread's row of them into TMEM: every
    // product with the old ones is done once the last scores have been read.
    auto take = [&]() {
      for (; w.valid() && w.nb == 0; w.next()) {
        const int r0 = w.rb * RP;
        const long slot = ((static_cast<long>(w.b) * a.c.n_kv_heads + w.h) * a.n_splits + w.sidx) * a.rows + r0;
        if (grp == 0 && row < min(a.rows - r0, RP)) __stcg(&a.part_ml[slot + row], make_float2(kNoKey, 0.f));
      }
      if (!w.valid() || !w.fresh) return;
      w.fresh = false;
      const int r0 = w.rb * RP;
      const bool have = row < min(a.rows - r0, RP);
      const long at = (static_cast<long>(w.b) * a.c.n_kv_heads + w.h) * a.rows + r0 + row;
      p = w.L + a.q_offset + (r0 + row) / a.G;
      qs = have ? a.q_scale[at] : 0.f;
      qs = qs == qs ? qs * a.scale_log2 : 0.f;        // a NaN row's result is set at the end
      const long plane = static_cast<long>(a.B) * a.c.n_kv_heads * a.rows;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q_codes + (at + c * plane) * D + cg * (D / 2));
        uint32_t v[D / 32][4];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 x = have ? __ldcg(src + i) : make_uint4(0, 0, 0, 0);
          v[i][0] = x.x;
          v[i][1] = x.y;
          v[i][2] = x.z;
          v[i][3] = x.w;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          tmem_st8(t_lane + C::kColQ + c * (D / 4) + cg * (D / 8) + i * 8, *reinterpret_cast<uint32_t(*)[8]>(v[2 * i]));
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };
    take();
    while (w.valid()) {
      const int r0 = w.rb * RP, nrows = min(a.rows - r0, RP);
      const long slot = ((static_cast<long>(w.b) * a.c.n_kv_heads + w.h) * a.n_splits + w.sidx) * a.rows + r0;
      const bool half_used = rh * 32 < nrows;         // these warps hold rows
      const bool mine = row < nrows;
      const int row_lo = max(w.lo, a.window > 0 ? p - a.window + 1 : 0), row_hi = min(w.hi, p);
      const float* ks = ks_s + (item & 1) * kMaxScales;
      const float* vs = vs_s + (item & 1) * kMaxScales;
      fwait(&sc_full[item & 1], (item >> 1) & 1, a.c.status, fail);
      float mref = kNoKey, l = 0.f;
      for (int j = 0; j < w.nb; ++j, ++g) {
        const int kb = (w.blk0 + j) << kLgBlk, key0 = kb + grp * KW;
        constexpr int NE = KW / 16;                   // scales of the keys (one or two of 16-token blocks)
        float s[KW], f[NE], vsc[NE];
#pragma unroll
        for (int u = 0; u < NE; ++u) {
          const int e = ((j << kLgBlk) + grp * KW + 16 * u) >> lg_bt;
          vsc[u] = vs[e];
          f[u] = fminf(fmaxf(qs * ks[e], 1e-30f), 3e38f);
        }
        fwait(&s_full[g % SB], (g / SB) & 1, a.c.status, fail);
        __syncwarp();
        tc_fence_after();
        if (half_used) {
          const uint32_t t_s = t_lane + C::kColS + (g % SB) * kBlk + grp * KW;
#pragma unroll
          for (int c = 0; c < KW; c += 8) tmem_ld8_nowait(t_s + c, *reinterpret_cast<uint32_t(*)[8]>(&s[c]));
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[g % SB]);
        if (half_used) {
          bool edge = key0 < row_lo || key0 + KW - 1 > row_hi;
#pragma unroll
          for (int u = 0; u < NE; ++u) edge |= vsc[u] < 0.f;
          if (edge) {
#pragma unroll
            for (int c = 0; c < KW; ++c)
              if (key0 + c < row_lo || key0 + c > row_hi || vsc[c >> 4] < 0.f) s[c] = -INFINITY;
          }
          float cand = -INFINITY;
#pragma unroll
          for (int u = 0; u < NE; ++u) {
            float m4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = fmaxf(fmaxf(s[16 * u + c], s[16 * u + 4 + c]), fmaxf(s[16 * u + 8 + c], s[16 * u + 12 + c]));
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            // log2 of the scale, rounded up to a whole number, within the range the sums can take
            const uint32_t ub = __float_as_uint(vsc[u]);
            int lv = static_cast<int>(ub >> 23) - 127 + ((ub & 0x7fffffu) ? 1 : 0);
            lv = vsc[u] < 0.f ? 0 : max(-100, min(100, lv));
            cand = fmaxf(cand, fmaf(mx, f[u], static_cast<float>(lv)));
          }
          __syncwarp();
          if (bar_red_or(bar_rows, kRowThreads, mine && cand > mref + kLazy)) {
            red_r[grp * 32 + lane] = cand;
            named_bar(bar_rows, kRowThreads);
            float bm = red_r[lane];
#pragma unroll
            for (int e = 1; e < NG; ++e) bm = fmaxf(bm, red_r[e * 32 + lane]);
            float al = 1.f;
            if (mine && bm > mref + kLazy) {
              al = ex2(mref - bm);            // 0 while the row had no key
              mref = bm;
              l *= al;
            }
            if (j > 0 && sums && __any_sync(0xffffffffu, al != 1.f)) {
              // the running sums of the moved rows (all earlier P V done)
              fwait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, a.c.status, fail);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = cg * (D / 2); c < (cg + 1) * (D / 2); c += 32) {
                uint32_t r8[4][8];
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_ld8_nowait(t_lane + c + 8 * e, r8[e]);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                  for (int x = 0; x < 8; ++x) r8[e][x] = __float_as_uint(__uint_as_float(r8[e][x]) * al);
                  tmem_st8(t_lane + c + 8 * e, r8[e]);
                }
              }
              tmem_st_wait();
            }
          }
        }
        uint32_t w0[KW / 4], w1[KW / 4];
        if (half_used) {
#pragma unroll
          for (int c = 0; c < KW; c += 2) {
            const float fa = f[c >> 4], vb = fmaxf(vsc[c >> 4], 0.f) * kUnit;
            const float p0 = ex2(fmaf(s[c], fa, -mref)), p1 = ex2(fmaf(s[c + 1], fa, -mref));
            l += p0;
            l += p1;
            const __half2 x = __floats2half2_rn(p0 * vb, p1 * vb);
            uint16_t c0, c1;
            uint32_t back;
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c0) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c0));
            const __half2 rest = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(kLow));
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c1) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
            if ((c & 2) == 0) {
              w0[c >> 2] = c0;
              w1[c >> 2] = c1;
            } else {
              w0[c >> 2] |= static_cast<uint32_t>(c0) << 16;
              w1[c >> 2] |= static_cast<uint32_t>(c1) << 16;
            }
          }
        }
        // the P buffer was last read by P V of block g - PB
        if (g >= PB) fwait(&pv_done[(g - PB) & 1], ((g - PB) >> 1) & 1, a.c.status, fail);
        if (mine) {
          uint8_t* pp = pbuf + (g % PB) * kPBytes;
#pragma unroll
          for (int u = 0; u < NE; ++u) {
            *reinterpret_cast<uint4*>(pp + swz128(row, NE * grp + u)) =
                make_uint4(w0[4 * u], w0[4 * u + 1], w0[4 * u + 2], w0[4 * u + 3]);
            *reinterpret_cast<uint4*>(pp + swz128(64 + row, NE * grp + u)) =
                make_uint4(w1[4 * u], w1[4 * u + 1], w1[4 * u + 2], w1[4 * u + 3]);
          }
        }
        // ---- value rows no row of the item may use: zero them (two threads per key)
        {
          const int key = kb + (st >> 1);
          if (key < w.lo || key > w.hi || vs[((j << kLgBlk) + (st >> 1)) >> lg_bt] < 0.f) {
            const int u = value_unit(g);
            fwait(&u_full[u % NU], (u / NU) & 1, a.c.status, fail);
            uint8_t* vrow = ring + (u % NU) * C::kUnitBytes + (st >> 1) * 128;
#pragma unroll
            for (int t = 0; t < ATOMS; ++t)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4*>(vrow + t * kAtom + ((st & 1) * 4 + c) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g & 1]);
      }
      // ---- on to the next item's queries, then this one's (m, l) and o = (o0 +
      // o1 / 16) / kUnit: quadrants 0, 1 hold o0 and 2, 3 o1; each finishes half
      // of the columns and passes its sums of the others through shared memory
      // (this row half's part of the P buffer, which no MMA reads now)
      w.next();
      take();
      fwait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, a.c.status, fail);
      __syncwarp();
      tc_fence_after();
      if (half_used) {
        red_r[grp * 32 + lane] = l;           // every warp is past the last block's reductions
        named_bar(bar_rows, kRowThreads);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < NG; e += 4)
          sum += (red_r[e * 32 + lane] + red_r[e * 32 + 32 + lane]) + (red_r[e * 32 + 64 + lane] + red_r[e * 32 + 96 + lane]);
        if (grp == 0 && mine && !*fail) __stcg(&a.part_ml[slot + row], make_float2(mref, sum));
        if (sums) {
          constexpr int CW = RP == 32 ? 32 : 16;       // columns a warp finishes at a time
          const bool low = quad >= 2;
          float* give = reinterpret_cast<float*>(pbuf + (64 * cg + 32 * rh) * 128) + (low ? 0 : CW * 32) + lane;
          const float* get = reinterpret_cast<const float*>(pbuf + (64 * cg + 32 * rh) * 128) + (low ? CW * 32 : 0) + lane;
          float* po = a.part_o + (slot + row) * D;
#pragma unroll 1
          for (int c0 = cg * (D / 2); c0 < (cg + 1) * (D / 2); c0 += 2 * CW) {
            const int mine0 = c0 + (low ? CW : 0), other0 = c0 + (low ? 0 : CW);
            uint32_t o[CW / 8][8], x[CW / 8][8];
#pragma unroll
            for (int c = 0; c < CW / 8; ++c) {
              tmem_ld8_nowait(t_lane + mine0 + 8 * c, o[c]);
              tmem_ld8_nowait(t_lane + other0 + 8 * c, x[c]);
            }
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < CW; ++c) give[c * 32] = __uint_as_float(x[c >> 3][c & 7]);
            named_bar(bar_cg, 64);
            float y[CW];
            const float f_own = low ? 1.f / (kUnit * kLow) : 1.f / kUnit, f_get = low ? 1.f / kUnit : 1.f / (kUnit * kLow);
#pragma unroll
            for (int c = 0; c < CW; ++c) y[c] = get[c * 32];
#pragma unroll
            for (int c = 0; c < CW; ++c) y[c] = fmaf(y[c], f_get, __uint_as_float(o[c >> 3][c & 7]) * f_own);
            if (mine && !*fail) {
#pragma unroll
              for (int c = 0; c < CW; c += 4)
                __stcg(reinterpret_cast<float4*>(po + mine0 + c), make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]));
            }
            named_bar(bar_cg, 64);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free);
        mbar_arrive(&sc_empty[item & 1]);
      }
      ++item;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the splits of a row.
// Four parts by absolute split index mod 4, each in ascending order, then the
// parts in order: splits without a key of the row add nothing at fixed places,
// so the order does not depend on where the list of splits starts.  One warp per
// part, a CTA per row.
__global__ void __launch_bounds__(128) qattn_combine_kernel(const __grid_constant__ QAttnArgs a) {
  __shared__ float o_s[4][256];
  __shared__ float l_s[4], m_s[4];
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x % a.rows, bh = blockIdx.x / a.rows;
  const int h = bh % a.c.n_kv_heads, b = bh / a.c.n_kv_heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = a.c.dim, i = r / a.G, hq = h * a.G + r % a.G;
  uint16_t* dst = a.out + ((static_cast<int64_t>(b) * a.n + i) * (a.c.n_kv_heads * a.G) + hq) * D;
  const SeqKeys k = seq_keys(a, a.c.seq_lens[b]);
  const int64_t slot0 = static_cast<int64_t>(bh) * a.n_splits * a.rows + r;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < k.splits; s += 128) M = fmaxf(M, __ldcg(&a.part_ml[slot0 + static_cast<int64_t>(s) * a.rows]).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (lane == 0) m_s[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
  float o[8], l = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  const int sf = k.splits ? k.lo / a.split : 0, per = D / 32;
  for (int s = ((warp - sf) & 3); s < k.splits; s += 4) {
    const float2 ml = __ldcg(&a.part_ml[slot0 + static_cast<int64_t>(s) * a.rows]);
    if (ml.x <= kNoKey) continue;
    const float wt = exp2f(ml.x - M);
    const float* po = a.part_o + (slot0 + static_cast<int64_t>(s) * a.rows) * D + lane * per;
    l = fmaf(wt, ml.y, l);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(po));
    o[0] = fmaf(wt, x.x, o[0]);
    o[1] = fmaf(wt, x.y, o[1]);
    o[2] = fmaf(wt, x.z, o[2]);
    o[3] = fmaf(wt, x.w, o[3]);
    if (per == 8) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(po + 4));
      o[4] = fmaf(wt, y.x, o[4]);
      o[5] = fmaf(wt, y.y, o[5]);
      o[6] = fmaf(wt, y.z, o[6]);
      o[7] = fmaf(wt, y.w, o[7]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < per) o_s[warp][lane * per + e] = o[e];
  if (lane == 0) l_s[warp] = l;
  __syncthreads();
  const float den = (l_s[0] + l_s[1]) + (l_s[2] + l_s[3]);
  const float qs = a.q_scale[static_cast<int64_t>(bh) * a.rows + r];
  for (int d = threadIdx.x; d < D; d += 128) {
    const float x = ((o_s[0][d] + o_s[1][d]) + o_s[2][d]) + o_s[3][d];
    dst[d] = den == 0.f ? 0 : f32_to_bf16(qs == qs ? x / den : qs);   // no key: zero
  }
}

template <int D, int RP>
cudaError_t launch_one(int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                       const QAttnArgs& a, cudaStream_t st) {
  auto kern = qattn_kernel<D, RP>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, st, tk, tv, a);
}

template <int D>
cudaError_t launch_dim(int rp, int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                       const QAttnArgs& a, cudaStream_t st) {
  if (rp == 32) return launch_one<D, 32>(grid, tk, tv, a, st);
  return launch_one<D, 64>(grid, tk, tv, a, st);
}

}  // namespace

cudaError_t launch_qcache_attn(const QAttnArgs& a, cudaStream_t st) {
  const int D = a.c.dim, rp = a.rows <= 32 ? 32 : 64;
  const uint64_t rows = static_cast<uint64_t>(a.c.num_pages) * a.c.n_kv_heads * kPg;
  CUtensorMap tk, tv;
  if (!make_tmap_u8_2d(&tk, a.c.k, rows, D, kPg, 128) || !make_tmap_u8_2d(&tv, a.c.v, rows, D, kPg, 128))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.B) * a.c.n_kv_heads * ((a.rows + rp - 1) / rp) * a.n_splits;
  const int grid = static_cast<int>(items < sms ? items : sms);
  e = D == 256 ? launch_dim<256>(rp, grid, tk, tv, a, st) : launch_dim<128>(rp, grid, tk, tv, a, st);
  if (e != cudaSuccess) return e;
  return launch_k(qattn_combine_kernel, dim3(a.B * a.c.n_kv_heads * a.rows), dim3(128), 0, st, a);
}

}  // namespace sv
