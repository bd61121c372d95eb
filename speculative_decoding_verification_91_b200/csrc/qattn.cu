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
// w1 / 16 (w1 the rounding error of w0, other rows of the same M tile, so one
// pass gives both sums, in lanes RP / 4 apart of the accumulator; RP = 128: below).
//
// Work item = (sequence, KV head, block of RP query rows, absolute split of
// split_tokens keys); items are ordered and every CTA (one per SM) takes those
// whose middle lies in an equal share of their cost.  12 warps:
//   warp 0     TMA producer: keys and values of 128-key blocks (two pages) into
//              a ring of kUnits units of 128 x dim bytes.
//   warp 1     allocates TMEM; one thread issues S[128][128 keys] = Q K^T (A = Q
//              from TMEM, B = K, K-major).  With Q in shared memory too the two
//              operands took all of its bandwidth.
//   warp 2     finds the CTA's items and describes them in shared memory, with
//              their pages and then their scales, up to kItems ahead.
//   warp 3     one thread issues O[rows][dim] += P V (A = P in shared memory,
//              K-major, B = V as stored, MN-major).
//   warps 4-11 softmax: a thread takes one query row and RP / 2 of the block's
//              keys.  The queries sit 128 / RP times in the 128 lanes of Q, so
//              every TMEM lane quadrant, and with it every scheduler, takes an
//              equal part of the keys (one copy left all of the work to one or
//              two schedulers, at 4300 clocks a block).  A row's
//              reference m moves only when a block exceeds it by 2^kLazy (one
//              barrier vote per block); the v scale is folded into m and p
//              (p v_scale <= 2^kLazy), so blocks of any scale share one
//              accumulator; the sum of p is kept in binary32.
//
// Per block of 128 keys (D = 256), in SM clocks: the scores' MMAs 1024, P V 512 (1536
// with RP = 128), a softmax warp 1650 with RP = 32, 2350 with 64 (exponentials and
// codes 930, the largest score 250, the store of P 270, the rest latency between
// them) and 6100 with 128, DRAM 2840 with every SM at work.  So long items of few rows
// run at the pace of DRAM (64 decodes of 1k to 16k, 16 / 8 heads, 2.29 GB: 432 to 465 us
// on one GPU or another, 4.9 to 5.3 TB/s, the clock down to 1.45 GHz at the power
// limit), prompt chunks at that of the softmax (256 rows over 8k, 32 / 4 heads, 2
// sequences: 214 us),
// and calls of some items a CTA also pay for the unequal shares of whole splits.  Not
// kept: 16 softmax warps, a vote after the exponentials instead of before (3%
// slower), a larger kLazy (1 to 4% faster, coarser small weights).
//
// RP = 128 (prompt chunks) has no lanes left for w1's rows: its weights are three e5m2
// codes in tiles of their own, w0 + w1 + w2, summed in one accumulator.  e5m2 is
// binary16's upper byte, so the first two are masks instead of conversions, and its
// range holds a weight to 2^-9 of itself down to 2^-18 of the reference, under which an
// item keeps up to 16384 keys.  (Two e4m3 codes without a scale between them kept
// weights above 2^-15 only: 182 us for the chunk below instead of 212, but beside a sink
// of 95 % results were off by 35 to 45 %.  w1 as e5m2 beside an e4m3 w0: 3 % where the
// others weigh the same.  Blocks of 64 rows: 215 us.)
//
// Value rows of keys outside the item's range or on pages that were not loaded
// are zeroed in shared memory before P V, so stale slots (NaN codes among them)
// never reach it.  Key blocks start at absolute multiples of 128 and a row's
// weights depend on its own scores only, so a row's partial depends neither on n
// nor on the batch, its row slot or the CTA: sums of p are kept by 16 keys of a
// block, whatever RP, and added in key order.  Every wait is bounded.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "qcache.h"
#include "tc_common.cuh"

namespace sv {

namespace {

constexpr int kBlk = kQBlk;                // keys per block
constexpr int kLgBlk = 7;
constexpr int kPg = SPEC_PAGE_SIZE;
constexpr int kSoftWarps = 8;
constexpr int kFirstSoft = 4;
constexpr int kThreads = (kFirstSoft + kSoftWarps) * 32;
constexpr uint32_t kSmemMax = 227u * 1024u;
constexpr int kItems = 4;                  // items described ahead in shared memory
constexpr uint32_t kTail = 17408;
constexpr uint32_t kPBytes = 128 * kBlk;
constexpr int kMaxScales = 256;            // scales of one item: 4096 keys / 16
constexpr int kMaxPg = 256;                // its pages: 16384 keys / 64
// p v_scale <= 2^kLazy; in code units times kUnit: at most 362 < 448, with RP = 128
// 23170 (e5m2 goes to 57344).  A larger kLazy moves the reference less often, a larger
// kUnit keeps smaller weights: the least steps are 2^-9 / (32 kLow) = 2^-18 and 2^-16 /
// 2048 = 2^-27 of the reference.  (RP <= 64 in units of 128 and 256, kLazy 1.8 and 0.8:
// 8 sequences 96 -> 107 and 109 us, the references move more often.)
constexpr float kLazy = 3.5f;
template <int RP>
constexpr float kUnit = RP == 128 ? 2048.f : 32.f;
constexpr float kLow = 16.f;               // w1 is stored times 16
constexpr float kNoKey = -0x1.fffffep127f;   // reference of a row that has seen no key
// References further than this from 0 are off by 1/4 and more, and with them 2^(s - m);
// a row that comes to one ends as NaN.
constexpr float kFar = 0x1p22f;
constexpr float kMostFactor = 4e30f;       // of a score's e4m3 products (below 2^26): the score stays finite

// Waits for this thread's loads from TMEM, v's among them.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[N]) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));   // no use of v before
}
// 16 TMEM lanes by 32 columns: v[4 k + 2 i + z] is lane (thread / 4 + 8 i), column
// 8 k + 2 (thread % 4) + z
__device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, uint32_t (&v)[32]) {
  tmem_ld16x256(taddr, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
  tmem_ld16x256(taddr + 32, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
}
// Added to a weight before it is coded (RP <= 64), by its key's place: each 16 keys take 16 values spread evenly
// over one least step of w1 around 0, in an order of their own.  So weights below that step are dropped or raised
// to it in shares that sum to what they are.  Rounded to nearest, thousands of small weights beside a dominant one
// (an attention sink) all went the same way, while the sum of p below the line kept them: results were off by 2 to
// 8 % (a sink of 99 % beside 4096 keys), now 0.2.  Values are spread evenly over every second, fourth and eighth
// key too, and the order changes from 16 keys to the next: values that recur with the key's place (one order for
// all: 2 to 8 % off for periods of 2 to 16) do not meet it.  Less than half a step: a weight of 0 stays 0.  From
// shared memory, 8 reads a thread and block of 64 rows: 8 sequences 95.5 -> 98.5 us, blocks of 32 rows unchanged.
__device__ __forceinline__ float spread(int order, int c) {
  return (static_cast<float>((5 * c & 15) ^ order) - 7.5f) / 16.f * (0x1p-9f / kLow);
}
__device__ __forceinline__ uint32_t spread_order(int key) { return static_cast<uint32_t>(key >> 4) * 0x9e3779b1u >> 28; }
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
// Instruction descriptor, kind::f8f6f4: D binary32, A e4m3 or e5m2, B e4m3, M = 128,
// N = n, A K-major, B K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int n, bool b_mn, bool a_e5m2) {
  return (1u << 4) | (a_e5m2 ? (1u << 7) : 0u) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

template <int D, int RP>
struct Cfg {
  static constexpr uint32_t kUnitBytes = kBlk * D;              // one block's keys or values
  static constexpr int kPBufs = D == 128 ? 2 : 1;
  static constexpr int kUnits = D == 128 ? (RP == 128 ? 7 : 11) : RP == 128 ? 5 : 6;
  static constexpr uint32_t kPTile = RP == 128 ? 3 * kPBytes : kPBytes;   // both codes' rows in one tile, or three tiles
  static constexpr uint32_t kOffRing = kPBufs * kPTile;
  static constexpr uint32_t kOffTail = kOffRing + kUnits * kUnitBytes;
  static constexpr uint32_t kSmem = 1024 + kOffTail + kTail + (RP == 128 ? 0 : 1024);
  static_assert(kSmem <= kSmemMax, "shared memory");
  // TMEM columns: output, scores, both codes of the queries (4 dims a column)
  static constexpr int kSBufs = D == 128 ? 2 : 1;
  static constexpr uint32_t kColS = D;
  static constexpr uint32_t kColQ = kColS + kSBufs * kBlk;
  static_assert(kColQ + 2 * D / 4 <= 512, "tensor memory");
};

// One work item as the roles see it; nb < 0: the end.
struct Item {
  int h, r0, nrows, p0;    // KV head, first row of the block, its rows, the sequence's first position
  int lo, hi, blk0, nb;    // its keys and blocks
  int fresh, pad;          // the queries differ from the item before
  long slot;               // partial of its first row
  long q_row;              // row of its first query among all
  long out0;               // row of the sequence's first result
};

// Walks the items of one CTA.
struct Walker {
  const QAttnArgs* a;
  int RP, RB;              // rows of a block, row blocks
  int b, h, rb, sidx, L;
  int split0, p0, p1;      // the sequence's first split; positions of the row block's first and last row
  SeqKeys k;
  int base, end, pos;      // cost before (b, h, rb); where the CTA stops; this item's middle
  int lo, hi, blk0, nb;    // this item's keys and blocks (nb = 0: none)
  bool fresh;
  __device__ bool valid() const { return b < a->B && pos < end; }
  __device__ void load_seq(int len) {
    L = len;
    k = seq_keys(*a, L);
    split0 = a->by_split(k.lo >> kLgBlk);
  }
  // from the first split of (b, h, rb) that is wanted: its rows, then its keys
  __device__ void derive(bool rows) {
    if (rows) {
      const int r0 = rb * RP, r1 = min(a->rows, r0 + RP) - 1;
      p0 = L + a->q_offset + a->by_G(r0);
      p1 = L + a->q_offset + a->by_G(r1);
      fresh = true;
    }
    const int s0 = (split0 + sidx) * a->split, start = max(s0, k.lo);
    const int b0 = start >> kLgBlk, b1 = min(s0 + a->split - 1, k.hi) >> kLgBlk;
    pos = base + 2 * (b0 - (k.lo >> kLgBlk) + sidx) + (b1 - b0 + 2);
    lo = a->window > 0 ? max(start, p0 - a->window + 1) : start;
    hi = min(min(s0 + a->split - 1, k.hi), p1);
    blk0 = lo >> kLgBlk;
    nb = hi >= lo ? (hi >> kLgBlk) - blk0 + 1 : 0;
  }
  __device__ void next() {
    bool rows = false;
    if (++sidx >= k.splits) {     // the next (b, h, rb) that has keys
      rows = true;
      sidx = 0;
      base += k.cost();
      if (++rb == RB) {
        rb = 0;
        if (++h == a->c.n_kv_heads) {
          h = 0;
          do {
            if (++b >= a->B) return;
            load_seq(__ldcg(&a->c.seq_lens[b]));
          } while (k.blocks == 0);
        }
      }
    }
    derive(rows);
  }
};

// Ring units of block g's keys and values: K0 K1 V0 K2 V1 K3 V2 ..
__device__ __forceinline__ int key_unit(int g) { return g == 0 ? 0 : 2 * g - 1; }
__device__ __forceinline__ int value_unit(int g) { return 2 * g + 2; }

// Bounded wait that gives up at once after a timeout anywhere in the CTA.  The
// part past the first test is kept out of line: inlined at every wait (and with
// a walker in every role) the kernel had 200 KB of code, and its roles spent
// half of their time on instruction fetches.
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, unsigned* status, volatile int* fail) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (*fail) return false;
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitNs) {
      flag_status(status, SPEC_DEV_TIMEOUT);
      *fail = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool fwait(uint64_t* bar, uint32_t parity, unsigned* status, volatile int* fail) {
  return mbar_try_wait(bar, parity) || wait_more(bar, parity, status, fail);
}

template <int D, int RP>
__global__ void __launch_bounds__(kThreads, 1) qattn_kernel(const __grid_constant__ CUtensorMap tk,
                                                            const __grid_constant__ CUtensorMap tv,
                                                            const __grid_constant__ QAttnArgs a) {
  using C = Cfg<D, RP>;
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
  uint64_t* p_full = s_free + 2;                           // [2] by block parity
  uint64_t* pv_done = p_full + 2;                          // [2]
  uint64_t* it_full = pv_done + 2;                         // [kItems] by item
  uint64_t* sc_full = it_full + kItems;                    // [kItems] its scales
  uint64_t* it_empty = sc_full + kItems;                   // [kItems]
  uint64_t* q_ready = it_empty + kItems;
  uint64_t* o_free = q_ready + 1;
  uint64_t* mma_done = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  volatile int* fail = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Item* items = reinterpret_cast<Item*>(tail + 512);       // [kItems]
  float* red = reinterpret_cast<float*>(tail + 1024);      // [threads of a row][rows]
  float* alpha_s = red + 256;                              // [rows]
  float* l_s = alpha_s + 128;                              // [16 keys of a block][rows]: sums of p
  float* bad_s = l_s + 512;                                // [rows]
  float* ks_s = reinterpret_cast<float*>(tail + 5120);     // [kItems][kMaxScales]
  float* vs_s = ks_s + kItems * kMaxScales;                // < 0: page not there
  int* pg_s = reinterpret_cast<int*>(vs_s + kItems * kMaxScales);   // [kItems][kMaxPg]; < 0: not there
  float* spread_s = reinterpret_cast<float*>(tail + kTail);         // [orders][16 keys] (RP <= 64)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(sizeof(Item) * kItems <= 512, "items");

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
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&sc_full[i], 1);
      mbar_init(&it_empty[i], kSoftWarps + 2);
    }
    mbar_init(q_ready, kSoftWarps);
    mbar_init(o_free, kSoftWarps);
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *fail = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_trigger();
  // Lengths, block table, pages and scales are read at once, the softmax warps
  // alone wait for the query kernel: it lets this one start only once every kernel
  // before it is done (it triggers after its own wait), so what it does not write
  // itself is final, and nothing earlier still reads the partials.  (Those loads
  // pass by L1, which nothing has ordered yet.)
  // Barriers and TMEM are there once all warps have passed this; warp 2 comes with
  // its first item in hand.
  uint32_t tmem = 0;
  const auto ready = [&]() {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *tmem_slot;
  };
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return fwait(bar, parity, a.c.status, fail); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    ready();
    if (lane == 0) {
      // keys shared by several row blocks: normal priority in L2
      const uint64_t pol = a.rows > RP ? policy_evict_normal() : policy_evict_first();
      int gk = 0, gv = 0, jk = 0, jv = 0, ik = 0, iv = 0;   // blocks, block in item, item: of keys, of values
      bool ok = true, more = true;                          // more: there may be keys left
      // order of the copies: K0 K1 V0 K2 V1 ..: values are needed a softmax
      // later than their keys, and would hold a slot meanwhile
      for (;;) {
        const bool key = more && gk < gv + 2;
        if (!key && gv == gk) break;
        const int i = key ? ik : iv, j = key ? jk : jv, u = key ? key_unit(gk) : value_unit(gv), s = u % NU;
        if (key && j == 0 && !(ok = wait(&it_full[i % kItems], (i / kItems) & 1))) break;
        const Item& x = items[i % kItems];
        if (x.nb < 0) {
          more = false;
          continue;
        }
        int y[2];
        uint32_t bytes = 0;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int id = pg_s[(i % kItems) * kMaxPg + j * 2 + p];
          y[p] = id >= 0 ? (id * a.c.n_kv_heads + x.h) * kPg : -1;
          if (id >= 0) bytes += kPg * D;
        }
        if (u >= NU && !(ok = wait(&u_empty[s], ((u / NU) - 1) & 1))) break;
        mbar_arrive_expect_tx(&u_full[s], bytes);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (y[p] >= 0)
#pragma unroll
            for (int t = 0; t < ATOMS; ++t)
              tma_load_2d(ring + s * C::kUnitBytes + t * kAtom + p * (kPg * 128), key ? &tk : &tv, &u_full[s], t * 128,
                          y[p], pol);
        if (key) {
          ++gk;
          if (++jk == x.nb) jk = 0, ++ik;
        } else {
          ++gv;
          if (++jv == x.nb) {
            jv = 0;
            mbar_arrive(&it_empty[iv % kItems]);
            ++iv;
          }
        }
      }
      // every issued copy must land before the CTA may exit (a slot's last unit)
      for (int i = 0; i < NU; ++i) {
        int last = -1;
        for (int g = max(0, gk - NU); g < gk; ++g)
          if (key_unit(g) % NU == i) last = max(last, key_unit(g));
        for (int g = max(0, gv - NU); g < gv; ++g)
          if (value_unit(g) % NU == i) last = max(last, value_unit(g));
        if (last >= 0) mbar_wait(&u_full[i], (last / NU) & 1, a.c.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- scores
    ready();
    if (lane == 0) {
      const uint32_t id_qk = idesc_e4m3(kBlk, false, false);
      int s = 0, su = 0, g = 0, nq = 0;     // ring slot and its round, block, query groups begun
      for (int i = 0;; ++i) {
        if (!wait(&it_full[i % kItems], (i / kItems) & 1)) break;
        const int nb = items[i % kItems].nb;
        bool ok = nb >= 0 && (!items[i % kItems].fresh || wait(q_ready, nq++ & 1));
        for (int j = 0; ok && j < nb; ++j, ++g) {
          ok = (g < SB || wait(&s_free[g % SB], ((g / SB) - 1) & 1)) && wait(&u_full[s], su & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k_addr = smem_u32(ring + s * C::kUnitBytes);
          const uint32_t t_s = tmem + C::kColS + (g % SB) * kBlk;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_e4m3_ta(t_s, tmem + C::kColQ + c * (D / 4) + kk * 8,
                           sw128_desc(k_addr + (kk >> 2) * kAtom + (kk & 3) * 32), id_qk, (c > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&s_full[g % SB]);
          umma_commit(&u_empty[s]);
          s += g == 0 ? 1 : 2;              // K0 K1 V0 K2 V1 ..
          if (s >= NU) s -= NU, ++su;
        }
        if (!ok) break;
      }
      umma_commit(&mma_done[0]);            // nothing may be in flight when TMEM is freed
      mbar_wait(&mma_done[0], 0, a.c.status);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- P V
    ready();
    // (a thread of its own: one thread that issued both spent 600 clocks from
    // the last MMA of one product to the first of the other)
    if (lane == 0) {
      const uint32_t id_pv = idesc_e4m3(D, true, RP == 128);
      int s = 2, su = 0, g = 0;
      for (int i = 0;; ++i) {
        if (!wait(&it_full[i % kItems], (i / kItems) & 1)) break;
        const int nb = items[i % kItems].nb;
        bool ok = nb >= 0 && (i == 0 || wait(o_free, (i - 1) & 1));
        for (int j = 0; ok && j < nb; ++j, ++g) {
          ok = wait(&u_full[s], su & 1) && wait(&p_full[g & 1], (g >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v_addr = smem_u32(ring + s * C::kUnitBytes);
          const uint32_t p_addr = smem_u32(pbuf + (g % PB) * C::kPTile);
#pragma unroll
          for (uint32_t t = 0; t < C::kPTile; t += kPBytes)
#pragma unroll
            for (int kk = 0; kk < kBlk / 32; ++kk)
              umma_e4m3(tmem, sw128_desc(p_addr + t + kk * 32), sw128_desc_mn(v_addr + kk * 4096, kAtom), id_pv,
                        (j > 0 || kk > 0 || t > 0) ? 1u : 0u);
          umma_commit(&pv_done[g & 1]);
          umma_commit(&u_empty[s]);
          s += 2;
          if (s >= NU) s -= NU, ++su;
        }
        if (!ok) break;
        mbar_arrive(&it_empty[i % kItems]);
      }
      umma_commit(&mma_done[1]);
      mbar_wait(&mma_done[1], 0, a.c.status);
    }
  } else if (warp == 2) {
    // --------------------------------------------------- items and scales
    const int RB = (a.rows + RP - 1) / RP, per_b = a.c.n_kv_heads * RB;
    // this CTA's share [x0, x1) of the cost of all items and its first item
    const auto length = [&](int b) { return b < a.B ? __ldcg(&a.c.seq_lens[b]) : 0; };
    const auto cost = [&](int b, int L) { return b < a.B ? seq_keys(a, L).cost() * per_b : 0; };
    int L = length(lane), n = cost(lane, L), total = 0;
    for (int b = lane; b - lane < a.B; b += 32) {
      if (b >= 32) n = cost(b, L = length(b));
      if (blockIdx.x == 0 && b < a.B &&
          (L < 0 || static_cast<int64_t>(L) + a.kv_extra > static_cast<int64_t>(a.c.max_pages) * kPg))
        flag_status(a.c.status, SPEC_DEV_BAD_LENGTH);
      total += __reduce_add_sync(0xffffffffu, n);
    }
    const int me = blockIdx.x, per = total / gridDim.x, rest = total % gridDim.x;
    const int x0 = me * per + min(me, rest), x1 = x0 + per + (me < rest ? 1 : 0);
    Walker w{};
    w.a = &a;
    w.RP = RP;
    w.RB = RB;
    w.b = a.B;
    w.end = x1;
    int pre = 0;
    for (int b = lane; b - lane < a.B && w.b == a.B && x1 > x0; b += 32) {
      if (a.B > 32) n = cost(b, L = length(b));
      int incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const int excl = pre + incl - n;
      const unsigned bal = __ballot_sync(0xffffffffu, n > 0 && x0 >= excl && x0 < excl + n);
      if (bal) {
        const int src = __ffs(bal) - 1;
        w.b = b - lane + src;
        w.base = __shfl_sync(0xffffffffu, excl, src);
        w.load_seq(__shfl_sync(0xffffffffu, L, src));
      }
      pre += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (w.b < a.B) {
      const int rem = x0 - w.base, hr = rem / w.k.cost(), r = rem - hr * w.k.cost();
      w.h = hr / RB;
      w.rb = hr - w.h * RB;
      w.base += hr * w.k.cost();
      // the first split whose middle is at or after cost r of the sequence: no middle
      // of a split before the one that cost r falls into is
      const int first = w.k.lo >> kLgBlk, bps = a.split >> kLgBlk;
      w.sidx = static_cast<int>(a.by_cost(r / 2 + (first - w.split0 * bps)));
      w.sidx = min(w.sidx, w.k.splits - 1);
      w.derive(true);
      while (w.b < a.B && w.pos < x0) w.next();
      w.fresh = true;
    }
    const int lg_bt = 31 - __clz(a.c.block), lg_pg = 31 - __clz(kPg);
    bool fresh = true;
    for (int i = 0;; w.next()) {
      const bool end = !w.valid();
      const int r0 = w.rb * RP, nrows = end ? 0 : min(a.rows - r0, RP);
      const long bh = static_cast<long>(w.b) * a.c.n_kv_heads + w.h;
      const long slot = (bh * a.n_splits + w.sidx) * a.rows + r0;
      fresh |= w.fresh;
      w.fresh = false;
      if (!end && w.nb == 0) {            // no key for this row block in this split
        for (int r = lane; r < nrows; r += 32) {
          if (a.n_splits > 1) {
            __stcg(&a.part_ml[slot + r], make_float2(kNoKey, 0.f));
          } else {
            const long o = (static_cast<long>(w.b) * a.n + (r0 + r) / a.G) * (a.c.n_kv_heads * a.G) + w.h * a.G + (r0 + r) % a.G;
            for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(a.out + o * D + c) = make_uint4(0, 0, 0, 0);
          }
        }
        continue;
      }
      const int q = i % kItems;
      // (given up: the slot is not touched, the softmax warps may be about to read it)
      if (i >= kItems && !__all_sync(0xffffffffu, wait(&it_empty[q], ((i / kItems) - 1) & 1))) break;
      if (lane == 0) {
        Item& x = items[q];
        x.h = w.h;
        x.r0 = r0;
        x.nrows = nrows;
        x.p0 = w.L + a.q_offset;
        x.lo = w.lo;
        x.hi = w.hi;
        x.blk0 = w.blk0;
        x.nb = end ? -1 : w.nb;
        x.fresh = fresh;
        x.slot = slot;
        x.q_row = bh * a.rows + r0;
        x.out0 = static_cast<long>(w.b) * a.n;
      }
      // its pages, all asked for at once (one at a time by the producer they cost an
      // L2 latency a block), then its scales; the copies start before those are here
      if (!end) {
        const int32_t* bt = a.c.block_table + static_cast<int64_t>(w.b) * a.c.max_pages;
        for (int e = lane; e < 2 * w.nb; e += 32) {
          const int pg = 2 * w.blk0 + e;
          int id = -1;
          if (pg * kPg <= w.hi && pg * kPg + kPg - 1 >= w.lo) {
            id = __ldcg(&bt[pg]);
            if (id < 0 || id >= a.c.num_pages) {
              id = -1;
              flag_status(a.c.status, SPEC_DEV_BAD_PAGE);
            }
          }
          pg_s[q * kMaxPg + e] = id;
        }
      }
      __syncwarp();
      if (i == 0) ready();
      if (lane == 0) mbar_arrive(&it_full[q]);
      if (!end) {
        fresh = false;
        const int count = w.nb * (kBlk / a.c.block), lg_per = lg_pg - lg_bt;
        for (int e = lane; e < count; e += 32) {
          const int id = pg_s[q * kMaxPg + (e >> lg_per)];
          float ks = 0.f, vs = -1.f;
          if (id >= 0) {
            const int64_t sc = ((static_cast<int64_t>(id) * a.c.n_kv_heads + w.h) << lg_per) + (e & ((1 << lg_per) - 1));
            ks = __ldcg(&a.c.ks[sc]);
            vs = __ldcg(&a.c.vs[sc]);
          }
          ks_s[q * kMaxScales + e] = ks;
          vs_s[q * kMaxScales + e] = vs;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[q]);
      if (end || *fail) break;
      ++i;
    }
  } else {
    // ------------------------------------------------------------- softmax
    ready();
    constexpr int KW = RP / 2;                 // keys of a block a thread takes
    constexpr int NG = kBlk / KW;              // threads of a row
    const int quad = warp & 3, cg = (warp - kFirstSoft) >> 2;     // TMEM lane quadrant; first or second half of its keys
    const int rh = RP == 128 ? quad : RP == 64 ? quad & 1 : 0;    // rows 32 rh + lane
    const int grp = (RP == 128 ? 0 : RP == 64 ? quad >> 1 : quad) * 2 + cg;   // keys KW grp .. of the block
    const int row = rh * 32 + lane;
    const int st = (warp - kFirstSoft) * 32 + lane;               // 0..255
    // Rows of P and of the output: row r in quadrant r / RQ, lane r % RQ for w0,
    // RQ + r % RQ for w1 (128 rows: the same lane of a second tile).  The row of this
    // thread's lane:
    constexpr int RQ = RP / 4;
    const int o_row = quad * RQ + lane % RQ;
    const int p_row = (row / RQ) * 32 + row % RQ;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    constexpr int kSoft = kSoftWarps * 32;
    const int lg_bt = 31 - __clz(a.c.block);
    float* l_r = l_s + rh * 32;
    float* red_r = red + rh * 32;              // [thread of the row][RP rows]
    int g = 0, p = 0;
    float qs = 0.f;
    bool bad_q = false;
    // Takes item i; where the queries change, this thread's row of them into
    // TMEM: every product with the old ones is done once the last scores have
    // been read.  False: there is none.
    auto take = [&](int i) -> bool {
      if (!wait(&it_full[i % kItems], (i / kItems) & 1)) return false;
      const Item& x = items[i % kItems];
      if (x.nb < 0) return false;
      if (!x.fresh) return true;
      const bool have = row < x.nrows;
      const int r = x.r0 + row, i_pos = a.by_G(r);
      p = x.p0 + i_pos;
      const long at = x.q_row + row, plane = static_cast<long>(a.B) * a.c.n_kv_heads * a.rows;
      const float scale = have ? __ldcg(&a.q_scale[at]) : 0.f;
      uint32_t v[2][D / 32][4];                       // all loads in flight at once
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q_codes + (at + c * plane) * D + cg * (D / 2));
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const uint4 z = have ? __ldcg(src + e) : make_uint4(0, 0, 0, 0);
          v[c][e][0] = z.x;
          v[c][e][1] = z.y;
          v[c][e][2] = z.z;
          v[c][e][3] = z.w;
        }
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          tmem_st8(t_lane + C::kColQ + c * (D / 4) + cg * (D / 8) + e * 8,
                   *reinterpret_cast<uint32_t(*)[8]>(v[c][2 * e]));
      bad_q = scale != scale;                         // a NaN row's result is set at the end
      qs = bad_q ? 0.f : scale * a.scale_log2;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      __syncwarp();
      return true;
    };
    // rows of P that no query row owns stay zero (what they held cost power: P V is
    // done for all 128)
    for (int i = st; i < PB * static_cast<int>(C::kPTile) / 16; i += kSoftWarps * 32)
      reinterpret_cast<uint4*>(pbuf)[i] = make_uint4(0, 0, 0, 0);
    if (RP < 128) spread_s[st] = spread(st >> 4, st & 15);
    named_bar(1, kSoftWarps * 32);
    pdl_wait();
    bool have_item = take(0);
    int item = 0;
    // a thread's keys are coded and stored in parts: registers (RP = 128 all at once: 231 us for the chunk, two parts 218)
    constexpr int PARTS = RP == 128 ? 4 : 1, KP = KW / PARTS;
    constexpr int NE = KW / 16;                       // 16-key groups of a thread (one scale each)
    constexpr int NL = RP == 128 ? 1 : NE;            // sums of p: by 16 keys where rows must not depend on RP
    float l_was[NL] = {}, m_was = 0.f;                // of the item before
    bool bad_was = false;
    // Ends the item before: (m, l) and o = (o0 + o1 / 16) / kUnit.  Loads of 16
    // lanes leave w0's and w1's sums of a row and a column in one thread (rows lane
    // / 4 and 8 more, two columns of 8).
    auto finish = [&]() {
      const Item& x = items[(item - 1) % kItems];
      wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
#pragma unroll
      for (int u = 0; u < NL; ++u) l_r[(grp * NL + u) * RP + lane] = l_was[u];
      if (grp == 0) bad_s[row] = bad_was ? 1.f : 0.f;
      named_bar(1, kSoft);
      tc_fence_after();
      if (grp == 0 && row < x.nrows && a.n_splits > 1 && !*fail) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < NG * NL; ++e) sum += l_r[e * RP + lane];
        __stcg(&a.part_ml[x.slot + row], make_float2(m_was, sum));
      }
      if (quad * RQ < x.nrows) {
        constexpr int NR = RQ / 8;                    // rows of a thread
        float* po[NR];
        uint16_t* dst[NR];
        float sum[NR];
        bool have[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = quad * RQ + lane / 4 + 8 * i;
          have[i] = r < x.nrows && !*fail;
          po[i] = a.part_o + (x.slot + r) * D + lane % 4 * 2;
          if (a.n_splits == 1) {
            const int pos = a.by_G(x.r0 + r);
            dst[i] = a.out + ((x.out0 + pos) * (a.c.n_kv_heads * a.G) + x.h * a.G + (x.r0 + r - pos * a.G)) * D + lane % 4 * 2;
            sum[i] = 0.f;
#pragma unroll
            for (int e = 0; e < NG * NL; ++e) sum[i] += l_s[e * RP + r];
            if (bad_s[r] != 0.f && sum[i] != 0.f) sum[i] = __int_as_float(0x7fffffff);    // a NaN query (no key: zero)
          }
        }
        // 64 columns of eight rows at a time, or 32 of 16 or (w0 and w1 summed already) 32
        auto readout = [&](auto direct) {
          constexpr int NC = NR == 1 ? 64 : 32, NK = NC / 8, NO = NR == 1 ? 1 : 2;
#pragma unroll 1
          for (int c0 = cg * (D / 2); c0 < (cg + 1) * (D / 2); c0 += NC) {
            uint32_t o[NO][NC / 2];
#pragma unroll
            for (int i = 0; i < NO; ++i) tmem_ld16x256(t_lane + (static_cast<uint32_t>(16 * i) << 16) + c0, o[i]);
#pragma unroll
            for (int i = 0; i < NO; ++i) tmem_ld_wait_for(o[i]);
            float2 y[NR][NK];
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
              for (int i = 0; i < NR; ++i) {
                const int e0 = NR == 4 ? 0 : 4 * k + 2 * i, e1 = NR == 1 ? 4 * k + 2 : e0;
                const auto sum_of = [&](int z) {
                  if (NR == 4) return __uint_as_float(o[NO > 1 ? i >> 1 : 0][4 * k + 2 * (i & 1) + z]) * (1.f / kUnit<RP>);
                  return fmaf(__uint_as_float(o[NO - 1][e1 + z]), 1.f / (kUnit<RP> * kLow), __uint_as_float(o[0][e0 + z]) * (1.f / kUnit<RP>));
                };
                y[i][k] = make_float2(sum_of(0), sum_of(1));
              }
#pragma unroll
            for (int i = 0; i < NR; ++i)
              if (have[i]) {
#pragma unroll
                for (int k = 0; k < NK; ++k)
                  if constexpr (decltype(direct)::value)
                    *reinterpret_cast<uint32_t*>(dst[i] + c0 + 8 * k) =
                        sum[i] == 0.f ? 0u : pack_bf16x2(y[i][k].x / sum[i], y[i][k].y / sum[i]);
                  else
                    __stcg(reinterpret_cast<float2*>(po[i] + c0 + 8 * k), y[i][k]);
              }
            __syncwarp();
          }
        };
        if (a.n_splits == 1)
          readout(std::true_type{});
        else
          readout(std::false_type{});
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free);
        mbar_arrive(&it_empty[(item - 1) % kItems]);
      }
    };
    // An item is ended between the weights of the next one's first block and their
    // store, which hides the wait for its last P V (one pass more ends the last).
    // All warps stop together, also after a timeout that only some have seen.
    for (;; ++item) {
      const bool more = !bar_red_or(2, kSoft, !have_item);
      if (!more && item == 0) break;
      const Item& x = items[item % kItems];
      const int nrows = more ? x.nrows : 0, x_lo = x.lo, x_hi = x.hi, blk0 = x.blk0, nb = more ? x.nb : 1;
      const bool half_used = rh * 32 < nrows;         // these warps hold rows
      const bool mine = row < nrows;
      const int row_lo = max(x_lo, a.window > 0 ? p - a.window + 1 : 0), row_hi = min(x_hi, p);
      const float* ks = ks_s + (item % kItems) * kMaxScales;
      const float* vs = vs_s + (item % kItems) * kMaxScales;
      if (more) wait(&sc_full[item % kItems], (item / kItems) & 1);
      float mref = kNoKey, l[NL] = {};
      for (int j = 0; j < nb; ++j, ++g) {
        const int kb = (blk0 + j) << kLgBlk, key0 = kb + grp * KW;
        float s[KW], f[NE], vsc[NE], cand = -INFINITY;
        uint32_t w0[KP / 4], w1[KP / 4], w2[RP == 128 ? KP / 4 : 1];   // of a part
        if (more) {
#pragma unroll
          for (int u = 0; u < NE; ++u) {
            const int e = ((j << kLgBlk) + grp * KW + 16 * u) >> lg_bt;
            vsc[u] = vs[e];
            f[u] = fminf(fmaxf(qs * ks[e], 1e-30f), kMostFactor);
          }
          wait(&s_full[g % SB], (g / SB) & 1);
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
          }
          if (j == 0 || bar_red_or(1, kSoft, mine && cand > mref + kLazy)) {
            red_r[grp * RP + lane] = cand;
            named_bar(1, kSoft);
            float bm = red_r[lane];
#pragma unroll
            for (int e = 1; e < NG; ++e) bm = fmaxf(bm, red_r[e * RP + lane]);
            float al = 1.f;
            if (mine && bm > mref + kLazy) {
              al = ex2(mref - bm);              // 0 while the row had no key
              mref = bm;
#pragma unroll
              for (int u = 0; u < NL; ++u) l[u] *= al;
              if (fabsf(bm) > kFar) l[0] = __int_as_float(0x7fffffff);
            }
            if (j > 0) {
              // the running sums of the rows that moved (all earlier P V done)
              if (grp == 0) alpha_s[row] = al;
              wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
              named_bar(1, kSoft);
              tc_fence_after();
              al = o_row < nrows ? alpha_s[o_row] : 1.f;
              if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll 1
                for (int c = cg * (D / 2); c < (cg + 1) * (D / 2); c += 32) {
                  uint32_t r8[4][8];
#pragma unroll
                  for (int e = 0; e < 4; ++e) tmem_ld8_nowait(t_lane + c + 8 * e, r8[e]);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int z = 0; z < 8; ++z) r8[e][z] = __float_as_uint(__uint_as_float(r8[e][z]) * al);
                    tmem_st8(t_lane + c + 8 * e, r8[e]);
                  }
                }
                tmem_st_wait();
              }
            }
          }
        }
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          if (more && half_used) {
            float4 add;                               // of four keys
#pragma unroll
            for (int e = 0; e < KP; e += 2) {
              const int c = part * KP + e;
              if (RP < 128 && c % 4 == 0)
                add = reinterpret_cast<const float4*>(spread_s)[spread_order(key0 + (c & ~15)) * 4 + c % 16 / 4];
              const float fa = f[c >> 4], vb = fmaxf(vsc[c >> 4], 0.f) * kUnit<RP>;
              const float p0 = ex2(fmaf(s[c], fa, -mref)), p1 = ex2(fmaf(s[c + 1], fa, -mref));
              l[NL > 1 ? c >> 4 : 0] += p0;
              l[NL > 1 ? c >> 4 : 0] += p1;
              if constexpr (RP == 128) {
                const __half2 x = __floats2half2_rn(p0 * vb, p1 * vb);
                const uint32_t c0 = *reinterpret_cast<const uint32_t*>(&x) & 0xff00ff00u;
                const __half2 rest = __hsub2(x, *reinterpret_cast<const __half2*>(&c0));
                const uint32_t c1 = *reinterpret_cast<const uint32_t*>(&rest) & 0xff00ff00u;
                const __half2 last = __hsub2(rest, *reinterpret_cast<const __half2*>(&c1));
                const uint32_t c2 = *reinterpret_cast<const uint32_t*>(&last) + 0x00800080u;
                // four keys a word: the upper bytes of two pairs
                w0[e >> 2] = c & 2 ? __byte_perm(w0[e >> 2], c0, 0x7531) : c0;
                w1[e >> 2] = c & 2 ? __byte_perm(w1[e >> 2], c1, 0x7531) : c1;
                w2[e >> 2] = c & 2 ? __byte_perm(w2[e >> 2], c2, 0x7531) : c2;
              } else {
                const __half2 x = __floats2half2_rn(fmaf(p0, vb, c & 2 ? add.z : add.x), fmaf(p1, vb, c & 2 ? add.w : add.y));
                uint16_t c0, c1;
                uint32_t back;
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c0) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c0));
                const __half2 rest = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(kLow));
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c1) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
                if ((c & 2) == 0) {
                  w0[e >> 2] = c0;
                  w1[e >> 2] = c1;
                } else {
                  w0[e >> 2] |= static_cast<uint32_t>(c0) << 16;
                  w1[e >> 2] |= static_cast<uint32_t>(c1) << 16;
                }
              }
            }
          }
          if (part == 0) {
            if (j == 0 && item > 0) finish();
            // the P buffer was last read by P V of block g - PB
            if (more && g >= PB) wait(&pv_done[(g - PB) & 1], ((g - PB) >> 1) & 1);
          }
          if (more && mine) {
            uint8_t* pp = pbuf + (g % PB) * C::kPTile;
#pragma unroll
            for (int u = 0; u < NE / PARTS; ++u) {
              const int at = NE * grp + part * (NE / PARTS) + u;
              *reinterpret_cast<uint4*>(pp + swz128(p_row, at)) = make_uint4(w0[4 * u], w0[4 * u + 1], w0[4 * u + 2], w0[4 * u + 3]);
              *reinterpret_cast<uint4*>(pp + (RP == 128 ? kPBytes + swz128(p_row, at) : swz128(p_row + RQ, at))) =
                  make_uint4(w1[4 * u], w1[4 * u + 1], w1[4 * u + 2], w1[4 * u + 3]);
              if constexpr (RP == 128)
                *reinterpret_cast<uint4*>(pp + 2 * kPBytes + swz128(p_row, at)) =
                    make_uint4(w2[4 * u], w2[4 * u + 1], w2[4 * u + 2], w2[4 * u + 3]);
            }
          }
        }
        if (!more) break;
        // ---- value rows no row of the item may use: zero them (two threads per key)
        {
          const int key = kb + (st >> 1);
          if (key < x_lo || key > x_hi || vs[((j << kLgBlk) + (st >> 1)) >> lg_bt] < 0.f) {
            const int u = value_unit(g);
            wait(&u_full[u % NU], (u / NU) & 1);
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
      if (!more) break;
#pragma unroll
      for (int u = 0; u < NL; ++u) l_was[u] = l[u];
      m_was = mref;
      bad_was = bad_q;
      have_item = take(item + 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the splits of a row, V
// dims a thread.  Four sums are kept by split index mod 4, each in ascending order,
// and added in the order of the absolute index: by one thread (P = 1) or by four
// (P = 4), which changes no bit, nor do V and U.  Splits without a key of the row
// add nothing at fixed places, so the order does not depend on where the list of
// splits starts.  The time is a chain of memory latencies: the sequence's length,
// the references and the first P U splits' partials are all asked for at once,
// those beyond the sequence's last split (whatever the workspace holds) are dropped.
template <int P, int V, int U>
__global__ void __launch_bounds__(256) qattn_combine_kernel(const __grid_constant__ QAttnArgs a) {
  constexpr int NT = 256 / P, NA = 4 / P;
  constexpr int kTile = P * U < 32 ? 32 : P * U;   // splits whose weights are held at a time
  constexpr int kRows = NT * V / 128 < 1 ? 1 : NT * V / 128;
  __shared__ float w_s[kRows][kTile], l_s[kRows][kTile], m_s[8], d_s[P > 1 ? P : 1][P > 1 ? NT : 1];
  __shared__ int n_s[8];
  __shared__ float y_s[P > 1 ? P : 1][P > 1 ? NT * V : 1];
  pdl_trigger();
  const int D = a.c.dim, lr = min(D / V, NT), lg = 31 - __clz(lr);   // threads of a row and sum
  const int p = threadIdx.x / NT, el = threadIdx.x % NT, rr = el >> lg;
  const int me = p * lr + (el & (lr - 1)), all = P * lr;             // among the row's threads
  const int64_t flat = (static_cast<int64_t>(blockIdx.x) * NT + el) * V;
  const int at = static_cast<int>(flat >> (D == 256 ? 8 : 7)), c = static_cast<int>(flat) & (D - 1);
  const bool have = at < a.B * a.c.n_kv_heads * a.rows;
  const int bh = have ? at / a.rows : 0, r = have ? at - bh * a.rows : 0, b = bh / a.c.n_kv_heads, h = bh - b * a.c.n_kv_heads;
  const int64_t slot0 = static_cast<int64_t>(bh) * a.n_splits * a.rows + r;
  const int L = __ldcg(&a.c.seq_lens[b]);                   // (final: see the split kernel's start)
  const SeqKeys k = seq_keys(a, L);
  const int64_t step = static_cast<int64_t>(a.rows) * D;
  const float* po = a.part_o + slot0 * D + p * step + c;
  float x[U][V];
  auto load = [&](int s0) {
    const float* at_s = po + s0 * step;
#pragma unroll
    for (int u = 0; u < U; ++u, at_s += P * step) {
      if (have && s0 + P * u + p < a.n_splits) {
        if (V == 4) {
          const float4 z = __ldcg(reinterpret_cast<const float4*>(at_s));
          x[u][0] = z.x;
          x[u][V > 1 ? 1 : 0] = z.y;
          x[u][V > 2 ? 2 : 0] = z.z;
          x[u][V > 3 ? 3 : 0] = z.w;
        } else {
          x[u][0] = __ldcg(at_s);
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[u][v] = 0.f;
      }
    }
  };
  auto load_tile = [&](int s0) {                   // references into w_s, sums into l_s
    for (int s = me; s < kTile; s += all) {
      const float2 ml = have && s0 + s < a.n_splits ? __ldcg(&a.part_ml[slot0 + static_cast<int64_t>(s0 + s) * a.rows])
                                                    : make_float2(kNoKey, 0.f);
      w_s[rr][s] = ml.x;
      l_s[rr][s] = ml.y;
    }
  };
  pdl_wait();
  load(0);
  const float qs = have ? __ldcg(&a.q_scale[at]) : 0.f;
  load_tile(0);
  float M = kNoKey;
  for (int s0 = 0; s0 < k.splits; s0 += kTile) {
    if (s0 > 0) load_tile(s0);                     // each thread reads back what it wrote
    for (int s = me; s < min(kTile, k.splits - s0); s += all) M = fmaxf(M, w_s[rr][s]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    m_s[warp] = M;
    n_s[warp] = k.splits;
  }
  __syncthreads();
  // (a row's threads are whole warps: lr / 32 next to each other for each sum)
  const int wr = lr >> 5, w0 = rr * wr;
#pragma unroll
  for (int q = 0; q < P; ++q)
    for (int i = 0; i < wr; ++i) M = fmaxf(M, m_s[q * (NT / 32) + w0 + i]);
  float acc[NA][V], den[NA];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    den[q] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[q][v] = 0.f;
  }
  int most = k.splits;                             // of the CTA's rows
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, n_s[i]);
  for (int s0 = 0; s0 < most; s0 += kTile) {
    const int ns = min(kTile, k.splits - s0);
    if (most > kTile) {
      __syncthreads();
      load_tile(s0);
    }
    for (int s = me; s < ns; s += all) {
      const float m = w_s[rr][s];
      w_s[rr][s] = m <= kNoKey ? 0.f : exp2f(m - M);
    }
    __syncthreads();
    for (int u0 = 0; u0 < ns; u0 += P * U) {
      if (s0 + u0 > 0) load(s0 + u0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = u0 + P * u + p;
        const float w = s < ns ? w_s[rr][s] : 0.f;
        if (w > 0.f) {                             // (a split without keys of the row has no sums)
          den[u % NA] = fmaf(w, l_s[rr][s], den[u % NA]);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[u % NA][v] = fmaf(w, x[u][v], acc[u % NA][v]);
        }
      }
    }
  }
  // the four sums in the order of the absolute split index
  const int turn = k.splits ? a.by_split(k.lo / kBlk) & 3 : 0;
  auto ordered = [&](float q0, float q1, float q2, float q3) {
    const float z0 = turn == 0 ? q0 : turn == 1 ? q3 : turn == 2 ? q2 : q1;
    const float z1 = turn == 0 ? q1 : turn == 1 ? q0 : turn == 2 ? q3 : q2;
    const float z2 = turn == 0 ? q2 : turn == 1 ? q1 : turn == 2 ? q0 : q3;
    const float z3 = turn == 0 ? q3 : turn == 1 ? q2 : turn == 2 ? q1 : q0;
    return ((z0 + z1) + z2) + z3;
  };
  float y[V], l;
  if (P == 1) {
    l = ordered(den[0], den[1 % NA], den[2 % NA], den[3 % NA]);
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = ordered(acc[0][v], acc[1 % NA][v], acc[2 % NA][v], acc[3 % NA][v]);
  } else {
    d_s[p][el] = den[0];
#pragma unroll
    for (int v = 0; v < V; ++v) y_s[p][v * NT + el] = acc[0][v];
    __syncthreads();
    if (p > 0) return;
    l = ordered(d_s[0][el], d_s[1 % P][el], d_s[2 % P][el], d_s[3 % P][el]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * NT + el;
      y[v] = ordered(y_s[0][i], y_s[1 % P][i], y_s[2 % P][i], y_s[3 % P][i]);
    }
  }
  if (!have) return;
#pragma unroll
  for (int v = 0; v < V; ++v) y[v] = l == 0.f ? 0.f : qs == qs ? y[v] / l : qs;     // no key: zero
  const int pos = a.by_G(r);
  uint16_t* dst = a.out + ((static_cast<int64_t>(b) * a.n + pos) * (a.c.n_kv_heads * a.G) + h * a.G + (r - pos * a.G)) * D + c;
  if (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y[0], y[1 % V]), pack_bf16x2(y[2 % V], y[3 % V]));
  else
    *dst = f32_to_bf16(y[0]);
}

template <int P, int V, int U>
cudaError_t launch_combine(const QAttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.c.n_kv_heads * a.rows, per = 256 / P * V;
  return launch_k(qattn_combine_kernel<P, V, U>, dim3(static_cast<unsigned>((rows * a.c.dim + per - 1) / per)), dim3(256), 0, st, a);
}

template <int D, int RP>
cudaError_t launch_one(int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                       const QAttnArgs& a, cudaStream_t st) {
  auto kern = qattn_kernel<D, RP>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, Cfg<D, RP>::kSmem, allowed);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(grid), dim3(kThreads), Cfg<D, RP>::kSmem, st, tk, tv, a);
}

template <int D>
cudaError_t launch_dim(int rp, int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                       const QAttnArgs& a, cudaStream_t st) {
  if (rp == 32) return launch_one<D, 32>(grid, tk, tv, a, st);
  if (rp == 128) return launch_one<D, 128>(grid, tk, tv, a, st);
  return launch_one<D, 64>(grid, tk, tv, a, st);
}

}  // namespace

cudaError_t launch_qcache_attn(const QAttnArgs& a, cudaStream_t st) {
  const int D = a.c.dim, rp = qattn_rows(a.n, a.rows);
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
  if (a.n_splits == 1) return cudaSuccess;     // the results are out
  // few splits: one thread has them all in flight; more: four threads; very many of
  // few rows: one dim a thread, for more CTAs (131k tokens, 36 rows of 129 splits: 10.5
  // us against 20 for four dims; 8 sequences of 33: 16 against 64)
  if (a.n_splits <= 4) return launch_combine<1, 4, 4>(a, st);
  if (a.n_splits <= 8) return launch_combine<1, 4, 8>(a, st);
  const int64_t all = static_cast<int64_t>(a.B) * a.c.n_kv_heads * a.rows;
  if (a.n_splits > 40 && all * D <= 4 * sms * 64) return launch_combine<4, 1, 32>(a, st);
  return launch_combine<4, 4, 8>(a, st);
}

}  // namespace sv
