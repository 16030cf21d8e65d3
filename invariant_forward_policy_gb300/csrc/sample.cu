// Sampling a token from a row of logits, and the logprob of a given token under the same
// truncated distribution.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §2 asks that a rollout's discrete choices
// and its logprobs come out the same in any batch and in the training recompute; here that holds
// for a sampled choice too.  For a row x[V] at temperature T the token masses are
// w_i = exp((x_i - max x) / T), tokens are ordered by (x descending, index ascending), and the
// kept set is a prefix of that order cut in turn by min-p (w_i >= min_p), top-k (the first k) and
// top-p (the shortest prefix with at least p of the mass that is left).  With u in [0, 1) the
// token is the first in index order whose running kept mass exceeds u times the kept mass S, and
// its logprob is (x_i - max x) / T - ln S.
//
// A token choice sits next to a border of a running sum: a relative error e of the masses moves
// the choice in about 2 e sqrt(N) of the rows over N tokens of like mass, so fp32 masses (6e-8)
// would change one row in 25,000 at N = 1e5, and top-p cuts likewise.  The masses are therefore
// fixed-point integers of about 2^56 for the largest: 2^(j/64) from a table (Tang's table-driven
// exponential, ACM TOMS 15, 1989) times a cubic in the remainder, whose argument is reduced in two
// floats, about 5e-10 relative.  Integer sums have no order, every quantity below is defined by
// them alone, and so a row's bits depend neither on how many CTAs share it, nor on which of the
// ways to its cut below was taken, nor on the batch.
//
// A row is shared by a cluster of 1, 2, 4 or 8 CTAs, each with a contiguous share that its passes stream
// (the first from HBM, the others from L2).  The first pass finds the maximum.  Then
//  - nothing cut but by min-p: one pass sums the masses;
//  - top_k up to 1024: in each CTA the k'-th largest of the threads' own maxima (known from the read),
//    k' (384 at most) somewhat above the CTA's share of k, lets through somewhat more than k' logits; one
//    CTA orders what the CTAs let through and does the rest, provided that the k-th of them is not below
//    any CTA's bound;
//  - top-p: a histogram of counts and mean depths (bins of 1/32 octave) predicts where the cut is; one
//    pass sums the masses and lists the logits next to the prediction, and one CTA orders the list
//    and finds the cut, exactly;
//  - anything else (larger top_k or k', top_k or top-p over logits beyond 2^13 octaves, a list that overflows, a
//    missed prediction, u = 0): one CTA finds the cut from global memory by histograms with masses, on octaves
//    first and on the float's bits then, until the bin fits the sort or holds equal values only, whose
//    first few by index are counted out.
// The draw finds the CTA, then the warp, then the token whose running mass crosses u S.
//
// What bounds it.  Large batches: the chain of a CTA's own passes (read, barrier, masses from L2, barrier) with two
// CTAs an SM to overlap; neither memory nor issue is full (HBM at 42 % and issue 42 % active at temperature alone,
// issue 53 % with top-p).  Reading the logits once would take 39 us for
// 512 fp32 rows of 129280 and 78 us for 2048 bf16 rows of them or 4096 fp32 rows of 32000.  At temperature
// alone the calls take 96, 242 and 168 us (23 instructions a logit), with top_k 180 us for the bf16 rows (the second
// pass only compares), with top-p 492 and 378 us for the last two: 49 instructions a logit (12 of them the counts, two
// shared atomics among them), 24,000 warp instructions a row beside them, and a dozen barriers.  Small calls: that
// chain alone, 12.0 us for one row of 4096 with top-k (launch and exit are 2.5 of them), 14.5 us for 16 rows of
// 129280 at temperature alone, 29 us with top-p.  The last way costs a row of 129280 some 180 us.  Measured and
// dropped: rows resident in shared memory (the passes after the first ran no faster than from L2, and fewer rows
// were in flight); 256 threads and four CTAs an SM, or three of 512 (spills); loads of the next batch under the work
// of this one; finer bins with counts alone (longer lists); packed two-element arithmetic (the same issue slots).
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <string>
#include <type_traits>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace bi {

typedef unsigned long long u64;
typedef unsigned __int128 Sum;  // of masses

constexpr int kSmpThreads = 512;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpBins = 1024;             // bins of top-p's counts (1/32 octave); the last one is open
constexpr int kSmpMaxBins = 256;           // bins of the threads' maxima
constexpr int kSmpMassBins = kSmpThreads;          // bins of a histogram with masses (count and five 12-bit limbs)
constexpr int kSmpMassShift = 2;           // 32 octaves of 1/64 over them
constexpr int kSmpMassBits = 9;            // log2 of them
constexpr int kSmpList = 2048;             // candidates that one CTA orders
constexpr int kSmpMaxK = 1024;             // top_k up to which the kept set goes straight to the list
constexpr int kSmpMaxShareK = kSmpThreads * 3 / 4;        // and each CTA's bound is the k'-th maximum for k' up to this
constexpr int kSmpMaxV = 1 << 18;
// The table's mantissa of 1 is 380000000: about the largest for which its products with 2^(f/64) - 1 round
// by the magic number (2 * 380000000 * (2^(1/128) - 1) is below 2^22).
constexpr int kSmpFrac = 27;               // mass = mantissa (below 2^29.6) << 27 >> octaves below the largest
                                           // (a small unit: 1e5 small masses, each cut by half a unit on average,
                                           // must not move the running sum by as much as one of them)
constexpr int kSmpTabLanes = 16;           // table copies: 8-byte reads of a half-warp have no bank conflict
constexpr int kSmpSmem = 64 * kSmpTabLanes * 8 + 8192 + kSmpList * 8;  // table, counts, list
constexpr float kSmpMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to an integer in the low bits
constexpr int kSmpMagicBits = 0x4B400000;

// round(380000000 * 2^(j / 64))
__constant__ uint32_t kExp2Tab[64] = {
    380000000, 384137929, 388320916, 392549454, 396824037, 401145168, 405513352, 409929103,
    414392938, 418905382, 423466962, 428078215, 432739681, 437451907, 442215446, 447030857,
    451898704, 456819558, 461793997, 466822604, 471905969, 477044688, 482239364, 487490606,
    492799031, 498165260, 503589924, 509073659, 514617108, 520220921, 525885755, 531612276,
    537401154, 543253069, 549168707, 555148762, 561193935, 567304937, 573482482, 579727297,
    586040114, 592421672, 598872721, 605394018, 611986326, 618650420, 625387082, 632197101,
    639081276, 646040414, 653075333, 660186857, 667375821, 674643067, 681989449, 689415827,
    696923073, 704512068, 712183701, 719938873, 727778493, 735703482, 743714767, 751813290};

// Device pointers of one call.
struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V, share;  // share: logits per CTA, a multiple of 8
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int64_t n_params;
  const int32_t* param_row;
  bool bf16;              // logits are bf16
  const float* u;         // draw
  int64_t u_ld, u_rows;   // row stride and rows of u
  const int32_t* u_row;
  const int32_t* ids_in;  // score (NULL: draw)
  int32_t* ids_out;
  float* lp_out;
  const int32_t* dst;     // results of row t go to index dst[t] (or t)
  int* status;
};

struct SmpCut {  // an element is kept iff its key is larger, or equal and its index not above idx
  uint32_t key;
  int32_t idx;   // -1: no cut was found
  Sum mass;      // mass through the cut
};
struct SmpFind { // a bin and what lies before it and in it
  int32_t bin;
  uint32_t before, inside;
  Sum before_mass;
};

// Static shared memory of one CTA.
struct SmpShared {
  // the row's parameters, by one thread
  double log_min_p;               // T ln(min_p)
  float c_hi, c_lo, r_hi, r_lo;   // 64 log2(e) / T and 1 / T, each in two floats
  float floor_abs, floor_rel;     // the mass functions' lowest arguments
  float p, u, min_p, x_id;
  int32_t k_eff, id, ok;
  // the warps' values
  float wmax[kSmpWarps], wmin[kSmpWarps];
  Sum wsum[kSmpWarps], wsum2[kSmpWarps];
  uint32_t wlow[kSmpWarps];       // of sums of list entries, with whigh
  u64 whigh[kSmpWarps];
  uint32_t wcnt[kSmpWarps];
  // written by the cluster's CTAs, each at its rank: what is needed of all of them is then at hand locally
  float cta_max[8], cta_bound[8];
  Sum cta_sum[8], cta_sum2[8];
  uint32_t cta_n[8];
  float x_lo, x_hi;               // top-p's prediction
  SmpCut cut;
  // this CTA's own
  uint32_t list_n;
  float x_cut;
  SmpFind find;
  Sum total, total2;
  int32_t pos;
};

BI_DEV uint32_t smp_key(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
BI_DEV float smp_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
BI_DEV float smp_max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
BI_DEV float smp_max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// floor(f S) for 0 <= f < 1 and S < 2^76, exactly; *rest: whether f S is no integer.
BI_DEV Sum smp_mul_floor(float f, Sum S, bool* rest) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const uint32_t mant = ex ? ((b & 0x7fffffu) | 0x800000u) : (b & 0x7fffffu);
  const int sh = 150 - (ex ? ex : 1);  // f = mant 2^-sh, sh >= 24
  const Sum v = S * mant;              // below 2^100
  const Sum q = sh < 128 ? v >> sh : 0;
  *rest = v != (sh < 128 ? q << sh : 0);
  return q;
}
// Sums below 2^96 between lanes
BI_DEV Sum smp_shfl_up(Sum v, int o) {
  const u64 l = __shfl_up_sync(0xffffffffu, (u64)v, o);
  const uint32_t h = __shfl_up_sync(0xffffffffu, (uint32_t)(v >> 64), o);
  return (Sum)h << 64 | l;
}
BI_DEV Sum smp_shfl_xor(Sum v, int o) {
  const u64 l = __shfl_xor_sync(0xffffffffu, (u64)v, o);
  const uint32_t h = __shfl_xor_sync(0xffffffffu, (uint32_t)(v >> 64), o);
  return (Sum)h << 64 | l;
}
BI_DEV Sum smp_warp_scan(Sum v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum y = smp_shfl_up(v, o);
    if (lane >= o) v += y;
  }
  return v;
}
BI_DEV Sum smp_warp_total(Sum upto) {  // of an inclusive scan: the last lane's
  const u64 l = __shfl_sync(0xffffffffu, (u64)upto, 31);
  const uint32_t h = __shfl_sync(0xffffffffu, (uint32_t)(upto >> 64), 31);
  return (Sum)h << 64 | l;
}
BI_DEV Sum smp_warp_sum(Sum v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += smp_shfl_xor(v, o);
  return v;
}

// x - m and its rounding error
BI_DEV float smp_diff(float x, float m, float* err) {
  const float d = __fsub_rn(x, m);
  const float b = __fsub_rn(d, x);
  *err = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
  return d;
}

// A row's mass function.  Both forms split 64 log2(e) x / T into an integer k and a remainder f, |f| <= 1/2
// (in units of 1/64 octave, to 2^-25): the integer by adding a large constant, the remainder by fused
// multiply-adds against c = 64 log2(e) / T in two floats.  ABS takes x itself and serves rows whose
// largest |64 log2(e) m / T| is below 2^19; the other takes x - m with its rounding error (six more
// operations) and serves the rest.  The form is the row's, so it changes no bits between calls.
template <bool ABS>
struct SmpMass {
  // 2^(f/64) - 1: the series to the third power of f ln2 / 64 (below 0.0055; the next term is 4e-11)
  static constexpr float a1 = 0.0108304247f, a2 = 5.86490496e-05f, a3 = 2.11731372e-07f;
  float m, c_hi, c_lo;
  float floor_;  // for k_of, ABS: logits below it are raised to it (-2^20 / c); else: x - m at or below it has no mass
                 // (-4096 / c)
  int k_top;     // k of the maximum
  int oct_top;   // its octave
  int shift0;    // (shift0 - bits of the rounded sum) >> 6 = 32 - kSmpFrac + octaves below the top one
  BI_DEV void init(float m_, const SmpShared& sh) {
    m = m_;
    c_hi = sh.c_hi;
    c_lo = sh.c_lo;
    floor_ = ABS ? sh.floor_abs : sh.floor_rel;
    k_top = ABS ? k_of(m) : 0;
    oct_top = k_top >> 6;
    shift0 = (oct_top + 32 - kSmpFrac) * 64 + 63 + kSmpMagicBits;
  }
  // k of an element; lower elements than the masses reach may have any k far below k_top
  BI_DEV int k_of(float x) const {
    if (ABS) return __float_as_int(__fmaf_rn(fmaxf(x, floor_), c_hi, kSmpMagic)) - kSmpMagicBits;
    return __float_as_int(__fmaf_rn(fmaxf(__fsub_rn(x, m), floor_), c_hi, kSmpMagic)) - kSmpMagicBits;
  }
  // x = (k + f) / c with k in the low bits of the rounded sum q.  2^(k/64) is a table entry and a shift by octaves;
  // the entry's product with g = 2^(f/64) - 1 is rounded to an integer by the magic number (which the table's
  // integers lack).  The mass is (mantissa 2^32) >> s; a shift of 64 or more gives 0, as it does for every logit that
  // is too low for the rounded sum, -inf among them.
  BI_DEV u64 mass(float x, const uint2* tab) const {
    float q, f;
    if (ABS) {
      q = __fmaf_rn(x, c_hi, kSmpMagic);
      f = __fmaf_rn(x, c_hi, __fsub_rn(kSmpMagic, q));
      f = __fmaf_rn(x, c_lo, f);
    } else {
      float dl;
      float d = smp_diff(x, m, &dl);
      if (!(d > floor_)) {  // -inf among them
        d = floor_;
        dl = 0.f;
      }
      q = __fmaf_rn(d, c_hi, kSmpMagic);
      f = __fmaf_rn(d, c_hi, __fsub_rn(kSmpMagic, q));
      f = __fmaf_rn(d, c_lo, f);
      f = __fmaf_rn(dl, c_hi, f);
    }
    const float g = __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, a3, a2), a1));
    const int bits = __float_as_int(q);
    const uint2 t = tab[(bits & 63) * kSmpTabLanes];
    const uint32_t M = t.x + (uint32_t)__float_as_int(__fmaf_rn(__uint_as_float(t.y), g, kSmpMagic));
    u64 w;
    asm("shr.b64 %0, %1, %2;" : "=l"(w) : "l"((u64)M << 32), "r"(((uint32_t)shift0 - (uint32_t)bits) >> 6));
    return w;
  }
};

// v = (h + l) 2^e to 48 bits: h 24 bits in [2^23, 2^24), l the next 24
BI_DEV void smp_split(Sum v, float& h, float& l, int& e) {
  const bool wide = (u64)(v >> 64) != 0ull;  // below 2^96
  const int z = wide ? __clzll((long long)(v >> 32)) : __clzll((long long)v);
  const u64 n = (wide ? (u64)(v >> 32) : (u64)v) << z;
  h = (float)(uint32_t)(n >> 40);
  l = __fmul_rn((float)((uint32_t)(n >> 16) & 0xffffffu), 0x1p-24f);
  e = (wide ? 72 : 40) - z;
}
// ln of a kept token's probability: (x - m) / T - ln(S / W), W the mass of the maximum; both terms in two
// floats until the last sum.
BI_DEV float smp_logprob(float x, float m, float r_hi, float r_lo, Sum S, Sum W) {
  float dl;
  float d = smp_diff(x, m, &dl);
  if (d == -INFINITY) {  // x - m beyond fp32, which (x - m) / T need not be: of the halves
    d = smp_diff(0.5f * x, 0.5f * m, &dl);
    r_hi *= 2.f;
    r_lo *= 2.f;
  }
  const float ah = __fmul_rn(d, r_hi);
  if (ah == -INFINITY) return ah;  // a logit of the lowest value at T < 1: the logprob is beyond fp32
  const float al = __fadd_rn(__fmaf_rn(d, r_hi, -ah), __fmaf_rn(d, r_lo, __fmul_rn(dl, r_hi)));
  float sh, sl, wh, wl;
  int es, ew;
  smp_split(S, sh, sl, es);
  smp_split(W, wh, wl, ew);
  // S / W = (qh + ql) 2^e with qh in [0.75, 1.5)
  float qh = __fdiv_rn(sh, wh);  // in (1/2, 2)
  float ql = __fdiv_rn(__fadd_rn(__fmaf_rn(-qh, wh, sh), __fmaf_rn(-qh, wl, sl)), wh);
  int e = es - ew;
  if (qh >= 1.5f || qh < 0.75f) {
    const float by = qh >= 1.5f ? 0.5f : 2.f;
    e += qh >= 1.5f ? 1 : -1;
    qh = __fmul_rn(qh, by);
    ql = __fmul_rn(ql, by);
  }
  const float ln2h = 45426.f / 65536.f, ln2l = 1.4286068203e-6f;  // e * ln2h is exact
  const float s = __fsub_rn(__fmaf_rn(-(float)e, ln2h, ah), logf(qh));
  return __fadd_rn(s, __fsub_rn(__fsub_rn(al, __fmul_rn((float)e, ln2l)), __fdiv_rn(ql, qh)));
}

// ln of the probability of token (i, x) and the write of a row's results, by one thread.
struct SmpOut {
  const SampleArgs& a;
  int64_t row;
  BI_DEV void write(int32_t id, float lp) const {
    const int64_t o = a.dst ? (int64_t)a.dst[row] : row;
    if (!a.ids_in && a.ids_out) a.ids_out[o] = id;
    if (a.lp_out) a.lp_out[o] = lp;
  }
  template <bool ABS>
  BI_DEV void token(const SmpMass<ABS>& ms, const SmpShared& sh, const uint2* tab, int32_t id, float x, Sum S) const {
    write(id, smp_logprob(x, ms.m, sh.r_hi, sh.r_lo, S, ms.mass(ms.m, tab)));
  }
};

// ceil(p S), at least 1: the mass at which top-p stops
BI_DEV Sum smp_top_p_target(float p, Sum S) {
  if (!(p > 0.f)) return 1;
  bool rest;
  const Sum q = smp_mul_floor(p, S, &rest);
  return q + (rest || q == 0 ? 1 : 0);
}
// floor(u S) + 1: the running mass that the drawn token is the first to reach
BI_DEV Sum smp_draw_target(float u, Sum S) {
  bool rest;
  return smp_mul_floor(u, S, &rest) + 1;
}
// ceil(a / b) of a quotient below 2^18
BI_DEV u64 smp_div_up(Sum a, u64 b) {
  u64 q = 0;
  for (int i = 18; i >= 0; --i)
    if ((Sum)(q + (1ull << i)) * b < a) q += 1ull << i;
  return q + 1ull;
}
// candidates: (key descending, index ascending) as one ascending 64-bit key
BI_DEV u64 smp_entry(float x, int32_t i) { return (u64)(~smp_key(x)) << 32 | (uint32_t)i; }
BI_DEV float smp_entry_x(u64 e) { return smp_unkey(~(uint32_t)(e >> 32)); }

// ---------------------------------------------------------------- one CTA's helpers
// Inclusive sum over the CTA's threads; *total: all of it.  wsum: a value per warp.
BI_DEV Sum smp_block_scan(Sum w, Sum* wsum, Sum* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  w = smp_warp_scan(w);
  __syncthreads();
  if (lane == 31) wsum[warp] = w;
  __syncthreads();
  Sum before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSmpWarps; ++i) {
    const Sum t = wsum[i];
    if (i < warp) before += t;
    all += t;
  }
  *total = all;
  return w + before;
}
// Sorts one value per thread, thread 0 the smallest: a bitonic network over the first n2 threads (a power of
// two, uniform; the others' values must be ~0).  Strides within a warp exchange by shuffles, wider ones through
// buf[kSmpThreads].
BI_DEV u64 smp_sort_threads(u64 v, int n2, u64* buf) {
  const int tid = threadIdx.x;
  for (int size = 2; size <= n2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      u64 y;
      if (stride >= 32) {
        __syncthreads();
        buf[tid] = v;
        __syncthreads();
        y = buf[tid ^ stride];
      } else {
        y = __shfl_xor_sync(0xffffffffu, v, stride);
      }
      const bool up = ((tid & size) == 0) == ((tid & stride) == 0);  // this thread keeps the smaller
      v = (v < y) == up ? v : y;
    }
  }
  return v;
}
// Sorts l[0, n) ascending, n <= kSmpList.
BI_DEV void smp_sort(u64* l, int n) {
  int n2 = 2;
  while (n2 < n) n2 <<= 1;
  for (int i = n + threadIdx.x; i < n2; i += kSmpThreads) l[i] = ~0ull;
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int t = threadIdx.x; t < n2 / 2; t += kSmpThreads) {
        const int i = 2 * t - (t & (stride - 1)), j = i + stride;
        const u64 x = l[i], y = l[j];
        if ((x > y) == ((i & size) == 0)) {
          l[i] = y;
          l[j] = x;
        }
      }
      __syncthreads();
    }
}
// Masses of l[0, n) in order (mass_of(entry)), then the first entry at which the running mass (or, for !by_mass,
// the number of entries) reaches target_of(total mass): its position (n: none) and the mass through it, to every
// thread.
template <typename F, typename G>
BI_DEV int smp_list_find(SmpShared& sh, const u64* l, int n, bool by_mass, F mass_of, G target_of, Sum* through) {
  constexpr int EPT = kSmpList / kSmpThreads;
  const int tid = threadIdx.x;
  u64 w[EPT];
  Sum ws = 0;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = tid * EPT + i;
    w[i] = e < n ? mass_of(l[e]) : 0ull;
    ws += w[i];
  }
  if (tid == 0) sh.pos = n;
  Sum total;
  Sum run = smp_block_scan(ws, sh.wsum, &total) - ws;
  const Sum target = target_of(total);
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = tid * EPT + i;
    const Sum next = run + w[i];
    if (e < n && (by_mass ? (run < target && target <= next) : (Sum)(e + 1) == target)) {
      sh.pos = e;
      sh.total = next;
    }
    run = next;
  }
  __syncthreads();
  const int pos = sh.pos;
  *through = pos == n ? total : sh.total;
  __syncthreads();
  return pos;
}

// ---------------------------------------------------------------- a contiguous share of a row, in global memory
// Positions count from a 16-byte boundary at or before the share; those outside it read as -inf.  A warp walks
// slabs of 128 positions, a contiguous and even number of them.
template <typename TL>
struct SmpShare {
  static constexpr int VE = 16 / sizeof(TL);  // logits of a 16-byte vector
  const TL* src0;      // position 0
  int base;            // its row index
  int p_lo, p_hi;      // the share's positions
  int slabs, per;      // slabs of the share, and of each warp
  int warp, lane;
  BI_DEV SmpShare(const SampleArgs& a, int64_t row, int lo, int n) {
    const TL* src = static_cast<const TL*>(a.logits) + row * a.ld + lo;
    p_lo = (int)((reinterpret_cast<uintptr_t>(src) / sizeof(TL)) % VE);
    p_hi = p_lo + n;
    base = lo - p_lo;
    src0 = src - p_lo;
    slabs = (p_hi + 255) / 256 * 2;
    per = (slabs / 2 + kSmpWarps - 1) / kSmpWarps * 2;
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
  }
  BI_DEV int slab_lo(int w) const { return min(slabs, w * per); }
  BI_DEV int slab_hi(int w) const { return min(slabs, w * per + per); }
  BI_DEV static void expand(const uint4& raw, float (&x)[VE]) {
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (VE == 4) {
        x[i] = __uint_as_float(r[i]);
      } else {
        x[2 * i] = bf16lo(r[i]);
        x[2 * i + 1] = bf16hi(r[i]);
      }
    }
  }
  template <int N>
  BI_DEV void edge(int p, float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p + i >= p_lo && p + i < p_hi ? (float)src0[p + i] : -INFINITY;
  }
  // A lane's four logits of a slab, in index order over the lanes.
  BI_DEV void slab4(int slab, float (&x)[4]) const { edge<4>(slab * 128 + lane * 4, x); }
  // A lane's vectors of one batch: plain loads inside the share, logit by logit (-inf outside it) at its ends.  Returns
  // how many of them the warp has.
  template <int U>
  BI_DEV int batch(int p_warp, uint4 (&raw)[U]) const {
    constexpr int STEP = 32 * VE;  // a warp's vector
    const int p = p_warp + lane * VE, p1 = min(p_hi, slab_hi(warp) * 128);
    if (p_warp >= p_lo && p_warp + STEP * U <= p1) {
#pragma unroll
      for (int j = 0; j < U; ++j) raw[j] = *reinterpret_cast<const uint4*>(src0 + p + j * STEP);
      return U;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int v = p_warp + j * STEP;
      if (v >= p_lo && v + STEP <= p1) {
        raw[j] = *reinterpret_cast<const uint4*>(src0 + p + j * STEP);
      } else if (v < p1) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = p + j * STEP + i * (VE / 4);
          if constexpr (VE == 4) {
            r[i] = q >= p_lo && q < p1 ? reinterpret_cast<const uint32_t*>(src0)[q] : 0xff800000u;
          } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(src0);
            r[i] = (q >= p_lo && q < p1 ? h[q] : 0xff80u) | (q + 1 >= p_lo && q + 1 < p1 ? h[q + 1] : 0xff80u) << 16;
          }
        }
        raw[j] = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
    return min(U, (p1 - p_warp + STEP - 1) / STEP);
  }
  // visit(first position, four logits) for this warp's slabs (converged), in any order; a batch of U vectors at a time,
  // after which flush() is called: 8 visits at most in between.  Positions outside the share read as -inf.
  template <int U, typename F, typename G>
  BI_DEV void each4(F visit, G flush) const {
    static_assert(U * VE <= 32, "the visitors' sums of masses below 2^57 stay below 2^62");
    constexpr int STEP = 32 * VE;
    const int p1 = slab_hi(warp) * 128;
    for (int p = slab_lo(warp) * 128; p < p1; p += STEP * U) {
      uint4 raw[U];
      const int n = batch<U>(p, raw);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (j < n) {
          float x[VE];
          expand(raw[j], x);
#pragma unroll
          for (int i = 0; i < VE; i += 4) {
            const float y[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
            visit(p + lane * VE + j * STEP + i, y);
          }
        }
      }
      flush();
    }
  }
  template <int U, typename F>
  BI_DEV void each4(F visit) const {
    each4<U>(visit, [] {});
  }
};

// ---------------------------------------------------------------- the rare way: one CTA
template <typename TL, bool ABS>
struct SmpSolo {
  SmpOut out;
  SmpShare<TL> all;  // the whole row
  SmpShared& sh;
  const uint2* tab;
  u64* list;       // 16 KB: kSmpList entries, or the counters
  SmpMass<ABS> ms;
  float x_min;
  int tid, warp, lane;

  // visit(index, logit)
  template <typename F>
  BI_DEV void each(F visit) {
    all.template each4<2>([&](int p0, const float (&x)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) visit(all.base + p0 + i, x[i]);
    });
  }
  // The element, in index order, at which the running weight(index, x) reaches target_of(sum): found(index, x, sum).
  template <typename F, typename G, typename H>
  BI_DEV void locate(F weight, G target_of, H found) {
    Sum w = 0;
    each([&](int i, float x) { w += weight(i, x); });
    w = smp_warp_sum(w);
    __syncthreads();
    if (lane == 0) sh.wsum2[warp] = w;
    __syncthreads();
    Sum b = 0, sum = 0;
    for (int i = 0; i < kSmpWarps; ++i) {
      if (i < warp) b += sh.wsum2[i];
      sum += sh.wsum2[i];
    }
    const Sum target = target_of(sum);
    if (b < target && target <= b + w) {  // one warp
      for (int s = all.slab_lo(warp); b < target && s < all.slabs; ++s) {
        const int i0 = all.base + s * 128 + lane * 4;
        float x[4];
        all.slab4(s, x);
        u64 y[4];
        Sum inc = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = weight(i0 + i, x[i]);
          inc += y[i];
        }
        const Sum upto = smp_warp_scan(inc);
        Sum run = b + upto - inc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (run < target && target <= run + y[i]) found(i0 + i, x[i], sum);
          run += y[i];
        }
        b += smp_warp_total(upto);
      }
    }
    __syncthreads();
  }
  // The cut at which the running count or mass (top_p: of the mass `target` that is left, 0 for all) reaches target.
  BI_DEV SmpCut select(bool by_mass, float p, Sum target) {
    uint32_t* h = reinterpret_cast<uint32_t*>(list);  // counts and five 12-bit limbs of the masses
    uint32_t lo = 0, hi = 0xffffffffu;  // keys of the active elements, once the bins are on keys
    int bin = -1, shift = 0, level = 0; // bins of 1/16 octave first
    Sum before_c = 0, before_w = 0;
    while (true) {
      auto active = [&](float x) {
        if (!(x >= x_min)) return false;
        if (level == 0) return true;
        if (level == 1) return min((ms.k_top - ms.k_of(x)) >> kSmpMassShift, kSmpMassBins - 1) == bin;
        const uint32_t k = smp_key(x);
        return k >= lo && k <= hi;
      };
      __syncthreads();
      for (int i = tid; i < 6 * kSmpMassBins; i += kSmpThreads) h[i] = 0u;
      __syncthreads();
      each([&](int, float x) {
        if (active(x)) {
          const int b = level == 0 ? min((ms.k_top - ms.k_of(x)) >> kSmpMassShift, kSmpMassBins - 1)
                                   : (int)((hi - smp_key(x)) >> shift);
          const u64 w = ms.mass(x, tab);
          atomicAdd(&h[b], 1u);
          // twelve-bit limbs: 2^18 of them sum to less than 2^30
#pragma unroll
          for (int i = 0; i < 5; ++i) atomicAdd(&h[(i + 1) * kSmpMassBins + b], (uint32_t)(w >> (12 * i)) & 0xfffu);
        }
      });
      __syncthreads();
      static_assert(kSmpMassBins == kSmpThreads, "a bin per thread");
      const uint32_t c = h[tid];
      Sum w = 0;
#pragma unroll
      for (int i = 0; i < 5; ++i) w += (Sum)h[(i + 1) * kSmpMassBins + tid] << (12 * i);
      Sum tot_c, tot_w;
      const Sum ic = smp_block_scan(c, sh.wsum, &tot_c);
      const Sum iw = smp_block_scan(w, sh.wsum, &tot_w);
      if (level == 0 && by_mass) target = smp_top_p_target(p, target ? target : tot_w);
      const Sum want = target - (by_mass ? before_w : before_c);
      if (want > (by_mass ? tot_w : tot_c)) return SmpCut{smp_key(x_min), 0x7fffffff, tot_w};  // too few: all stay
      if (by_mass ? (iw - w < want && want <= iw) : (ic - c < want && want <= ic))
        sh.find = SmpFind{tid, (uint32_t)(ic - c), c, iw - w};
      __syncthreads();
      const SmpFind f = sh.find;
      before_c += f.before;
      before_w += f.before_mass;
      if (level == 0) {
        bin = f.bin;
      } else {
        hi = hi - ((uint32_t)f.bin << shift);
        lo = hi - min((1u << shift) - 1u, hi - lo);
      }
      ++level;
      if (level == 1 || f.inside > (uint32_t)kSmpList) {  // smallest and largest key of the bin
        uint32_t kmin = 0xffffffffu, kmax = 0u;
        each([&](int, float x) {
          if (active(x)) {
            const uint32_t k = smp_key(x);
            kmin = min(kmin, k);
            kmax = max(kmax, k);
          }
        });
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        __syncthreads();
        if (lane == 0) {
          sh.wcnt[warp] = kmin;
          sh.wsum[warp] = kmax;
        }
        __syncthreads();
        for (int i = 0; i < kSmpWarps; ++i) {
          kmin = min(kmin, sh.wcnt[i]);
          kmax = max(kmax, (uint32_t)sh.wsum[i]);
        }
        lo = kmin;
        hi = kmax;
        level = 2;
        shift = max(0, 32 - __clz(kmax - kmin) - kSmpMassBits);
      }
      const Sum left = target - (by_mass ? before_w : before_c);
      if (lo == hi) {  // equal values: the first `need` of them by index
        const float x1 = smp_unkey(lo);
        const u64 w1 = ms.mass(x1, tab);
        const u64 need = by_mass ? smp_div_up(left, w1) : (u64)left;  // a bin that mass reached has some
        locate([&](int, float x) { return x >= x_min && x == x1 ? 1ull : 0ull; }, [&](Sum) { return (Sum)need; },
               [&](int i, float, Sum) { sh.pos = i; });
        return SmpCut{lo, sh.pos, before_w + (Sum)need * w1};
      }
      if (f.inside <= (uint32_t)kSmpList) {
        __syncthreads();
        if (tid == 0) sh.list_n = 0;
        __syncthreads();
        each([&](int i, float x) {
          if (active(x)) list[atomicAdd(&sh.list_n, 1u)] = smp_entry(x, i);
        });
        __syncthreads();
        smp_sort(list, (int)f.inside);
        Sum through;
        const int pos = smp_list_find(sh, list, (int)f.inside, by_mass,
                                      [&](u64 e) { return ms.mass(smp_entry_x(e), tab); }, [&](Sum) { return left; },
                                      &through);
        const u64 e = list[pos];
        return SmpCut{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, before_w + through};
      }
    }
  }
  BI_DEV void run() {
    tid = threadIdx.x;
    warp = tid >> 5;
    lane = tid & 31;
    SmpCut cut{smp_key(x_min), 0x7fffffff, 0};
    Sum left = 0;
    if (sh.k_eff < out.a.V) {
      cut = select(false, 1.f, (Sum)sh.k_eff);
      left = cut.mass;
      __syncthreads();
    }
    if (sh.p < 1.f) {
      const SmpCut c = select(true, sh.p, left);
      if (c.key > cut.key || (c.key == cut.key && c.idx < cut.idx)) cut = c;
      __syncthreads();
    }
    const float cut_x = smp_unkey(cut.key);
    const int32_t id = sh.id;
    const bool first = !out.a.ids_in && sh.u == 0.f;
    auto kept = [&](int i, float x) { return x > cut_x || (x == cut_x && i <= cut.idx); };
    locate([&](int i, float x) { return kept(i, x) ? ms.mass(x, tab) : 0ull; },
           [&](Sum S) { return out.a.ids_in || first ? S : smp_draw_target(sh.u, S); },
           [&](int i, float x, Sum S) {
             if (out.a.ids_in || first) sh.total2 = S;
             else out.token(ms, sh, tab, i, x, S);
           });
    if (first) {
      // u = 0: the first kept token of any mass, also one below the unit: 64 bits hold masses above 2^-1075, which
      // round to 2^-1074 and more
      const float x_pos = __double2float_ru((double)ms.m - 745.13321910194122 / ((double)sh.r_hi + (double)sh.r_lo));
      locate([&](int i, float x) { return kept(i, x) && x >= x_pos ? 1ull : 0ull; }, [](Sum) { return (Sum)1; },
             [&](int i, float x, Sum) { out.token(ms, sh, tab, i, x, sh.total2); });
    }
    if (out.a.ids_in && tid == 0) {
      const float x = sh.x_id;
      if (x > cut_x || (x == cut_x && id <= cut.idx)) out.token(ms, sh, tab, id, x, sh.total2);
      else out.write(id, -INFINITY);
    }
  }
};
template <typename TL, bool ABS>
__device__ __noinline__ void smp_solo(SmpOut out, SmpShared& sh, const uint2* tab, u64* list, SmpMass<ABS> ms,
                                      float x_min) {
  SmpSolo<TL, ABS> r{out, SmpShare<TL>(out.a, out.row, 0, out.a.V), sh, tab, list, ms, x_min};
  r.run();
}

// ---------------------------------------------------------------- one row per cluster of CS CTAs
template <typename TL, int CS>
struct SmpRow {
  SmpOut out;
  SmpShare<TL> mine;   // this CTA's part of the row
  SmpShared& sh;
  uint2* table;        // [64][kSmpTabLanes]
  const uint2* tab;    // this lane's copy of it
  unsigned char* area; // 8 KB: counts; 16 KB: list
  cg::cluster_group cl;
  int tid, warp, lane, rank;
  float m, x_min;      // row maximum; smallest logit that min-p keeps (above -inf)
  bool score;

  BI_DEV uint32_t* counts() { return reinterpret_cast<uint32_t*>(area); }
  BI_DEV u64* list() { return reinterpret_cast<u64*>(area + 8192); }
  static constexpr int kWide = 32 / SmpShare<TL>::VE;  // vectors in flight in passes that keep few registers
  static constexpr int kSegment = kSmpList / CS;  // a CTA's part of rank 0's list

  BI_DEV void csync() {
    if (CS == 1) __syncthreads();
    else cl.sync();
  }
  template <typename P>
  BI_DEV P* at(P* ptr, int r) {
    if (CS == 1) return ptr;
    return cl.map_shared_rank(ptr, r);
  }
  // Appends to this CTA's segment of rank 0's list, a lane for itself; entries beyond it are counted only.  (Few groups
  // of 128 logits have more than one: with the warp's lanes voting on all of a group's 4096 fp32 rows of 32000 under
  // top-p took 403 us instead of 378, 2048 bf16 rows of 129280 under all rules 331 instead of 320.)
  BI_DEV void append(float x, int p, u64* segment, u64* own) {
    const uint32_t o = atomicAdd(&sh.list_n, 1u);
    if (o < (uint32_t)kSegment) {
      const u64 e = smp_entry(x, mine.base + p);
      segment[o] = e;
      if (own) own[o] = e;
    }
  }
  // Rank 0: the segments' entries joined at the front of the list (no barrier after it); their number, or -1 when
  // a segment overflowed.
  BI_DEV int join() {
    u64* l = list();
    uint32_t n = 0;
    bool fits = true;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const uint32_t nr = sh.cta_n[r];
      fits = fits && nr <= (uint32_t)kSegment;
      if (r > 0 && fits)  // moves down: a segment never starts before the entries so far end
        for (uint32_t i0 = 0; i0 < nr; i0 += kSmpThreads) {
          const bool mine_too = i0 + tid < nr;
          const u64 e = mine_too ? l[r * kSegment + i0 + tid] : 0ull;
          __syncthreads();
          if (mine_too) l[n + i0 + tid] = e;
        }
      n += nr;
    }
    __syncthreads();
    return fits ? (int)n : -1;
  }

  // ---- sums over the row, and the draw.  weight4(index of the first, x, w) gives four elements' weights.
  // Warp sums to sh.wsum; then, with publish(), the CTA's sum to every rank's sh.cta_sum.
  template <typename F>
  BI_DEV void warp_sums(F weight4) {
    Sum sum = 0;
    u64 some = 0;
    mine.template each4<4>(
        [&](int p0, const float (&x)[4]) {
          u64 w[4];
          weight4(mine.base + p0, x, w);
          some += (w[0] + w[1]) + (w[2] + w[3]);
        },
        [&] {
          sum += some;
          some = 0;
        });
    sum = smp_warp_sum(sum);
    if (lane == 0) sh.wsum[warp] = sum;
  }
  BI_DEV void publish() {
    __syncthreads();
    if (tid < CS) {
      Sum t = 0;
#pragma unroll
      for (int i = 0; i < kSmpWarps; ++i) t += sh.wsum[i];
      at(sh.cta_sum, tid)[rank] = t;
    }
    csync();
  }
  BI_DEV Sum row_sum() {
    Sum t = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) t += sh.cta_sum[r];
    return t;
  }
  // After publish(): the element, in index order, at which the running weight reaches target (>= 1); the CTA that
  // holds it calls found(index, x).  Its warp's slabs are taken by a warp each.
  template <typename F, typename H>
  BI_DEV void locate(F weight4, Sum target, H found) {
    Sum b = 0, own = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const Sum t = sh.cta_sum[r];
      if (r < rank) b += t;
      if (r == rank) own = t;
    }
    if (!(b < target && target <= b + own)) return;
    int unit = 0;
    for (; unit < kSmpWarps - 1; ++unit) {
      const Sum t = sh.wsum[unit];
      if (target <= b + t) break;
      b += t;
    }
    const int s1 = mine.slab_hi(unit);
    for (int sb = mine.slab_lo(unit); sb < s1; sb += kSmpWarps) {
      const int i0 = mine.base + (sb + warp) * 128 + lane * 4;
      float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      u64 y[4] = {0, 0, 0, 0};
      if (sb + warp < s1) {
        mine.slab4(sb + warp, x);
        weight4(i0, x, y);
      }
      const u64 y4 = (y[0] + y[1]) + (y[2] + y[3]);
      Sum all;
      Sum run = b + smp_block_scan(y4, sh.wsum2, &all) - y4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (run < target && target <= run + y[i]) found(i0 + i, x[i]);
        run += y[i];
      }
      b += all;
      if (target <= b) break;
    }
  }
  template <bool ABS>
  struct Kept {  // masses of the kept elements
    const SmpMass<ABS>& ms;
    const uint2* tab;
    float x;
    int32_t idx;
    BI_DEV void operator()(int i0, const float (&v)[4], u64 (&w)[4]) const {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = ms.mass(v[i], tab);
        if (!(v[i] > x || (v[i] == x && i0 + i <= idx))) w[i] = 0ull;
      }
    }
  };
  // The draw from the kept set, after publish().
  template <bool ABS>
  BI_DEV void draw(const SmpMass<ABS>& ms, float cut_x, int32_t cut_i) {
    const Sum S = row_sum();
    locate(Kept<ABS>{ms, tab, cut_x, cut_i}, smp_draw_target(sh.u, S),
           [&](int i, float x) { out.token(ms, sh, tab, i, x, S); });
  }

  // ---- what follows from the row's maximum; false: the row is answered (rank 0)
  BI_DEV bool row_max() {
    float mx = sh.cta_max[0];
#pragma unroll
    for (int r = 1; r < CS; ++r) mx = smp_max_nan(mx, sh.cta_max[r]);
    m = mx;
    const bool bad = !(m < INFINITY);  // NaN or +inf
    if (bad || m == -INFINITY) {
      if (rank == 0 && tid == 0) {
        if (bad) report(out.a.status, DEV_BAD_VALUE);
        out.write(-1, bad ? NAN : -INFINITY);
      }
      return false;
    }
    // the smallest float whose mass is at least min_p
    const float mp = sh.min_p;
    x_min = -FLT_MAX;
    if (mp >= 1.f) x_min = m;
    else if (mp > 0.f) x_min = fmaxf(-FLT_MAX, __double2float_ru((double)m + sh.log_min_p));
    if (score && !(sh.x_id >= x_min)) {
      if (rank == 0 && tid == 0) out.write(sh.id, -INFINITY);
      return false;
    }
    return true;
  }
  BI_DEV bool absolute() { return fabsf(m) * sh.c_hi < 524288.f; }
  BI_DEV void solo() {
    if (absolute()) {
      SmpMass<true> ms;
      ms.init(m, sh);
      smp_solo<TL>(out, sh, tab, list(), ms, x_min);
    } else {
      SmpMass<false> ms;
      ms.init(m, sh);
      smp_solo<TL>(out, sh, tab, list(), ms, x_min);
    }
  }

  // ---- top-k up to kSmpMaxK.  k: the CTA's bound is the k-th largest of its threads' maxima.
  BI_DEV void few(int k, float t_max, float cta_max, float cta_min) {
    // bins linear in x, from the CTA's maximum to the smallest of the threads' maxima (counts() is zeroed)
    const float scale = fminf(__fdiv_rn((float)(kSmpMaxBins - 2), __fsub_rn(cta_max, cta_min)), FLT_MAX);
    if (t_max > -INFINITY) {
      const float y = __fmul_rn(__fsub_rn(cta_max, t_max), scale);
      atomicAdd(&counts()[y < (float)(kSmpMaxBins - 1) ? (int)y : kSmpMaxBins - 1], 1u);
    }
    __syncthreads();
    // lane l holds bins 8 l .. 8 l + 7 (every warp for itself)
    uint32_t c[8], n = 0;
    *reinterpret_cast<uint4*>(c) = reinterpret_cast<const uint4*>(counts())[lane * 2];
    *reinterpret_cast<uint4*>(c + 4) = reinterpret_cast<const uint4*>(counts())[lane * 2 + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) n += c[i];
    uint32_t run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    run -= n;
    int bin = kSmpMaxBins - 1;  // fewer maxima than k: every logit is let through
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (run < (uint32_t)k && (uint32_t)k <= run + c[i]) bin = lane * 8 + i;
      run += c[i];
    }
    bin = __reduce_min_sync(0xffffffffu, bin);
    // k of the maxima lie in the bins up to this one: none is below its end (made lower by more than the roundings)
    const float depth = __fmul_rn(__fdiv_rn((float)(bin + 1), scale), 1.000001f);
    const float bound = bin == kSmpMaxBins - 1 ? -FLT_MAX : fmaxf(-FLT_MAX, __fsub_rd(cta_max, depth));
    u64* segment = at(list(), 0) + rank * kSegment;
    mine.template each4<kWide>([&](int p0, const float (&x)[4]) {
      const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      if (top >= bound) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (x[i] >= bound) append(x[i], p0 + i, segment, nullptr);
      }
    });
    __syncthreads();
    if (tid == 0) {
      at(sh.cta_n, 0)[rank] = sh.list_n;
      at(sh.cta_max, 0)[rank] = cta_max;
      at(sh.cta_bound, 0)[rank] = bound;
    }
    csync();
    if (rank > 0) return;
    if (!row_max()) return;
    const int total = join();
    bool done = false;
    if (total >= 0 && absolute()) {
      float need = sh.cta_bound[0];  // every logit that is not below this is in the list
#pragma unroll
      for (int r = 1; r < CS; ++r) need = fmaxf(need, sh.cta_bound[r]);
      SmpMass<true> ms;
      ms.init(m, sh);
      done = total <= kSmpThreads ? small(ms, total, need) : small_sorted(ms, total, need);
    }
    if (!done) solo();
  }
  // The row's kept set lies in the list of n entries, a thread each (rank 0).  False: it may not.
  BI_DEV bool small(const SmpMass<true>& ms, int n, float need) {
    u64* l = list();
    u64* wl = l + kSmpThreads;  // [kSmpThreads], also the sort's buffer
    int n2 = 32;
    while (n2 < n) n2 <<= 1;
    u64 e = tid < n ? l[tid] : ~0ull;
    if (tid < n && smp_entry_x(e) < x_min) e = ~0ull;  // min-p
    e = smp_sort_threads(e, n2, wl);
    const bool some = e != ~0ull;
    const float x = smp_entry_x(e);
    u64 w = some ? ms.mass(x, tab) : 0ull;
    bool kept = some && tid < sh.k_eff;
    if (!kept) w = 0;
    Sum S;
    Sum run = smp_block_scan(w, sh.wsum, &S) - w;
    // the k-th of the list, and below it nothing that a CTA held back; or the row has fewer logits above min-p
    const bool full = __syncthreads_or(some && tid == sh.k_eff - 1 && x >= need);
    if (!full && !(need <= x_min)) return false;
    if (sh.p < 1.f) {
      const Sum target = smp_top_p_target(sh.p, S);
      kept = kept && run < target;
      if (kept && target <= run + w) sh.total2 = run + w;
      if (!kept) w = 0;
      __syncthreads();
      S = sh.total2;
    }
    if (score) {
      const bool it = kept && (int32_t)(uint32_t)e == sh.id;
      if (it) out.token(ms, sh, tab, sh.id, x, S);
      if (!__syncthreads_or(it) && tid == 0) out.write(sh.id, -INFINITY);
      return true;
    }
    // index order: the kept entries come first, so threads beyond the last of them are through
    const int count = __syncthreads_count(kept);
    wl[tid] = w;
    l[tid] = e;
    __syncthreads();
    if (tid < count) {
      Sum before = 0;
#pragma unroll 4
      for (int j = 0; j < count; ++j) {
        const u64 y = wl[j];
        if ((uint32_t)l[j] < (uint32_t)e) before += y;
      }
      const Sum target = smp_draw_target(sh.u, S);
      if (before < target && target <= before + w) out.token(ms, sh, tab, (int32_t)(uint32_t)e, x, S);
    }
    return true;
  }
  // The same for up to kSmpList entries.
  BI_DEV bool small_sorted(const SmpMass<true>& ms, int n, float need) {
    u64* l = list();
    smp_sort(l, n);
    const u64 worst = smp_entry(x_min, 0x7fffffff);
    if (tid == 0) sh.pos = n;
    __syncthreads();
    for (int i = tid; i < n; i += kSmpThreads)  // min-p: the first entry beyond it
      if (l[i] > worst && (i == 0 || l[i - 1] <= worst)) sh.pos = i;
    __syncthreads();
    const int above = sh.pos;
    __syncthreads();
    const int k = min(above, sh.k_eff);
    if (!(k == sh.k_eff ? smp_entry_x(l[k - 1]) >= need : need <= x_min)) return false;
    Sum S;
    int last = smp_list_find(sh, l, k, true, [&](u64 e) { return ms.mass(smp_entry_x(e), tab); },
                             [&](Sum total) { return sh.p < 1.f ? smp_top_p_target(sh.p, total) : total + 1; }, &S);
    if (last == k) last = k - 1;  // no top-p: all of them, with or without mass
    if (score) {
      if (tid == 0) {
        if (smp_entry(sh.x_id, sh.id) <= l[last]) out.token(ms, sh, tab, sh.id, sh.x_id, S);
        else out.write(sh.id, -INFINITY);
      }
      return true;
    }
    // index order: (index, key)
    for (int i = tid; i <= last; i += kSmpThreads) {
      const u64 e = l[i];
      l[i] = (e << 32) | (uint32_t)~(uint32_t)(e >> 32);
    }
    __syncthreads();
    smp_sort(l, last + 1);
    Sum through;
    const int pos = smp_list_find(sh, l, last + 1, true, [&](u64 e) { return ms.mass(smp_unkey((uint32_t)e), tab); },
                                  [&](Sum total) { return smp_draw_target(sh.u, total); }, &through);
    if (tid == 0) {
      out.token(ms, sh, tab, (int32_t)(l[pos] >> 32), smp_unkey((uint32_t)l[pos]), S);
    }
    return true;
  }

  // ---- top-p over the whole row: predicted cut, exact sums
  BI_DEV void nucleus(const SmpMass<true>& ms) {
    for (int i = tid; i < 2 * kSmpBins; i += kSmpThreads) counts()[i] = 0u;
    __syncthreads();
    // depth below the maximum in units of 2^-17 octave: a bin is 2^12 of them, and takes the count and the sum of
    // the depths within it
    // (with 128 more, more than the rounding of `zero` takes off; a lower bound on the logits bounds the depths)
    const float c11 = __fmul_rn(ms.c_hi, -2048.f), zero = __fmaf_rn(-m, c11, 8388736.f);
    const float bottom = fminf(fmaxf(__fmaf_rn(x_min, c11, zero) - 8388608.f, 0.f) + 2.f, 4096.f * (kSmpBins - 1));
    const uint32_t deepest = (uint32_t)bottom;
    uint32_t* depths = counts() + kSmpBins;
    uint32_t bits = 0;
    mine.template each4<4>([&](int, const float (&x)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (SmpShare<TL>::VE == 4) bits |= __float_as_uint(x[i]);
        const uint32_t d = (uint32_t)__float_as_int(__fmaf_rn(x[i], c11, zero)) - 0x4B000000u;
        if (d < deepest) {  // the open bin would only serialise
          atomicAdd(&counts()[d >> 12], 1u);
          atomicAdd(&depths[d >> 12], d & 4095u);
        }
      }
    });
    // 16-bit logits, as they are or widened, stand in few places: a bin's are not spread over it
    const bool coarse = !__syncthreads_or(SmpShare<TL>::VE == 4 && (bits & 0x1fffu) != 0u);
    csync();
    if (rank == 0) {
      // a bin's mass to second order from its count and mean depth; the open bin's is left out of the prediction
      constexpr int BPT = kSmpBins / kSmpThreads;
      float w[BPT], sum = 0.f;
      bool dense[BPT];
      const uint32_t many = coarse ? 1024 : 64;
      static_assert(BPT == 2, "a pair of bins per thread");
      uint32_t c[BPT] = {0, 0}, d[BPT] = {0, 0};
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        const uint2 v = reinterpret_cast<const uint2*>(at(counts(), r))[tid];
        const uint2 z = reinterpret_cast<const uint2*>(at(counts(), r))[kSmpBins / BPT + tid];
        c[0] += v.x;
        c[1] += v.y;
        d[0] += z.x;
        d[1] += z.y;
      }
      const float scale = exp2f((float)tid * -0.0625f);
#pragma unroll
      for (int i = 0; i < BPT; ++i) {
        const float n = (float)c[i], z = (float)d[i] * 5.2882933e-6f;  // times ln 2 / 2^17
        // in units of the maximum's mass; the variance of many depths across a bin adds 2e-5
        const float r = c[i] ? __fdividef(0.5f * z * z - 1.96e-5f, n) + (1.f + 1.96e-5f) * n - z : 0.f;
        w[i] = r * (i ? scale * 0.97857206f : scale);  // 2^(-1/32)
        dense[i] = c[i] >= many;
        sum += w[i];
      }
      float run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) sh.wmax[warp] = run;
      if (tid == 0) {  // no prediction
        sh.x_hi = -INFINITY;
        sh.x_lo = -INFINITY;
      }
      __syncthreads();
      float total = 0.f;
      run -= sum;
#pragma unroll
      for (int i = 0; i < kSmpWarps; ++i) {
        const float y = sh.wmax[i];
        if (i < warp) run += y;
        total += y;
      }
      // what the roundings above leave open, with room
      const float guess = sh.p * total, open = total * 1e-5f;
      const float g_hi = fmaxf(guess - open, total * 1e-12f), g_lo = fminf(guess + open, total * 0.9999999f);
      const float k_m = __fmaf_rn(m, ms.c_hi, 0.0625f),  // the depths' 128 more
                   per_k = __fdividef(1.f, ms.c_hi);
#pragma unroll
      for (int i = 0; i < BPT; ++i) {
        const float next = run + w[i];
        const int b = tid * BPT + i;
        if (b < kSmpBins - 2) {
          // within a bin of many, at the fraction of its mass, give or take what n places at random leave open
          // (2.2 / sqrt(n) of a bin); else at the bin's end; and a little further.  (Whole bins of up to 1024 for
          // coarse logits, whose ties a fraction misses: 2048 bf16 rows of 129280 719 -> 499 us; for others their
          // longer list costs more than it saves: 4096 fp32 rows of 32000 390 -> 434 us.)
          const float give = 0.1f + (dense[i] ? 4.4f * rsqrtf((float)c[i]) : 0.f);
          if (run < g_hi && g_hi <= next) {
            const float part = dense[i] ? __fdividef(g_hi - run, w[i]) : 0.f;
            sh.x_hi = (k_m - 2.f * ((float)b + part) + give) * per_k;
          }
          if (run < g_lo && g_lo <= next) {
            const float part = dense[i] ? __fdividef(g_lo - run, w[i]) : 1.f;
            sh.x_lo = (k_m - 2.f * ((float)b + part) - give) * per_k;
          }
        }
        run = next;
      }
      __syncthreads();
      if (tid == 0) {
        if (sh.x_hi == -INFINITY || sh.x_lo == -INFINITY) {
          sh.x_hi = -INFINITY;
        } else {
          sh.x_lo = fmaxf(x_min, sh.x_lo);
          sh.x_hi = fmaxf(sh.x_lo, sh.x_hi);
        }
      }
      __syncthreads();
      if (tid > 0 && tid < CS) {
        *at(&sh.x_lo, tid) = sh.x_lo;
        *at(&sh.x_hi, tid) = sh.x_hi;
      }
    }
    csync();
    const float x_lo = sh.x_lo, x_hi = sh.x_hi;
    if (x_hi == -INFINITY) {
      if (rank == 0) solo();
      return;
    }
    Sum all = 0, above = 0;
    u64* segment = at(list(), 0) + rank * kSegment;
    // the draw looks at this CTA's entries once more (alone, in the list itself)
    u64* own = CS == 1 || score ? nullptr : reinterpret_cast<u64*>(counts());
    static_assert(CS == 1 || kSegment * 8 <= 8192, "own entries take the counts' place");
    u64 some = 0, some_above = 0;
    const float mid = 0.5f * x_lo + 0.5f * x_hi, half = fmaxf(x_hi - mid, mid - x_lo) * 1.00001f;
    auto pass = [&](auto with_min_p) {
      mine.template each4<4>(
          [&](int p0, const float (&x)[4]) {
            float near = INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const u64 w = ms.mass(x[i], tab);
              if (!decltype(with_min_p)::value || x[i] >= x_min) some += w;
              if (x[i] > x_hi) some_above += w;
              near = fminf(near, fabsf(x[i] - mid));
            }
            if (near <= half) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (x[i] <= x_hi && x[i] >= x_lo) append(x[i], p0 + i, segment, own);
            }
          },
          [&] {
            all += some;
            above += some_above;
            some = some_above = 0;
          });
    };
    if (x_min == -FLT_MAX) pass(std::false_type{});
    else pass(std::true_type{});
    all = smp_warp_sum(all);
    above = smp_warp_sum(above);
    if (lane == 0) {
      sh.wsum[warp] = all;
      sh.wsum2[warp] = above;
      sh.wlow[warp] = 0u;
      sh.whigh[warp] = 0ull;
    }
    __syncthreads();
    if (tid == 0) {
      Sum t = 0, t2 = 0;
#pragma unroll
      for (int i = 0; i < kSmpWarps; ++i) {
        t += sh.wsum[i];
        t2 += sh.wsum2[i];
      }
      at(sh.cta_sum, 0)[rank] = t;
      at(sh.cta_sum2, 0)[rank] = t2;
      at(sh.cta_n, 0)[rank] = sh.list_n;
    }
    csync();
    if (rank == 0) {
      Sum total = 0, over = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        total += sh.cta_sum[r];
        over += sh.cta_sum2[r];
      }
      const Sum target = smp_top_p_target(sh.p, total);
      if (tid == 0) sh.cut = SmpCut{0u, -1, 0};
      const int n = join();
      if (n >= 0 && over < target) list_cut(ms, n, over, target);
      __syncthreads();
      const SmpCut c = sh.cut;
      if (c.idx < 0) {  // missed
        if (!score && tid > 0 && tid < CS) *at(&sh.cut, tid) = c;
        if (!score) csync();
        solo();
        return;
      }
      if (score) {
        if (tid == 0) {
          if (smp_entry(sh.x_id, sh.id) <= ((u64)(~c.key) << 32 | (uint32_t)c.idx))
            out.token(ms, sh, tab, sh.id, sh.x_id, c.mass);
          else
            out.write(sh.id, -INFINITY);
        }
        return;
      }
      if (tid > 0 && tid < CS) *at(&sh.cut, tid) = c;
    }
    if (score) return;
    csync();
    const SmpCut cut = sh.cut;
    if (cut.idx < 0) return;
    // the warps' kept sums: what lies above the prediction, and the kept entries next to it
    const float cut_x = smp_unkey(cut.key);
    const u64 last = (u64)(~cut.key) << 32 | (uint32_t)cut.idx;
    for (uint32_t i = tid; i < sh.list_n; i += kSmpThreads) {
      const u64 e = CS == 1 ? list()[i] : own[i];
      if (e <= last) {
        const int at_ = ((int)(uint32_t)e - mine.base) / 128 / mine.per;
        const u64 w = ms.mass(smp_entry_x(e), tab);
        atomicAdd(&sh.wlow[at_], (uint32_t)w & 0xfffffu);
        atomicAdd(&sh.whigh[at_], w >> 20);
      }
    }
    __syncthreads();
    if (tid < kSmpWarps) sh.wsum[tid] = sh.wsum2[tid] + ((Sum)sh.whigh[tid] << 20) + sh.wlow[tid];
    publish();
    draw(ms, cut_x, cut.idx);
  }
  // The entry of list[0, n) at which the mass in order, from `over` on, reaches target, to sh.cut (rank 0).
  BI_DEV void list_cut(const SmpMass<true>& ms, int n, Sum over, Sum target) {
    u64* l = list();
    if (n <= kSmpThreads) {
      int n2 = 32;
      while (n2 < n) n2 <<= 1;
      const u64 e = smp_sort_threads(tid < n ? l[tid] : ~0ull, n2, l + kSmpThreads);
      const u64 w = tid < n ? ms.mass(smp_entry_x(e), tab) : 0ull;
      Sum total;
      const Sum run = over + smp_block_scan(w, sh.wsum, &total) - w;
      if (tid < n && run < target && target <= run + w)
        sh.cut = SmpCut{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, run + w};
    } else {
      smp_sort(l, n);
      Sum through;
      const int pos = smp_list_find(sh, l, n, true, [&](u64 e) { return ms.mass(smp_entry_x(e), tab); },
                                    [&](Sum) { return target - over; }, &through);
      if (tid == 0 && pos < n) {
        const u64 e = l[pos];
        sh.cut = SmpCut{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, over + through};
      }
    }
  }

  // ---- nothing cut but by min-p
  template <bool ABS>
  BI_DEV void plain() {
    SmpMass<ABS> ms;
    ms.init(m, sh);
    if (x_min == -FLT_MAX)
      warp_sums([&](int, const float (&x)[4], u64 (&w)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ms.mass(x[i], tab);
      });
    else warp_sums(Kept<ABS>{ms, tab, x_min, 0x7fffffff});
    publish();
    if (!score) draw(ms, x_min, 0x7fffffff);
    else if (rank == 0 && tid == 0) out.token(ms, sh, tab, sh.id, sh.x_id, row_sum());
  }

  // The row's parameters and constants, by one thread.  Returns the scored token's logit, on its way.
  BI_DEV float setup() {
    const SampleArgs& a = out.a;
    const int64_t row = out.row;
    const int64_t pr = a.param_row ? (int64_t)a.param_row[row] : row;
    bool ok = !(a.temperature || a.top_k || a.top_p || a.min_p) || (pr >= 0 && pr < a.n_params);
    float T = 1.f, mp = 0.f, q = 1.f, u = 0.f, x = 0.f;
    int32_t k = 0, id = 0;
    if (ok) {
      if (a.temperature) T = a.temperature[pr];
      if (a.top_k) k = a.top_k[pr];
      if (a.top_p) q = a.top_p[pr];
      if (a.min_p) mp = a.min_p[pr];
    }
    if (score) {
      id = a.ids_in[row];
      if (id >= 0 && id < a.V) x = (float)static_cast<const TL*>(a.logits)[row * a.ld + id];
      else ok = false;
    } else {
      const int64_t ur = a.u_row ? (int64_t)*a.u_row : 0;
      // (-0 -> +0: the products with u take it apart without a sign)
      if (ur >= 0 && ur < a.u_rows)
        u = __fadd_rn(a.u[ur * a.u_ld + (a.dst ? (int64_t)a.dst[row] : row)], 0.f);
      else ok = false;
      ok = ok && u >= 0.f && u < 1.f;
    }
    ok = ok && (T == 0.f || (T >= 0x1p-64f && T <= 0x1p64f)) && q == q && mp == mp;
    if (T == 0.f) {
      T = 1.f;
      k = 1;
      q = 1.f;
      mp = 0.f;
    }
    // 1 / T and 64 log2(e) / T in two floats each: the remainders of fused multiply-adds are exact
    const float r_hi = __frcp_rn(T), r_lo = __fmul_rn(__fmaf_rn(-T, r_hi, 1.f), r_hi);
    const float l_hi = 92.33248138427734f, l_lo = 1.2326163e-06f;  // 64 log2(e)
    const float c_hi = __fmul_rn(l_hi, r_hi);
    sh.c_hi = c_hi;
    sh.c_lo = __fadd_rn(__fmaf_rn(l_hi, r_hi, -c_hi), __fmaf_rn(l_hi, r_lo, __fmul_rn(l_lo, r_hi)));
    sh.r_hi = r_hi;
    sh.r_lo = r_lo;
    sh.floor_rel = __fmul_rn(T, -4096.f / 92.332481f);
    sh.floor_abs = __fmul_rn(T, -1048576.f / 92.332481f);
    sh.log_min_p = mp > 0.f && mp < 1.f ? (double)T * log((double)mp) : 0.0;
    sh.p = q;
    sh.u = u;
    sh.min_p = mp;
    sh.id = id;
    sh.k_eff = k <= 0 || k > a.V ? a.V : k;
    sh.ok = ok;
    sh.list_n = 0;
    return x;
  }

  BI_DEV float prepare() {
    for (int i = tid; i < 64 * kSmpTabLanes; i += kSmpThreads) {
      const uint32_t t = kExp2Tab[i / kSmpTabLanes];
      table[i] = make_uint2(t - (uint32_t)kSmpMagicBits, __float_as_uint((float)t));
    }
    if (tid < kSmpMaxBins) counts()[tid] = 0u;
    return tid == kSmpThreads - 1 ? setup() : 0.f;
  }
  BI_DEV void run() {
    const SampleArgs& a = out.a;
    score = a.ids_in != nullptr;
    if (CS > 1) cl.barrier_arrive();  // with the wait below: every CTA runs before any writes to another
    float mx = -INFINITY;  // NaN once one is seen
    const float x_id = prepare();
    mine.template each4<kWide>([&](int, const float (&x)[4]) {
      mx = smp_max3_nan(smp_max3_nan(mx, x[0], x[1]), x[2], x[3]);
    });
    if (tid == kSmpThreads - 1) sh.x_id = x_id;
    const float t_max = mx;
    float t_min = mx == -INFINITY ? INFINITY : mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = smp_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      t_min = fminf(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
    }
    if (lane == 0) {
      sh.wmax[warp] = mx;
      sh.wmin[warp] = t_min;
    }
    __syncthreads();
    if (CS > 1) cl.barrier_wait();
    if (!sh.ok) {  // the same in every CTA of the cluster
      if (rank == 0 && tid == 0) {
        report(a.status, DEV_BAD_INDEX);
        out.write(-1, NAN);
      }
      return;
    }
    mx = sh.wmax[lane & (kSmpWarps - 1)];
    t_min = sh.wmin[lane & (kSmpWarps - 1)];
#pragma unroll
    for (int o = kSmpWarps / 2; o > 0; o >>= 1) {
      mx = smp_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      t_min = fminf(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
    }
    const int k_eff = sh.k_eff;
    const bool first = !score && sh.u == 0.f && k_eff > 1;  // masses do not tell: the rare way
    if (!first && k_eff < a.V && k_eff <= kSmpMaxK) {
      // a CTA's share of k, with four of its standard deviations
      const float part = (float)k_eff / CS;
      const int k = CS == 1 ? k_eff : min(k_eff, (int)(part + 4.f * sqrtf(part)) + 8);
      if (k <= kSmpMaxShareK) {
        few(k, t_max, mx, t_min);
        return;
      }
    }
    if (tid < CS) at(sh.cta_max, tid)[rank] = mx;
    csync();
    if (!row_max()) return;
    if (first) {
      if (rank == 0) solo();
    } else if (k_eff == a.V && sh.p >= 1.f) {
      if (absolute()) plain<true>();
      else plain<false>();
    } else if (k_eff == a.V && absolute()) {
      SmpMass<true> ms;
      ms.init(m, sh);
      nucleus(ms);
    } else if (rank == 0) {
      solo();
    }
  }
};

template <typename TL, int CS>
__global__ void __launch_bounds__(kSmpThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smp_dyn[];
  __shared__ SmpShared sh;
  uint2* tab = reinterpret_cast<uint2*>(smp_dyn);
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int rank = CS == 1 ? 0 : (int)cl.block_rank();
  const int64_t row = blockIdx.x / CS;
  const int lo = min(a.V, rank * a.share);
  SmpRow<TL, CS> r{SmpOut{a, row}, SmpShare<TL>(a, row, lo, min(a.V, lo + a.share) - lo), sh, tab,
                   tab + (threadIdx.x & (kSmpTabLanes - 1)), smp_dyn + 64 * kSmpTabLanes * 8, cl};
  r.tid = threadIdx.x;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  r.rank = rank;
  r.run();
}

template <typename TL, int CS>
static bi_status launch_sample(const SampleArgs& a, int64_t T, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(T * CS));
  cfg.blockDim = dim3(kSmpThreads);
  cfg.dynamicSmemBytes = kSmpSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, sample_kernel<TL, CS>, a), "sample_kernel");
}

template <typename TL>
static bi_status dispatch_sample_as(SampleArgs& a, int64_t T, cudaStream_t st) {
  // Bits do not depend on the split.  A row is split while the rows alone leave CTA slots (two per SM) idle, down to
  // 2K logits a CTA: 64 rows of 129280 with top-k and top-p take 25, 23, 22 and 30 us on 1, 2, 4 and 8 CTAs a row (4 is
  // the rule's), and 4096 rows of 32000 at temperature alone 168 us on one and 281 us on two (1 is).  The rule does not
  // always find the best: 37 bf16 rows of 50261 under mixed rules take 27 us on its 8, 23 us on 4.
  int cs = 1;
  while (cs < 8 && cdiv(a.V, cs) > 2048 && T * cs * 2 <= 2 * num_sms()) cs *= 2;
  // The rows in flight have to stay in L2 until their last pass: a row of more than 256 KB is split too (512 fp32 rows
  // of 129280 at temperature alone: 103 us unsplit, 98 us on two CTAs).
  if (cs == 1 && a.V * (int64_t)sizeof(TL) > 256 * 1024) cs = a.V * (int64_t)sizeof(TL) > 512 * 1024 ? 4 : 2;
  a.share = (int)(cdiv(cdiv(a.V, cs), 8) * 8);
  switch (cs) {
    case 1: return launch_sample<TL, 1>(a, T, st);
    case 2: return launch_sample<TL, 2>(a, T, st);
    case 4: return launch_sample<TL, 4>(a, T, st);
    default: return launch_sample<TL, 8>(a, T, st);
  }
}
static bi_status dispatch_sample(SampleArgs& a, int64_t T, cudaStream_t st) {
  return a.bf16 ? dispatch_sample_as<__nv_bfloat16>(a, T, st) : dispatch_sample_as<float>(a, T, st);
}

// Checks that both entry points share; fills the row-independent arguments.
static bi_status sample_args(const char* who, const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                             const bi_sampling* sp, const int32_t* param_row, SampleArgs* a) {
  auto bad = [&](bi_status st, const char* what) { return fail(st, std::string(who) + ": " + what); };
  if (!logits) return bad(BI_ERR_INVALID_ARG, "null logits");
  if (dtype != BI_DTYPE_FP32 && dtype != BI_DTYPE_BF16)
    return bad(BI_ERR_INVALID_ARG, "dtype must be BI_DTYPE_FP32 or BI_DTYPE_BF16");
  if (V < 1 || ld < V) return bad(BI_ERR_INVALID_ARG, "V must be positive and ld at least V");
  static_assert(kSmpMaxV == kMaxSampleVocab, "vocabulary limit");
  if (V > kSmpMaxV) return bad(BI_ERR_UNSUPPORTED_SHAPE, "V must be at most 262144");
  if (T > 0x7fffffff / 8) return bad(BI_ERR_INVALID_ARG, "T too large");
  if (ld > (int64_t(1) << 40)) return bad(BI_ERR_INVALID_ARG, "ld too large");
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == BI_DTYPE_FP32 ? 4 : 2))
    return bad(BI_ERR_INVALID_ARG, "logits must be aligned to their type");
  a->logits = logits;
  a->bf16 = dtype == BI_DTYPE_BF16;
  a->ld = ld;
  a->V = (int)V;
  if (sp) {
    const bool any = sp->temperature || sp->top_k || sp->top_p || sp->min_p;
    if (any && sp->n < 1) return bad(BI_ERR_INVALID_ARG, "sampling parameters need n >= 1");
    if (any && !param_row && sp->n < T)
      return bad(BI_ERR_INVALID_ARG, "fewer sampling parameters than rows and no param_row");
    a->temperature = sp->temperature;
    a->top_k = sp->top_k;
    a->top_p = sp->top_p;
    a->min_p = sp->min_p;
    a->n_params = sp->n;
  }
  a->param_row = param_row;
  a->status = device_status_ptr();
  return BI_OK;
}

bi_status sample_rows(const float* logits, int64_t T, int64_t V, const bi_sampling* sampling, const int32_t* param_row,
                      const float* u, int64_t u_ld, int64_t u_rows, const int32_t* u_row, const int32_t* ids_in,
                      const int32_t* dst, int32_t* ids_out, float* lp_out, cudaStream_t st) {
  if (T == 0) return BI_OK;
  SampleArgs a{};
  BI_TRY(sample_args(__func__, logits, BI_DTYPE_FP32, T, V, V, sampling, param_row, &a));
  a.u = u;
  a.u_ld = u_ld;
  a.u_rows = u_rows;
  a.u_row = u_row;
  a.ids_in = ids_in;
  a.dst = dst;
  a.ids_out = ids_out;
  a.lp_out = lp_out;
  return dispatch_sample(a, T, st);
}

}  // namespace bi

extern "C" {

bi_status bi_sample(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const bi_sampling* sampling,
                    const int32_t* param_row, const float* u, int64_t u_rows, const int32_t* u_row, int32_t* ids_out,
                    float* logprob_out, void* stream) {
  using namespace bi;
  BI_REQUIRE(T >= 0, "T < 0");
  if (T == 0) return BI_OK;
  BI_REQUIRE(u && ids_out, "null pointer");
  BI_REQUIRE(u_rows >= 1, "u_rows must be positive");
  SampleArgs a{};
  BI_TRY(sample_args(__func__, logits, dtype, T, V, ld, sampling, param_row, &a));
  a.u = u;
  a.u_ld = T;
  a.u_rows = u_rows;
  a.u_row = u_row;
  a.ids_out = ids_out;
  a.lp_out = logprob_out;
  return dispatch_sample(a, T, as_stream(stream));
}

bi_status bi_sample_logprob(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                            const bi_sampling* sampling, const int32_t* param_row, const int32_t* ids,
                            float* logprob_out, void* stream) {
  using namespace bi;
  BI_REQUIRE(T >= 0, "T < 0");
  if (T == 0) return BI_OK;
  BI_REQUIRE(ids && logprob_out, "null pointer");
  SampleArgs a{};
  BI_TRY(sample_args(__func__, logits, dtype, T, V, ld, sampling, param_row, &a));
  a.ids_in = ids;
  a.lp_out = logprob_out;
  return dispatch_sample(a, T, as_stream(stream));
}

}  // extern "C"
