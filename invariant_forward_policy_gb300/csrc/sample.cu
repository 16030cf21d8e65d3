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
// fixed-point integers of about 2^44 for the largest: 2^(j/64) from a table (Tang's table-driven
// exponential, ACM TOMS 15, 1989) times a cubic in the remainder, whose argument is reduced in two
// floats, about 5e-10 relative.  Integer sums have no order, every quantity below is defined by
// them alone, and so a row's bits depend neither on how many CTAs share it, nor on which of the
// ways to its cut below was taken, nor on T.
//
// A row is read once, into the shared memory of a cluster of 1, 2, 4 or 8 CTAs (fp32).  Then
//  - nothing cut but by min-p: one pass sums the masses;
//  - top_k up to 1024: the k-th largest of the threads' own maxima (known from the read) bounds the
//    k-th largest logit from below, so that only a few more than k logits pass it; one CTA orders
//    those and does the rest;
//  - top-p: a histogram of counts over k = 64 log2 w (1/64 octave) predicts where the cut is; one
//    pass sums the masses and lists the logits next to the prediction, and one CTA orders the list
//    and finds the cut, exactly;
//  - anything else (top_k above 1024, lists that overflow, a missed prediction): the cut by
//    histograms with masses, on octaves first and on the float's bits then, until the bin fits the
//    sort or holds equal values only, whose first few by index are counted out.
// The draw finds the CTA, then the warp, then the token whose running mass crosses u S.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <string>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace bi {

typedef unsigned long long u64;

constexpr int kSmpThreads = 512;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpBins = 2048;             // bins of top-p's counts; the last one is open
constexpr int kSmpMaxBins = 256;           // bins of the threads' maxima
constexpr int kSmpMassBins = 1024;         // bins of a histogram with masses (count and three 16-bit limbs)
constexpr int kSmpList = 2048;             // candidates that one CTA orders
constexpr int kSmpLocal = 1024;            // candidates that one CTA of several lists
constexpr int kSmpMaxK = 1024;             // top_k up to which the kept set goes straight to the list
constexpr int kSmpMaxShare = 32768;        // logits of one CTA: a limb's sum stays below 2^31
constexpr int kSmpMaxV = 8 * kSmpMaxShare; // 2^18 masses below 2^44.6 sum to less than 2^63
constexpr int kSmpOne = 380000000;         // mantissa of 1: the largest for which the table's products below round
                                           // by the magic number (|2 kSmpOne (2^(1/128) - 1)| < 2^22), with some room
constexpr int kSmpFrac = 15;               // mass = mantissa (below 2^29.6) << 15 >> octaves below the largest
constexpr int kSmpTabLanes = 16;           // table copies: 8-byte reads of a half-warp have no bank conflict
constexpr float kSmpMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to an integer in the low bits
constexpr int kSmpMagicBits = 0x4B400000;

// round(kSmpOne * 2^(j / 64))
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
  u64 mass;      // mass through the cut
};
struct SmpFind { // a bin and what lies before it
  int32_t bin;   // -1: the target is beyond the total
  uint32_t before, inside;
  u64 before_mass, inside_mass;
};

// Static shared memory of one CTA.
struct SmpShared {
  // the row's parameters, by one thread
  double log_min_p;               // T ln(min_p)
  float c_hi, c_lo, r_hi, r_lo;   // 64 log2(e) / T and 1 / T, each in two floats
  float p, u, min_p, x_id;
  int32_t k_eff, id, ok;
  float wmax[kSmpWarps], wmin[kSmpWarps];
  // written by the cluster's CTAs, each at its rank: what all of them need is then at hand locally
  float cta_max[8], cta_min[8];
  u64 cta_sum[8];
  int32_t cta_idx[8];
  // values that the cluster's other CTAs read, or write here
  u64 wsum[kSmpWarps], wsum2[kSmpWarps];
  uint32_t wcnt[kSmpWarps];
  u64 pub_sum[2];                 // two sets, used in turn
  uint32_t pub_cnt[2], pub_lo[2], pub_hi[2];
  uint32_t list_n;                // entries of this CTA's own list (rank 0: of the joint list)
  SmpFind find;
  SmpCut cut;
  // one CTA's results
  float x_cut;
  u64 total, total2;
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

// floor(f S) for 0 <= f < 1, exactly; *rest: whether f S is no integer.
BI_DEV u64 smp_mul_floor(float f, u64 S, bool* rest) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const u64 mant = ex ? ((b & 0x7fffffu) | 0x800000u) : (b & 0x7fffffu);
  const int sh = 150 - (ex ? ex : 1);  // f = mant 2^-sh, sh >= 24
  const u64 hi = __umul64hi(mant, S), lo = mant * S;
  u64 q, r;
  if (sh < 64) {
    q = (hi << (64 - sh)) | (lo >> sh);
    r = lo << (64 - sh);
  } else {
    const int s2 = sh - 64;
    q = s2 < 64 ? hi >> s2 : 0ull;
    r = lo | (s2 < 64 ? (s2 ? hi << (64 - s2) : 0ull) : hi);
  }
  *rest = r != 0ull;
  return q;
}

template <typename T>
BI_DEV T smp_warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x - m and its rounding error
BI_DEV float smp_diff(float x, float m, float* err) {
  const float d = __fsub_rn(x, m);
  const float b = __fsub_rn(d, x);
  *err = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
  return d;
}

BI_DEV u64 smp_pair(float lo, float hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BI_DEV void smp_unpair(u64 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
BI_DEV u64 smp_fma2(u64 a, u64 b, u64 c) {  // two floats at once, each rounded as fma
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
BI_DEV u64 smp_mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  float floor_;  // ABS: logits below it are raised to it; else: x - m at or below it has no mass
  int k_top;     // k of the maximum
  int oct_top;   // its octave
  int shift0;    // (shift0 - bits of the rounded sum) >> 6 = 32 - kSmpFrac + octaves below the top one
  BI_DEV void init(float m_, float hi, float lo) {
    m = m_;
    c_hi = hi;
    c_lo = lo;
    floor_ = __fdiv_rn(ABS ? -1048576.f : -4096.f, c_hi);
    k_top = ABS ? k_of(m) : 0;
    oct_top = k_top >> 6;
    shift0 = (oct_top + 32 - kSmpFrac) * 64 + 63 + kSmpMagicBits;
  }
  // k of an element; lower elements than the masses reach may have any k far below k_top
  BI_DEV int k_of(float x) const {
    if (ABS) return __float_as_int(__fmaf_rn(fmaxf(x, floor_), c_hi, kSmpMagic)) - kSmpMagicBits;
    return __float_as_int(__fmaf_rn(fmaxf(__fsub_rn(x, m), floor_), c_hi, kSmpMagic)) - kSmpMagicBits;
  }
  BI_DEV int bin(float x) const { return min(k_top - k_of(x), kSmpBins - 1); }
  // The mass from the rounded sum (k in its low bits) and g = 2^(f/64) - 1: the table's 2^(k mod 64 / 64) and its
  // product with g, rounded to an integer by the magic number (taken off the table's integers), then shifted by
  // the octave: (mantissa 2^32) >> s, where a shift of 64 or more gives 0.
  BI_DEV u64 scale(int q, float g, const uint2* tab) const {
    const uint2 t = tab[(q & 63) * kSmpTabLanes];
    const uint32_t M = t.x + (uint32_t)__float_as_int(__fmaf_rn(__uint_as_float(t.y), g, kSmpMagic));
    u64 w;
    asm("shr.b64 %0, %1, %2;" : "=l"(w) : "l"((u64)M << 32), "r"((shift0 - q) >> 6));
    return w;
  }
  BI_DEV u64 mass(float x, const uint2* tab) const {
    float q, f;
    if (ABS) {
      x = fmaxf(x, floor_);
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
    return scale(__float_as_int(q), g, tab);
  }
  // Four masses, the same bits: the float operations of ABS on two logits at a time.
  BI_DEV void mass4(const float (&x)[4], const uint2* tab, u64 (&w)[4]) const {
    if (!ABS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = mass(x[i], tab);
      return;
    }
    const u64 hi = smp_pair(c_hi, c_hi), lo = smp_pair(c_lo, c_lo), magic = smp_pair(kSmpMagic, kSmpMagic);
    const u64 minus = smp_pair(-1.f, -1.f), b1 = smp_pair(a1, a1), b2 = smp_pair(a2, a2), b3 = smp_pair(a3, a3);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const u64 v = smp_pair(fmaxf(x[i], floor_), fmaxf(x[i + 1], floor_));
      const u64 q = smp_fma2(v, hi, magic);
      u64 f = smp_fma2(v, hi, smp_fma2(q, minus, magic));
      f = smp_fma2(v, lo, f);
      const u64 g = smp_mul2(f, smp_fma2(f, smp_fma2(f, b3, b2), b1));
      float q0, q1, g0, g1;
      smp_unpair(q, q0, q1);
      smp_unpair(g, g0, g1);
      w[i] = scale(__float_as_int(q0), g0, tab);
      w[i + 1] = scale(__float_as_int(q1), g1, tab);
    }
  }
};

// ln of a kept token's probability: (x - m) / T - ln(S / W), W the mass of the maximum; both terms in two
// floats until the last sum.
BI_DEV float smp_logprob(float x, float m, float r_hi, float r_lo, u64 S, u64 W) {
  float dl;
  const float d = smp_diff(x, m, &dl);
  const float ah = __fmul_rn(d, r_hi);
  const float al = __fadd_rn(__fmaf_rn(d, r_hi, -ah), __fmaf_rn(d, r_lo, __fmul_rn(dl, r_hi)));
  // q = S / W in two floats, S and W each split into 24 and 40 bits
  const float sh = __ull2float_rz(S & ~0xffffffffffull), sl = __ull2float_rn(S & 0xffffffffffull);
  const float wh = __ull2float_rz(W & ~0xffffffull), wl = __ull2float_rn(W & 0xffffffull);  // W < 2^45
  float qh = __fdiv_rn(__fadd_rn(sh, sl), __fadd_rn(wh, wl));
  const float rem = __fadd_rn(__fmaf_rn(-qh, wh, sh), __fmaf_rn(-qh, wl, sl));
  float ql = __fdiv_rn(rem, wh);
  // S may exceed 2^40 sums of 24 bits: sh holds 23 bits above bit 40, exact
  int e = (__float_as_int(qh) >> 23) - 127;
  const float scale = __int_as_float((127 - e) << 23);
  qh = __fmul_rn(qh, scale);  // in [1, 2)
  ql = __fmul_rn(ql, scale);
  if (qh >= 1.5f) {
    qh = __fmul_rn(qh, 0.5f);
    ql = __fmul_rn(ql, 0.5f);
    ++e;
  }
  const float ln2h = 45426.f / 65536.f, ln2l = 1.4286068203e-6f;  // e * ln2h is exact
  const float s = __fsub_rn(__fmaf_rn(-(float)e, ln2h, ah), logf(qh));
  return __fadd_rn(s, __fsub_rn(__fsub_rn(al, __fmul_rn((float)e, ln2l)), __fdiv_rn(ql, qh)));
}

// One row per cluster of CS CTAs.
template <int CS>
struct SmpRow {
  const SampleArgs& a;
  SmpShared& sh;
  float* xs;         // this CTA's logits, -inf before and after them
  uint2* table;      // [64][kSmpTabLanes]
  const uint2* tab;  // this lane's copy of it
  unsigned char* area;  // 24 KB: own list or counts [kSmpBins] (8 KB); list or masses [4][kSmpMassBins] (16 KB)
  cg::cluster_group cl;
  int tid, warp, lane, rank;
  int base;          // row index of position 0 of xs
  int slabs, per;    // slabs of 128 positions of this CTA, and of each of its warps
  int par;           // set of the published values in use
  float m, x_min;    // row maximum; smallest logit that min-p keeps (above -inf)
  int64_t row;
  int k_eff;
  float p;
  bool score;

  BI_DEV uint32_t* counts() { return reinterpret_cast<uint32_t*>(area); }
  BI_DEV u64* own_list() { return reinterpret_cast<u64*>(area); }
  BI_DEV u64* list() { return reinterpret_cast<u64*>(area + kSmpLocal * 8); }

  BI_DEV void csync() {
    if (CS == 1) __syncthreads();
    else cl.sync();
  }
  template <typename P>
  BI_DEV P* at(P* ptr, int r) {
    if (CS == 1) return ptr;
    return cl.map_shared_rank(ptr, r);
  }
  BI_DEV int slab_lo(int w) { return min(slabs, w * per); }
  BI_DEV int slab_hi(int w) { return min(slabs, w * per + per); }

  // visit(position, x) for this warp's elements
  template <typename F>
  BI_DEV void each(F visit) {
    const int s1 = slab_hi(warp);
    for (int s = slab_lo(warp); s < s1; ++s) {
      const int p0 = s * 128 + lane * 4;
      const float4 v = *reinterpret_cast<const float4*>(xs + p0);
      visit(p0, v.x);
      visit(p0 + 1, v.y);
      visit(p0 + 2, v.z);
      visit(p0 + 3, v.w);
    }
  }

  // Inclusive sums over the CTA's threads, and their totals.
  BI_DEV void block_scan(uint32_t& c, u64& w, uint32_t* tot_c, u64* tot_w) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t c2 = __shfl_up_sync(0xffffffffu, c, o);
      const u64 w2 = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) {
        c += c2;
        w += w2;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sh.wcnt[warp] = c;
      sh.wsum[warp] = w;
    }
    __syncthreads();
    uint32_t bc = 0, tc = 0;
    u64 bw = 0, tw = 0;
#pragma unroll
    for (int i = 0; i < kSmpWarps; ++i) {
      const uint32_t ci = sh.wcnt[i];
      const u64 wi = sh.wsum[i];
      if (i < warp) {
        bc += ci;
        bw += wi;
      }
      tc += ci;
      tw += wi;
    }
    c += bc;
    w += bw;
    *tot_c = tc;
    *tot_w = tw;
  }
  // Publishes this CTA's (count, mass); sums over lower ranks and over all ranks.
  uint32_t base_c, tot_c;
  u64 base_w, tot_w;
  BI_DEV void cluster_scan(uint32_t c, u64 w) {
    par ^= 1;
    if (tid == 0) {
      sh.pub_cnt[par] = c;
      sh.pub_sum[par] = w;
    }
    csync();
    base_c = tot_c = 0;
    base_w = tot_w = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const uint32_t cr = *at(&sh.pub_cnt[par], r);
      const u64 wr = *at(&sh.pub_sum[par], r);
      if (r < rank) {
        base_c += cr;
        base_w += wr;
      }
      tot_c += cr;
      tot_w += wr;
    }
  }
  // Rank r sums bins [r slice, (r + 1) slice) over the cluster (sum(b, &count, &mass)) and leaves their
  // inclusive prefix sums in its own shared memory (put); base_* and tot_* then hold the ranks' sums.
  template <int NB, typename F, typename G>
  BI_DEV void reduce(F sum, G put) {
    constexpr int slice = NB / CS;
    constexpr int BPT = slice > kSmpThreads ? slice / kSmpThreads : 1;
    uint32_t c[BPT], cs = 0;
    u64 w[BPT], ws = 0;
    const bool mine = tid * BPT < slice;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      c[i] = 0;
      w[i] = 0;
      if (mine) sum(rank * slice + tid * BPT + i, c[i], w[i]);
      cs += c[i];
      ws += w[i];
      c[i] = cs;
      w[i] = ws;
    }
    uint32_t ic = cs, tc;
    u64 iw = ws, tw;
    block_scan(ic, iw, &tc, &tw);
    if (mine) {
#pragma unroll
      for (int i = 0; i < BPT; ++i) put(rank * slice + tid * BPT + i, ic - cs + c[i], iw - ws + w[i]);
    }
    cluster_scan(tc, tw);
  }
  // The bin where the running count or mass reaches target (>= 1), to every rank: get(b, &count, &mass) reads
  // the prefix sums of reduce.
  template <int NB, typename G>
  BI_DEV SmpFind find(bool by_mass, u64 target, G get) {
    constexpr int slice = NB / CS;
    for (int i = tid; i < slice; i += kSmpThreads) {
      const int b = rank * slice + i;
      uint32_t c0 = base_c, c1;
      u64 w0 = base_w, w1;
      if (i > 0) {
        get(b - 1, c1, w1);
        c0 += c1;
        w0 += w1;
      }
      get(b, c1, w1);
      c1 += base_c;
      w1 += base_w;
      if (by_mass ? (w0 < target && target <= w1) : (c0 < target && target <= c1)) {
        const SmpFind f{b, c0, c1 - c0, w0, w1 - w0};
        for (int r = 0; r < CS; ++r) *at(&sh.find, r) = f;
      }
    }
    csync();
    return (by_mass ? tot_w : (u64)tot_c) < target ? SmpFind{-1, 0, 0, 0ull, 0ull} : sh.find;
  }

  // ---- lists of candidates: (key descending, index ascending) as one ascending 64-bit key
  BI_DEV u64 entry(float x, int pos) { return (u64)(~smp_key(x)) << 32 | (uint32_t)(base + pos); }
  BI_DEV static float entry_x(u64 e) { return smp_unkey(~(uint32_t)(e >> 32)); }
  // Appends (warp-converged) to a list of at most cap entries; those beyond are counted only.
  BI_DEV void append(bool take, float x, int pos, uint32_t* n, u64* l, uint32_t cap) {
    const unsigned who = __ballot_sync(0xffffffffu, take);
    if (who == 0u) return;
    uint32_t o = 0;
    if (lane == 0) o = atomicAdd(n, (uint32_t)__popc(who));
    o = __shfl_sync(0xffffffffu, o, 0) + __popc(who & ((1u << lane) - 1u));
    if (take && o < cap) l[o] = entry(x, pos);
  }
  // Bitonic sort of list[0, n) ascending (one CTA).
  BI_DEV void sort(int n) {
    u64* l = list();
    int n2 = 2;
    while (n2 < n) n2 <<= 1;
    for (int i = n + tid; i < n2; i += kSmpThreads) l[i] = ~0ull;
    __syncthreads();
    for (int size = 2; size <= n2; size <<= 1)
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        for (int t = tid; t < n2 / 2; t += kSmpThreads) {
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
  // Masses of list[0, n) in order (mass_of(entry)), then the first entry at which the running mass (or, for
  // !by_mass, the number of entries) reaches target_of(total mass): its position (n: none) and the mass through
  // it, to every thread of the CTA.
  template <typename F, typename G>
  BI_DEV int list_find(int n, bool by_mass, F mass_of, G target_of, u64* through) {
    constexpr int EPT = kSmpList / kSmpThreads;
    const u64* l = list();
    u64 w[EPT], ws = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = tid * EPT + i;
      w[i] = e < n ? mass_of(l[e]) : 0ull;
      ws += w[i];
    }
    uint32_t c = 0, tc;
    u64 run = ws, total;
    if (tid == 0) sh.pos = n;
    block_scan(c, run, &tc, &total);
    run -= ws;
    const u64 target = target_of(total);
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = tid * EPT + i;
      const u64 next = run + w[i];
      if (e < n && (by_mass ? (run < target && target <= next) : (u64)(e + 1) == target)) {
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

  // ceil(p S), at least 1: the mass at which top-p stops
  BI_DEV u64 top_p_target(u64 S) {
    if (!(p > 0.f)) return 1ull;
    bool rest;
    const u64 q = smp_mul_floor(p, S, &rest);
    return q + (rest || q == 0ull ? 1ull : 0ull);
  }
  BI_DEV u64 draw_target(u64 S) {
    bool rest;
    return smp_mul_floor(sh.u, S, &rest) + 1ull;
  }


  BI_DEV void write(int32_t out_id, float lp) {
    const int64_t o = a.dst ? (int64_t)a.dst[row] : row;
    if (!score && a.ids_out) a.ids_out[o] = out_id;
    if (a.lp_out) a.lp_out[o] = lp;
  }
  template <bool ABS>
  BI_DEV void write_token(const SmpMass<ABS>& ms, int32_t i, float x, u64 S) {
    write(i, smp_logprob(x, m, sh.r_hi, sh.r_lo, S, ms.mass(m, tab)));
  }
  BI_DEV float value(int32_t i) {
    const int64_t at = row * a.ld + i;
    return a.bf16 ? bf2f(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
  }

  // ---- sums over the row, and the draw.  weight4(index of the first, x, w) gives four elements' weights.
  // Warp sums to sh.wsum; then, with publish(), the CTA's sum to every rank's sh.cta_sum.
  template <typename F>
  BI_DEV void warp_sums(F weight4) {
    u64 sum = 0;
    const int s1 = slab_hi(warp);
    for (int s = slab_lo(warp); s < s1; ++s) {
      const int p0 = s * 128 + lane * 4;
      const float4 v = *reinterpret_cast<const float4*>(xs + p0);
      const float x[4] = {v.x, v.y, v.z, v.w};
      u64 w[4];
      weight4(base + p0, x, w);
      sum += (w[0] + w[1]) + (w[2] + w[3]);
    }
    sum = smp_warp_sum(sum);
    if (lane == 0) sh.wsum[warp] = sum;
  }
  BI_DEV void publish() {
    __syncthreads();
    if (CS > 1) {
      if (tid < CS) {
        u64 t = 0;
#pragma unroll
        for (int i = 0; i < kSmpWarps; ++i) t += sh.wsum[i];
        at(sh.cta_sum, tid)[rank] = t;
      }
      csync();
    } else {
      if (tid == 0) {
        u64 t = 0;
#pragma unroll
        for (int i = 0; i < kSmpWarps; ++i) t += sh.wsum[i];
        sh.cta_sum[0] = t;
      }
      __syncthreads();
    }
  }
  BI_DEV u64 row_sum() {
    u64 t = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) t += sh.cta_sum[r];
    return t;
  }
  // After publish(): the element, in index order, at which the running weight reaches target (>= 1); the CTA that
  // holds it calls found(index, x).  A warp's slabs are taken by a warp each, then the one slab by one warp.
  template <typename F, typename H>
  BI_DEV void locate(F weight4, u64 target, H found) {
    u64 b = 0, mine = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const u64 t = sh.cta_sum[r];
      if (r < rank) b += t;
      if (r == rank) mine = t;
    }
    if (!(b < target && target <= b + mine)) return;
    int unit = 0;
    for (; unit < kSmpWarps - 1; ++unit) {
      const u64 t = sh.wsum[unit];
      if (target <= b + t) break;
      b += t;
    }
    const int s0 = slab_lo(unit), s1 = slab_hi(unit);
    for (int sb = s0; sb < s1; sb += kSmpWarps) {  // one round, for up to 16 slabs a warp
      const int s = sb + warp;
      float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      const int p0 = s * 128 + lane * 4;
      u64 y[4] = {0, 0, 0, 0}, inc;
      if (s < s1) {
        const float4 v = *reinterpret_cast<const float4*>(xs + p0);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
        weight4(base + p0, x, y);
      }
      inc = (y[0] + y[1]) + (y[2] + y[3]);
      u64 run = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 z = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += z;
      }
      run = inc - run;
      if (lane == 31) sh.wsum2[warp] = inc;
      __syncthreads();
      u64 before = b, all = b;
#pragma unroll
      for (int i = 0; i < kSmpWarps; ++i) {
        const u64 t = sh.wsum2[i];
        if (i < warp) before += t;
        all += t;
      }
      run += before;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (run < target && target <= run + y[i]) found(base + p0 + i, x[i]);
        run += y[i];
      }
      if (target <= all) break;
      b = all;
      __syncthreads();
    }
  }

  // ---- the cut by histograms with masses, for whatever the quicker ways do not take
  template <bool ABS>
  BI_DEV SmpCut select(const SmpMass<ABS>& ms, bool by_mass, bool top_p, u64 target, uint32_t* all_c, u64* all_w) {
    uint32_t* h = reinterpret_cast<uint32_t*>(list());
    uint32_t lo = 0, hi = 0xffffffffu;  // keys of the active elements, once the bins are on keys
    int bin = -1, shift = 0;            // bin of the octave histogram, then shift of the key histograms
    int level = 0;
    u64 before_c = 0, before_w = 0;
    while (true) {
      auto active = [&](float x) {
        if (!(x >= x_min)) return false;
        if (level == 0) return true;
        if (level == 1) return min(ms.bin(x) >> 1, kSmpMassBins - 1) == bin;
        const uint32_t k = smp_key(x);
        return k >= lo && k <= hi;
      };
      csync();  // the counters' memory is free in every rank
      for (int i = tid; i < 4 * kSmpMassBins; i += kSmpThreads) h[i] = 0u;
      __syncthreads();
      each([&](int, float x) {
        if (active(x)) {
          const int b = level == 0 ? ms.bin(x) >> 1 : (int)((hi - smp_key(x)) >> shift);
          const u64 w = ms.mass(x, tab);
          atomicAdd(&h[b], 1u);
          atomicAdd(&h[kSmpMassBins + b], (uint32_t)w & 0xffffu);
          atomicAdd(&h[2 * kSmpMassBins + b], (uint32_t)(w >> 16) & 0xffffu);
          atomicAdd(&h[3 * kSmpMassBins + b], (uint32_t)(w >> 32));
        }
      });
      csync();
      reduce<kSmpMassBins>(
          [&](int b, uint32_t& c, u64& w) {
            for (int r = 0; r < CS; ++r) {
              const uint32_t* g = at(h, r);
              c += g[b];
              w += (u64)g[kSmpMassBins + b] + ((u64)g[2 * kSmpMassBins + b] << 16) +
                   ((u64)g[3 * kSmpMassBins + b] << 32);
            }
          },
          [&](int b, uint32_t c, u64 w) {
            h[b] = c;
            h[kSmpMassBins + b] = (uint32_t)w;
            h[2 * kSmpMassBins + b] = (uint32_t)(w >> 32);
          });
      if (level == 0) {
        *all_c = tot_c;
        *all_w = tot_w;
        if (top_p) target = top_p_target(target ? target : tot_w);  // target: the mass that top-k left, or 0
      }
      const SmpFind f = find<kSmpMassBins>(by_mass, target - (by_mass ? before_w : before_c),
                                           [&](int b, uint32_t& c, u64& w) {
                                             c = h[b];
                                             w = (u64)h[2 * kSmpMassBins + b] << 32 | h[kSmpMassBins + b];
                                           });
      if (f.bin < 0) return SmpCut{smp_key(x_min), 0x7fffffff, tot_w};  // fewer elements than asked for: all stay
      before_c += f.before;
      before_w += f.before_mass;
      if (level == 0) {
        bin = f.bin;
      } else {
        hi = hi - ((uint32_t)f.bin << shift);
        const uint32_t width = (1u << shift) - 1u;
        lo = hi - min(width, hi - lo);
      }
      ++level;
      if (level == 1 || f.inside > (uint32_t)kSmpList) {
        // smallest and largest key of the bin
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
        if (lane == 0) {
          sh.wcnt[warp] = kmin;
          sh.wsum[warp] = kmax;
        }
        __syncthreads();
        par ^= 1;
        if (tid == 0) {
          for (int i = 0; i < kSmpWarps; ++i) {
            kmin = min(kmin, sh.wcnt[i]);
            kmax = max(kmax, (uint32_t)sh.wsum[i]);
          }
          sh.pub_lo[par] = kmin;
          sh.pub_hi[par] = kmax;
        }
        csync();
        for (int r = 0; r < CS; ++r) {
          kmin = min(kmin, *at(&sh.pub_lo[par], r));
          kmax = max(kmax, *at(&sh.pub_hi[par], r));
        }
        lo = kmin;
        hi = kmax;
        level = 2;
        shift = max(0, 32 - __clz(kmax - kmin) - 10);
      }
      const u64 left = target - (by_mass ? before_w : before_c);
      if (lo == hi) {  // equal values: the first `need` of them by index
        const float x1 = smp_unkey(lo);
        const u64 w1 = ms.mass(x1, tab);
        const u64 need = by_mass ? (left + w1 - 1) / w1 : left;  // a bin that mass reached has some
        auto one = [&](int, const float (&x)[4], u64 (&w)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = x[i] >= x_min && x[i] == x1 ? 1ull : 0ull;
        };
        warp_sums(one);
        publish();
        locate(one, need, [&](int i, float) {
          for (int r = 0; r < CS; ++r) at(&sh.cut, r)->idx = i;
        });
        csync();
        const SmpCut c{lo, sh.cut.idx, before_w + need * w1};
        csync();
        return c;
      }
      if (f.inside <= (uint32_t)kSmpList) {
        u64* l = at(list(), 0);
        uint32_t* n = at(&sh.list_n, 0);
        if (tid == 0) sh.list_n = 0;
        csync();
        each([&](int pos, float x) {
          if (active(x)) l[atomicAdd(n, 1u)] = entry(x, pos);
        });
        csync();
        if (rank == 0) {
          sort((int)f.inside);
          u64 through;
          const int pos = list_find((int)f.inside, by_mass, [&](u64 e) { return ms.mass(entry_x(e), tab); },
                                    [&](u64) { return left; }, &through);
          if (tid == 0) {
            const u64 e = list()[pos];
            const SmpCut c{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, before_w + through};
            for (int r = 0; r < CS; ++r) *at(&sh.cut, r) = c;
          }
        }
        csync();
        const SmpCut c = sh.cut;
        csync();
        return c;
      }
    }
  }
  template <bool ABS>
  __device__ __noinline__ SmpCut general(SmpMass<ABS> ms) {
    uint32_t all_c;
    u64 all_w;
    SmpCut cut{smp_key(x_min), 0x7fffffff, 0ull};
    u64 left = 0;
    if (k_eff < a.V) {
      cut = select(ms, false, false, (u64)k_eff, &all_c, &all_w);
      left = cut.mass;
    }
    if (p < 1.f) {
      const SmpCut c = select(ms, true, true, left, &all_c, &all_w);
      if (c.key > cut.key || (c.key == cut.key && c.idx < cut.idx)) cut = c;
    }
    return cut;
  }

  // ---- top-k up to kSmpMaxK: candidates by the threads' maxima.  False: too many of them.
  template <bool ABS>
  BI_DEV bool few(const SmpMass<ABS>& ms, float t_max, float row_min) {
    // bins linear in x, from the row's maximum to the smallest of the threads' maxima (counts() is zeroed)
    const float scale = fminf(__fdiv_rn((float)(kSmpMaxBins - 2), __fsub_rn(m, row_min)), FLT_MAX);
    if (t_max >= x_min) {
      const float y = __fmul_rn(__fsub_rn(m, t_max), scale);
      atomicAdd(&counts()[y < (float)(kSmpMaxBins - 1) ? (int)y : kSmpMaxBins - 1], 1u);
    }
    csync();
    if (warp == 0) {
      // lane l sums bins 8 l .. 8 l + 7 of the cluster's CTAs
      uint32_t c[8], n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        const uint4* q = reinterpret_cast<const uint4*>(at(counts(), r)) + lane * 2;
        const uint4 v0 = q[0], v1 = q[1];
        c[0] += v0.x;
        c[1] += v0.y;
        c[2] += v0.z;
        c[3] += v0.w;
        c[4] += v1.x;
        c[5] += v1.y;
        c[6] += v1.z;
        c[7] += v1.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) n += c[i];
      uint32_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      uint32_t run = inc - n;
      int bin = kSmpMaxBins - 1;  // fewer maxima than k: every logit is a candidate
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (run < (uint32_t)k_eff && (uint32_t)k_eff <= run + c[i]) bin = lane * 8 + i;
        run += c[i];
      }
      bin = __reduce_min_sync(0xffffffffu, bin);
      // k_eff of the maxima lie in the bins up to this one, so the k_eff largest logits are not below its end
      // (made lower by more than the roundings above)
      if (lane == 0) {
        const float depth = __fmul_rn(__fdiv_rn((float)(bin + 1), scale), 1.000001f);
        sh.x_cut = bin == kSmpMaxBins - 1 ? x_min : fmaxf(x_min, __fsub_rd(m, depth));
      }
    }
    __syncthreads();
    const float x_cut = sh.x_cut;
    uint32_t* n = at(&sh.list_n, 0);
    u64* l = at(list(), 0);
    const int s1 = slab_hi(warp);
    for (int s = slab_lo(warp); s < s1; ++s) {
      const int p0 = s * 128 + lane * 4;
      const float4 v = *reinterpret_cast<const float4*>(xs + p0);
      const float top = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
      if (__any_sync(0xffffffffu, top >= x_cut)) {
        append(v.x >= x_cut, v.x, p0, n, l, kSmpList);
        append(v.y >= x_cut, v.y, p0 + 1, n, l, kSmpList);
        append(v.z >= x_cut, v.z, p0 + 2, n, l, kSmpList);
        append(v.w >= x_cut, v.w, p0 + 3, n, l, kSmpList);
      }
    }
    csync();
    const uint32_t total = *n;
    if (total > (uint32_t)kSmpList) return false;
    if (rank == 0) {
      if (total <= (uint32_t)kSmpThreads / 4) small<4>(ms, (int)total);
      else if (total <= (uint32_t)kSmpThreads) small<1>(ms, (int)total);
      else {
        SmpRow other = *this;  // as in finish()
        other.small_sorted(ms, (int)total);
      }
    }
    return true;
  }
  // The row's kept set lies in the list of at most kSmpThreads entries (one CTA): G threads (or one) per entry sum
  // what comes before it in order, then in index order.
  template <int G, typename F>
  BI_DEV u64 sum_before(int n, int g, const u64* wl, F before, int* count) {
    const u64* l = list();
    u64 w = 0;
    int c = 0;
#pragma unroll 4
    for (int j = g; j < n; j += G) {
      const u64 y = wl[j];
      if (before(l[j])) {
        w += y;
        ++c;
      }
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    *count = c;
    return w;
  }
  template <int G, bool ABS>
  BI_DEV void small(const SmpMass<ABS>& ms, int n) {
    u64* l = list();
    u64* wl = l + kSmpThreads;
    const int i = tid / G, g = tid % G;
    const bool mine = i < n;
    const u64 e = mine ? l[i] : 0ull;
    const float x = entry_x(e);
    u64 w = mine ? ms.mass(x, tab) : 0ull;
    if (g == 0) wl[i] = w;
    if (tid == 0) sh.total2 = 0ull;
    __syncthreads();
    const int k = min(n, k_eff);
    int before = 0;
    u64 before_w = 0;
    if (warp * 32 / G < n) {
      before_w = sum_before<G>(n, g, wl, [&](u64 y) { return y < e; }, &before);
      if (mine && before == k - 1) sh.total = before_w + w;  // the mass that top-k leaves
    }
    __syncthreads();
    bool kept = mine && before < k;
    if (p < 1.f) {
      const u64 target = top_p_target(sh.total);
      kept = kept && before_w < target;
      if (kept && target <= before_w + w) sh.total2 = before_w + w;
    }
    if (!kept) w = 0;
    if (g == 0) wl[i] = w;
    const bool it = kept && score && (int32_t)(uint32_t)e == sh.id && g == 0;
    const int any = __syncthreads_or(it);
    const u64 S = p < 1.f ? sh.total2 : sh.total;
    if (score) {
      if (it) write_token(ms, sh.id, x, S);
      if (!any && tid == 0) write(sh.id, -INFINITY);  // cut off, or not among the candidates
    } else if (warp * 32 / G < n) {
      const u64 run = sum_before<G>(n, g, wl, [&](u64 y) { return (uint32_t)y < (uint32_t)e; }, &before);
      const u64 target = draw_target(S);
      if (g == 0 && run < target && target <= run + w) write_token(ms, (int32_t)(uint32_t)e, x, S);
    }
  }
  // The same for up to kSmpList entries, by sorts.
  template <bool ABS>
  __device__ __noinline__ void small_sorted(SmpMass<ABS> ms, int n) {
    u64* l = list();
    sort(n);
    n = min(n, k_eff);
    u64 S;
    int last = list_find(n, true, [&](u64 e) { return ms.mass(entry_x(e), tab); },
                         [&](u64 total) { return p < 1.f ? top_p_target(total) : total + 1ull; }, &S);
    if (last == n) last = n - 1;  // no top-p: all of them, with or without mass
    if (score) {
      const u64 e = (u64)(~smp_key(sh.x_id)) << 32 | (uint32_t)sh.id;
      if (tid == 0) {
        if (e <= l[last]) write_token(ms, sh.id, sh.x_id, S);
        else write(sh.id, -INFINITY);
      }
      return;
    }
    // index order: (index, mass) in one key (18 and 46 bits)
    for (int i = tid; i <= last; i += kSmpThreads) {
      const u64 e = l[i];
      l[i] = (e << 46) | ms.mass(entry_x(e), tab);
    }
    __syncthreads();
    sort(last + 1);
    u64 through;
    const int pos = list_find(last + 1, true, [&](u64 e) { return e & ((1ull << 46) - 1ull); },
                              [&](u64 total) { return draw_target(total); }, &through);
    if (tid == 0) {
      const int32_t best = (int32_t)(l[pos] >> 46);
      write_token(ms, best, value(best), S);
    }
  }

  // ---- top-p over the whole row: predicted cut, exact sums.  False: the prediction missed, or a list is full.
  template <bool ABS>
  BI_DEV bool nucleus(const SmpMass<ABS>& ms) {
    for (int i = tid; i < kSmpBins; i += kSmpThreads) counts()[i] = 0u;
    __syncthreads();
    each([&](int, float x) {
      const int b = ms.k_top - ms.k_of(x);
      if (x >= x_min && b < kSmpBins - 1) atomicAdd(&counts()[b], 1u);  // the open bin would only serialise
    });
    csync();
    // a bin's mass is about its count times 2^(k / 64); the open bin's is left out of the prediction
    u64* est = list();
    reduce<kSmpBins>(
        [&](int b, uint32_t& c, u64& w) {
#pragma unroll
          for (int r = 0; r < CS; ++r) c += at(counts(), r)[b];
          const int k = ms.k_top - b;
          if (b < kSmpBins - 1) w = ((u64)c * kExp2Tab[k & 63]) << kSmpFrac >> (ms.oct_top - (k >> 6));
        },
        [&](int b, uint32_t, u64 w) { est[b - rank * (kSmpBins / CS)] = w; });
    __syncthreads();
    const u64 guess = top_p_target(tot_w);
    const SmpFind f = find<kSmpBins>(true, guess, [&](int b, uint32_t& c, u64& w) {
      c = 0;
      w = est[b - rank * (kSmpBins / CS)];
    });
    if (f.bin < 0 || f.bin >= kSmpBins - 2) return false;
    // a bin of many logits is cut at the fraction of its mass that is still wanted, to within 0.15 of it;
    // one of few, anywhere in it or next to it
    const float k_bin = (float)(ms.k_top - f.bin);
    float hi = k_bin + 1.5f, lo = k_bin - 1.5f;
    if (f.inside_mass >= 64ull * ((u64)kExp2Tab[(ms.k_top - f.bin) & 63] << kSmpFrac >>
                                  (ms.oct_top - ((ms.k_top - f.bin) >> 6)))) {
      const float mid = k_bin + 0.5f - __fdiv_rn((float)(guess - f.before_mass), (float)f.inside_mass);
      hi = mid + 0.15f;
      lo = mid - 0.15f;
    }
    const float x_lo = fmaxf(x_min, ABS ? __fdiv_rn(lo, ms.c_hi) : __fadd_rn(m, __fdiv_rn(lo, ms.c_hi)));
    const float x_hi = fmaxf(x_lo, ABS ? __fdiv_rn(hi, ms.c_hi) : __fadd_rn(m, __fdiv_rn(hi, ms.c_hi)));
    u64 all = 0, above = 0;
    const int s1 = slab_hi(warp);
    u64* ml = CS == 1 ? list() : own_list();
    constexpr uint32_t cap = CS == 1 ? kSmpList : kSmpLocal;
    for (int s = slab_lo(warp); s < s1; ++s) {
      const int p0 = s * 128 + lane * 4;
      const float4 v = *reinterpret_cast<const float4*>(xs + p0);
      const float x[4] = {v.x, v.y, v.z, v.w};
      bool near = false;
      u64 w[4];
      ms.mass4(x, tab, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (x[i] >= x_min) all += w[i];
        if (x[i] > x_hi) above += w[i];
        near |= x[i] <= x_hi && x[i] >= x_lo;
      }
      if (__any_sync(0xffffffffu, near)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) append(x[i] <= x_hi && x[i] >= x_lo, x[i], p0 + i, &sh.list_n, ml, cap);
      }
    }
    all = smp_warp_sum(all);
    above = smp_warp_sum(above);
    if (lane == 0) {
      sh.wsum[warp] = all;
      sh.wsum2[warp] = above;
    }
    csync();
    // rank 0 collects the sums and the lists
    if (rank == 0) {
      if (warp == 0) {
        u64 t = 0, t2 = 0;
        for (int g = lane; g < CS * kSmpWarps; g += 32) {
          t += at(sh.wsum, g / kSmpWarps)[g % kSmpWarps];
          t2 += at(sh.wsum2, g / kSmpWarps)[g % kSmpWarps];
        }
        t = smp_warp_sum(t);
        t2 = smp_warp_sum(t2);
        if (lane == 0) {
          sh.total = t;
          sh.total2 = t2;
        }
      }
      uint32_t n = 0;
      bool fits = true;
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        const uint32_t nr = *at(&sh.list_n, r);
        fits = fits && nr <= cap && n + nr <= (uint32_t)kSmpList;
        if (CS > 1 && fits)
          for (uint32_t i = tid; i < nr; i += kSmpThreads) list()[n + i] = at(own_list(), r)[i];
        n += nr;
      }
      __syncthreads();
      const u64 over = sh.total2, target = top_p_target(sh.total);
      if (tid == 0) sh.cut = SmpCut{0u, -1, 0ull};
      __syncthreads();
      if (fits && over < target) list_cut(ms, (int)n, over, target);
      __syncthreads();
      const SmpCut c = sh.cut;
      if (tid < CS && tid > 0) *at(&sh.cut, tid) = c;
      if (score && c.idx >= 0 && tid == 0) {
        const u64 e = (u64)(~smp_key(sh.x_id)) << 32 | (uint32_t)sh.id;
        if (e <= ((u64)(~c.key) << 32 | (uint32_t)c.idx)) write_token(ms, sh.id, sh.x_id, c.mass);
        else write(sh.id, -INFINITY);
      }
    }
    csync();
    const SmpCut cut = sh.cut;
    if (cut.idx < 0) return false;
    if (score) return true;
    // the warps' kept sums: what lies above the list, and the list's kept entries
    const u64 last = (u64)(~cut.key) << 32 | (uint32_t)cut.idx;
    for (uint32_t i = tid; i < sh.list_n; i += kSmpThreads) {
      const u64 e = ml[i];
      if (e <= last) atomicAdd(&sh.wsum2[((int)(uint32_t)e - base) / 128 / per], ms.mass(entry_x(e), tab));
    }
    __syncthreads();
    if (tid < kSmpWarps) sh.wsum[tid] = sh.wsum2[tid];
    publish();
    draw(ms, cut);
    return true;
  }
  // The entry of list[0, n) at which the mass in order, from `over` on, reaches target, to sh.cut (one CTA).
  template <bool ABS>
  BI_DEV void list_cut(const SmpMass<ABS>& ms, int n, u64 over, u64 target) {
    u64* l = list();
    if (n <= kSmpThreads) {
      u64* wl = l + kSmpThreads;
      const u64 e = tid < n ? l[tid] : 0ull;
      const u64 w = tid < n ? ms.mass(entry_x(e), tab) : 0ull;
      wl[tid] = w;
      __syncthreads();
      if (warp * 32 < n) {
        u64 run = over;
        for (int j = 0; j < n; ++j)
          if (l[j] < e) run += wl[j];
        if (tid < n && run < target && target <= run + w)
          sh.cut = SmpCut{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, run + w};
      }
    } else {
      sort(n);
      u64 through;
      const int pos = list_find(n, true, [&](u64 e) { return ms.mass(entry_x(e), tab); },
                                [&](u64) { return target - over; }, &through);
      if (tid == 0 && pos < n) {
        const u64 e = l[pos];
        sh.cut = SmpCut{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, over + through};
      }
    }
  }

  template <bool ABS>
  struct Kept {  // masses of the kept elements
    const SmpMass<ABS>& ms;
    const uint2* tab;
    float x;
    int32_t idx;
    BI_DEV void operator()(int i0, const float (&v)[4], u64 (&w)[4]) const {
      ms.mass4(v, tab, w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(v[i] > x || (v[i] == x && i0 + i <= idx))) w[i] = 0ull;
    }
  };
  // The draw from the kept set, after publish().
  template <bool ABS>
  BI_DEV void draw(const SmpMass<ABS>& ms, const SmpCut& cut) {
    const u64 S = row_sum();
    locate(Kept<ABS>{ms, tab, smp_unkey(cut.key), cut.idx}, draw_target(S),
           [&](int i, float x) { write_token(ms, i, x, S); });
  }

  // False: nothing in this CTA's shared memory is reached by others any more.
  template <bool ABS>
  BI_DEV bool finish(float t_max, float row_min) {
    SmpMass<ABS> ms;
    ms.init(m, sh.c_hi, sh.c_lo);
    SmpCut cut{smp_key(x_min), 0x7fffffff, 0ull};
    if (k_eff < a.V || p < 1.f) {
      if constexpr (ABS) {
        if (k_eff < a.V && k_eff <= kSmpMaxK) {
          if (few(ms, t_max, row_min)) return true;
        } else if (k_eff == a.V) {
          if (nucleus(ms)) return true;
        }
      }
      SmpRow other = *this;  // the rare way's own copy, so that this one stays in registers
      cut = other.general(ms);
      if (score) {
        if (rank == 0 && tid == 0) {
          const u64 e = (u64)(~smp_key(sh.x_id)) << 32 | (uint32_t)sh.id;
          if (e <= ((u64)(~cut.key) << 32 | (uint32_t)cut.idx)) write_token(ms, sh.id, sh.x_id, cut.mass);
          else write(sh.id, -INFINITY);
        }
        return true;
      }
      warp_sums(Kept<ABS>{ms, tab, smp_unkey(cut.key), cut.idx});
    } else if (x_min == -FLT_MAX) {
      warp_sums([&](int, const float (&x)[4], u64 (&w)[4]) { ms.mass4(x, tab, w); });
    } else {
      warp_sums(Kept<ABS>{ms, tab, x_min, 0x7fffffff});
    }
    publish();
    if (!score) draw(ms, cut);
    else if (rank == 0 && tid == 0) write_token(ms, sh.id, sh.x_id, row_sum());
    return false;
  }

  // The row's parameters and constants, by one thread.
  BI_DEV void setup() {
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
      if (id >= 0 && id < a.V) x = value(id);
      else ok = false;
    } else {
      const int64_t ur = a.u_row ? (int64_t)*a.u_row : 0;
      if (ur >= 0 && ur < a.u_rows) u = a.u[ur * a.u_ld + (a.dst ? (int64_t)a.dst[row] : row)];
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
    sh.log_min_p = mp > 0.f && mp < 1.f ? (double)T * log((double)mp) : 0.0;
    sh.p = q;
    sh.u = u;
    sh.min_p = mp;
    sh.x_id = x;
    sh.id = id;
    sh.k_eff = k <= 0 || k > a.V ? a.V : k;
    sh.ok = ok;
    sh.list_n = 0;
  }

  template <typename TL>
  BI_DEV void run() {
    score = a.ids_in != nullptr;
    // ---- load: 16-byte vectors aligned to memory; positions before and after the share hold -inf
    constexpr int VE = 16 / sizeof(TL), UNROLL = 8;
    const int lo = min(a.V, rank * a.share), n = min(a.V, lo + a.share) - lo;
    const TL* src = static_cast<const TL*>(a.logits) + row * a.ld + lo;
    const int a0 = (int)((reinterpret_cast<uintptr_t>(src) / sizeof(TL)) % VE);
    base = lo - a0;
    slabs = (n + a0 + 127) / 128;
    per = (slabs + kSmpWarps - 1) / kSmpWarps;
    const TL* src0 = src - a0;
    const int v_lo = a0 > 0 ? 1 : 0, v_hi = (a0 + n) / VE, v_end = slabs * (128 / VE);  // whole vectors: [v_lo, v_hi)
    float mx = -INFINITY;  // NaN once one is seen
    auto put = [&](int v, const float (&x)[VE]) {
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        mx = smp_max3_nan(smp_max3_nan(mx, x[i], x[i + 1]), x[i + 2], x[i + 3]);
        *reinterpret_cast<float4*>(xs + v * VE + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    };
    bool first = true;
    for (int v0 = v_lo + tid; v0 - tid < v_hi || first; v0 += kSmpThreads * UNROLL) {
      uint4 raw[UNROLL];
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        const int v = v0 + j * kSmpThreads;
        if (v < v_hi) raw[j] = *reinterpret_cast<const uint4*>(src0 + v * VE);
      }
      if (first) {  // while the loads are on their way
        for (int i = tid; i < 64 * kSmpTabLanes; i += kSmpThreads) {
          const uint32_t t = kExp2Tab[i / kSmpTabLanes];
          table[i] = make_uint2(t - (uint32_t)kSmpMagicBits, __float_as_uint((float)t));
        }
        if (tid == kSmpThreads - 1) setup();
      }
      first = false;
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        const int v = v0 + j * kSmpThreads;
        if (v < v_hi) {
          const uint32_t r[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          float x[VE];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (VE == 4) {
              x[i] = __uint_as_float(r[i]);
            } else {
              x[2 * i] = bf16lo(r[i]);
              x[2 * i + 1] = bf16hi(r[i]);
            }
          }
          put(v, x);
        }
      }
    }
    // the partial vectors at both ends, and -inf up to the end of the last slab
    for (int v = tid; v < v_lo + (v_end - max(v_lo, v_hi)); v += kSmpThreads) {
      const int q = v < v_lo ? v : max(v_lo, v_hi) + v - v_lo;
      float x[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const int at = q * VE + i;
        x[i] = at >= a0 && at < a0 + n ? (float)src0[at] : -INFINITY;
      }
      put(q, x);
    }
    if (tid < kSmpMaxBins) counts()[tid] = 0u;
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
    if (warp == 0) {  // the CTA's to every rank
      mx = sh.wmax[lane & (kSmpWarps - 1)];
      t_min = sh.wmin[lane & (kSmpWarps - 1)];
#pragma unroll
      for (int o = kSmpWarps / 2; o > 0; o >>= 1) {
        mx = smp_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        t_min = fminf(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
      }
      if (lane < CS) {
        at(sh.cta_max, lane)[rank] = mx;
        at(sh.cta_min, lane)[rank] = t_min;
      }
    }
    par = 0;
    csync();
    if (!sh.ok) {  // the same in every CTA of the cluster
      if (rank == 0 && tid == 0) {
        report(a.status, DEV_BAD_INDEX);
        write(-1, NAN);
      }
      return;
    }
    mx = sh.cta_max[0];
    t_min = sh.cta_min[0];
#pragma unroll
    for (int r = 1; r < CS; ++r) {
      mx = smp_max_nan(mx, sh.cta_max[r]);
      t_min = fminf(t_min, sh.cta_min[r]);
    }
    m = mx;
    k_eff = sh.k_eff;
    p = sh.p;
    const bool bad = !(m < INFINITY);  // NaN or +inf
    if (bad || m == -INFINITY) {
      if (rank == 0 && tid == 0) {
        if (bad) report(a.status, DEV_BAD_VALUE);
        write(-1, bad ? NAN : -INFINITY);
      }
      return;
    }
    // the smallest float whose mass is at least min_p
    const float mp = sh.min_p;
    x_min = -FLT_MAX;
    if (mp >= 1.f) x_min = m;
    else if (mp > 0.f) x_min = fmaxf(-FLT_MAX, __double2float_ru((double)m + sh.log_min_p));

    if (score && !(sh.x_id >= x_min)) {
      if (rank == 0 && tid == 0) write(sh.id, -INFINITY);
      return;
    }
    if (k_eff == 1) {  // the first maximum; its logprob is 0
      int32_t at_max = 0x7fffffff;
      each([&](int pos, float x) {
        if (x == m) at_max = min(at_max, base + pos);
      });
      at_max = __reduce_min_sync(0xffffffffu, at_max);
      if (lane == 0) sh.wcnt[warp] = (uint32_t)at_max;
      __syncthreads();
      if (tid == 0) {
        for (int i = 1; i < kSmpWarps; ++i) at_max = min(at_max, (int32_t)sh.wcnt[i]);
        at(sh.cta_idx, 0)[rank] = at_max;
      }
      csync();
      if (rank == 0 && tid == 0) {
        for (int r = 0; r < CS; ++r) at_max = min(at_max, sh.cta_idx[r]);
        write(at_max, score && sh.id != at_max ? -INFINITY : 0.f);
      }
      return;
    }
    if (fabsf(m) * sh.c_hi < 524288.f ? finish<true>(t_max, t_min) : finish<false>(t_max, t_min))
      csync();  // no CTA leaves while another may still reach its shared memory
  }
};

template <typename TL, int CS>
__global__ void __launch_bounds__(kSmpThreads, 2) sample_kernel(const SampleArgs a, int positions) {
  extern __shared__ __align__(16) unsigned char smp_dyn[];
  __shared__ SmpShared sh;
  float* xs = reinterpret_cast<float*>(smp_dyn);
  uint2* tab = reinterpret_cast<uint2*>(xs + positions);
  pdl_trigger();
  pdl_wait();
  SmpRow<CS> r{a, sh, xs, tab, tab + (threadIdx.x & (kSmpTabLanes - 1)),
               reinterpret_cast<unsigned char*>(tab + 64 * kSmpTabLanes), cg::this_cluster()};
  r.tid = threadIdx.x;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  r.rank = CS == 1 ? 0 : (int)r.cl.block_rank();
  r.row = blockIdx.x / CS;
  r.template run<TL>();
}

static int smp_positions(int64_t share) { return (int)(cdiv(share + 8, 128) * 128); }
static size_t smp_dyn_bytes(int64_t share) {
  return (size_t)smp_positions(share) * 4 + 64 * kSmpTabLanes * 8 + kSmpLocal * 8 + kSmpList * 8;
}

template <typename TL, int CS>
static bi_status launch_sample(const SampleArgs& a, int64_t T, cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(sample_kernel<TL, CS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smp_dyn_bytes(kSmpMaxShare));
  });
  if (err != cudaSuccess) return fail(BI_ERR_CUDA, std::string("sample_kernel smem attribute: ") + cudaGetErrorString(err));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(T * CS));
  cfg.blockDim = dim3(kSmpThreads);
  cfg.dynamicSmemBytes = smp_dyn_bytes(a.share);
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
  return launched(cudaLaunchKernelEx(&cfg, sample_kernel<TL, CS>, a, smp_positions(a.share)), "sample_kernel");
}

static bi_status dispatch_sample(SampleArgs& a, int64_t T, cudaStream_t st) {
  // Bits do not depend on the split.  A CTA takes at most 16K logits (64 KB, so that two CTAs share an SM);
  // while the rows leave SMs idle, a row is split further, down to 2K logits a CTA.
  int cs = 1;
  while (cs < 8 && cdiv(a.V, cs) > 16384) cs *= 2;
  while (cs < 8 && cdiv(a.V, cs) > 2048 && T * cs * 2 <= num_sms()) cs *= 2;
  a.share = (int)(cdiv(cdiv(a.V, cs), 8) * 8);
  switch (cs * 2 + (a.bf16 ? 1 : 0)) {
    case 2: return launch_sample<float, 1>(a, T, st);
    case 4: return launch_sample<float, 2>(a, T, st);
    case 8: return launch_sample<float, 4>(a, T, st);
    case 16: return launch_sample<float, 8>(a, T, st);
    case 3: return launch_sample<__nv_bfloat16, 1>(a, T, st);
    case 5: return launch_sample<__nv_bfloat16, 2>(a, T, st);
    case 9: return launch_sample<__nv_bfloat16, 4>(a, T, st);
    default: return launch_sample<__nv_bfloat16, 8>(a, T, st);
  }
}

// Checks that both entry points share; fills the row-independent arguments.
static bi_status sample_args(const char* who, const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                             const bi_sampling* sp, const int32_t* param_row, SampleArgs* a) {
  auto bad = [&](bi_status st, const char* what) { return fail(st, std::string(who) + ": " + what); };
  if (!logits) return bad(BI_ERR_INVALID_ARG, "null logits");
  if (dtype != BI_DTYPE_FP32 && dtype != BI_DTYPE_BF16) return bad(BI_ERR_INVALID_ARG, "dtype must be BI_DTYPE_FP32 or BI_DTYPE_BF16");
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
    if (any && !param_row && sp->n < T) return bad(BI_ERR_INVALID_ARG, "fewer sampling parameters than rows and no param_row");
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
