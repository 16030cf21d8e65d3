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
// fixed-point integers in units of 2^-45 of the largest one: 2^(k/64) from a table (Tang's
// table-driven exponential, ACM TOMS 15, 1989) times a cubic in the remainder, with the argument
// reduced in two floats, about 3e-10 relative.  Integer sums have no order, so a row's bits depend
// neither on how many CTAs share it nor on T, and histograms may use atomics.
//
// A row is held in the shared memory of a cluster of 1, 2, 4 or 8 CTAs (fp32, read once).  The cut
// comes from a histogram over k = 64 log2 w (2048 bins, 1/64 octave), summed over the cluster through
// distributed shared memory, and a sort of the one bin that holds the border; a bin with more
// candidates than the sort holds is refined on the float's bits first, down to equal values, whose
// first few by index are counted out.  The draw finds the CTA, then the warp, then the token whose
// running mass crosses u S.
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
constexpr int kSmpBins = 2048;             // histogram bins of 1/64 octave; the last one is open
constexpr int kSmpRefineBins = 1024;       // bins of a refinement on the float's bits
constexpr int kSmpList = 2048;             // candidates that one CTA sorts
constexpr int kSmpMaxK = 1024;             // top_k up to which the kept set goes straight to the list
constexpr int kSmpMaxShare = 32768;        // logits of one CTA
constexpr int kSmpMaxV = 8 * kSmpMaxShare; // 2^18 masses of at most 2^45 sum to at most 2^63
constexpr int kSmpFrac = 45;               // the largest mass is 2^45
constexpr float kSmpMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to an integer in the low bits
constexpr int kSmpMagicBits = 0x4B400000;

// round(2^30 * 2^(j / 64))
__constant__ uint32_t kExp2Tab[64] = {
    0x40000000, 0x40B268FA, 0x4166C34C, 0x421D1462, 0x42D561B4, 0x438FB0CB, 0x444C0740, 0x450A6ABB,
    0x45CAE0F2, 0x468D6FAE, 0x47521CC6, 0x4818EE22, 0x48E1E9BA, 0x49AD1598, 0x4A7A77D4, 0x4B4A169C,
    0x4C1BF829, 0x4CF022CA, 0x4DC69CDD, 0x4E9F6CD4, 0x4F7A9930, 0x50582888, 0x51382182, 0x521A8AD7,
    0x52FF6B55, 0x53E6C9DA, 0x54D0AD5A, 0x55BD1CDB, 0x56AC1F75, 0x579DBC57, 0x5891FAC1, 0x5988E209,
    0x5A82799A, 0x5B7EC8F2, 0x5C7DD7A4, 0x5D7FAD59, 0x5E8451D0, 0x5F8BCCDB, 0x60962665, 0x61A3666D,
    0x62B39509, 0x63C6BA64, 0x64DCDEC3, 0x65F60A7F, 0x6712460B, 0x683199ED, 0x69540EC9, 0x6A79AD56,
    0x6BA27E65, 0x6CCE8AE1, 0x6DFDDBCC, 0x6F307A41, 0x70666F76, 0x719FC4B9, 0x72DC8374, 0x741CB528,
    0x75606374, 0x76A7980F, 0x77F25CCE, 0x7940BB9E, 0x7A92BE8B, 0x7BE86FBA, 0x7D41D96E, 0x7E9F0606};

// Device pointers of one call.
struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V, share;  // share: logits per CTA, a multiple of 8
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int64_t n_params;
  const int32_t* param_row;
  const float* u;         // draw
  int64_t u_ld, u_rows;   // row stride and rows of u
  const int32_t* u_row;
  const int32_t* ids_in;  // score
  int32_t* ids_out;
  float* lp_out;
  const int32_t* dst;     // results of row t go to index dst[t] (or t)
  int* status;
};

struct SmpCut {  // an element is kept iff its key is larger, or equal and its index not above idx
  uint32_t key;
  int32_t idx;
  u64 mass;      // mass through the cut
};
struct SmpFind { // a bin and what lies before it
  int32_t bin;   // -1: the target is beyond the total
  uint32_t before, inside;
  u64 before_mass;
};

// Static shared memory of one CTA.
struct SmpShared {
  double log_min_p;               // T ln(min_p)
  float c_hi, c_lo, r_hi, r_lo;   // 64 log2(e) / T and 1 / T, each in two floats
  float wmax[kSmpWarps];
  u64 wsum[kSmpWarps];
  uint32_t wcnt[kSmpWarps];
  u64 tail;                       // mass of the open bin
  // values that the cluster's other CTAs read, or write here
  float pub_max[2];
  int pub_bad[2];
  u64 pub_sum[2];
  uint32_t pub_cnt[2], pub_lo[2], pub_hi[2];
  uint32_t list_n;
  SmpFind find;
  SmpCut cut;
  // one CTA's results
  u64 total;
  int32_t pos;
};

BI_DEV uint32_t smp_key(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
BI_DEV float smp_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// floor(f S) and ceil(f S) for 0 <= f < 1, exactly.
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

// The row-wide constants and the two value functions.
struct SmpScale {
  float m;           // row maximum
  float c_hi, c_lo;  // 64 log2(e) / T
  float dmin;        // x - m at or below which the mass is zero

  // k = round(64 log2 w): an integer <= 0, for x - m above dmin
  BI_DEV int bin(float x) const {
    const float d = __fsub_rn(x, m);
    if (!(d > dmin)) return kSmpBins - 1;
    const int k = __float_as_int(__fmaf_rn(d, c_hi, kSmpMagic)) - kSmpMagicBits;
    return min(-k, kSmpBins - 1);
  }
  // Mass mantissa M in [2^30, 2^31) and octave shift e: w = M 2^-30 2^-e.  The difference x - m is
  // taken with its rounding error (two-sum), the product with 64 log2(e) / T reduced against the
  // nearest integer by fused multiply-adds, and 2^(f/64) - 1 is a cubic, |f| <= 1/2.  False: no mass.
  BI_DEV bool mantissa(float x, const uint2* tab, uint32_t& M, int& k) const {
    const float d = __fsub_rn(x, m);
    if (!(d > dmin)) return false;
    const float b = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
    const float q = __fmaf_rn(d, c_hi, kSmpMagic);
    float f = __fmaf_rn(d, c_hi, -__fsub_rn(q, kSmpMagic));
    f = __fmaf_rn(d, c_lo, f);
    f = __fmaf_rn(dl, c_hi, f);
    k = __float_as_int(q) - kSmpMagicBits;
    constexpr float a1 = 0.0108304247f, a2 = 5.86490496e-05f, a3 = 2.11731372e-07f;  // (ln2/64)^n / n!
    const float g = __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, a3, a2), a1));
    const uint2 t = tab[(k & 63) * 32];
    M = t.x + (uint32_t)__float2int_rn(__fmul_rn(__uint_as_float(t.y), g));
    return true;
  }
  BI_DEV u64 mass(float x, const uint2* tab) const {
    uint32_t M;
    int k;
    if (!mantissa(x, tab, M, k)) return 0ull;
    return ((u64)M << (kSmpFrac - 30)) >> min(-(k >> 6), 63);
  }
};

// ln of the token's probability: (x - m) / T - ln(S 2^-45), in two floats, rounded once more at the end.
BI_DEV float smp_logprob(float x, float m, float r_hi, float r_lo, u64 S) {
  const float d = __fsub_rn(x, m);
  const float b = __fsub_rn(d, x);
  const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
  const float ah = __fmul_rn(d, r_hi);
  const float al = __fadd_rn(__fmaf_rn(d, r_hi, -ah), __fmaf_rn(d, r_lo, __fmul_rn(dl, r_hi)));
  const int z = __clzll((long long)S);
  const u64 n = S << z;                               // leading bit at 63
  float mh = __ull2float_rz(n >> 40);                 // 24 bits, exact
  float ml = __ull2float_rn(n & 0xffffffffffull);     // the 40 below
  int e = 63 - z - kSmpFrac;
  mh = __fmul_rn(mh, 0x1p-23f);                       // in [1, 2)
  ml = __fmul_rn(ml, 0x1p-63f);
  if (mh >= 1.5f) {
    mh = __fmul_rn(mh, 0.5f);
    ml = __fmul_rn(ml, 0.5f);
    ++e;
  }
  const float ln2h = 45426.f / 65536.f, ln2l = 1.4286068203e-6f;  // e * ln2h is exact
  const float s = __fsub_rn(__fmaf_rn(-(float)e, ln2h, ah), logf(mh));
  return __fadd_rn(s, __fsub_rn(__fsub_rn(al, __fmul_rn((float)e, ln2l)), __fdiv_rn(ml, mh)));
}

// One row per cluster of CS CTAs.
template <typename TL, int CS, bool SCORE>
struct SmpRow {
  const SampleArgs& a;
  SmpShared& sh;
  float* xs;         // this CTA's logits, -inf before and after them
  const uint2* tab;  // this lane's copy of the table (stride 32)
  uint32_t* hist;    // [3][kSmpBins]
  u64* list;         // [kSmpList], also the refinement's [4][kSmpRefineBins] counters
  cg::cluster_group cl;
  int tid, warp, lane, rank;
  int base;          // row index of position 0 of xs
  int slab_lo, slab_hi;  // this warp's slabs of 128 positions
  int par;           // parity of the published values in use
  SmpScale sc;
  float x_min;       // smallest logit that min-p keeps (above -inf)
  int64_t row;
  int k_eff;
  float p;

  BI_DEV void csync() {
    if (CS == 1) __syncthreads();
    else cl.sync();
  }
  template <typename P>
  BI_DEV P* at(P* ptr, int r) {
    if (CS == 1) return ptr;
    return cl.map_shared_rank(ptr, r);
  }

  // visit(position, x) for this warp's elements
  template <typename F>
  BI_DEV void each(F visit) {
    for (int s = slab_lo; s < slab_hi; ++s) {
      const int p0 = s * 128 + lane * 4;
      const float4 v = *reinterpret_cast<const float4*>(xs + p0);
      visit(p0, v.x);
      visit(p0 + 1, v.y);
      visit(p0 + 2, v.z);
      visit(p0 + 3, v.w);
    }
  }

  // Inclusive block scan over threads of (count, mass); totals to sh.wcnt / sh.wsum users through return values.
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

  // Publishes this CTA's (count, mass); returns the sums over lower ranks and over all ranks.
  BI_DEV void cluster_scan(uint32_t c, u64 w, uint32_t* base_c, u64* base_w, uint32_t* tot_c, u64* tot_w) {
    par ^= 1;
    if (tid == 0) {
      sh.pub_cnt[par] = c;
      sh.pub_sum[par] = w;
    }
    csync();
    uint32_t bc = 0, tc = 0;
    u64 bw = 0, tw = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const uint32_t cr = *at(&sh.pub_cnt[par], r);
      const u64 wr = *at(&sh.pub_sum[par], r);
      if (r < rank) {
        bc += cr;
        bw += wr;
      }
      tc += cr;
      tw += wr;
    }
    *base_c = bc;
    *base_w = bw;
    *tot_c = tc;
    *tot_w = tw;
  }

  // Sum of a per-warp (count, mass) over the CTA (all threads get it); sh.wcnt / sh.wsum keep the warps' values.
  BI_DEV void block_sum(uint32_t c, u64 w, uint32_t* tot_c, u64* tot_w) {
    c = smp_warp_sum(c);
    w = smp_warp_sum(w);
    __syncthreads();
    if (lane == 0) {
      sh.wcnt[warp] = c;
      sh.wsum[warp] = w;
    }
    __syncthreads();
    uint32_t tc = 0;
    u64 tw = 0;
#pragma unroll
    for (int i = 0; i < kSmpWarps; ++i) {
      tc += sh.wcnt[i];
      tw += sh.wsum[i];
    }
    *tot_c = tc;
    *tot_w = tw;
  }

  // ---- first histogram, over bins of k
  // Count (and, for MASS, mass mantissas in two 16-bit limbs: at most 2^15 elements a CTA, so no limb
  // overflows) of every bin.  A bin's elements share their octave, so its mass is one shift of its sum;
  // the open last bin's is summed apart.
  template <bool MASS>
  BI_DEV void histogram() {
    for (int i = tid; i < (MASS ? 3 : 1) * kSmpBins; i += kSmpThreads) hist[i] = 0u;
    __syncthreads();
    u64 tail = 0;
    each([&](int, float x) {
      if (!(x >= x_min)) return;
      if (MASS) {
        uint32_t M;
        int k;
        if (sc.mantissa(x, tab, M, k) && -k < kSmpBins - 1) {
          atomicAdd(&hist[-k], 1u);
          atomicAdd(&hist[kSmpBins - k], M & 0xffffu);
          atomicAdd(&hist[2 * kSmpBins - k], M >> 16);
        } else {
          atomicAdd(&hist[kSmpBins - 1], 1u);
          tail += sc.mass(x, tab);
        }
      } else {
        atomicAdd(&hist[sc.bin(x)], 1u);
      }
    });
    if (MASS) {
      uint32_t c;
      block_sum(0u, tail, &c, &tail);
      if (tid == 0) sh.tail = tail;
    }
    csync();
  }

  // Rank r sums bins [r slice, (r + 1) slice) over the cluster and leaves their inclusive prefix sums in its
  // own counters; base_*: what the lower ranks hold, tot_*: everything.  bin_sum(b, &count, &mass) reads one bin.
  uint32_t base_c, tot_c;
  u64 base_w, tot_w;
  template <int NB, typename F, typename G>
  BI_DEV void reduce(F bin_sum, G put) {
    constexpr int slice = NB / CS;
    constexpr int BPT = slice > kSmpThreads ? slice / kSmpThreads : 1;
    uint32_t c[BPT];
    u64 w[BPT];
    uint32_t cs = 0;
    u64 ws = 0;
    const bool mine = tid * BPT < slice;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      c[i] = 0;
      w[i] = 0;
      if (mine) bin_sum(rank * slice + tid * BPT + i, c[i], w[i]);
      cs += c[i];
      ws += w[i];
      c[i] = cs;
      w[i] = ws;
    }
    uint32_t ic = cs, tc;
    u64 iw = ws, tw;
    block_scan(ic, iw, &tc, &tw);
    // the barriers in block_scan put every read of this slice before the writes
    if (mine) {
#pragma unroll
      for (int i = 0; i < BPT; ++i) put(rank * slice + tid * BPT + i, ic - cs + c[i], iw - ws + w[i]);
    }
    cluster_scan(tc, tw, &base_c, &base_w, &tot_c, &tot_w);
  }
  // The bin where the running count or mass reaches target, to every rank (sh.find; bin -1: nowhere).
  template <int NB, typename G>
  BI_DEV void find(bool by_mass, u64 target, G get) {
    constexpr int slice = NB / CS;
    if (tid == 0) sh.find.bin = -1;
    csync();
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
        const SmpFind f{b, c0, c1 - c0, w0};
        for (int r = 0; r < CS; ++r) *at(&sh.find, r) = f;
      }
    }
    csync();
  }
  template <bool MASS>
  BI_DEV void reduce_first() {
    reduce<kSmpBins>(
        [&](int b, uint32_t& c, u64& w) {
          u64 s = 0;
#pragma unroll
          for (int r = 0; r < CS; ++r) {
            const uint32_t* h = at(hist, r);
            c += h[b];
            if (MASS) s += ((u64)h[2 * kSmpBins + b] << 16) + h[kSmpBins + b];
          }
          if (MASS) {
            if (b == kSmpBins - 1) {
              for (int r = 0; r < CS; ++r) w += *at(&sh.tail, r);
            } else {
              const int e = (b + 63) >> 6;
              w = e <= kSmpFrac - 30 ? s << (kSmpFrac - 30 - e) : s >> (e - (kSmpFrac - 30));
            }
          }
        },
        [&](int b, uint32_t c, u64 w) {
          hist[b] = c;
          if (MASS) {
            hist[kSmpBins + b] = (uint32_t)w;
            hist[2 * kSmpBins + b] = (uint32_t)(w >> 32);
          }
        });
  }
  template <bool MASS>
  BI_DEV void find_first(bool by_mass, u64 target) {
    find<kSmpBins>(by_mass, target, [&](int b, uint32_t& c, u64& w) {
      c = hist[b];
      w = MASS ? ((u64)hist[2 * kSmpBins + b] << 32 | hist[kSmpBins + b]) : 0ull;
    });
  }

  // ---- candidate list, held by rank 0: (key descending, index ascending) as one ascending 64-bit key
  template <typename F>
  BI_DEV void gather(F pred) {
    if (tid == 0 && rank == 0) sh.list_n = 0;
    csync();
    uint32_t* n = at(&sh.list_n, 0);
    u64* l = at(list, 0);
    each([&](int pos, float x) {
      const bool take = pred(x);
      const unsigned who = __ballot_sync(0xffffffffu, take);
      if (who == 0u) return;
      uint32_t o = 0;
      const int lead = __ffs(who) - 1;
      if (lane == lead) o = atomicAdd(n, (uint32_t)__popc(who));
      o = __shfl_sync(0xffffffffu, o, lead) + __popc(who & ((1u << lane) - 1u));
      if (take && o < (uint32_t)kSmpList) l[o] = (u64)(~smp_key(x)) << 32 | (uint32_t)(base + pos);
    });
    csync();
  }
  // Bitonic sort of list[0, n) ascending (one CTA).
  BI_DEV void sort(int n) {
    int n2 = 2;
    while (n2 < n) n2 <<= 1;
    for (int i = n + tid; i < n2; i += kSmpThreads) list[i] = ~0ull;
    __syncthreads();
    for (int size = 2; size <= n2; size <<= 1)
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        for (int t = tid; t < n2 / 2; t += kSmpThreads) {
          const int i = 2 * t - (t & (stride - 1)), j = i + stride;
          const u64 x = list[i], y = list[j];
          if ((x > y) == ((i & size) == 0)) {
            list[i] = y;
            list[j] = x;
          }
        }
        __syncthreads();
      }
  }
  // Masses of list[0, n) in order (mass_of(entry)), then the first entry at which the running mass (or, for
  // !by_mass, the number of entries) reaches target_of(total mass), or the last one: its position and the mass
  // through it, to every thread of the CTA.
  template <typename F, typename G>
  BI_DEV void list_find(int n, bool by_mass, F mass_of, G target_of, int* pos, u64* through) {
    constexpr int EPT = kSmpList / kSmpThreads;
    u64 w[EPT], ws = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = tid * EPT + i;
      w[i] = e < n ? mass_of(list[e]) : 0ull;
      ws += w[i];
    }
    uint32_t c = 0, tc;
    u64 run = ws, total;
    if (tid == 0) sh.pos = -1;
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
    *pos = sh.pos < 0 ? n - 1 : sh.pos;
    *through = sh.pos < 0 ? total : sh.total;
    __syncthreads();
  }

  BI_DEV u64 entry_mass(u64 e) { return sc.mass(smp_unkey(~(uint32_t)(e >> 32)), tab); }
  // ceil(p S), at least 1: the mass at which top-p stops
  BI_DEV u64 top_p_target(u64 S) {
    if (!(p > 0.f)) return 1ull;
    bool rest;
    const u64 q = smp_mul_floor(p, S, &rest);
    return q + (rest || q == 0ull ? 1ull : 0ull);
  }

  // The whole row's kept set lies in the list (one CTA): top-k, top-p and the token.
  BI_DEV void small(int32_t id, float x_id, float u) {
    int n = (int)min(sh.list_n, (uint32_t)kSmpList);
    sort(n);
    n = min(n, k_eff);
    int last;
    u64 S;
    list_find(n, true, [&](u64 e) { return entry_mass(e); },
              [&](u64 total) { return p < 1.f ? top_p_target(total) : total; }, &last, &S);
    if (p >= 1.f) last = n - 1;  // masses of zero after the total is reached are still kept
    if constexpr (SCORE) {
      const u64 e = (u64)(~smp_key(x_id)) << 32 | (uint32_t)id;
      if (tid == 0) write(id, e <= list[last] ? logprob(x_id, S) : -INFINITY);
    } else {
      draw_small(last, S, u);
    }
  }
  BI_DEV void draw_small(int last, u64 S, float u) {
    // index order: (index, mass) in one key (18 and 46 bits)
    for (int i = tid; i <= last; i += kSmpThreads) {
      const u64 e = list[i];
      list[i] = (e << 46) | entry_mass(e);
    }
    __syncthreads();
    sort(last + 1);
    constexpr u64 kMassMask = (1ull << 46) - 1ull;
    int pos;
    u64 through;
    list_find(last + 1, true, [&](u64 e) { return e & kMassMask; },
              [&](u64 total) {
                bool rest;
                return smp_mul_floor(u, total, &rest) + 1ull;
              },
              &pos, &through);
    if (tid == 0) {
      const int32_t best = (int32_t)(list[pos] >> 46);
      write(best, logprob(value(best), S));
    }
  }

  // ---- the cut where the running count or mass of the whole row reaches target
  BI_DEV SmpCut select(bool by_mass, u64 target) {
    find_first<true>(by_mass, target);
    SmpFind f = sh.find;
    uint32_t lo = 0, hi = 0xffffffffu;  // key range of the active elements, once the bins are on keys
    int bin = f.bin;
    bool on_keys = false;
    if (bin < 0) {  // beyond the total: everything eligible is kept
      return SmpCut{smp_key(x_min), 0x7fffffff, tot_w};
    }
    while (true) {
      auto active = [&](float x) {
        if (!(x >= x_min)) return false;
        if (!on_keys) return sc.bin(x) == bin;
        const uint32_t k = smp_key(x);
        return k >= lo && k <= hi;
      };
      if (f.inside <= (uint32_t)kSmpList) {
        gather(active);
        if (rank == 0) {
          const int n = (int)min(sh.list_n, (uint32_t)kSmpList);
          sort(n);
          int pos;
          u64 through;
          const u64 left = by_mass ? target - f.before_mass : target - f.before;
          list_find(n, by_mass, [&](u64 e) { return entry_mass(e); }, [&](u64) { return left; }, &pos, &through);
          if (tid == 0) {
            const u64 e = list[pos];
            const SmpCut c{~(uint32_t)(e >> 32), (int32_t)(uint32_t)e, f.before_mass + through};
            for (int r = 0; r < CS; ++r) *at(&sh.cut, r) = c;
          }
        }
        csync();
        const SmpCut c = sh.cut;
        csync();
        return c;
      }
      // smallest and largest key of the active elements
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
      par ^= 1;
      if (tid == 0) {
        uint32_t a0 = 0xffffffffu, a1 = 0u;
        for (int i = 0; i < kSmpWarps; ++i) {
          a0 = min(a0, sh.wcnt[i]);
          a1 = max(a1, (uint32_t)sh.wsum[i]);
        }
        sh.pub_lo[par] = a0;
        sh.pub_hi[par] = a1;
      }
      csync();
      for (int r = 0; r < CS; ++r) {
        kmin = min(kmin, *at(&sh.pub_lo[par], r));
        kmax = max(kmax, *at(&sh.pub_hi[par], r));
      }
      lo = kmin;
      hi = kmax;
      on_keys = true;
      if (kmin == kmax) {  // equal values: the first `need` of them by index
        const u64 w1 = sc.mass(smp_unkey(kmin), tab);
        u64 need;
        if (by_mass) {
          const u64 left = target - f.before_mass;
          need = w1 ? (left + w1 - 1) / w1 : 1ull;
        } else {
          need = target - f.before;
        }
        if (need < 1) need = 1;
        if (need > f.inside) need = f.inside;
        locate([&](int, float x) { return x >= x_min && smp_key(x) == kmin ? 1ull : 0ull; }, need);
        const SmpCut c{kmin, sh.cut.idx, f.before_mass + need * w1};
        csync();
        return c;
      }
      // refine on the key: at least ten more bits of it
      uint32_t* h = reinterpret_cast<uint32_t*>(list);
      const int s = max(0, 32 - __clz(kmax - kmin) - 10);
      for (int i = tid; i < 4 * kSmpRefineBins; i += kSmpThreads) h[i] = 0u;
      __syncthreads();
      each([&](int, float x) {
        if (active(x)) {
          const uint32_t b = (kmax - smp_key(x)) >> s;
          const u64 w = sc.mass(x, tab);
          atomicAdd(&h[b], 1u);
          atomicAdd(&h[kSmpRefineBins + b], (uint32_t)w & 0xffffu);
          atomicAdd(&h[2 * kSmpRefineBins + b], (uint32_t)(w >> 16) & 0xffffu);
          atomicAdd(&h[3 * kSmpRefineBins + b], (uint32_t)(w >> 32));
        }
      });
      csync();
      const uint32_t keep_c = base_c, keep_tc = tot_c;  // the first histogram's, for a later select
      const u64 keep_w = base_w, keep_tw = tot_w;
      reduce<kSmpRefineBins>(
          [&](int b, uint32_t& c, u64& w) {
            for (int r = 0; r < CS; ++r) {
              const uint32_t* g = at(h, r);
              c += g[b];
              w += (u64)g[kSmpRefineBins + b] + ((u64)g[2 * kSmpRefineBins + b] << 16) +
                   ((u64)g[3 * kSmpRefineBins + b] << 32);
            }
          },
          [&](int b, uint32_t c, u64 w) {
            h[b] = c;
            h[kSmpRefineBins + b] = (uint32_t)w;
            h[2 * kSmpRefineBins + b] = (uint32_t)(w >> 32);
          });
      // a target that rounding put just past this set's mass belongs to its last element
      u64 left = by_mass ? target - f.before_mass : target - f.before;
      if (by_mass && left > tot_w) left = tot_w;
      if (by_mass && left == 0) left = 1;
      if (by_mass && tot_w == 0) {  // no mass at all: cut at the first by order
        by_mass = false;
        left = 1;
        target = (u64)f.before + 1;
      }
      find<kSmpRefineBins>(by_mass, left, [&](int b, uint32_t& c, u64& w) {
        c = h[b];
        w = (u64)h[2 * kSmpRefineBins + b] << 32 | h[kSmpRefineBins + b];
      });
      const SmpFind g = sh.find;
      base_c = keep_c;
      tot_c = keep_tc;
      base_w = keep_w;
      tot_w = keep_tw;
      if (by_mass) target = f.before_mass + left;
      f.before += g.before;
      f.before_mass += g.before_mass;
      f.inside = g.inside;
      hi = kmax - ((uint32_t)g.bin << s);
      lo = hi - ((s ? (1u << s) : 1u) - 1u);
      if (lo < kmin || lo > hi) lo = kmin;
      csync();  // every rank has read its counters' owner before the list is used again
    }
  }

  // The element, in index order, at which the running sum of weight(index, x) reaches target (>= 1): its index and
  // value to every rank's sh.cut.idx / sh.cut.key.  Returns the sum over the row.
  template <typename F>
  BI_DEV u64 sums(F weight) {
    u64 w = 0;
    each([&](int pos, float x) { w += weight(base + pos, x); });
    uint32_t c;
    u64 tot;
    block_sum(0u, w, &c, &tot);
    uint32_t bc, tc;
    u64 all;
    cluster_scan(0u, tot, &bc, &loc_base, &tc, &all);
    return all;
  }
  u64 loc_base;
  template <typename F>
  BI_DEV void locate_in(F weight, u64 target) {
    // sh.wsum holds the warps' sums, loc_base what the lower ranks hold
    u64 b = loc_base;
#pragma unroll
    for (int i = 0; i < kSmpWarps; ++i)
      if (i < warp) b += sh.wsum[i];
    if (b < target && target <= b + sh.wsum[warp]) {  // one warp of the cluster
      for (int s = slab_lo; s < slab_hi; ++s) {
        const int p0 = s * 128 + lane * 4;
        const float4 v = *reinterpret_cast<const float4*>(xs + p0);
        const float x[4] = {v.x, v.y, v.z, v.w};
        u64 w[4], ws = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = weight(base + p0 + i, x[i]);
          ws += w[i];
        }
        u64 inc = ws;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        u64 run = b + inc - ws;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u64 next = run + w[i];
          if (run < target && target <= next) {
            for (int r = 0; r < CS; ++r) {
              SmpCut* c = at(&sh.cut, r);
              c->idx = base + p0 + i;
              c->key = smp_key(x[i]);
            }
          }
          run = next;
        }
        b += __shfl_sync(0xffffffffu, inc, 31);
        if (b >= target) break;
      }
    }
    csync();
  }
  template <typename F>
  BI_DEV void locate(F weight, u64 target) {
    sums(weight);
    locate_in(weight, target);
  }

  BI_DEV void write(int32_t id, float lp) {
    const int64_t o = a.dst ? (int64_t)a.dst[row] : row;
    if (!SCORE && a.ids_out) a.ids_out[o] = id;
    if (a.lp_out) a.lp_out[o] = lp;
  }
  BI_DEV float value(int32_t id) {
    const TL* r = static_cast<const TL*>(a.logits) + row * a.ld;
    return (float)r[id];
  }
  // (x - m) / T - ln S of the row's token.
  BI_DEV float logprob(float x, u64 S) { return smp_logprob(x, sc.m, sh.r_hi, sh.r_lo, S); }

  BI_DEV void run() {
    // ---- the row's parameters (uniform over the cluster)
    const int64_t pr = a.param_row ? (int64_t)a.param_row[row] : row;
    bool ok = !(a.temperature || a.top_k || a.top_p || a.min_p) || (pr >= 0 && pr < a.n_params);
    float T = 1.f, mp = 0.f, u = 0.f;
    int k = 0;
    p = 1.f;
    int32_t id = 0;
    if (ok) {
      if (a.temperature) T = a.temperature[pr];
      if (a.top_k) k = a.top_k[pr];
      if (a.top_p) p = a.top_p[pr];
      if (a.min_p) mp = a.min_p[pr];
    }
    if (SCORE) {
      id = a.ids_in[row];
      ok = ok && id >= 0 && id < a.V;
    } else {
      const int64_t ur = a.u_row ? (int64_t)*a.u_row : 0;
      if (ur >= 0 && ur < a.u_rows) u = a.u[ur * a.u_ld + (a.dst ? (int64_t)a.dst[row] : row)];
      else ok = false;
      ok = ok && u >= 0.f && u < 1.f;
    }
    ok = ok && (T == 0.f || (T >= 0x1p-64f && T <= 0x1p64f)) && p == p && mp == mp;
    if (T == 0.f) {
      T = 1.f;
      k = 1;
      p = 1.f;
      mp = 0.f;
    }
    k_eff = k <= 0 || k > a.V ? a.V : k;
    if (tid == kSmpThreads - 1 && ok) {  // 64-bit constants, by one thread
      const double c = 64.0 * 1.4426950408889634074 / (double)T, r = 1.0 / (double)T;
      sh.c_hi = (float)c;
      sh.c_lo = (float)(c - (double)sh.c_hi);
      sh.r_hi = (float)r;
      sh.r_lo = (float)(r - (double)sh.r_hi);
      sh.log_min_p = mp > 0.f && mp < 1.f ? (double)T * log((double)mp) : 0.0;
    }
    if (!ok) {
      if (rank == 0 && tid == 0) {
        report(a.status, DEV_BAD_INDEX);
        write(-1, NAN);
      }
      return;
    }

    // ---- load: 16-byte vectors aligned to memory; positions before and after the share hold -inf
    constexpr int VE = 16 / sizeof(TL);
    const int lo = min(a.V, rank * a.share), n = min(a.V, lo + a.share) - lo;
    const TL* src = static_cast<const TL*>(a.logits) + row * a.ld + lo;
    const int a0 = (int)((reinterpret_cast<uintptr_t>(src) / sizeof(TL)) % VE);
    base = lo - a0;
    const int slabs = (n + a0 + 127) / 128;
    const int per = (slabs + kSmpWarps - 1) / kSmpWarps;
    slab_lo = min(slabs, warp * per);
    slab_hi = min(slabs, slab_lo + per);
    float mx = -INFINITY;
    bool bad = false;
    const TL* src0 = src - a0;
    for (int v = tid; v < slabs * (128 / VE); v += kSmpThreads) {
      const int p0 = v * VE;
      float x[VE];
      if (p0 >= a0 && p0 + VE <= a0 + n) {
        const uint4 raw = *reinterpret_cast<const uint4*>(src0 + p0);
        const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (VE == 4) {
            x[i] = __uint_as_float(r[i]);
          } else {
            x[2 * i] = bf16lo(r[i]);
            x[2 * i + 1] = bf16hi(r[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) x[i] = p0 + i >= a0 && p0 + i < a0 + n ? (float)src0[p0 + i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        bad |= !(x[i] < INFINITY);  // NaN and +inf
        mx = fmaxf(mx, x[i]);
      }
#pragma unroll
      for (int i = 0; i < VE; i += 4)
        *reinterpret_cast<float4*>(xs + p0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) sh.wmax[warp] = mx;
    const int any_bad = __syncthreads_or(bad);
    par = 0;
    if (tid == 0) {
      for (int i = 0; i < kSmpWarps; ++i) mx = fmaxf(mx, sh.wmax[i]);
      sh.pub_max[0] = mx;
      sh.pub_bad[0] = any_bad;
    }
    csync();
    float m = -INFINITY;
    int row_bad = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      m = fmaxf(m, *at(&sh.pub_max[0], r));
      row_bad |= *at(&sh.pub_bad[0], r);
    }
    sc.m = m;
    sc.c_hi = sh.c_hi;
    sc.c_lo = sh.c_lo;
    sc.dmin = -4096.f / sc.c_hi;
    if (row_bad || m == -INFINITY) {
      if (rank == 0 && tid == 0) {
        if (row_bad) report(a.status, DEV_BAD_VALUE);
        write(-1, row_bad ? NAN : -INFINITY);
      }
      csync();
      return;
    }
    // the smallest float whose mass is at least min_p
    x_min = -FLT_MAX;
    if (mp >= 1.f) {
      x_min = m;
    } else if (mp > 0.f) {
      const double t = (double)m + sh.log_min_p;
      x_min = __double2float_ru(t);
      if (!(x_min >= -FLT_MAX)) x_min = -FLT_MAX;
    }

    const float x_id = SCORE ? value(id) : 0.f;
    if (SCORE && !(x_id >= x_min)) {
      if (rank == 0 && tid == 0) write(id, -INFINITY);
      csync();
      return;
    }
    if (k_eff == 1) {  // the first maximum; its logprob is 0
      const float top = m;
      locate([&](int, float x) { return x == top ? 1ull : 0ull; }, 1ull);
      if (rank == 0 && tid == 0) {
        const int32_t best = sh.cut.idx;
        write(best, SCORE && id != best ? -INFINITY : 0.f);
      }
      csync();
      return;
    }
    SmpCut cut{smp_key(x_min), 0x7fffffff, 0ull};
    bool have_cut = false;
    u64 S = 0;
    if (k_eff <= kSmpMaxK) {
      // the bins down to the k-th largest hold few elements: the rest of the work is one CTA's
      histogram<false>();
      reduce_first<false>();
      find_first<false>(false, (u64)k_eff);
      const SmpFind f = sh.find;
      const int bin = f.bin < 0 ? kSmpBins - 1 : f.bin;
      const uint32_t cand = f.bin < 0 ? tot_c : f.before + f.inside;
      if (cand <= (uint32_t)kSmpList) {
        gather([&](float x) { return x >= x_min && sc.bin(x) <= bin; });
        if (rank == 0) small(id, x_id, u);
        csync();
        return;
      }
      csync();
    }
    if (k_eff < a.V || p < 1.f) {
      histogram<true>();
      reduce_first<true>();
      S = tot_w;
      if ((uint32_t)k_eff < tot_c) {
        cut = select(false, (u64)k_eff);
        have_cut = true;
        S = cut.mass;
      }
      if (p < 1.f) {
        const SmpCut c = select(true, top_p_target(S));
        if (!have_cut || c.key > cut.key || (c.key == cut.key && c.idx < cut.idx)) cut = c;
        have_cut = true;
        S = cut.mass;
      }
    }
    const float cut_x = smp_unkey(cut.key);
    const int32_t cut_i = cut.idx;
    auto kept = [&](int i, float x) { return x > cut_x || (x == cut_x && i <= cut_i); };
    if (SCORE) {
      if (!have_cut) S = sums([&](int i, float x) { return kept(i, x) ? sc.mass(x, tab) : 0ull; });
      if (rank == 0 && tid == 0) write(id, kept(id, x_id) ? logprob(x_id, S) : -INFINITY);
    } else {
      auto weight = [&](int i, float x) { return kept(i, x) ? sc.mass(x, tab) : 0ull; };
      const u64 all = sums(weight);
      if (!have_cut) S = all;
      bool rest;
      locate_in(weight, smp_mul_floor(u, all, &rest) + 1ull);
      if (rank == 0 && tid == 0) write(sh.cut.idx, logprob(smp_unkey(sh.cut.key), S));
    }
    csync();
  }
};

template <typename TL, int CS, bool SCORE>
__global__ void __launch_bounds__(kSmpThreads) sample_kernel(const SampleArgs a, int positions) {
  extern __shared__ __align__(16) unsigned char smp_dyn[];
  __shared__ SmpShared sh;
  float* xs = reinterpret_cast<float*>(smp_dyn);
  uint2* tab = reinterpret_cast<uint2*>(xs + positions);
  uint32_t* hist = reinterpret_cast<uint32_t*>(tab + 64 * 32);
  u64* list = reinterpret_cast<u64*>(hist + 3 * kSmpBins);
  pdl_trigger();
  // one copy of the table per lane: the reads have no bank conflicts
  for (int i = threadIdx.x; i < 64 * 32; i += kSmpThreads) {
    const uint32_t m = kExp2Tab[i >> 5];
    tab[i] = make_uint2(m, __float_as_uint((float)m));
  }
  pdl_wait();
  SmpRow<TL, CS, SCORE> r{a, sh, xs, tab + (threadIdx.x & 31), hist, list, cg::this_cluster()};
  r.tid = threadIdx.x;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  r.rank = CS == 1 ? 0 : (int)r.cl.block_rank();
  r.row = blockIdx.x / CS;
  r.run();
}

static int smp_positions(int64_t share) { return (int)(cdiv(share + 8, 128) * 128); }
static size_t smp_dyn_bytes(int64_t share) {
  return (size_t)smp_positions(share) * 4 + 64 * 32 * 8 + 3 * kSmpBins * 4 + kSmpList * 8;
}

template <typename TL, int CS, bool SCORE>
static bi_status launch_sample(const SampleArgs& a, int64_t T, cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(sample_kernel<TL, CS, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  return launched(cudaLaunchKernelEx(&cfg, sample_kernel<TL, CS, SCORE>, a, smp_positions(a.share)), "sample_kernel");
}

template <typename TL, bool SCORE>
static bi_status dispatch_sample(SampleArgs& a, int64_t T, cudaStream_t st) {
  // Bits do not depend on the split.  A CTA takes at most 16K logits (64 KB, so that two CTAs share an SM);
  // while the rows leave SMs idle, a row is split further, down to 2K logits a CTA.
  int cs = 1;
  while (cs < 8 && cdiv(a.V, cs) > 16384) cs *= 2;
  while (cs < 8 && cdiv(a.V, cs) > 2048 && T * cs * 2 <= num_sms()) cs *= 2;
  a.share = (int)(cdiv(cdiv(a.V, cs), 8) * 8);
  switch (cs) {
    case 1: return launch_sample<TL, 1, SCORE>(a, T, st);
    case 2: return launch_sample<TL, 2, SCORE>(a, T, st);
    case 4: return launch_sample<TL, 4, SCORE>(a, T, st);
    default: return launch_sample<TL, 8, SCORE>(a, T, st);
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
  return ids_in ? dispatch_sample<float, true>(a, T, st) : dispatch_sample<float, false>(a, T, st);
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
  return dtype == BI_DTYPE_FP32 ? dispatch_sample<float, false>(a, T, as_stream(stream))
                                : dispatch_sample<__nv_bfloat16, false>(a, T, as_stream(stream));
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
  return dtype == BI_DTYPE_FP32 ? dispatch_sample<float, true>(a, T, as_stream(stream))
                                : dispatch_sample<__nv_bfloat16, true>(a, T, as_stream(stream));
}

}  // extern "C"
