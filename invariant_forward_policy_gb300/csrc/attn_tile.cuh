// Per-row arithmetic of paged attention, shared by every schedule (decode, prefill, drafted trees).
#pragma once
#include "common.cuh"

namespace bi {

constexpr int kKeys = 64;  // keys per tile = cache block

// Per-row arithmetic (the decode, prefill and tree schedules alike):
// a split of S positions is cut into at most four "lanes" of lane_len =
// roundup(S / 4, 64) positions.  Inside a lane, 64-key tiles are taken in
// ascending order with an fp32 online softmax from a fresh (m, l, acc); the
// lane results are then merged in lane order 0, 1, 2, 3 (lanes with no key
// at or before the row's position are skipped).  The schedule decides only
// who computes a lane (all four warps in parallel for a decode tile, one warp
// after another for a prefill tile), never the arithmetic.

// Shared-memory byte offset of 16-byte chunk `ch` of key row `key` inside a
// 64-key tile: HD/64 boxes of 64 keys x 128 bytes, the chunks of each row
// XOR-swizzled by (key mod 8).  This is the layout a TMA copy with 128-byte
// swizzle writes for a 64x64 bf16 box at a 1024-byte aligned address, and the
// one the cp.async loader below reproduces; ldmatrix reads of 8 consecutive
// keys at one chunk hit 8 different bank groups.
template <int HD>
__device__ __forceinline__ uint32_t kv_off(int key, int ch) {
  return (uint32_t)((ch >> 3) * (kKeys * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
}

// P = 2^x for the attention probabilities: the hardware's ex2 with results
// below 2^-126 flushed to zero (and 2^-inf = +0).  Every schedule, decode and
// prefill, takes P through this one instruction, so their bits stay equal.
__device__ __forceinline__ float exp2_p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The warp's query rows: NH = 2 holds 16 rows per tile (thread (g, qd) rows g and
// g + 8), NH = 1 only rows 0..7 (decode tiles of at most 8 rows: GQA group x
// tokens).  At NH = 1 the m16n8k16 MMAs get zero A rows 8..15 and their D rows
// 8..15 are discarded; a D element depends only on its own A row and B column, so
// rows 0..7 are the same bits either way.
template <int NH>
__device__ __forceinline__ void mma_rows(float (&d)[2 * NH], const uint32_t (&a)[2 * NH], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (NH == 2) {
    mma_bf16_16816(d, a, b0, b1);
  } else {
    float t2, t3;  // rows 8..15 of D: discarded
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%10,%11};"
        : "+f"(d[0]), "+f"(d[1]), "=f"(t2), "=f"(t3)
        : "r"(a[0]), "r"(0u), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1), "f"(0.f), "f"(0.f));
  }
}

// S = Q K^T for the warp's query rows and one 64-key tile (fp32, unscaled).
// qf[kk]: the rows' A fragment of head dims 16 kk .. 16 kk + 15 (h-th row half
// at [h] for dims + 0..7 and at [NH + h] for dims + 8..15).
template <int HD, int NH = 2>
__device__ __forceinline__ void attn_scores(uint32_t sk, const uint32_t (&qf)[HD / 16][2 * NH], int lane,
                                            float (&sc)[8][2 * NH]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < 2 * NH; ++c) sc[j][c] = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int kk = 0; kk < HD / 16; kk += 2) {
      const int key = j * 8 + (lane & 7);
      const int ch = kk * 2 + (lane >> 3);
      uint32_t b0, b1, b2, b3;
      ldsm_x4(sk + kv_off<HD>(key, ch), b0, b1, b2, b3);
      mma_rows<NH>(sc[j], qf[kk], b0, b1);
      mma_rows<NH>(sc[j], qf[kk + 1], b2, b3);
    }
  }
}

// Fold one tile's scores into the online-softmax state of the warp's rows:
// masking by select, fp32 rescaling, then O += P V with P rounded to bf16.
// vsm (FP8 cache only): the tile's V scales; P is then multiplied by its key's
// scale before the bf16 rounding (exact: a power of two), so that P' V_codes has
// the products P (V_codes scale) term for term.
template <int HD, int NH = 2>
__device__ __forceinline__ void attn_update(uint32_t sv, float (&sc)[8][2 * NH], int key0, const bool (&row_valid)[2],
                                            const int (&row_pos)[2], float scale_log2, int lane, float (&m)[2],
                                            float (&l)[2], float (&acc)[HD / 8][2 * NH],
                                            const float* vsm = nullptr) {
  const int tq = lane & 3;
  float pr[8][2 * NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    float tmax = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kp = key0 + j * 8 + tq * 2 + e;
        const bool ok = row_valid[h] && kp <= row_pos[h];
        const float v = ok ? __fmul_rn(sc[j][h * 2 + e], scale_log2) : -INFINITY;
        sc[j][h * 2 + e] = v;
        tmax = fmaxf(tmax, v);
      }
    }
    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
    const float m_new = fmaxf(m[h], tmax);
    const float alpha = (m_new == m[h]) ? 1.0f : exp2f(__fsub_rn(m[h], m_new));
    float rs = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = sc[j][h * 2 + e];
        const float pv = (v == -INFINITY) ? 0.f : exp2_p(__fsub_rn(v, m_new));
        pr[j][h * 2 + e] = pv;
        rs = __fadd_rn(rs, pv);
      }
    }
    rs = __fadd_rn(rs, __shfl_xor_sync(0xffffffffu, rs, 1));
    rs = __fadd_rn(rs, __shfl_xor_sync(0xffffffffu, rs, 2));
    l[h] = __fadd_rn(__fmul_rn(l[h], alpha), rs);
    m[h] = m_new;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      acc[j][h * 2] = __fmul_rn(acc[j][h * 2], alpha);
      acc[j][h * 2 + 1] = __fmul_rn(acc[j][h * 2 + 1], alpha);
    }
  }
  if (vsm) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 vv = *reinterpret_cast<const float2*>(vsm + j * 8 + tq * 2);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        pr[j][h * 2] = __fmul_rn(pr[j][h * 2], vv.x);
        pr[j][h * 2 + 1] = __fmul_rn(pr[j][h * 2 + 1], vv.y);
      }
    }
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {  // 64 keys = 4 k-steps of 16
    uint32_t pa[2 * NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      pa[h] = pack_bf16x2(pr[2 * kk][h * 2], pr[2 * kk][h * 2 + 1]);
      pa[NH + h] = pack_bf16x2(pr[2 * kk + 1][h * 2], pr[2 * kk + 1][h * 2 + 1]);
    }
#pragma unroll
    for (int j = 0; j < HD / 8; j += 2) {
      const int key = kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
      const int ch = j + (lane >> 4);
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(sv + kv_off<HD>(key, ch), b0, b1, b2, b3);
      mma_rows<NH>(acc[j], pa, b0, b1);
      mma_rows<NH>(acc[j + 1], pa, b2, b3);
    }
  }
}

// One 64-key tile into the online-softmax state of 16 query rows (one warp).
// ksm / vsm (FP8 cache only): the tile holds unscaled e4m3 values and these are
// its per-key K and V scales.  A score column is multiplied by its key's K
// scale: Q (codes x 2^k)^T = 2^k (Q codes^T) exactly.
template <int HD, int NH = 2>
__device__ __forceinline__ void attn_tile(uint32_t sk, uint32_t sv, int key0, const uint32_t (&qf)[HD / 16][2 * NH],
                                          const bool (&row_valid)[2], const int (&row_pos)[2], float scale_log2,
                                          int lane, float (&m)[2], float (&l)[2], float (&acc)[HD / 8][2 * NH],
                                          const float* ksm = nullptr, const float* vsm = nullptr) {
  float sc[8][2 * NH];
  attn_scores<HD, NH>(sk, qf, lane, sc);
  if (ksm) {
    const int tq = lane & 3;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 kk = *reinterpret_cast<const float2*>(ksm + j * 8 + tq * 2);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        sc[j][h * 2] = __fmul_rn(sc[j][h * 2], kk.x);
        sc[j][h * 2 + 1] = __fmul_rn(sc[j][h * 2 + 1], kk.y);
      }
    }
  }
  attn_update<HD, NH>(sv, sc, key0, row_valid, row_pos, scale_log2, lane, m, l, acc, vsm);
}

// Per-thread state of one lane (its NH row halves), as stored in shared memory
// between lanes.
template <int HD, int NH = 2>
struct LaneState {
  float m[NH], l[NH];
  float acc[HD / 8][2 * NH];
};

// P <- P (+) Q for the rows a thread holds; an empty Q leaves P unchanged, an
// empty P takes Q as it is.
template <int HD, int NH = 2>
__device__ __forceinline__ void lane_merge(LaneState<HD, NH>& P, const float* mq, const float* lq,
                                           const float (&accq)[HD / 8][2 * NH]) {
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    if (mq[h] == -INFINITY) continue;
    if (P.m[h] == -INFINITY) {
      P.m[h] = mq[h];
      P.l[h] = lq[h];
#pragma unroll
      for (int j = 0; j < HD / 8; ++j) {
        P.acc[j][h * 2] = accq[j][h * 2];
        P.acc[j][h * 2 + 1] = accq[j][h * 2 + 1];
      }
      continue;
    }
    const float M = fmaxf(P.m[h], mq[h]);
    const float a = (P.m[h] == M) ? 1.0f : exp2f(__fsub_rn(P.m[h], M));
    const float b = (mq[h] == M) ? 1.0f : exp2f(__fsub_rn(mq[h], M));
    P.l[h] = __fadd_rn(__fmul_rn(P.l[h], a), __fmul_rn(lq[h], b));
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = h * 2 + e;
        P.acc[j][c] = __fadd_rn(__fmul_rn(P.acc[j][c], a), __fmul_rn(accq[j][c], b));
      }
    }
    P.m[h] = M;
  }
}

}  // namespace bi
