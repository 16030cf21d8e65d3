// RoPE tables scaled for long contexts, and the rotation of q and k with a K/V write at given cache slots.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §4.2: every phase writes the cache through one path.
// A step that drafts a tree writes a node's K and V at a slot that is not its position, so slots are an
// input here (bi_tree_slot_map or bi_slot_map makes them); the arithmetic is bi_rope_kv_write's.
#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"

namespace bi {

constexpr int kMaxRot = 256;

// Angle a position of pair i in units of 2^-64 turns, so that the angle of position p is w[i] * p modulo one
// turn, exactly: the reduction of far positions costs an integer product.
struct TurnRates {
  uint64_t w[kMaxRot / 2];
};

// cos and sin of t * 2^-64 turns, times the amplitude amp (1 + rho) (a 64-bit number; one float alone may be half a unit
// away), each within 0.6 * 2^-23 of the amplitude.
// The offset from the nearest quarter turn is a sum s + e of two floats (|s| <= pi/4); sin = s + (e (1 - s^2/2) + s^3
// P(s^2)), cos = (1 - s^2/2) + (s^4 Q(s^2) - s e) with the roundings of s^2 and of 1 - s^2/2 carried along, P and Q the
// Taylor series (next terms below 2^-29).  The table is bound by its instructions (about 14 on integers, which run at
// half rate, and 30 on floats a pair) next to its 8 bytes a pair, so the reduction works on the high word: the quarter
// is its two high bits after adding an eighth of a turn, and its offset converts as 24 bits that a float holds exactly
// and the 32 bits behind them.
template <bool AMP>
BI_DEV void turn_cos_sin(uint64_t t, float amp, float rho, float& c_out, float& s_out) {
  const uint32_t hi = (uint32_t)(t >> 32) + 0x20000000u, lo = (uint32_t)t;
  const int r = (int)(hi & 0x3FFFFFFFu) - 0x20000000;  // the offset's high word, in 2^-32 turns
  const float a = (float)(r & ~0x3F) * 0x1p-32f;
  const float b = (float)__funnelshift_l(lo, (uint32_t)r, 26) * 0x1p-58f;
  constexpr float kH = 6.28318548202514648f;   // 2 pi rounded to fp32, and the rest
  constexpr float kL = -1.74845553146951715e-7f;
  const float xh = a * kH;
  const float xl = __fmaf_rn(a, kH, -xh) + __fmaf_rn(a, kL, b * kH);
  const float s = xh + xl;
  const float e = xl - (s - xh);
  const float z = s * s;
  const float zl = __fmaf_rn(s, s, -z);
  const float h = -0.5f * z;
  const float w = 1.0f + h;
  const float wt = (1.0f - w) + h;
  const float P = __fmaf_rn(z, __fmaf_rn(z, __fmaf_rn(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
  const float Q = __fmaf_rn(z, __fmaf_rn(z, __fmaf_rn(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
  const float st = __fmaf_rn(e, w, AMP ? s * __fmaf_rn(z, P, rho) : s * z * P);
  const float ct = (AMP ? __fmaf_rn(rho, w, wt) : wt) + __fmaf_rn(z * z, Q, __fmaf_rn(-s, e, -0.5f * zl));
  const float sn = AMP ? __fmaf_rn(amp, s, amp * st) : s + st;
  const float cs = AMP ? __fmaf_rn(amp, w, amp * ct) : w + ct;
  const bool odd = hi & 0x40000000u;
  c_out = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ ((hi + 0x40000000u) & 0x80000000u));
  s_out = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ (hi & 0x80000000u));
}

// A thread holds V neighbouring pairs and walks positions, all CTAs side by side; a CTA's `rows_step` row groups are
// neighbours.
template <int V, bool AMP>
__global__ void __launch_bounds__(256) rope_scaled_table_kernel(float* __restrict__ table, int64_t max_pos, int half,
                                                                float amp, float rho,
                                                                const __grid_constant__ TurnRates rates) {
  pdl_trigger();
  pdl_wait();
  const int nq = half / V;
  const int rows_step = 256 / nq;
  const int q = threadIdx.x % nq, r = threadIdx.x / nq;
  if (r >= rows_step) return;
  uint64_t w[V], t[V];
  int64_t p = (int64_t)blockIdx.x * rows_step + r;
  const int64_t step = (int64_t)gridDim.x * rows_step;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    w[k] = rates.w[q * V + k];
    t[k] = w[k] * (uint64_t)p;
    w[k] *= (uint64_t)step;
  }
  for (; p < max_pos; p += step) {
    float c[V], s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      turn_cos_sin<AMP>(t[k], amp, rho, c[k], s[k]);
      t[k] += w[k];
    }
    float* row = table + p * (2 * half) + q * V;
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(row + half) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      row[0] = c[0];
      row[half] = s[0];
    }
  }
}

// ---------------------------------------------------------------- rotation and write at slots
struct SlotWriteArgs {
  const __nv_bfloat16* qkv;  // [T, ld]
  int64_t ld;
  const int32_t* pos;
  const int64_t* slots;
  const float* table;  // [max_pos, rot]
  int64_t max_pos, n_slots;
  __nv_bfloat16* q_out;  // [T, Hq, hd]
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;  // [n_blocks, Hkv, 64, hd]
  int Hq, Hkv, hd, rot;
  uint32_t per_inv, hv_inv;  // 2^32 / divisor, rounded up (0: divisor 1)
  int* status;
};

// i / d for i d < 2^32, inv = 2^32 / d rounded up
BI_DEV int fast_div(int i, uint32_t inv) { return inv ? (int)__umulhi((uint32_t)i, inv) : i; }

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), every product and sum rounded, one rounding to bf16: bi_rope_kv_write's
BI_DEV void rotate_pair(float x1, float x2, float c, float s, float& y1, float& y2) {
  y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
}

// One CTA a row; 16-byte vectors of 8 elements.  The items of a row are, per q and k head, its rotated vectors (half
// layout: a vector of the first half with its partner; interleaved: a vector of four pairs) and the vectors of its
// unrotated part, then the vectors of v.  Bound by the loads' latency with as many rows in flight as the SMs hold: a
// thread reads two items before it needs the row's numbers, whose loads run beside them.
template <bool INTER>
__global__ void __launch_bounds__(128) rope_slot_write_kernel(const SlotWriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int64_t pos = a.pos[row];
  const int64_t slot = a.slots[row];
  const uint4* src = reinterpret_cast<const uint4*>(a.qkv + row * a.ld);
  const int hv = a.hd / 8, half = a.rot / 2;
  const int nrot = INTER ? a.rot / 8 : a.rot / 16;  // rotated items of a head
  const int per = hv - a.rot / 8 + nrot;
  const int n_qk = (a.Hq + a.Hkv) * per, n = n_qk + a.Hkv * hv;
  struct Item {
    int h, k;   // head (q, k, then v), vector of it
    bool turn;  // rotated
    uint4 x, y; // the vector, and (half layout) its partner
  };
  auto read = [&](int i) {
    Item t;
    if (i >= n_qk) {
      t.h = fast_div(i - n_qk, a.hv_inv);
      t.k = i - n_qk - t.h * hv;
      t.h += a.Hq + a.Hkv;
      t.turn = false;
    } else {
      t.h = fast_div(i, a.per_inv);
      t.k = i - t.h * per;
      t.turn = t.k < nrot;
      if (!t.turn) t.k += a.rot / 8 - nrot;
    }
    t.x = src[t.h * hv + t.k];
    if (!INTER && t.turn) t.y = src[t.h * hv + t.k + nrot];
    return t;
  };
  const int tid = threadIdx.x;
  Item one{}, two{};
  if (tid < n) one = read(tid);
  if (tid + 128 < n) two = read(tid + 128);
  if (pos < 0 || pos >= a.max_pos) {
    if (tid == 0) report(a.status, DEV_BAD_INDEX);
    return;
  }
  const bool slot_ok = slot >= 0 && slot < a.n_slots;
  if (!slot_ok && tid == 0) report(a.status, DEV_BAD_INDEX);
  const float* cs = a.table + pos * a.rot;
  uint4* qd = reinterpret_cast<uint4*>(a.q_out) + row * a.Hq * hv;
  // vector 0 of kv head 0 at this slot; the next head's is 64 hv further
  const int64_t kv0 = ((slot >> 6) * a.Hkv * 64 + (slot & 63)) * hv;
  auto write = [&](const Item& t) {
    if (t.h >= a.Hq && !slot_ok) return;
    uint4* y = t.h < a.Hq ? qd + t.h * hv
               : t.h < a.Hq + a.Hkv
                   ? reinterpret_cast<uint4*>(a.k_cache) + kv0 + (int64_t)(t.h - a.Hq) * 64 * hv
                   : reinterpret_cast<uint4*>(a.v_cache) + kv0 + (int64_t)(t.h - a.Hq - a.Hkv) * 64 * hv;
    if (!t.turn) {
      y[t.k] = t.x;
      return;
    }
    const uint32_t w1[4] = {t.x.x, t.x.y, t.x.z, t.x.w};
    uint32_t o1[4], o2[4];
    if constexpr (INTER) {
      const float4 c = *reinterpret_cast<const float4*>(cs + t.k * 4);
      const float4 s = *reinterpret_cast<const float4*>(cs + half + t.k * 4);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y1, y2;
        rotate_pair(bf16lo(w1[e]), bf16hi(w1[e]), cc[e], ss[e], y1, y2);
        o1[e] = pack_bf16x2(y1, y2);
      }
    } else {
      const uint32_t w2[4] = {t.y.x, t.y.y, t.y.z, t.y.w};
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float4 c = *reinterpret_cast<const float4*>(cs + t.k * 8 + e * 2);
        const float4 s = *reinterpret_cast<const float4*>(cs + half + t.k * 8 + e * 2);
        float a1, a2, b1, b2;
        rotate_pair(bf16lo(w1[e]), bf16lo(w2[e]), c.x, s.x, a1, b1);
        rotate_pair(bf16hi(w1[e]), bf16hi(w2[e]), c.y, s.y, a2, b2);
        o1[e] = pack_bf16x2(a1, a2);
        o2[e] = pack_bf16x2(b1, b2);
        rotate_pair(bf16lo(w1[e + 1]), bf16lo(w2[e + 1]), c.z, s.z, a1, b1);
        rotate_pair(bf16hi(w1[e + 1]), bf16hi(w2[e + 1]), c.w, s.w, a2, b2);
        o1[e + 1] = pack_bf16x2(a1, a2);
        o2[e + 1] = pack_bf16x2(b1, b2);
      }
      y[t.k + nrot] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
    }
    y[t.k] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  };
  if (tid < n) write(one);
  if (tid + 128 < n) write(two);
  for (int i = tid + 256; i < n; i += 128) write(read(i));
}

// Angle a position of pair i, in turns (64 bits).
static double turns_a_position(int i, int rot, double theta, const bi_rope_scaling& s) {
  const double kTwoPi = 6.283185307179586476925;
  if (s.kind == BI_ROPE_BASE) theta *= pow(s.factor, (double)rot / (rot - 2));
  double w = pow(theta, -2.0 * i / rot);
  if (s.kind == BI_ROPE_LINEAR) w /= s.factor;
  if (s.kind == BI_ROPE_TURNS) {
    const double keep = std::min(std::max((s.orig_len * w / kTwoPi - s.low) / (s.high - s.low), 0.0), 1.0);
    w = w * keep + w / s.factor * (1 - keep);
  }
  if (s.kind == BI_ROPE_DIMS) {
    auto dim = [&](double turns) { return rot * log(s.orig_len / (kTwoPi * turns)) / (2 * log(theta)); };
    const double first = std::max(floor(dim(s.high)), 0.0), last = std::min(ceil(dim(s.low)), (double)rot - 1);
    const double ramp = std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
    w = w * (1 - ramp) + w / s.factor * ramp;
  }
  return w / kTwoPi;
}

}  // namespace bi

extern "C" {

bi_status bi_rope_scaled_table(float* rope_table, int64_t max_pos, int rot, double theta,
                               const bi_rope_scaling* scaling, void* stream) {
  using namespace bi;
  BI_REQUIRE(rope_table, "null table");
  BI_REQUIRE(max_pos > 0 && max_pos <= int64_t(1) << 31, "max_pos must be in [1, 2^31]");
  BI_REQUIRE(rot >= 2 && rot % 2 == 0, "rot must be even and positive");
  BI_REQUIRE_SHAPE(rot <= kMaxRot, "rot must be at most 256");
  BI_REQUIRE(std::isfinite(theta) && theta > 1, "theta must be above 1");
  const bi_rope_scaling s = scaling ? *scaling : bi_rope_scaling{BI_ROPE_PLAIN, 1, 1, 1, 2, 1};
  BI_REQUIRE(s.kind >= BI_ROPE_PLAIN && s.kind <= BI_ROPE_DIMS, "unknown kind of scaling");
  BI_REQUIRE(std::isfinite(s.amplitude) && std::isfinite((float)s.amplitude), "amplitude must be finite");
  if (s.kind != BI_ROPE_PLAIN)
    BI_REQUIRE(std::isfinite(s.factor) && s.factor > 0, "factor must be positive");
  if (s.kind == BI_ROPE_BASE) {
    BI_REQUIRE(rot > 2, "a scaled base needs rot > 2");
    const double base = theta * pow(s.factor, (double)rot / (rot - 2));
    BI_REQUIRE(std::isfinite(base) && base > 1, "the scaled base must be above 1 and finite");
  }
  if (s.kind == BI_ROPE_TURNS || s.kind == BI_ROPE_DIMS)
    BI_REQUIRE(std::isfinite(s.orig_len) && std::isfinite(s.high) && s.orig_len > 0 && s.low > 0 && s.high > s.low,
               "orig_len > 0 and 0 < low < high are needed");
  TurnRates rates = {};
  for (int i = 0; i < rot / 2; ++i) {
    double w = turns_a_position(i, rot, theta, s);
    BI_REQUIRE(std::isfinite(w), "the scaled angles must be finite");
    w -= floor(w);
    rates.w[i] = w < 1 ? (uint64_t)ldexp(w, 64) : 0;
  }
  const int half = rot / 2;
  const bool vec = half % 4 == 0 && aligned16(rope_table);
  const int rows_step = 256 / (half / (vec ? 4 : 1));
  const int64_t blocks = std::min<int64_t>(cdiv(max_pos, rows_step), 5 * (int64_t)num_sms());
  const bool amp = s.amplitude != 1.0;
  const float near = (float)s.amplitude;
  const float rho = near != 0 ? (float)((s.amplitude - (double)near) / (double)near) : 0.f;
  auto kernel = vec ? (amp ? rope_scaled_table_kernel<4, true> : rope_scaled_table_kernel<4, false>)
                    : (amp ? rope_scaled_table_kernel<1, true> : rope_scaled_table_kernel<1, false>);
  return launched(launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, as_stream(stream), rope_table, max_pos,
                             half, near, rho, rates),
                  "bi_rope_scaled_table");
}

bi_status bi_rope_slot_write(const void* qkv, int64_t T, int64_t ld, const int32_t* row_pos, const int64_t* slots,
                             int Hq, int Hkv, int hd, int rot, int layout, const float* rope_table, int64_t max_pos,
                             int64_t n_blocks, void* q_out, void* k_cache, void* v_cache, void* stream) {
  using namespace bi;
  BI_REQUIRE(T >= 0, "T < 0");
  if (T == 0) return BI_OK;
  BI_REQUIRE(qkv && row_pos && slots && rope_table && q_out && k_cache && v_cache, "null pointer");
  BI_REQUIRE(Hq > 0 && Hkv > 0 && hd > 0 && max_pos > 0 && n_blocks > 0, "non-positive size");
  BI_REQUIRE(layout == BI_ROPE_HALF || layout == BI_ROPE_INTERLEAVED, "bad layout");
  BI_REQUIRE_SHAPE(hd % 8 == 0 && hd <= 1024, "head_dim must be a multiple of 8, at most 1024");
  BI_REQUIRE_SHAPE(Hq <= 4096 && Hkv <= 4096, "at most 4096 heads");
  BI_REQUIRE(rot >= 0 && rot <= hd, "rot must be in [0, head_dim]");
  BI_REQUIRE_SHAPE(rot % (layout == BI_ROPE_HALF ? 16 : 8) == 0,
                   "rot must be a multiple of 16 (half layout) or 8 (interleaved)");
  BI_REQUIRE(ld >= (int64_t)(Hq + 2 * Hkv) * hd, "ld is shorter than a row");
  BI_REQUIRE_SHAPE(ld % 8 == 0, "ld must be a multiple of 8");
  BI_REQUIRE(aligned16(qkv) && aligned16(q_out) && aligned16(k_cache) && aligned16(v_cache) && aligned16(rope_table),
             "pointers must be 16-byte aligned");
  BI_REQUIRE(T <= 0x7fffffff && n_blocks <= 0x7fffffff, "too many rows or blocks");
  auto inverse = [](int d) { return d > 1 ? (uint32_t)(((uint64_t(1) << 32) + d - 1) / d) : 0u; };
  SlotWriteArgs a{static_cast<const __nv_bfloat16*>(qkv), ld, row_pos, slots, rope_table, max_pos, n_blocks * 64,
                  static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_cache),
                  static_cast<__nv_bfloat16*>(v_cache), Hq, Hkv, hd, rot,
                  inverse(hd / 8 - rot / 8 + rot / (layout == BI_ROPE_HALF ? 16 : 8)), inverse(hd / 8),
                  device_status_ptr()};
  auto kernel = layout == BI_ROPE_INTERLEAVED ? rope_slot_write_kernel<true> : rope_slot_write_kernel<false>;
  return launched(launch_pdl(kernel, dim3((unsigned)T), dim3(128), 0, as_stream(stream), a), "bi_rope_slot_write");
}

}  // extern "C"
