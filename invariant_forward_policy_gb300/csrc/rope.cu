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

// cos and sin of t * 2^-64 turns, times amp, each within 0.6 units of the last place (amp = 1).
// r = the offset from the nearest quarter turn, as a sum s + e of two floats (|s| <= pi/4);
// sin = s + (e (1 - s^2/2) + s^3 P(s^2)), cos = (1 - s^2/2) + (s^4 Q(s^2) - s e) with the roundings of s^2 and
// of 1 - s^2/2 carried along, P and Q the Taylor series (next terms below 2^-29).
BI_DEV void turn_cos_sin(uint64_t t, float amp, float& c_out, float& s_out) {
  const uint64_t quarter = (t + (1ull << 61)) >> 62;
  const int64_t r = (int64_t)(t - (quarter << 62));
  // |r| = a 2^37 + b 2^5 (+ less than 2^5): a fits a float's 24 bits, and of a small angle b holds 24 bits
  const uint64_t u = (uint64_t)(r < 0 ? -r : r);
  const float a = (float)(int)(u >> 37) * 0x1p-27f;
  const float b = (float)(uint32_t)((u & ((1ull << 37) - 1)) >> 5) * 0x1p-59f;
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
  const float st = __fmaf_rn(e, w, s * z * P);
  const float ct = wt + __fmaf_rn(z * z, Q, __fmaf_rn(-s, e, -0.5f * zl));
  const float sp = __fmaf_rn(amp, s, amp * st);
  const float sn = r < 0 ? -sp : sp;
  const float cs = __fmaf_rn(amp, w, amp * ct);
  const bool odd = quarter & 1;
  const float c0 = odd ? sn : cs, s0 = odd ? cs : sn;
  c_out = (quarter + 1) & 2 ? -c0 : c0;
  s_out = quarter & 2 ? -s0 : s0;
}

// A thread holds V neighbouring pairs and walks positions; a block's `rows_step` row groups are neighbours.
template <int V>
__global__ void __launch_bounds__(256) rope_scaled_table_kernel(float* __restrict__ table, int64_t max_pos, int half,
                                                                int iters, float amp,
                                                                const __grid_constant__ TurnRates rates) {
  pdl_trigger();
  pdl_wait();
  const int nq = half / V;
  const int rows_step = 256 / nq;
  const int q = threadIdx.x % nq, r = threadIdx.x / nq;
  if (r >= rows_step) return;
  uint64_t w[V], t[V];
  int64_t p = (int64_t)blockIdx.x * rows_step * iters + r;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    w[k] = rates.w[q * V + k];
    t[k] = w[k] * (uint64_t)p;
    w[k] *= (uint64_t)rows_step;
  }
  for (int i = 0; i < iters && p < max_pos; ++i, p += rows_step) {
    float c[V], s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      turn_cos_sin(t[k], amp, c[k], s[k]);
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
  int* status;
};

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), every product and sum rounded, one rounding to bf16: bi_rope_kv_write's
BI_DEV void rotate_pair(float x1, float x2, float c, float s, float& y1, float& y2) {
  y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
}

// One CTA a row; 16-byte vectors of 8 elements.  The items of a row are, per q and k head, its rotated vectors
// (half layout: a vector of the first half with its partner; interleaved: a vector of four pairs), then the
// vectors of its unrotated part, then the vectors of v.
template <bool INTER>
__global__ void __launch_bounds__(128) rope_slot_write_kernel(const SlotWriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int64_t pos = a.pos[row];
  const int64_t slot = a.slots[row];
  if (pos < 0 || pos >= a.max_pos) {
    if (threadIdx.x == 0) report(a.status, DEV_BAD_INDEX);
    return;
  }
  const bool slot_ok = slot >= 0 && slot < a.n_slots;
  if (!slot_ok && threadIdx.x == 0) report(a.status, DEV_BAD_INDEX);
  const uint4* src = reinterpret_cast<const uint4*>(a.qkv + row * a.ld);
  const float* cs = a.table + pos * a.rot;
  const int hv = a.hd / 8, half = a.rot / 2;
  const int nrot = INTER ? a.rot / 8 : a.rot / 16;  // rotated items of a head
  const int rest = hv - a.rot / 8;
  const int per = nrot + rest;
  const int n_qk = (a.Hq + a.Hkv) * per;
  uint4* qd = reinterpret_cast<uint4*>(a.q_out) + row * a.Hq * hv;
  // vector 0 of kv head 0 at this slot, and the distance of the next head
  const int64_t page = slot >> 6;
  const int64_t kv0 = (page * a.Hkv * 64 + (slot & 63)) * hv;
  uint4* kd = reinterpret_cast<uint4*>(a.k_cache) + kv0;
  uint4* vd = reinterpret_cast<uint4*>(a.v_cache) + kv0;
  for (int i = threadIdx.x; i < n_qk + a.Hkv * hv; i += blockDim.x) {
    if (i >= n_qk) {
      const int j = i - n_qk;
      if (slot_ok) vd[(int64_t)(j / hv) * 64 * hv + j % hv] = src[(a.Hq + a.Hkv) * hv + j];
      continue;
    }
    const int h = i / per, k = i % per;
    if (h >= a.Hq && !slot_ok) continue;
    const uint4* x = src + h * hv;
    uint4* y = h < a.Hq ? qd + h * hv : kd + (int64_t)(h - a.Hq) * 64 * hv;
    if (k >= nrot) {
      const int j = a.rot / 8 + k - nrot;
      y[j] = x[j];
      continue;
    }
    if constexpr (INTER) {
      const uint4 in = x[k];
      const float4 c = *reinterpret_cast<const float4*>(cs + k * 4);
      const float4 s = *reinterpret_cast<const float4*>(cs + half + k * 4);
      const uint32_t w[4] = {in.x, in.y, in.z, in.w};
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y1, y2;
        rotate_pair(bf16lo(w[e]), bf16hi(w[e]), cc[e], ss[e], y1, y2);
        o[e] = pack_bf16x2(y1, y2);
      }
      y[k] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      const uint4 in1 = x[k], in2 = x[k + nrot];
      const uint32_t w1[4] = {in1.x, in1.y, in1.z, in1.w}, w2[4] = {in2.x, in2.y, in2.z, in2.w};
      uint32_t o1[4], o2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c = *reinterpret_cast<const float2*>(cs + k * 8 + e * 2);
        const float2 s = *reinterpret_cast<const float2*>(cs + half + k * 8 + e * 2);
        float a1, a2, b1, b2;
        rotate_pair(bf16lo(w1[e]), bf16lo(w2[e]), c.x, s.x, a1, b1);
        rotate_pair(bf16hi(w1[e]), bf16hi(w2[e]), c.y, s.y, a2, b2);
        o1[e] = pack_bf16x2(a1, a2);
        o2[e] = pack_bf16x2(b1, b2);
      }
      y[k] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
      y[k + nrot] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
    }
  }
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
    w -= floor(w);
    rates.w[i] = w < 1 ? (uint64_t)ldexp(w, 64) : 0;
  }
  const int half = rot / 2;
  const bool vec = half % 4 == 0 && aligned16(rope_table);
  const int rows_step = 256 / (half / (vec ? 4 : 1));
  const int64_t iters = std::min<int64_t>(16, std::max<int64_t>(1, max_pos / ((int64_t)rows_step * 8 * num_sms())));
  const int64_t blocks = cdiv(max_pos, rows_step * iters);
  BI_REQUIRE_SHAPE(blocks <= 0x7fffffff, "table too large");
  auto kernel = vec ? rope_scaled_table_kernel<4> : rope_scaled_table_kernel<1>;
  return launched(launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, as_stream(stream), rope_table, max_pos,
                             half, (int)iters, (float)s.amplitude, rates),
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
  SlotWriteArgs a{static_cast<const __nv_bfloat16*>(qkv), ld, row_pos, slots, rope_table, max_pos, n_blocks * 64,
                  static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_cache),
                  static_cast<__nv_bfloat16*>(v_cache), Hq, Hkv, hd, rot, device_status_ptr()};
  auto kernel = layout == BI_ROPE_INTERLEAVED ? rope_slot_write_kernel<true> : rope_slot_write_kernel<false>;
  return launched(launch_pdl(kernel, dim3((unsigned)T), dim3(128), 0, as_stream(stream), a), "bi_rope_slot_write");
}

}  // extern "C"
