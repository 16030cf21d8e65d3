// Attention of the nodes of drafted trees over the paged cache and their own ancestors.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §4.2 (one read path, fixed absolute splits).  Node i of a
// sequence's tree has its key and value in the cache at position start + i, and stands itself at position start +
// depth.  It attends to positions 0 .. start - 1 and to its path, taken as if the path's nodes stood at positions
// start .. start + depth.  Every row repeats, operation for operation, the arithmetic of bi_attention on a cache
// that holds just that path (splits, lanes, 64-key tiles and 16-key MMA steps by position), so it has the bits
// that a plain decode of the path gives.
//
// Three launches.  Let E be the start of the lane (of bi_attention's partition) that holds position `start`.
//   * tree_tail_kernel: the lanes from E on, which differ by node, on mma.sync; a record (m, l, acc) for each row
//     and lane.
//   * tree_context_kernel: the lanes before E, which every node of a sequence sees whole, on tcgen05; a record for
//     each row and split.  It needs nothing of the tail kernel and runs beside it.
//   * tree_merge_kernel: folds and merges a row's records in order.
// What bounds it: a page of keys and values is read once for up to 128 query rows (nodes x q heads of a group), so
// HBM bounds small trees; with more rows the softmax's instructions and the split records (one for every 512
// positions of every row: as many bytes as the keys and values themselves at 256 rows) do.  Measured (GB300, 16 q heads on
// 4 kv heads of 128, us a call): 64 chains of up to 8 nodes, contexts of 1K to 32K, 229 (1.21 GB at 5.3 TB/s); 16 trees of
// 64 nodes, contexts of 6K to 8K, 150 (0.24 GB, 58.7 GFLOP); one tree of 37 nodes behind 32K positions 46; 16 trees of 16
// nodes, contexts up to 768, 8 heads of 64: 25.
#include <algorithm>
#include <mutex>
#include <string>

#include "attn_merge.cuh"
#include "attn_tile.cuh"
#include "common.cuh"
#include "tree.cuh"

namespace bi {

struct TreeArgs {
  const __nv_bfloat16* q;  // [T, Hq, hd]
  const int32_t *parent, *row0, *start, *block_table;
  float* part_o;    // [T, Hq, nsplit, hd]: the lanes before E
  float* part_ml;   // [T, Hq, nsplit, 2]
  float* tail_o;    // [T, Hq, ntail, hd]: the lanes from E on, one by one
  float* tail_ml;   // [T, Hq, ntail, 2]
  int32_t* row_pos; // [T]: a node's position, -1 when it has none
  const void *k_cache, *v_cache;
  __nv_bfloat16* out;
  int* status;
  int64_t T, max_blk, n_blocks;
  int B, max_nodes, Hq, Hkv, group, gshift, nsplit, ntail, split, lane_len, stages;
  float scale_log2;
  float neg_zero;  // -0, see mul2
};

constexpr int kMaxTailRecords = 32;  // the merge holds one a lane
constexpr int kTreeMaxSplit = 16384;  // positions of a split (positions near max_ctx stay 32-bit numbers)

// A sequence as the kernels see it: its rows, or none when its numbers cannot be right.
struct TreeSeq {
  int64_t row0;
  int n;
  int start;
  bool rows_ok;  // row range and node count: the rows can be written
  bool ok;       // and its positions lie in the block table
};
BI_DEV TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s;
  const int64_t r0 = __ldcg(a.row0 + b), r1 = __ldcg(a.row0 + b + 1);
  s.row0 = r0;
  s.start = __ldcg(a.start + b);
  s.rows_ok = r0 >= 0 && r1 >= r0 && r1 <= a.T && r1 - r0 <= a.max_nodes;
  s.n = s.rows_ok ? (int)(r1 - r0) : 0;
  s.ok = s.rows_ok && s.start >= 0 && (int64_t)s.start + s.n <= a.max_blk * kKeys;
  return s;
}

// E: the start of the lane that holds position `start`.
BI_DEV int tail_lane(const TreeArgs& a, int start) {
  const int kv = start / a.split * a.split;
  return kv + (start - kv) / a.lane_len * a.lane_len;
}
// The end of the lane that begins at `at`.
BI_DEV int lane_end(const TreeArgs& a, int at) {
  return min(at + a.lane_len, (at / a.split + 1) * a.split);
}

template <int HD>
__device__ __forceinline__ void clear(LaneState<HD>& st) {
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
#pragma unroll
  for (int j = 0; j < HD / 8; ++j) st.acc[j][0] = st.acc[j][1] = st.acc[j][2] = st.acc[j][3] = 0.f;
}

// The online softmax of one 64-key tile (attn_update's operations in its order) up to P, left in sc.
// MASK: positions behind a row's own are masked; without it every key counts for every row.
template <int HD, bool MASK>
__device__ __forceinline__ void tree_softmax(float (&sc)[8][4], int key0, const int (&row_pos)[2], float scale_log2,
                                             int lane, LaneState<HD>& st) {
  const int tq = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float tmax = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = __fmul_rn(sc[j][h * 2 + e], scale_log2);
        if (MASK) v = key0 + j * 8 + tq * 2 + e <= row_pos[h] ? v : -INFINITY;
        sc[j][h * 2 + e] = v;
        tmax = fmaxf(tmax, v);
      }
    }
    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
    const float m_new = fmaxf(st.m[h], tmax);
    const float alpha = (m_new == st.m[h]) ? 1.0f : exp2f(__fsub_rn(st.m[h], m_new));
    // a row without any key above -inf so far: 2^(-inf - 0) = 0
    const float sub = m_new == -INFINITY ? 0.f : m_new;
    float rs = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p = exp2_p(__fsub_rn(sc[j][h * 2 + e], sub));
        sc[j][h * 2 + e] = p;
        rs = __fadd_rn(rs, p);
      }
    }
    rs = __fadd_rn(rs, __shfl_xor_sync(0xffffffffu, rs, 1));
    rs = __fadd_rn(rs, __shfl_xor_sync(0xffffffffu, rs, 2));
    st.l[h] = __fadd_rn(__fmul_rn(st.l[h], alpha), rs);
    st.m[h] = m_new;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      st.acc[j][h * 2] = __fmul_rn(st.acc[j][h * 2], alpha);
      st.acc[j][h * 2 + 1] = __fmul_rn(st.acc[j][h * 2 + 1], alpha);
    }
  }
}

// Shared-memory address of 16-byte chunk ch of a key row that begins at `row` (rows of 128 bytes under the 128-byte
// swizzle; the second 64 head dims 8 KB on).
BI_DEV uint32_t row_chunk(uint32_t row, int ch) {
  return row + (ch >> 3) * (kKeys * 128) + ((((uint32_t)ch & 7) ^ ((row >> 7) & 7)) << 4);
}

// S = Q K^T of the first `groups` 8-key groups of a tile (0 for the others), in 16-wide steps of hd, the groups'
// chains side by side.  row(key): the address of the key's row.
template <int HD, typename Row>
__device__ __forceinline__ void tree_scores(const uint32_t (&qf)[HD / 16][4], int lane, float (&sc)[8][4], Row row,
                                            int groups) {
#pragma unroll
  for (int j = 0; j < 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
  for (int j0 = 0; j0 < 8; j0 += 4) {
    if (j0 >= groups) break;
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = row((j0 + j) * 8 + (lane & 7));
#pragma unroll
    for (int kk = 0; kk < HD / 16; kk += 2) {
      uint32_t k[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) ldsm_x4(row_chunk(r[j], kk * 2 + (lane >> 3)), k[j][0], k[j][1], k[j][2], k[j][3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_bf16_16816(sc[j0 + j], qf[kk], k[j][0], k[j][1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_bf16_16816(sc[j0 + j], qf[kk + 1], k[j][2], k[j][3]);
    }
  }
}

// acc += P V of the first `steps` 16-key steps of a tile, in order, P rounded to bf16.
template <int HD, typename Row>
__device__ __forceinline__ void tree_pv(const float (&p)[8][4], int lane, LaneState<HD>& st, Row row, int steps) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    if (kk >= steps) break;
    const uint32_t pa[4] = {pack_bf16x2(p[2 * kk][0], p[2 * kk][1]), pack_bf16x2(p[2 * kk][2], p[2 * kk][3]),
                            pack_bf16x2(p[2 * kk + 1][0], p[2 * kk + 1][1]),
                            pack_bf16x2(p[2 * kk + 1][2], p[2 * kk + 1][3])};
    const uint32_t r = row(kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8);
#pragma unroll
    for (int j = 0; j < HD / 8; j += 2) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(row_chunk(r, j + (lane >> 4)), b0, b1, b2, b3);
      mma_bf16_16816(st.acc[j], pa, b0, b1);
      mma_bf16_16816(st.acc[j + 1], pa, b2, b3);
    }
  }
}

// ------------------------------------------------------------------------ the lanes from E on
// A warp owns a node's q heads of one kv head (a 16-row tile; groups of 32 and 64 heads take two and four warps), a
// CTA of four warps neighbouring ones, whose keys and values come by TMA into its shared memory once: the pages of the first
// lane before position `start`, through a ring, then all pages that hold the tree's own keys at once.  ldmatrix takes
// an address for every key row, so a tile behind `start` is read as if the node's path stood in the cache: the page's
// row for a position before `start`, the path node's row behind it, a row of zeros behind the node (as a plain decode
// reads positions behind its own).  8-key groups of scores and 16-key steps of P V behind the node's position are
// left out.  Most of a 16-row tile is empty for small groups; the chain of one node's few tiles is the time (16 x 64
// nodes x 4 kv heads: 26 us, of which 7 beside the context kernel; a warp of four nodes that selects each node's results
// from its own MMAs took 51).
constexpr int kTailWarps = 4;

// Shared memory: the page ring; then barriers, depths, parents, the warps' path tables.  The zero row is 128 bytes
// behind the ring and, for the second half of 128 head dims, 128 bytes 8 KB on: where V would be of a K row kPage
// before them.
template <int HD>
struct TailLayout {
  static constexpr int kPage = kKeys * HD * 2;
  static constexpr int kStage = 2 * kPage;  // a K page and its V page
  static constexpr int kMaxStages = 12;
  static constexpr int kOffBar = 128, kOffDepth = 512, kOffParent = kOffDepth + 2 * kMaxTreeNodes,
                       kOffPath = kOffParent + 2 * kMaxTreeNodes,
                       kExtra = HD == 128 ? kKeys * 128 + 128 : kOffPath + kTailWarps * kKeys * 2;
  static_assert(kOffPath + kTailWarps * kKeys * 2 <= kKeys * 128, "the tables end before the second zero row");
  static int bytes(int stages) { return 1024 + stages * kStage + kExtra; }
};

template <int HD>
__global__ void __launch_bounds__(kTailWarps * 32, HD == 64 ? 4 : 2) tree_tail_kernel(const TreeArgs a,
                                                                    const __grid_constant__ CUtensorMap tmk,
                                                                    const __grid_constant__ CUtensorMap tmv) {
  using Lay = TailLayout<HD>;
  constexpr int WARPS = kTailWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NS = a.stages;
  uint8_t* extra = smem + NS * Lay::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(extra + Lay::kOffBar);  // [NS] the stage's pages have landed
  uint64_t* empty = full + Lay::kMaxStages;                            // [NS] the warps have read them
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + Lay::kMaxStages);
  volatile int* issued = abort_flag + 1;  // [NS] the page that was last asked for in each stage
  int16_t* depth_of = reinterpret_cast<int16_t*>(extra + Lay::kOffDepth);
  int16_t* parent_of = reinterpret_cast<int16_t*>(extra + Lay::kOffParent);
  uint16_t* paths = reinterpret_cast<uint16_t*>(extra + Lay::kOffPath);  // [WARPS][64]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y, kvh = blockIdx.z;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], WARPS);
      issued[i] = -1;
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 32) reinterpret_cast<uint32_t*>(extra)[tid] = 0u;
  if (HD == 128 && tid >= 32 && tid < 64) reinterpret_cast<uint32_t*>(extra + kKeys * 128)[tid - 32] = 0u;
  // the context kernel reads what this kernel's predecessors wrote without waiting for this one: it may start only
  // once they have completed
  pdl_wait();
  pdl_trigger();
  const TreeSeq sq = tree_seq(a, b);
  const bool speaks = kvh == 0;  // reports the sequence's faults and writes positions
  const int n = sq.n, start = sq.start;
  const int parts = (a.group + 15) / 16;  // warps of a node
  const int per_cta = WARPS / parts;      // nodes of a CTA
  const int node0 = blockIdx.x * per_cta;
  if (speaks && blockIdx.x == 0 && tid == 0 && !sq.ok) report(a.status, DEV_BAD_INDEX);
  if (node0 >= n) return;
  const int last_node = min(n, node0 + per_cta) - 1;
  if (!sq.ok) {
    if (speaks)
      for (int i = node0 + tid; i <= last_node; i += WARPS * 32) a.row_pos[sq.row0 + i] = -1;
    return;
  }
  const int E = tail_lane(a, start);
  const int tail_page0 = start / kKeys, tail0 = tail_page0 * kKeys;
  const int n_plain = (tail0 - E) / kKeys;  // whole pages of the first lane before `start`
  const int tail_pages = (start + last_node) / kKeys - tail_page0 + 1;
  const int n_issue = n_plain + tail_pages;
  const int rows_total = (int)(a.n_blocks * a.Hkv * kKeys);
  auto issue = [&](int j) {
    const int page = E / kKeys + j;
    const int32_t id = page < a.max_blk ? __ldcg(a.block_table + (int64_t)b * a.max_blk + page) : -1;
    int row = rows_total;  // past the end: the copy reads zeros
    if (id >= 0 && id < a.n_blocks) row = (int)(((int64_t)id * a.Hkv + kvh) * kKeys);
    else report(a.status, DEV_BAD_INDEX);
    const int slot = j % NS;
    uint8_t* sk = smem + slot * Lay::kStage;
    issued[slot] = j;
    mbar_arrive_expect_tx(&full[slot], Lay::kStage);
#pragma unroll
    for (int x = 0; x < HD / 64; ++x) {
      tma_load_2d(sk + x * (kKeys * 128), &tmk, &full[slot], x * 64, row);
      tma_load_2d(sk + Lay::kPage + x * (kKeys * 128), &tmv, &full[slot], x * 64, row);
    }
  };
  if (tid == 0)
    for (int j = 0; j < NS && j < n_issue; ++j) issue(j);
  if (warp == WARPS - 1) {
    const bool bad = tree_depths(a.parent + sq.row0, last_node + 1, depth_of, lane, parent_of);
    bool far = false;
    for (int i = node0 + lane; i <= last_node; i += 32) {
      const int d = depth_of[i];
      const bool fits = start + d < a.nsplit * a.split;
      far |= !fits;
      if (speaks) a.row_pos[sq.row0 + i] = d >= 0 && fits ? start + d : -1;
    }
    far = __any_sync(0xffffffffu, far);
    if (speaks && (bad || far)) report(a.status, DEV_BAD_INDEX);
  }

  // the rows that a thread holds: q heads g and g + 8 of the node's group (or of the warp's 16 of it)
  const int g = lane >> 2, tq = lane & 3;
  const int node = node0 + warp / parts;
  const int h0 = warp % parts * 16;
  const bool there = node <= last_node && warp < per_cta * parts;
  uint32_t qf[HD / 16][4];
  int row_head[2];
  bool row_valid[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    row_valid[h] = there && h0 + g + h * 8 < a.group;
    row_head[h] = kvh * a.group + h0 + g + h * 8;
    const __nv_bfloat16* qr = a.q + ((sq.row0 + node) * a.Hq + row_head[h]) * HD + tq * 2;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      qf[kk][h] = row_valid[h] ? __ldcg(reinterpret_cast<const uint32_t*>(qr + kk * 16)) : 0u;
      qf[kk][2 + h] = row_valid[h] ? __ldcg(reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8)) : 0u;
    }
  }
  __syncthreads();
  const int d = there ? depth_of[node] : -1;
  const bool live = d >= 0 && start + d < a.nsplit * a.split;
  const int pos = start + d;

  bool ok = true;
  auto wait_page = [&](int j) {
    if (!mbar_wait(&full[j % NS], (j / NS) & 1)) {
      report(a.status, DEV_TIMEOUT);
      *abort_flag = 1;
    }
    return (bool)__all_sync(0xffffffffu, *abort_flag == 0);
  };
  LaneState<HD> cur;
  clear(cur);
  for (int j = 0; ok && j < n_plain; ++j) {
    if (!(ok = wait_page(j))) break;
    const uint32_t sk = smem_u32(smem + j % NS * Lay::kStage);
    if (live) {
      float sc[8][4];
      tree_scores<HD>(qf, lane, sc, [&](int key) { return sk + key * 128; }, 8);
      const int all[2] = {0x7fffffff, 0x7fffffff};
      tree_softmax<HD, false>(sc, 0, all, a.scale_log2, lane, cur);
      tree_pv<HD>(sc, lane, cur, [&](int key) { return sk + Lay::kPage + key * 128; }, 4);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[j % NS]);
    if (tid == 0 && j + NS < n_issue) {  // the freed stage takes the page NS places on
      if (!mbar_wait(&empty[j % NS], (j / NS) & 1)) {
        report(a.status, DEV_TIMEOUT);
        *abort_flag = 1;
      } else {
        issue(j + NS);
      }
    }
    __syncwarp();
  }
  for (int i = 0; ok && i < tail_pages; ++i) ok = wait_page(n_plain + i);
  uint16_t* path = paths + warp * kKeys;
  const int first_slot = n_plain % NS;
  const uint32_t base = smem_u32(smem);
  const uint32_t zero = base + NS * Lay::kStage - Lay::kPage;  // its V is the zero row
  int lb = E;
  for (int t = 0; ok && live && t < a.ntail && lb <= pos; ++t) {
    const int le = lane_end(a, lb);
    for (int key0 = max(lb, tail0); key0 < min(le, pos + 1); key0 += kKeys) {
      // path[i]: the key row of position key0 + i, in units of 128 bytes of shared memory
      auto row_of = [&](int off) {  // off: from the first tail page's first row
        int slot = first_slot + off / kKeys;
        if (slot >= NS) slot -= NS;
        return (uint16_t)(slot * (Lay::kStage / 128) + off % kKeys);
      };
      __syncwarp();
      for (int i = lane; i < kKeys; i += 32)
        path[i] = key0 + i < start ? row_of(key0 + i - tail0) : (uint16_t)((zero - base) / 128);
      __syncwarp();
      if (lane == 0) {
        int x = node;
        for (int p = pos; p >= start && p >= key0; --p) {
          if (p < key0 + kKeys) path[p - key0] = row_of(start - tail0 + x);
          x = parent_of[x];
        }
      }
      __syncwarp();
      float sc[8][4];
      tree_scores<HD>(qf, lane, sc, [&](int key) { return base + path[key] * 128u; }, min(8, (pos - key0) / 8 + 1));
      const int at[2] = {pos, pos};
      tree_softmax<HD, true>(sc, key0, at, a.scale_log2, lane, cur);
      const int steps = min(4, (pos - key0) / 16 + 1);
      tree_pv<HD>(sc, lane, cur, [&](int key) { return base + Lay::kPage + path[key] * 128u; }, steps);
      if (steps < 4) {  // a step that is left out would have added +0: -0 becomes +0
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) cur.acc[j][c] = __fadd_rn(cur.acc[j][c], 0.f);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!row_valid[h]) continue;
      const int64_t at = ((sq.row0 + node) * a.Hq + row_head[h]) * a.ntail + t;
      float* po = a.tail_o + at * HD;
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
        *reinterpret_cast<float2*>(po + j * 8 + tq * 2) = make_float2(cur.acc[j][h * 2], cur.acc[j][h * 2 + 1]);
      if (tq == 0) *reinterpret_cast<float2*>(a.tail_ml + at * 2) = make_float2(cur.m[h], cur.l[h]);
    }
    clear(cur);
    lb = le;
  }
  __syncthreads();
  if (*abort_flag && tid == 0)  // the copies this CTA started land before it ends
    for (int i = 0; i < NS; ++i)
      if (issued[i] >= 0) mbar_wait(&full[i], (issued[i] / NS) & 1);
}

// ------------------------------------------------------------------------ the lanes before E
// A unit is (sequence, kv head, tile of 128 rows, split), numbered in that order; every CTA takes an equal run of the
// call's units, so contexts of any lengths spread evenly and a CTA's consecutive splits of one row tile go through
// one pipeline.  S = Q K^T (K = hd in 16-wide steps,
// ascending) and O = P V (64 keys in 16-wide steps, ascending) accumulate in TMEM; tcgen05.mma and mma.sync give
// the same fp32 bits for the same 16-wide steps.  A softmax thread holds one row: its 64 scores of a tile, and the
// split's running state in registers.  P goes back to TMEM, over the scores it came from, as the A operand of P V.
// The sums that a quad of mma.sync threads would form are formed by the one thread in the same order: s_q over the
// keys 8j + 2q + {0, 1}, then (s0 + s1) + (s2 + s3).  Products and sums go two at a time (f32x2: the same
// roundings).  S of a tile is computed while the one before it is in the softmax, and the accumulator of a finished
// lane is folded while the next lane's first scores are.
// Two CTAs share an SM (their chains softmax -> P V -> fold interleave): 113 KB of shared memory and 256 TMEM
// columns each, and 128 registers a thread at launch, which the warpgroups then split 224 to 32.  At 128 live rows a
// CTA takes 3400 clocks a tile: S 570 to wait for, scores 180, exponentials 720, P V 240 to wait for, fold 1900 a lane,
// scaling 530 a lane, a record 2000 a split; with two warps a scheduler the chains' latency is what bounds it (issue
// 41%, tensor pipe 27%).  One row tile's pages twice from memory (a second tile of 128 rows) is the rest: 422 MB read
// for 236.  Tried and slower: P in shared memory, more O columns a wait (both spill), row tiles in turn for every split
// (Q changes too often), one CTA an SM with warps of their own for scaling and folds (the fold's chain bounds it).
template <int HD>
struct CtxLayout {
  static constexpr int kQ = 128 * HD * 2;       // HD/64 boxes of 128 rows x 128 bytes
  static constexpr int kPage = kKeys * HD * 2;  // one K or V page
  static constexpr int kSlots = HD == 128 ? 5 : 11;
  static constexpr int kOffKV = kQ;
  static constexpr int kOffBar = kOffKV + kSlots * kPage;
  static constexpr int kBytes = kOffBar + 640;
  static constexpr int kThreads = 256;
  static constexpr int kSoftmaxRegs = 224, kOtherRegs = 32, kLaunchRegs = 128;
  static_assert(128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr uint32_t kCols = 256, kColS = 0, kColO = 128;  // S0, S1 (64 each; P over them), O (HD)
};

// D(tmem) (+)= A(tmem) * B(smem desc)^T: A holds two bf16 values of K in each 32-bit column.
BI_DEV void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A tile of K or V; `policy` is its L2 eviction priority.
BI_DEV void tma_load_2d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], "
      "[%2], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
// One lane of the (converged) warp.  The compiler knows that a branch on it has one thread: tcgen05.mma then issues in
// 55-80 clocks, against 200 in a branch on lane == 0 (whatever N and the accumulator: M = 128, N = 32..128).
BI_DEV bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
// Wait for this thread's TMEM loads; r: the registers of one, which nothing may read before.
template <int N>
BI_DEV void tmem_ld_wait_for(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 16)  // (the first waits; the others only tie their registers to it)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                   "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15])
                 :
                 : "memory");
}
// Eight floats, 32-byte aligned.
BI_DEV void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// Two products, each rounded once: x y + nz with nz = (-0, -0), a value that the compiler cannot see.  (It contracts
// mul.rn.f32x2 and a following add.rn.f32x2 into one rounding.)
BI_DEV float2 mul2(float2 x, float2 y, float nz) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %6};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(nz));
  return r;
}
BI_DEV float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 c, a, b;\n"
      " mov.b64 {%0, %1}, c;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// A CTA's place in the call's units: those of one (sequence, kv head, row tile) from split s on, and the rest of the run.
struct CtxCursor {
  TreeSeq sq;
  int b, kvh, tile, s;
  int n_split, n_tile;  // splits with lanes before E, and row tiles, of the sequence
  int64_t left;         // units of the CTA from here on
  // the sequence's units: n_split and n_tile of it are set
  BI_DEV int64_t sequence(const TreeArgs& a, int b_) {
    b = b_;
    sq = tree_seq(a, b);
    const int E = sq.ok ? tail_lane(a, sq.start) : 0;
    n_split = min(E / a.split + (E % a.split != 0), a.nsplit);  // (E may be near 2^31)
    n_tile = ((sq.n << a.gshift) + 127) >> 7;
    return (int64_t)n_split * n_tile * a.Hkv;
  }
  BI_DEV void at(int64_t v) {  // unit v of the sequence
    s = (int)(v % n_split);
    const int64_t w = v / n_split;
    tile = (int)(w % n_tile);
    kvh = (int)(w / n_tile);
  }
  BI_DEV int splits() const { return (int)min((int64_t)(n_split - s), left); }  // of this row tile
  // 64-key tiles of `splits()` splits from s on
  BI_DEV int tiles(const TreeArgs& a) const {
    const int E = tail_lane(a, sq.start);
    return (min(E, (s + splits()) * a.split) - s * a.split) / kKeys;
  }
  BI_DEV void next(const TreeArgs& a) {  // past this row tile's splits
    left -= splits();
    s = 0;
    if (++tile == n_tile) {
      tile = 0;
      ++kvh;
    }
    while (left > 0 && kvh == a.Hkv && b + 1 < a.B)
      if (sequence(a, b + 1) > 0) kvh = 0;
    if (kvh == a.Hkv) left = 0;
  }
};

// A row tile's consecutive splits, as the producer hands them to the other warps.
struct CtxSegment {
  int64_t row0;      // of the sequence
  int n, s0, s_end;  // 64-key tiles (0: the run has ended); splits s0 .. s_end - 1
  int r0, n_rows;    // the tile's first row, and the sequence's rows
  int head0;         // the kv head's first q head
};
constexpr int kSegments = 4;  // in flight

template <int HD>
__global__ void __launch_bounds__(CtxLayout<HD>::kThreads, 2)
    tree_context_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  using Lay = CtxLayout<HD>;
  constexpr int NS = Lay::kSlots;
  constexpr int kWarpTma = 4, kWarpMma = 5;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + Lay::kOffKV;  // tile i of K0, V0, K1, V1, ... in slot i % NS
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBar);
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;  // [2] MMA -> softmax: S of a tile is in TMEM
  uint64_t* p_full = s_full + 2;     // softmax -> MMA: P written, O folded or rescaled (4 warp arrivals)
  uint64_t* o_done = p_full + 1;     // MMA -> softmax, MMA: P V of a tile has completed
  uint64_t* q_full = o_done + 1;     // softmax -> MMA: Q of a row tile loaded (128 thread arrivals)
  uint64_t* seg_full = q_full + 1;   // [kSegments] TMA -> all: a segment stands in its place
  uint64_t* seg_empty = seg_full + kSegments;  // [kSegments] read (MMA thread and 4 warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_empty + kSegments);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first_b = reinterpret_cast<int*>(tmem_slot + 2);
  int64_t* first_v = reinterpret_cast<int64_t*>(tmem_slot + 4);
  int64_t* sums = first_v + 1;  // [8]
  CtxSegment* segs = reinterpret_cast<CtxSegment*>(sums + 8);
  static_assert((2 * NS + 5 + 2 * kSegments) * 8 + 16 + 72 + kSegments * sizeof(CtxSegment) <= Lay::kBytes - Lay::kOffBar,
                "barriers and segments fit");

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(q_full, 128);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 5);
    }
    *abort_flag = 0;
    *first_b = -1;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, Lay::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  // The launch before this one (tree_tail_kernel) starts it only after its own predecessors have completed, so q, the
  // caches and the tables may be read at once (through L2, where those wrote them); the end waits for it.
  CtxCursor cur;
  // the sum of a 256-sequence group's units over the threads before this one, and over all
  auto scan = [&](int64_t mine, int64_t& all) {
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t before = inc - mine;
    all = 0;
    for (int w = 0; w < 8; ++w) {
      before += w < warp ? sums[w] : 0;
      all += sums[w];
    }
    return before;
  };
  int64_t total = 0, mine0 = 0, before0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += 256) {
    const int64_t mine = b0 + tid < a.B ? cur.sequence(a, b0 + tid) : 0;
    int64_t all;
    const int64_t before = scan(mine, all);
    if (b0 == 0) mine0 = mine, before0 = before;
    total += all;
  }
  const int64_t u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  int64_t run_up = 0;
  for (int b0 = 0; b0 < a.B && u0 < u1; b0 += 256) {
    int64_t mine = mine0, before = before0, all = total;
    if (a.B > 256) {
      mine = b0 + tid < a.B ? cur.sequence(a, b0 + tid) : 0;
      before = scan(mine, all);
    }
    if (run_up + before <= u0 && u0 < run_up + before + mine) {
      *first_b = b0 + tid;
      *first_v = u0 - run_up - before;
    }
    run_up += all;
    if (run_up > u0) break;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  const int tpl = a.lane_len / kKeys;  // tiles of a lane
  const int ntf = a.split / kKeys;     // and of a whole split

  if (warp >= 4) {
    reg_alloc_dec<Lay::kOtherRegs>();
    if (warp == kWarpTma && elect_one()) {
      // ---------------- TMA producer: K and V pages in order
      const int rows_total = (int)(a.n_blocks * a.Hkv * kKeys);
      // the records are read back by the merge, the pages only by a neighbouring CTA at about the same time
      uint64_t policy;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      cur.left = *first_b < 0 ? 0 : u1 - u0;
      if (cur.left > 0) {
        cur.sequence(a, *first_b);
        cur.at(*first_v);
      }
      int i = 0;
      for (int q = 0; !*abort_flag; ++q, cur.next(a)) {
        const int place = q % kSegments;
        if (q >= kSegments && !mbar_wait(&seg_empty[place], ((q / kSegments) - 1) & 1)) {
          report(a.status, DEV_TIMEOUT);
          *abort_flag = 1;
        }
        segs[place].n = cur.left > 0 ? cur.tiles(a) : 0;
        if (cur.left > 0) {
          segs[place].row0 = cur.sq.row0;
          segs[place].s0 = cur.s;
          segs[place].s_end = cur.s + cur.splits();
          segs[place].r0 = cur.tile * 128;
          segs[place].n_rows = cur.sq.n << a.gshift;
          segs[place].head0 = cur.kvh * a.group;
        }
        mbar_arrive(&seg_full[place]);
        if (cur.left <= 0) break;
        const int32_t* bt = a.block_table + (int64_t)cur.b * a.max_blk;
        const int page0 = cur.s * ntf, page1 = page0 + cur.tiles(a);
        int32_t blk = page0 < a.max_blk ? __ldcg(bt + page0) : -1;
        for (int page = page0; page < page1 && !*abort_flag; ++page) {
          int row = rows_total;  // past the end: the copy reads zeros
          if (blk >= 0 && blk < a.n_blocks) row = (int)(((int64_t)blk * a.Hkv + cur.kvh) * kKeys);
          else report(a.status, DEV_BAD_INDEX);
          if (page + 1 < page1) blk = page + 1 < a.max_blk ? __ldcg(bt + page + 1) : -1;
          for (int v = 0; v < 2 && !*abort_flag; ++v) {
            const int slot = i % NS;
            if (i >= NS && !mbar_wait(&kv_empty[slot], ((i / NS) - 1) & 1)) {
              report(a.status, DEV_TIMEOUT);
              *abort_flag = 1;
              break;
            }
            uint8_t* dst = sKV + slot * Lay::kPage;
            mbar_arrive_expect_tx(&kv_full[slot], Lay::kPage);
#pragma unroll
            for (int x = 0; x < HD / 64; ++x)
              tma_load_2d_hint(dst + x * (kKeys * 128), v ? &tmv : &tmk, &kv_full[slot], x * 64, row, policy);
            ++i;
          }
        }
      }
      // the copies this CTA started land before it can exit
      for (int k = 0; k < NS && k < i; ++k) mbar_wait(&kv_full[(i - 1 - k) % NS], ((i - 1 - k) / NS) & 1);
    } else if (warp == kWarpMma && elect_one()) {
      // ---------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD) | (1u << 16);  // V read MN-major
      int t = 0;        // tiles so far
      bool ok = true;
      int seg = 0;      // row tiles so far
      // descriptors count addresses in 16 bytes, so one of another address is a sum away
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(sQ));
      const uint64_t k_desc = sw128_kmajor_desc(smem_u32(sKV));
      const uint64_t v_desc = sw128_mnmajor_desc(smem_u32(sKV), kKeys * 128, 1024);
      auto issue_s = [&](int t) -> bool {
        const int i = 2 * t;
        if (!mbar_wait(&kv_full[i % NS], (i / NS) & 1)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc + (uint32_t)(i % NS) * (Lay::kPage / 16);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          tc_mma_bf16(tmem + Lay::kColS + (t & 1) * kKeys, q_desc + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16,
                      kd + ((k >> 2) * (kKeys * 128) + (k & 3) * 32) / 16, idesc_s, k != 0 ? 1u : 0u);
        tc_commit(&s_full[t & 1]);
        tc_commit(&kv_empty[i % NS]);
        return true;
      };
      for (; ok && !*abort_flag; ++seg) {
        const int place = seg % kSegments;
        if (!(ok = mbar_wait(&seg_full[place], (seg / kSegments) & 1))) break;
        const int n = segs[place].n;
        mbar_arrive(&seg_empty[place]);
        if (n == 0) break;
        // S of tile t takes the columns that hold P of tile t - 2, whose P V the softmax had seen done before it gave
        // out P of tile t - 1
        ok = mbar_wait(q_full, seg & 1) && issue_s(t);
        int i_split = 0, i_lane = 0;
        for (int k = 0; ok && k < n && !*abort_flag; ++k, ++t) {
          if (k + 1 < n && ((t > 0 && !mbar_wait(o_done, (t - 1) & 1)) || !issue_s(t + 1))) {
            ok = false;
            break;
          }
          const int i = 2 * t + 1;
          if (!mbar_wait(p_full, t & 1) || !mbar_wait(&kv_full[i % NS], (i / NS) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t vd = v_desc + (uint32_t)(i % NS) * (Lay::kPage / 16);
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)  // a lane's first tile starts from nothing
            tc_mma_bf16_ts(tmem + Lay::kColO, tmem + Lay::kColS + (t & 1) * kKeys + x * 8, vd + x * (16 * 128 / 16),
                           idesc_o, x == 0 && i_lane == 0 ? 0u : 1u);
          tc_commit(o_done);
          tc_commit(&kv_empty[i % NS]);
          if (++i_lane == tpl) i_lane = 0;
          if (++i_split == ntf) i_split = i_lane = 0;
        }
      }
      if (!ok) {
        report(a.status, DEV_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    reg_alloc_inc<Lay::kSoftmaxRegs>();
    // ---------------- softmax: thread tid holds row tid of the tile (its TMEM lane)
    int seg_n = 0, seg_q = 0;  // tiles of the segment at hand; segments so far
    int64_t seg_rec = 0;       // this thread's row in it, as an index of q heads; -1: none
    int seg_s0 = 0, seg_end = 0;
    bool seg_live = false;     // a row of the warp exists
    // the next segment: its numbers, and its Q on the way to shared memory
    auto next_segment = [&]() -> bool {
      const int place = seg_q % kSegments;
      if (!__all_sync(0xffffffffu, mbar_wait(&seg_full[place], (seg_q / kSegments) & 1))) return false;
      const CtxSegment g = segs[place];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[place]);
      ++seg_q;
      seg_n = g.n;
      if (g.n == 0) return true;
      seg_s0 = g.s0;
      seg_end = g.s_end;
      seg_live = g.r0 + warp * 32 < g.n_rows;
      auto index = [&](int r) { return (g.row0 + (r >> a.gshift)) * a.Hq + g.head0 + (r & (a.group - 1)); };
      seg_rec = g.r0 + tid < g.n_rows ? index(g.r0 + tid) : -1;
#pragma unroll 4
      for (int i = tid; i < 128 * (HD / 8); i += 128) {
        const int qrow = i / (HD / 8), ch = i % (HD / 8);
        const bool there = g.r0 + qrow < g.n_rows;
        cp_async16(sQ + (ch >> 3) * (128 * 128) + qrow * 128 + (((ch & 7) ^ (qrow & 7)) << 4),
                   there ? a.q + index(g.r0 + qrow) * HD + ch * 8 : a.q, there);
      }
      cp_async_commit();
      return true;
    };
    auto q_ready = [&] {
      cp_async_wait<0>();
      fence_proxy_async();
      mbar_arrive(q_full);
    };
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + lane_base + Lay::kColO;
    const float nz = a.neg_zero;
    float run[HD], run_m = -INFINITY, run_l = 0.f;
#pragma unroll
    for (int c = 0; c < HD; ++c) run[c] = 0.f;
    float m = -INFINITY, l = 0.f;  // the lane in progress
    int64_t rec0 = -1;             // the row's records

    // run <- run (+) (lm, ll, O): lane_merge's formula, an empty run taking O as it is (0 * 0 + O * 1).  The last lane
    // of a split: the result is split s's record, and run starts over (s < 0: none).
    auto fold = [&](float lm, float ll, int s) {
      const float M = fmaxf(run_m, lm);
      const bool skip = lm == -INFINITY;  // an empty lane leaves the state as it is
      float fa = run_m == M ? 1.0f : exp2f(__fsub_rn(run_m, M));
      float fb = lm == M ? 1.0f : exp2f(__fsub_rn(lm, M));
      if (run_m == -INFINITY) fa = 0.f, fb = 1.f;
      if (skip) {
        fa = 1.f;
        fb = 0.f;
      } else {
        run_l = run_m == -INFINITY ? ll : __fadd_rn(__fmul_rn(run_l, fa), __fmul_rn(ll, fb));
        run_m = M;
      }
      const bool any_skip = __any_sync(0xffffffffu, skip);
      const float2 fa2 = make_float2(fa, fa), fb2 = make_float2(fb, fb);
      uint32_t ob[2][16];  // 16 columns at hand and the next on their way
      tmem_ld_32x32b_x16(tO, ob[0]);
#pragma unroll
      for (int c = 0; c < HD; c += 16) {
        uint32_t(&o)[16] = ob[(c / 16) & 1];
        tmem_ld_wait_for(o);
        if (c + 16 < HD) tmem_ld_32x32b_x16(tO + c + 16, ob[(c / 16 + 1) & 1]);
        if (any_skip) {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = skip ? 0u : o[k];
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float2 z = add2(mul2(make_float2(run[c + k], run[c + k + 1]), fa2, nz),
                                mul2(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), fb2, nz));
          run[c + k] = z.x;
          run[c + k + 1] = z.y;
        }
        if (s >= 0) {
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            if (rec0 >= 0) store8(a.part_o + (rec0 + s) * HD + c + k, run + c + k);
#pragma unroll
            for (int e = 0; e < 8; ++e) run[c + k + e] = 0.f;
          }
        }
      }
      if (s >= 0) {
        if (rec0 >= 0) *reinterpret_cast<float2*>(a.part_ml + (rec0 + s) * 2) = make_float2(run_m, run_l);
        run_m = -INFINITY;
        run_l = 0.f;
      }
    };

    int t = 0;  // tiles so far
    bool ok = next_segment();
    if (ok && seg_n > 0) q_ready();
    while (ok && seg_n > 0) {
      const int n = seg_n, s0 = seg_s0, s_last = seg_end - 1;
      const bool live = seg_live;
      rec0 = seg_rec < 0 ? -1 : seg_rec * a.nsplit;
      int i_split = 0, i_lane = 0, split = s0;  // the tile's place in its split and lane
      for (int k = 0; k < n; ++k, ++t) {
        ok = mbar_wait(&s_full[t & 1], (t >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const bool fresh = i_lane == 0;
        float alpha = 1.f;
        const float lm = m, ll = l;  // of the lane before, when this tile starts one
        if (k + 1 == n && !(ok = next_segment())) break;  // the last S of the row tile is there: Q may go
        if (live) {
          const uint32_t tS = tmem + lane_base + Lay::kColS + (t & 1) * kKeys;
          uint32_t s[64];
          uint32_t(&s_lo)[32] = *reinterpret_cast<uint32_t (*)[32]>(&s[0]);
          uint32_t(&s_hi)[32] = *reinterpret_cast<uint32_t (*)[32]>(&s[32]);
          tmem_ld_32x32b_x32(tS, s_lo);
          tmem_ld_32x32b_x32(tS + 32, s_hi);
          tmem_ld_wait_for(s);
          // the largest score is the largest product's (scale > 0 and rounding is monotone)
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 2)
            mx[(j >> 1) & 3] = fmaxf(mx[(j >> 1) & 3], fmaxf(__uint_as_float(s[j]), __uint_as_float(s[j + 1])));
          const float top = __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.scale_log2);
          const float m_old = fresh ? -INFINITY : m;
          const float m_new = fmaxf(m_old, top);
          alpha = m_new == m_old ? 1.0f : exp2f(__fsub_rn(m_old, m_new));
          const float2 sc = make_float2(a.scale_log2, a.scale_log2);
          // a row without any key above -inf so far: 2^(-inf - 0) = 0
          const float neg = m_new == -INFINITY ? 0.f : -m_new;
          const float2 ng = make_float2(neg, neg);
          float2 s01 = make_float2(0.f, 0.f), s23 = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              float p[8];
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 x = add2(
                    mul2(make_float2(__uint_as_float(s[h + j + e]), __uint_as_float(s[h + j + e + 1])), sc, nz), ng);
                p[e] = exp2_p(x.x);
                p[e + 1] = exp2_p(x.y);
                pk[(j + e) / 2] = pack_bf16x2(p[e], p[e + 1]);
              }
              s01 = add2(add2(s01, make_float2(p[0], p[2])), make_float2(p[1], p[3]));
              s23 = add2(add2(s23, make_float2(p[4], p[6])), make_float2(p[5], p[7]));
            }
            tmem_st_32x32b_x16(tS + h / 2, pk);
          }
          const float rs = __fadd_rn(__fadd_rn(s01.x, s01.y), __fadd_rn(s23.x, s23.y));
          l = __fadd_rn(__fmul_rn(fresh ? 0.f : l, alpha), rs);
          m = m_new;
        }
        if (k > 0) {
          ok = mbar_wait(o_done, (t - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          if (live && fresh) {
            fold(lm, ll, i_split == 0 ? split - 1 : -1);
          } else if (live && __any_sync(0xffffffffu, alpha != 1.0f)) {
            const float2 al = make_float2(alpha, alpha);
            uint32_t ob[2][16];
            tmem_ld_32x32b_x16(tO, ob[0]);
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
              uint32_t(&o)[16] = ob[(c / 16) & 1];
              tmem_ld_wait_for(o);
              if (c + 16 < HD) tmem_ld_32x32b_x16(tO + c + 16, ob[(c / 16 + 1) & 1]);
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 x = mul2(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), al, nz);
                o[j] = __float_as_uint(x.x);
                o[j + 1] = __float_as_uint(x.y);
              }
              tmem_st_32x32b_x16(tO + c, o);
            }
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        if (++i_lane == tpl) i_lane = 0;
        if (++i_split == ntf) {
          i_split = i_lane = 0;
          ++split;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (seg_n > 0) q_ready();
      ok = mbar_wait(o_done, (t - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (live) fold(m, l, s_last);
    }
    if (!ok) {
      if (lane == 0) report(a.status, DEV_TIMEOUT);
      *abort_flag = 1;
      cp_async_wait<0>();
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, Lay::kCols);
  pdl_wait();
}

// ------------------------------------------------------------------------ the merge
// A warp a (node, q head), HD / 32 neighbouring elements a lane.  The splits before E are merged as the attention merge
// does (a weight a lane, 32 at a time; sums in ascending order; places behind the last split add 0 * 0, and the sums,
// which start from +0, are never -0); the split that E cuts and those behind it are first folded from their lanes with
// lane_merge's formula.  Loads that do not depend on the row's position go out at once, and the next NB records while
// NB are added up.  Few rows wait for their records' latency and want many in flight, many rows want the registers for
// more warps: NB = 16, 8, 4 take 45.9, 47.6, 50.5 us a whole call for 592 rows of 64 splits, 24.6, 25.0, 25.1 for 2048
// of one, and 168, 153.5, 150.5 for 16384 of 14.  The rule's border (16 rows x heads an SM) lies between; nearest above
// it 4608 rows of 2 to 64 splits: 232, 228, 227, so that there 4 and 8 are as good as each other.
constexpr int kTreeMergeWarps = 4;

template <int HD, int NB>
__global__ void __launch_bounds__(kTreeMergeWarps * 32) tree_merge_kernel(const TreeArgs a) {
  constexpr int NE = HD / 32;
  __shared__ float2 weights[kTreeMergeWarps][32];  // (weight, l) of 32 splits
  pdl_trigger();
  pdl_wait();
  struct Vec {
    float v[NE];
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, i = blockIdx.x;
  const int head = blockIdx.z * kTreeMergeWarps + warp;
  if (head >= a.Hq) return;
  const TreeSeq sq = tree_seq(a, b);
  if (i >= sq.n) return;
  const int64_t row = sq.row0 + i;
  const int pos = __ldcg(a.row_pos + row);
  auto load = [&](const float* p, bool there) {
    Vec r = {};
    if constexpr (NE == 4) {
      const float4 x = there ? __ldcg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
      r.v[0] = x.x, r.v[1] = x.y, r.v[2] = x.z, r.v[3] = x.w;
    } else {
      const float2 x = there ? __ldcg(reinterpret_cast<const float2*>(p)) : make_float2(0.f, 0.f);
      r.v[0] = x.x, r.v[1] = x.y;
    }
    return r;
  };
  const bool ok = sq.ok;
  const int E = ok ? tail_lane(a, sq.start) : 0;
  const int sE = ok ? min(sq.start / a.split, a.nsplit) : 0;  // the split that E stands in
  const bool cut = E > sE * a.split && sE < a.nsplit;         // with lanes before E in it
  const int64_t rec = row * a.Hq + head;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + rec * a.nsplit;
  const float2* tml = reinterpret_cast<const float2*>(a.tail_ml) + rec * a.ntail;
  const float* po = a.part_o + rec * a.nsplit * HD + lane * NE;
  const float* to = a.tail_o + rec * a.ntail * HD + lane * NE;
  const float2 none = make_float2(-INFINITY, 0.f);
  float2 r = lane < sE ? __ldcg(ml + lane) : none;
  const float2 rc = cut ? __ldcg(ml + sE) : none;
  const float2 rt = lane < a.ntail ? __ldcg(tml + lane) : none;
  Vec v[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) v[k] = load(po + (int64_t)k * HD, k < sE);
  Vec P = load(po + (int64_t)sE * HD, cut);
  Vec Q = load(to, true);
  __nv_bfloat16* dst = a.out + rec * HD + lane * NE;
  auto store = [&](const Vec& x) {
    uint32_t w[NE / 2];
#pragma unroll
    for (int e = 0; e < NE; e += 2) w[e / 2] = pack_bf16x2(x.v[e], x.v[e + 1]);
    if constexpr (NE == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  };
  Vec O = {};
  if (!ok || pos < 0) {
    store(O);
    return;
  }
  // the largest score
  int n_tail = 0;
  for (int lb = E; lb <= pos && n_tail < a.ntail; lb = lane_end(a, lb)) ++n_tail;
  float M = fmaxf(r.x, rc.x);
  if (lane < n_tail) M = fmaxf(M, rt.x);
  for (int s = 32 + lane; s < sE; s += 32) M = fmaxf(M, __ldcg(ml + s).x);
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  for (int c0 = 0; c0 < sE; c0 += 32) {
    if (c0) r = c0 + lane < sE ? __ldcg(ml + c0 + lane) : none;
    __syncwarp();
    weights[warp][lane] = make_float2(merge_weight(r.x, M), r.y);
    __syncwarp();
    for (int k0 = 0; k0 < 32 && c0 + k0 < sE; k0 += NB) {
      Vec x[NB];
      const int ahead = c0 + k0 + NB;
#pragma unroll
      for (int k = 0; k < NB; ++k) x[k] = load(po + (int64_t)(ahead + k) * HD, ahead + k < sE);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float2 wl = weights[warp][k0 + k];
        L = merge_term(L, wl.y, wl.x);
#pragma unroll
        for (int e = 0; e < NE; ++e) O.v[e] = merge_term(O.v[e], v[k].v[e], wl.x);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) v[k] = x[k];
    }
  }
  // the split that E cuts, and those behind it
  float pm = rc.x, pl = rc.y;
  int lb = E;
  for (int t = 0; t < n_tail; ++t) {
    const float2 x = make_float2(__shfl_sync(0xffffffffu, rt.x, t), __shfl_sync(0xffffffffu, rt.y, t));
    if (t > 0) Q = load(to + (int64_t)t * HD, true);
    if (x.x != -INFINITY) {
      if (pm == -INFINITY) {
        pm = x.x;
        pl = x.y;
        P = Q;
      } else {
        const float m = fmaxf(pm, x.x);
        const float fa = pm == m ? 1.0f : exp2f(__fsub_rn(pm, m));
        const float fb = x.x == m ? 1.0f : exp2f(__fsub_rn(x.x, m));
        pl = __fadd_rn(__fmul_rn(pl, fa), __fmul_rn(x.y, fb));
#pragma unroll
        for (int e = 0; e < NE; ++e) P.v[e] = __fadd_rn(__fmul_rn(P.v[e], fa), __fmul_rn(Q.v[e], fb));
        pm = m;
      }
    }
    const int le = lane_end(a, lb);
    if (le % a.split == 0 || t + 1 == n_tail) {  // the split ends, or the row does
      const float w = merge_weight(pm, M);
      L = merge_term(L, pl, w);
#pragma unroll
      for (int e = 0; e < NE; ++e) O.v[e] = merge_term(O.v[e], P.v[e], w);
      P = {};
      pm = -INFINITY;
      pl = 0.f;
    }
    lb = le;
  }
#pragma unroll
  for (int e = 0; e < NE; ++e) O.v[e] = __fdiv_rn(O.v[e], L);
  store(O);
}

// Records of a row's lanes from E on: its positions there are at most `max_nodes` from anywhere in a lane.
// At most 8 (256 nodes, a split of 832: lanes of 256 and a last one of 64).
static int tail_records(int64_t max_nodes, int split, int lane_len) {
  const int shortest = split % lane_len ? split % lane_len : lane_len;
  return (int)((max_nodes - 1 + lane_len - 1) / shortest) + 1;
}
static int split_lane_len(int split) { return ((split + 3) / 4 + kKeys - 1) / kKeys * kKeys; }

template <int HD>
static bi_status launch_tree(TreeArgs args, int64_t B, cudaStream_t st) {
  using Tail = TailLayout<HD>;
  using Ctx = CtxLayout<HD>;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  static int ctx_regs = 0;
  constexpr int kMost = 227 * 1024;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(tree_tail_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (attr_err == cudaSuccess)
      attr_err = cudaFuncSetAttribute(tree_context_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ctx::kBytes);
    cudaFuncAttributes fa{};
    if (attr_err == cudaSuccess) attr_err = cudaFuncGetAttributes(&fa, tree_context_kernel<HD>);
    ctx_regs = fa.numRegs;
  });
  if (attr_err != cudaSuccess)
    return fail(BI_ERR_CUDA, std::string("tree attention attributes: ") + cudaGetErrorString(attr_err));
  // the warpgroups' register split must fit what the block launches with, or the increase would never be granted
  if (ctx_regs < Ctx::kLaunchRegs)
    return fail(BI_ERR_CUDA, "tree attention: compiled with fewer registers than its warpgroup split needs");
  CUtensorMap tmk, tmv;
  const uint64_t rows = (uint64_t)args.n_blocks * args.Hkv * kKeys;
  if (!encode_tmap_2d_bf16(&tmk, args.k_cache, HD, rows, HD * 2, 64, kKeys, true) ||
      !encode_tmap_2d_bf16(&tmv, args.v_cache, HD, rows, HD * 2, 64, kKeys, true))
    return fail(BI_ERR_CUDA, "bi_tree_attention: cuTensorMapEncodeTiled failed for the K/V cache");
  // pages that can hold a tile's nodes and their ancestors together with the last context tokens before them
  args.stages = std::max(3, (63 + args.max_nodes + 63) / 64);
  const int64_t r = (int64_t)args.max_nodes * args.group;
  const int per_cta = kTailWarps / ((args.group + 15) / 16);  // nodes of a CTA
  BI_TRY(launched(launch_pdl(tree_tail_kernel<HD>,
                             dim3((unsigned)cdiv(args.max_nodes, per_cta), (unsigned)B, (unsigned)args.Hkv),
                             dim3(kTailWarps * 32), Tail::bytes(args.stages), st, args, tmk, tmv),
                  "tree_tail_kernel"));
  // at most one CTA a unit, and what fits on the GPU at once
  const int64_t units = cdiv(r, 128) * B * args.Hkv * args.nsplit;
  BI_TRY(launched(launch_pdl(tree_context_kernel<HD>, dim3((unsigned)std::min<int64_t>(units, 2 * (int64_t)num_sms())),
                             dim3(Ctx::kThreads), Ctx::kBytes, st, args, tmk, tmv),
                  "tree_context_kernel"));
  const bool few = args.T * args.Hq <= 16 * (int64_t)num_sms();
  return launched(launch_pdl(few ? tree_merge_kernel<HD, 16> : tree_merge_kernel<HD, 4>,
                             dim3((unsigned)args.max_nodes, (unsigned)B, (unsigned)cdiv(args.Hq, kTreeMergeWarps)),
                             dim3(kTreeMergeWarps * 32), 0, st, args),
                  "tree_merge_kernel");
}

}  // namespace bi

extern "C" {

size_t bi_tree_attention_workspace_size(int64_t max_T, int Hq, int hd, int64_t max_ctx, int kv_split) {
  if (max_T <= 0 || Hq <= 0 || hd <= 0 || max_ctx <= 0 || kv_split < 64) return 0;
  const size_t recs = bi::cdiv(max_ctx, kv_split) +
                      bi::tail_records(bi::kMaxTreeNodes, kv_split, bi::split_lane_len(kv_split));
  return (size_t)max_T * Hq * recs * (hd + 2) * sizeof(float) + (size_t)max_T * sizeof(int32_t) + 256;
}

bi_status bi_tree_attention(const void* q, int64_t T, const int32_t* parent, const int32_t* row0, const int32_t* start,
                            int64_t B, int64_t max_nodes, int Hq, int Hkv, int hd, const void* k_cache,
                            const void* v_cache, const int32_t* block_table, int64_t max_blocks_per_seq,
                            int64_t n_blocks, int64_t max_ctx, int kv_split, float scale, void* workspace,
                            size_t ws_bytes, void* out, void* stream) {
  using namespace bi;
  BI_REQUIRE(T >= 0 && B >= 0, "T < 0 or B < 0");
  if (T == 0 || B == 0) return BI_OK;
  BI_REQUIRE(q && parent && row0 && start && k_cache && v_cache && block_table && workspace && out, "null pointer");
  BI_REQUIRE(max_nodes >= 1, "max_nodes must be positive");
  BI_REQUIRE_SHAPE(max_nodes <= kMaxTreeNodes, "max_nodes must be at most 256");
  BI_REQUIRE_SHAPE(hd == 64 || hd == 128, "head_dim must be 64 or 128");
  BI_REQUIRE(Hq > 0 && Hkv > 0 && Hq % Hkv == 0, "Hq must be a multiple of Hkv");
  const int group = Hq / Hkv;
  BI_REQUIRE_SHAPE(64 % group == 0, "64 must be a multiple of Hq/Hkv");
  BI_REQUIRE(kv_split >= 64 && kv_split % 64 == 0, "kv_split must be a positive multiple of 64");
  BI_REQUIRE_SHAPE(kv_split <= kTreeMaxSplit, "kv_split must be at most 16384");
  BI_REQUIRE(scale > 0, "scale must be positive");
  BI_REQUIRE(max_ctx > 0 && max_blocks_per_seq > 0 && n_blocks > 0, "bad max_ctx or cache shape");
  BI_REQUIRE_SHAPE(n_blocks < (int64_t(1) << 31) / 64 / Hkv && max_blocks_per_seq <= 0x7fffffff / 64 &&
                       max_ctx <= 0x7fffffff - 2 * kTreeMaxSplit,
                   "cache or context too large");
  BI_REQUIRE(aligned16(q) && aligned16(workspace) && aligned16(out) && aligned16(k_cache) && aligned16(v_cache),
             "pointers must be 16-byte aligned");
  const int64_t ns = cdiv(max_ctx, kv_split);
  BI_REQUIRE(B <= 65535 && Hkv * ns <= 65535 && T <= 0x7fffffff, "too many sequences, rows or splits");
  const int lane_len = split_lane_len(kv_split);
  const int nt = tail_records(max_nodes, kv_split, lane_len);
  BI_REQUIRE(nt <= kMaxTailRecords, "too many lanes behind the context");
  const size_t per = (size_t)T * Hq * ns, per_t = (size_t)T * Hq * nt;
  // records are written 32 bytes at a time
  const size_t skip = (32 - (reinterpret_cast<uintptr_t>(workspace) & 31)) & 31;
  BI_REQUIRE(ws_bytes >= skip + (per + per_t) * (hd + 2) * sizeof(float) + (size_t)T * sizeof(int32_t),
             "workspace too small (bi_tree_attention_workspace_size)");
  TreeArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.parent = parent;
  a.row0 = row0;
  a.start = start;
  a.block_table = block_table;
  a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + skip);
  a.tail_o = a.part_o + per * hd;
  a.part_ml = a.tail_o + per_t * hd;
  a.tail_ml = a.part_ml + per * 2;
  a.row_pos = reinterpret_cast<int32_t*>(a.tail_ml + per_t * 2);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = device_status_ptr();
  a.T = T;
  a.max_blk = max_blocks_per_seq;
  a.n_blocks = n_blocks;
  a.max_nodes = (int)max_nodes;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.B = (int)B;
  a.group = group;  // a power of two (a divisor of 64)
  a.gshift = 0;
  while ((1 << a.gshift) < group) ++a.gshift;
  a.nsplit = (int)ns;
  a.ntail = nt;
  a.lane_len = lane_len;
  a.split = kv_split;
  a.stages = 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.neg_zero = -0.f;
  return hd == 64 ? launch_tree<64>(a, B, as_stream(stream)) : launch_tree<128>(a, B, as_stream(stream));
}

}  // extern "C"
