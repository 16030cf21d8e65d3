// Attention of the nodes of drafted trees over the paged cache and their own ancestors.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §4.2 (one read path, fixed absolute splits).  Node i of a
// sequence's tree has its key and value in the cache at position start + i, and stands itself at position start +
// depth.  It attends to positions 0 .. start - 1 and to its path, taken as if the path's nodes stood at positions
// start .. start + depth.  Every row repeats, operation for operation, the arithmetic of bi_attention on a cache
// that holds just that path (splits, lanes, 64-key tiles and 16-key MMA steps by position), so it has the bits
// that a plain decode of the path gives.
//
// What bounds it: keys and values are read once for a tile of up to 64 query rows (nodes x q heads of a group),
// so small trees are bound by HBM, large ones by mma.sync and the shared-memory reads that feed it.
//
// A CTA owns (sequence, row tile, kv head, split).  The keys before `start` are the same for all rows: whole 64-key
// pages come by TMA into a ring and every warp runs its 16 rows over them.  Tiles that hold positions from
// `start` on differ by node: the pages that hold the tree's own keys are then all in the ring at once, and a
// node's tile is read by ldmatrix with a row address for each position (the page's row for a position before
// `start`, the path node's row behind it).  An 8-key group of scores or a 16-key step of P V whose positions all
// stand before `start` is done for the warp's 16 rows at once; the others once for each node of the warp, and a
// row keeps its own node's result.
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
  float* part_o;    // [T, Hq, nsplit, hd]
  float* part_ml;   // [T, Hq, nsplit, 2]
  int32_t* row_pos; // [T]: a node's position, -1 when it has none
  __nv_bfloat16* out;
  int* status;
  int64_t T, max_blk, n_blocks;
  int max_nodes, Hq, Hkv, group, nsplit, split, stages;
  float scale_log2;
};

constexpr int kTreeMaxSplit = 16384;  // positions of a split: 256 pages, whose ids stand in shared memory

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
  const int64_t r0 = a.row0[b], r1 = a.row0[b + 1];
  s.row0 = r0;
  s.start = a.start[b];
  s.rows_ok = r0 >= 0 && r1 >= r0 && r1 <= a.T && r1 - r0 <= a.max_nodes;
  s.n = s.rows_ok ? (int)(r1 - r0) : 0;
  s.ok = s.rows_ok && s.start >= 0 && (int64_t)s.start + s.n <= a.max_blk * kKeys;
  return s;
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

// acc += P V of one 64-key tile: four 16-key steps in order, P rounded to bf16.
template <int HD>
__device__ __forceinline__ void tree_pv(uint32_t sv, const float (&p)[8][4], int lane, LaneState<HD>& st) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint32_t pa[4] = {pack_bf16x2(p[2 * kk][0], p[2 * kk][1]), pack_bf16x2(p[2 * kk][2], p[2 * kk][3]),
                            pack_bf16x2(p[2 * kk + 1][0], p[2 * kk + 1][1]),
                            pack_bf16x2(p[2 * kk + 1][2], p[2 * kk + 1][3])};
#pragma unroll
    for (int j = 0; j < HD / 8; j += 2) {
      const int key = kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(sv + kv_off<HD>(key, j + (lane >> 4)), b0, b1, b2, b3);
      mma_bf16_16816(st.acc[j], pa, b0, b1);
      mma_bf16_16816(st.acc[j + 1], pa, b2, b3);
    }
  }
}

// Shared memory: the page ring, then barriers, a row of zeros, depths, parents, the warps' path
// tables and the page ids of the CTA.
template <int HD, int WARPS>
struct TreeLayout {
  static constexpr int kPage = kKeys * HD * 2;
  static constexpr int kStage = 2 * kPage;  // a K page and its V page
  static constexpr int kMaxStages = 12;
  static constexpr int kZero = HD * 2;      // a key row of zeros
  static int ids(int split) { return (split / kKeys + kMaxTreeNodes / kKeys + 2) * 4; }
  static int bytes(int stages, int split) {
    return 1024 + stages * kStage + 256 + kZero + kMaxTreeNodes * 4 + WARPS * 16 * kKeys * 2 + ids(split);
  }
};

// ROWS: 16-row warps of a row tile.  LANES: the split's four lanes on warps of their own (few rows: more warps to
// hide latency with), or 1: one after another.
template <int HD, int ROWS, int LANES>
__global__ void __launch_bounds__(ROWS * LANES * 32) tree_attention_kernel(const TreeArgs a,
                                                                           const __grid_constant__ CUtensorMap tmk,
                                                                           const __grid_constant__ CUtensorMap tmv) {
  constexpr int WARPS = ROWS * LANES;
  using Lay = TreeLayout<HD, WARPS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NS = a.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * Lay::kStage);  // [NS] the stage's pages have landed
  uint64_t* empty = full + Lay::kMaxStages;                               // [NS] its warps have read them
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + Lay::kMaxStages);
  int* max_depth = const_cast<int*>(abort_flag) + 1;
  volatile int* issued = abort_flag + 2;  // [NS] the page that was last asked for in each stage
  uint8_t* zero_row = smem + NS * Lay::kStage + 256;
  int16_t* depth_of = reinterpret_cast<int16_t*>(zero_row + Lay::kZero);
  int16_t* parent_of = depth_of + kMaxTreeNodes;
  uint16_t* paths = reinterpret_cast<uint16_t*>(parent_of + kMaxTreeNodes);  // [WARPS][16][64]
  int32_t* ids = reinterpret_cast<int32_t*>(paths + WARPS * 16 * kKeys);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y;
  const int kvh = (int)blockIdx.z % a.Hkv, s = (int)blockIdx.z / a.Hkv;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], ROWS);
      issued[i] = -1;
    }
    *abort_flag = 0;
    *max_depth = -1;
    fence_barrier_init();
  }
  for (int i = tid; i < Lay::kZero / 4; i += WARPS * 32) reinterpret_cast<uint32_t*>(zero_row)[i] = 0u;
  pdl_trigger();
  pdl_wait();
  const TreeSeq sq = tree_seq(a, b);
  const bool speaks = s == 0 && kvh == 0;  // the CTA that reports its sequence's faults and writes positions
  const int n = sq.n, start = sq.start;
  const int node0 = (int)((int64_t)blockIdx.x * ROWS * 16 / a.group);  // the tile's first node
  if (speaks && tid == 0 && !sq.ok) report(a.status, DEV_BAD_INDEX);
  if (node0 >= n) return;
  const int last_node = min(n, (int)(((int64_t)(blockIdx.x + 1) * ROWS * 16 + a.group - 1) / a.group)) - 1;
  if (!sq.ok) {
    if (speaks)
      for (int i = node0 + tid; i <= last_node; i += WARPS * 32) a.row_pos[sq.row0 + i] = -1;
    return;
  }
  const int kv_begin = s * a.split;
  // no position of this split is at or before any row's
  if (kv_begin > start + last_node) return;
  const int lane_len = ((a.split + 3) / 4 + kKeys - 1) / kKeys * kKeys;
  const int tail0 = start / kKeys * kKeys;  // the first tile with positions from `start` on
  // depths (and so the rows' own positions) matter to splits that reach such a tile, and to whoever writes them down
  const bool tail = kv_begin + a.split > tail0;
  const int n_plain = max(0, min(kv_begin + a.split, tail0) - kv_begin) / kKeys;
  const int tail_page0 = start / kKeys;
  const int tail_pages = tail ? (start + last_node) / kKeys - tail_page0 + 1 : 0;
  const int n_pages = n_plain + tail_pages;
  for (int i = tid; i < n_pages; i += WARPS * 32) {
    const int page = i < n_plain ? kv_begin / kKeys + i : tail_page0 + i - n_plain;
    ids[i] = page < a.max_blk ? a.block_table[(int64_t)b * a.max_blk + page] : -1;
  }
  if ((tail || speaks) && warp == WARPS - 1) {
    const bool bad = tree_depths(a.parent + sq.row0, last_node + 1, depth_of, lane, parent_of);
    int deep = -1;
    bool far = false;
    for (int i = node0 + lane; i <= last_node; i += 32) {
      const int d = depth_of[i];
      const bool fits = (int64_t)start + d < (int64_t)a.nsplit * a.split;
      far |= !fits;
      if (d >= 0 && fits) deep = max(deep, d);
      if (speaks) a.row_pos[sq.row0 + i] = d >= 0 && fits ? start + d : -1;
    }
    for (int o = 16; o; o >>= 1) deep = max(deep, __shfl_xor_sync(0xffffffffu, deep, o));
    if (lane == 0) *max_depth = deep;
    if (speaks && (bad || far)) report(a.status, DEV_BAD_INDEX);
  }
  __syncthreads();
  const int deep = tail ? *max_depth : 0;
  // logical tiles from tail0 on that some row of the tile sees in this split
  const int tail_begin = max(tail0, kv_begin);
  const int tail_end = tail ? min(kv_begin + a.split, start + deep + 1) : 0;
  if (n_plain == 0 && tail_end <= tail_begin) return;
  const int n_issue = tail_end > tail_begin ? n_pages : n_plain;

  // plain pages in the order in which they are used: round k holds page k of every lane that has one
  const int ppl = lane_len / kKeys;
  const int nl = (n_plain + ppl - 1) / ppl;
  const int last_cnt = n_plain - (nl - 1) * ppl;  // pages of the last lane
  auto order_of = [&](int ln, int k) {
    return LANES == 1 ? ln * ppl + k : (k < last_cnt ? k * nl + ln : last_cnt * nl + (k - last_cnt) * (nl - 1) + ln);
  };
  auto page_at = [&](int j) {
    if (LANES == 1 || j >= n_plain) return j;
    if (j < last_cnt * nl) return j % nl * ppl + j / nl;
    const int r = j - last_cnt * nl;
    return r % (nl - 1) * ppl + last_cnt + r / (nl - 1);
  };
  const int rows_total = (int)(a.n_blocks * a.Hkv * kKeys);
  auto issue = [&](int j) {
    const int32_t id = ids[page_at(j)];
    int row = rows_total;  // past the end: the copy reads zeros
    if (id >= 0 && id < a.n_blocks) row = (int)(((int64_t)id * a.Hkv + kvh) * kKeys);
    else report(a.status, DEV_BAD_INDEX);
    const int slot = j % NS;
    uint8_t* sk = smem + slot * Lay::kStage;
    __threadfence_block();
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

  // this warp's rows: node, q head and position of the two a thread holds
  const int g = lane >> 2, tq = lane & 3;
  const int rw = warp % ROWS, lw = warp / ROWS;
  int row_node[2], row_pos[2], row_head[2];
  bool row_valid[2];
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = (int64_t)blockIdx.x * ROWS * 16 + rw * 16 + g + h * 8;
    row_node[h] = (int)(r / a.group);
    row_valid[h] = row_node[h] < n;
    row_head[h] = kvh * a.group + (int)(r % a.group);
    const int d = row_valid[h] && tail ? depth_of[row_node[h]] : 0;
    row_pos[h] = row_valid[h] && d >= 0 && start + d < a.nsplit * a.split ? start + d : -1;
    const __nv_bfloat16* qr = a.q + ((sq.row0 + row_node[h]) * a.Hq + row_head[h]) * HD + tq * 2;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      qf[kk][h] = row_valid[h] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16) : 0u;
      qf[kk][2 + h] = row_valid[h] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8) : 0u;
    }
  }

  LaneState<HD> cur, run;
  clear(run);
  clear(cur);
  int prev = -1;  // the page (in order of use) that this group of warps read last
  bool ok = true;
  auto refill = [&]() {  // the freed stage takes the page NS places on
    if (rw == 0 && lane == 0 && prev >= 0 && prev + NS < n_issue) {
      if (!mbar_wait(&empty[prev % NS], (prev / NS) & 1)) {
        report(a.status, DEV_TIMEOUT);
        *abort_flag = 1;
      } else {
        issue(prev + NS);
      }
    }
    prev = -1;
  };
  auto wait_page = [&](int j) {
    bool there = true;
    if constexpr (LANES > 1) {
      // the stage's page before this one may be another group's, not landed yet: its phase must not be taken for this one's
      const unsigned long long t0 = globaltimer();
      while (there && issued[j % NS] != j) there = globaltimer() - t0 < kWaitLimitNs;
      __threadfence_block();
    }
    if (!there || !mbar_wait(&full[j % NS], (j / NS) & 1)) {
      report(a.status, DEV_TIMEOUT);
      *abort_flag = 1;
    }
    return (bool)__all_sync(0xffffffffu, *abort_flag == 0);
  };

  uint16_t* path = paths + warp * 16 * kKeys;
  const int per_node = min(a.group, 16);           // rows of a node in this warp
  const int n_slots = 16 / per_node;               // nodes of this warp
  const int64_t wr0 = (int64_t)blockIdx.x * ROWS * 16 + rw * 16;
  const int wnode0 = (int)(wr0 / a.group);
  const int wlast = min(n, wnode0 + n_slots) - 1;  // the warp's last node
  bool tail_here = false;
  const int lanes = (a.split + lane_len - 1) / lane_len;
  for (int ln = LANES == 1 ? 0 : lw; ok && ln < lanes; ln += LANES) {
    const int lb = kv_begin + ln * lane_len, le = min(lb + lane_len, kv_begin + a.split);
    const int plain = max(0, min(ppl, n_plain - ln * ppl));
    for (int k = 0; ok && k < plain; ++k) {
      const int j = order_of(ln, k);
      refill();
      if (!(ok = wait_page(j))) break;
      const uint32_t sk = smem_u32(smem + j % NS * Lay::kStage);
      float sc[8][4];
      attn_scores<HD, 2>(sk, qf, lane, sc);
      tree_softmax<HD, false>(sc, 0, row_pos, a.scale_log2, lane, cur);
      tree_pv<HD>(sk + Lay::kPage, sc, lane, cur);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[j % NS]);
      prev = j;
    }
    // tiles that hold positions from `start` on
    const int tb = max(lb, tail_begin), te = min(le, tail_end);
    if (ok && tb < te) {
      refill();
      if (!tail_here) {
        for (int i = 0; ok && i < tail_pages; ++i) ok = wait_page(n_plain + i);
        tail_here = true;
        if (!ok) break;
      }
      for (int key0 = tb / kKeys * kKeys; key0 < te; key0 += kKeys) {
        // path[slot][i]: the row, among the tail pages' rows, of position key0 + i (0xffff: none, a row of zeros)
        __syncwarp();
        for (int i = lane; i < n_slots * kKeys; i += 32) {
          const int p = key0 + i % kKeys;
          path[i] = p < start ? (uint16_t)(p - tail0) : (uint16_t)0xffff;
        }
        __syncwarp();
        if (lane < n_slots && wnode0 + lane <= wlast) {
          int node = wnode0 + lane;
          for (int p = start + depth_of[node]; p >= start && p >= key0; --p) {
            if (p < key0 + kKeys) path[lane * kKeys + p - key0] = (uint16_t)(start - tail0 + node);
            node = parent_of[node];
          }
        }
        __syncwarp();
        // byte address of chunk ch of position i of node slot ns; v: of the V page
        auto addr = [&](int ns, int i, int ch, bool v) -> uint32_t {
          const int off = path[ns * kKeys + i];
          if (off == 0xffff) return smem_u32(zero_row) + ch * 16;
          const int pg = n_plain + off / kKeys;
          return smem_u32(smem + pg % NS * Lay::kStage + (v ? Lay::kPage : 0)) + kv_off<HD>(off % kKeys, ch);
        };
        float sc[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
          const bool shared = key0 + j * 8 + 7 < start;
          for (int ns = 0; ns < (shared ? 1 : n_slots); ++ns) {
            if (!shared && (wnode0 + ns > wlast || start + depth_of[wnode0 + ns] < key0 + j * 8)) continue;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < HD / 16; kk += 2) {
              uint32_t b0, b1, b2, b3;
              ldsm_x4(addr(ns, j * 8 + (lane & 7), kk * 2 + (lane >> 3), false), b0, b1, b2, b3);
              mma_bf16_16816(d, qf[kk], b0, b1);
              mma_bf16_16816(d, qf[kk + 1], b2, b3);
            }
            const bool mine0 = shared || g / per_node == ns, mine1 = shared || (g + 8) / per_node == ns;
            sc[j][0] = mine0 ? d[0] : sc[j][0];
            sc[j][1] = mine0 ? d[1] : sc[j][1];
            sc[j][2] = mine1 ? d[2] : sc[j][2];
            sc[j][3] = mine1 ? d[3] : sc[j][3];
          }
        }
        tree_softmax<HD, true>(sc, key0, row_pos, a.scale_log2, lane, cur);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t pa[4] = {pack_bf16x2(sc[2 * kk][0], sc[2 * kk][1]), pack_bf16x2(sc[2 * kk][2], sc[2 * kk][3]),
                                  pack_bf16x2(sc[2 * kk + 1][0], sc[2 * kk + 1][1]),
                                  pack_bf16x2(sc[2 * kk + 1][2], sc[2 * kk + 1][3])};
          const bool shared = key0 + kk * 16 + 15 < start;
          for (int ns = 0; ns < (shared ? 1 : n_slots); ++ns) {
            if (wnode0 + ns > wlast) continue;
            const bool mine0 = shared || g / per_node == ns, mine1 = shared || (g + 8) / per_node == ns;
#pragma unroll
            for (int j = 0; j < HD / 8; j += 2) {
              const int key = kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
              uint32_t b0, b1, b2, b3;
              ldsm_x4_t(addr(ns, key, j + (lane >> 4), true), b0, b1, b2, b3);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float (&acc)[4] = cur.acc[j + x];
                float d[4] = {acc[0], acc[1], acc[2], acc[3]};
                mma_bf16_16816(d, pa, x ? b2 : b0, x ? b3 : b1);
                acc[0] = mine0 ? d[0] : acc[0];
                acc[1] = mine0 ? d[1] : acc[1];
                acc[2] = mine1 ? d[2] : acc[2];
                acc[3] = mine1 ? d[3] : acc[3];
              }
            }
          }
        }
      }
    }
    if constexpr (LANES == 1) {  // the finished lane folds into the split's state
      lane_merge<HD>(run, cur.m, cur.l, cur.acc);
      clear(cur);
    }
  }
  refill();
  if constexpr (LANES > 1) {
    // the lanes meet in shared memory, over the ring, once every warp is through with it
    __syncthreads();
    constexpr int NF = 4 + HD / 2;  // floats of a thread's state
    float* mine = reinterpret_cast<float*>(smem) + warp * NF * 32 + lane;
    if (*abort_flag == 0) {
      mine[0] = cur.m[0];
      mine[32] = cur.m[1];
      mine[64] = cur.l[0];
      mine[96] = cur.l[1];
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) mine[(4 + j * 4 + c) * 32] = cur.acc[j][c];
    }
    __syncthreads();
    if (lw == 0 && *abort_flag == 0) {
      for (int w = 0; w < min(lanes, LANES); ++w) {
        const float* o = reinterpret_cast<const float*>(smem) + (w * ROWS + rw) * NF * 32 + lane;
        cur.m[0] = o[0];
        cur.m[1] = o[32];
        cur.l[0] = o[64];
        cur.l[1] = o[96];
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) cur.acc[j][c] = o[(4 + j * 4 + c) * 32];
        lane_merge<HD>(run, cur.m, cur.l, cur.acc);
      }
    }
  } else {
    __syncthreads();
  }
  if (*abort_flag) {
    // the copies this CTA started land before it ends
    if (tid == 0)
      for (int i = 0; i < NS; ++i)
        if (issued[i] >= 0) mbar_wait(&full[i], (issued[i] / NS) & 1);
    return;
  }
  if (lw != 0) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!row_valid[h] || (tail && row_pos[h] < kv_begin)) continue;
    const int64_t at = ((sq.row0 + row_node[h]) * a.Hq + row_head[h]) * a.nsplit + s;
    float* po = a.part_o + at * HD;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j)
      *reinterpret_cast<float2*>(po + j * 8 + tq * 2) = make_float2(run.acc[j][h * 2], run.acc[j][h * 2 + 1]);
    if (tq == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(run.m[h], run.l[h]);
  }
}

// The split partials of a row, merged as the attention merge does: one CTA a node, a thread an element.
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a, int hd) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, i = blockIdx.x;
  const TreeSeq sq = tree_seq(a, b);
  if (i >= sq.n) return;
  const int64_t row = sq.row0 + i;
  const int pos = a.row_pos[row];
  for (int e = blockIdx.z * 128 + threadIdx.x; e < a.Hq * hd; e += gridDim.z * 128) {
    float v = 0.f;
    if (pos >= 0)
      v = merge_split_element(a.part_o, a.part_ml, (row * a.Hq + e / hd) * a.nsplit, pos / a.split + 1, hd, e % hd);
    a.out[row * a.Hq * hd + e] = f2bf(v);
  }
}

template <int HD, int ROWS, int LANES>
static bi_status launch_tree(TreeArgs args, int64_t B, int want_stages, int min_stages, const CUtensorMap& tmk,
                             const CUtensorMap& tmv, cudaStream_t st) {
  using Lay = TreeLayout<HD, ROWS * LANES>;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  constexpr int kMost = 227 * 1024;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(tree_attention_kernel<HD, ROWS, LANES>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (attr_err != cudaSuccess)
    return fail(BI_ERR_CUDA, std::string("tree attention smem attribute: ") + cudaGetErrorString(attr_err));
  args.stages = std::max(want_stages, min_stages);
  const int smem = Lay::bytes(args.stages, args.split);
  if (args.stages > Lay::kMaxStages || smem > kMost)
    return fail(BI_ERR_UNSUPPORTED_SHAPE, "bi_tree_attention: the tree does not fit shared memory");
  const dim3 grid((unsigned)cdiv((int64_t)args.max_nodes * args.group, ROWS * 16), (unsigned)B,
                  (unsigned)(args.Hkv * args.nsplit));
  return launched(launch_pdl(tree_attention_kernel<HD, ROWS, LANES>, grid, dim3(ROWS * LANES * 32), smem, st, args,
                             tmk, tmv),
                  "tree_attention_kernel");
}

}  // namespace bi

extern "C" {

size_t bi_tree_attention_workspace_size(int64_t max_T, int Hq, int hd, int64_t max_ctx, int kv_split) {
  if (max_T <= 0 || Hq <= 0 || hd <= 0 || max_ctx <= 0 || kv_split < 64) return 0;
  const size_t per = (size_t)max_T * Hq * bi::cdiv(max_ctx, kv_split);
  return per * (hd + 2) * sizeof(float) + (size_t)max_T * sizeof(int32_t) + 256;
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
  BI_REQUIRE(max_ctx > 0 && max_blocks_per_seq > 0 && n_blocks > 0, "bad max_ctx or cache shape");
  BI_REQUIRE_SHAPE(n_blocks < (int64_t(1) << 31) / 64 / Hkv && max_blocks_per_seq <= 0x7fffffff / 64 &&
                       max_ctx <= 0x7fffffff - 2 * kTreeMaxSplit,
                   "cache or context too large");
  BI_REQUIRE(aligned16(q) && aligned16(workspace) && aligned16(out) && aligned16(k_cache) && aligned16(v_cache),
             "pointers must be 16-byte aligned");
  const int64_t ns = cdiv(max_ctx, kv_split);
  BI_REQUIRE(B <= 65535 && Hkv * ns <= 65535 && T <= 0x7fffffff, "too many sequences, rows or splits");
  const size_t per = (size_t)T * Hq * ns;
  BI_REQUIRE(ws_bytes >= per * (hd + 2) * sizeof(float) + (size_t)T * sizeof(int32_t),
             "workspace too small (bi_tree_attention_workspace_size)");
  TreeArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.parent = parent;
  a.row0 = row0;
  a.start = start;
  a.block_table = block_table;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + per * hd;
  a.row_pos = reinterpret_cast<int32_t*>(a.part_ml + per * 2);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = device_status_ptr();
  a.T = T;
  a.max_blk = max_blocks_per_seq;
  a.n_blocks = n_blocks;
  a.max_nodes = (int)max_nodes;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = group;
  a.nsplit = (int)ns;
  a.split = kv_split;
  a.stages = 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  CUtensorMap tmk, tmv;
  const uint64_t rows = (uint64_t)n_blocks * Hkv * kKeys;
  if (!encode_tmap_2d_bf16(&tmk, k_cache, hd, rows, hd * 2, 64, kKeys, true) ||
      !encode_tmap_2d_bf16(&tmv, v_cache, hd, rows, hd * 2, 64, kKeys, true))
    return fail(BI_ERR_CUDA, "bi_tree_attention: cuTensorMapEncodeTiled failed for the K/V cache");
  cudaStream_t st = as_stream(stream);
  // pages that can hold a tree's nodes together with the last context tokens before them
  const int tail = (int)((63 + max_nodes + 63) / 64);
  const int64_t r = max_nodes * group;
  bi_status s;
  if (r <= 16)
    s = hd == 64 ? launch_tree<64, 1, 4>(a, B, 6, tail, tmk, tmv, st) : launch_tree<128, 1, 4>(a, B, 6, tail, tmk, tmv, st);
  else if (r <= 32)
    s = hd == 64 ? launch_tree<64, 2, 4>(a, B, 6, tail, tmk, tmv, st) : launch_tree<128, 2, 4>(a, B, 6, tail, tmk, tmv, st);
  else
    s = hd == 64 ? launch_tree<64, 4, 1>(a, B, 6, tail, tmk, tmv, st) : launch_tree<128, 4, 1>(a, B, 3, tail, tmk, tmv, st);
  BI_TRY(s);
  const dim3 mgrid((unsigned)max_nodes, (unsigned)B, (unsigned)std::min<int64_t>(cdiv(Hq * hd, 128), 65535));
  return launched(launch_pdl(tree_merge_kernel, mgrid, dim3(128), 0, st, a, hd), "tree_merge_kernel");
}

}  // extern "C"
