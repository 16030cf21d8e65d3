// The rows of a step that drafts a tree of tokens a sequence, and the acceptance of a path of it.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §2 ("the same discrete choices"): a drafted token is kept
// when it is the token that the model chose at its parent, so the rollout is the one that plain decoding gives;
// §4.2: the accepted rows then stand in the paged cache where plain decoding would have written them.
#include <algorithm>
#include <string>

#include "common.cuh"
#include "tree.cuh"

namespace bi {

constexpr int kPage = 64;

// ------------------------------------------------------------------------ rows of a step
// A warp a sequence; a CTA's eight sequences are neighbours, and its threads first add up the node counts before
// them.  A step has few rows, so the chain of loads (counts, parents, table) is the time.
constexpr int kSlotWarps = 8;

__global__ void __launch_bounds__(kSlotWarps * 32) tree_slot_map_kernel(
    const int32_t* __restrict__ parent, const int32_t* __restrict__ n_nodes, const int32_t* __restrict__ start, int B,
    int max_nodes, const int32_t* __restrict__ table, int64_t max_blk, int64_t n_blocks, int64_t T,
    int32_t* __restrict__ row0, int32_t* __restrict__ row_seq, int32_t* __restrict__ row_pos,
    int64_t* __restrict__ slots, int* status) {
  __shared__ long long sums[kSlotWarps];
  __shared__ int16_t depth_of[kSlotWarps][kMaxTreeNodes];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b0 = blockIdx.x * kSlotWarps, b = b0 + warp;
  long long before = 0;
  for (int i = tid; i < b0; i += kSlotWarps * 32) before += max(n_nodes[i], 0);
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) sums[warp] = before;
  __syncthreads();
  long long first = 0;
  for (int w = 0; w < kSlotWarps; ++w) first += sums[w];
  int mine = b0 + lane < B && lane < kSlotWarps ? max(n_nodes[b0 + lane], 0) : 0;
  long long own = lane < warp ? mine : 0;
  for (int o = 16; o; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  first += own;
  if (b >= B) return;
  const int n_in = n_nodes[b];
  const int n = max(n_in, 0);
  bool bad = n_in < 0 || n > max_nodes || first + n > T;
  if (lane == 0) {
    row0[b] = (int32_t)min(first, (long long)T);
    if (b == B - 1) row0[B] = (int32_t)min(first + n, (long long)T);
  }
  if (n > 0 && n <= max_nodes && first + n <= T) {
    bad |= tree_depths(parent + first, n, depth_of[warp], lane);
    const int64_t s = start[b];
    for (int i = lane; i < n; i += 32) {
      const int64_t row = first + i;
      const int d = depth_of[warp][i];
      const int64_t pos = d < 0 || s < 0 || s + d > 0x7fffffff ? -1 : s + d;
      const int64_t at = s + i;
      bad |= pos < 0;
      if (row_seq) row_seq[row] = b;
      if (row_pos) row_pos[row] = (int32_t)pos;
      if (slots) {
        int64_t slot = -1;
        if (s >= 0 && at / kPage < max_blk) {
          const int32_t id = table[(int64_t)b * max_blk + at / kPage];
          if (id >= 0 && id < n_blocks) slot = (int64_t)id * kPage + at % kPage;
        }
        bad |= slot < 0;
        slots[row] = slot;
      }
    }
  } else {
    // a refused sequence's rows: nothing may be written where an earlier step's rows of these buffers stood
    for (int64_t row = first + lane; row < min(first + n, (long long)T); row += 32) {
      if (row_pos) row_pos[row] = -1;
      if (slots) slots[row] = -1;
    }
  }
  if (bad) report(status, DEV_BAD_INDEX);
}

// ------------------------------------------------------------------------ acceptance
struct AcceptArgs {
  const int32_t *parent, *row0, *start, *tokens, *targets, *limit;
  int64_t T;
  int B, max_nodes, max_path;
  int32_t *n_out, *path, *tokens_out, *pos_out;
  // the caches [n_layers, n_blocks, Hkv, 64, hd], in 16-byte vectors
  uint4 *k, *v;
  const int32_t* table;
  int64_t max_blk, n_blocks, layer_vecs;
  int n_layers, Hkv, hv;
  int* status;
};

constexpr int kAcceptThreads = 256;

// CTA (x, b): every CTA of a sequence walks its tree (each child that carries the token chosen at its parent
// bids for it, the lowest index wins; then a chain of at most n shared-memory loads), the first one writes the
// result, and each moves its share of the accepted rows.  A thread moves one 16-byte vector of every row of the
// path, in path order, four rows read before they are written.  That order makes the move safe in place: row j goes
// to start + j, and a later row k > j comes from node path[k] >= k > j, so no row is written over before it is read.
// Bound by the chain of loads (row offsets; tree and block ids; rows): nothing else depends on the walk.
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const AcceptArgs a) {
  __shared__ int32_t next[kMaxTreeNodes], target[kMaxTreeNodes];
  __shared__ int32_t path[kMaxTreeNodes];
  __shared__ int64_t slot_of[kMaxTreeNodes];  // of cache position start + i, -1 without a block
  __shared__ int count;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, b = blockIdx.y;
  const bool first = blockIdx.x == 0;
  const int64_t r0 = a.row0[b], r1 = a.row0[b + 1];
  const int64_t start = a.start[b];
  const bool fine = r0 >= 0 && r1 >= r0 && r1 <= a.T && r1 - r0 <= a.max_nodes && start >= 0 &&
                    start + (r1 - r0) <= 0x7fffffff;  // (start + m is a 32-bit position)
  const int n = fine ? (int)(r1 - r0) : 0;
  bool bad = !fine;
  int par = -1, tok = 0;
  if (tid < n) {
    par = a.parent[r0 + tid];
    tok = a.tokens[r0 + tid];
    target[tid] = a.targets[r0 + tid];
    next[tid] = n;
    if (a.k) {
      const int64_t at = start + tid;
      const int32_t id = at / kPage < a.max_blk ? a.table[(int64_t)b * a.max_blk + at / kPage] : -1;
      slot_of[tid] = id >= 0 && id < a.n_blocks ? (int64_t)id * kPage + at % kPage : -1;
    }
  }
  if (tid == 0) count = 0;
  __syncthreads();
  const bool valid = tid < n && par >= -1 && par < tid;
  bad |= tid < n && !valid;
  if (valid && par >= 0 && tok == target[par]) atomicMin(&next[par], tid);
  bad |= tid == 0 && n > 0 && par != -1;
  __syncthreads();
  if (tid == 0 && n > 0 && par == -1) {
    const int most = min(min(n, a.max_path), a.limit ? a.limit[b] : n);
    int m = 0;
    for (int cur = 0; cur < n && m < most; cur = next[cur]) path[m++] = cur;
    count = m;
  }
  __syncthreads();
  const int m = count;
  if (first) {
    for (int j = tid; j < a.max_path; j += kAcceptThreads) {
      a.path[(int64_t)b * a.max_path + j] = j < m ? path[j] : -1;
      a.tokens_out[(int64_t)b * a.max_path + j] = j < m ? target[path[j]] : -1;
    }
    if (tid == 0) {
      a.n_out[b] = m;
      a.pos_out[b] = (int32_t)(start + m);
    }
  }
  if (a.k && m > 1) {
    if (tid < m && path[tid] != tid) bad |= slot_of[path[tid]] < 0 || slot_of[tid] < 0;
    const int items = 2 * a.n_layers * a.Hkv * a.hv;
    for (int i = blockIdx.x * kAcceptThreads + tid; i < items; i += gridDim.x * kAcceptThreads) {
      const int vec = i % a.hv;
      const int head = i / a.hv % a.Hkv;
      const int lay = i / (a.hv * a.Hkv);
      uint4* cache = (lay >= a.n_layers ? a.v + (lay - a.n_layers) * a.layer_vecs : a.k + lay * a.layer_vecs) + vec;
      auto at = [&](int64_t slot) { return cache + (((slot >> 6) * a.Hkv + head) * kPage + (slot & 63)) * a.hv; };
      for (int j0 = 1; j0 < m; j0 += 4) {
        uint4 x[4];
        int64_t to[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + e;
          to[e] = -1;
          if (j < m && path[j] != j && slot_of[path[j]] >= 0 && slot_of[j] >= 0) {
            to[e] = slot_of[j];
            x[e] = *at(slot_of[path[j]]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (to[e] >= 0) *at(to[e]) = x[e];
      }
    }
  }
  if (bad && first) report(a.status, DEV_BAD_INDEX);
}

}  // namespace bi

extern "C" {

bi_status bi_tree_slot_map(const int32_t* parent, const int32_t* n_nodes, const int32_t* start, int64_t B,
                           int64_t max_nodes, const int32_t* block_table, int64_t max_blocks_per_seq, int64_t n_blocks,
                           int64_t T, int32_t* row0, int32_t* row_seq, int32_t* row_pos, int64_t* slots, void* stream) {
  using namespace bi;
  BI_REQUIRE(B >= 0 && T >= 0, "B < 0 or T < 0");
  if (B == 0) return BI_OK;
  BI_REQUIRE(n_nodes && start && row0 && (parent || T == 0), "null pointer");
  BI_REQUIRE(!slots || block_table, "slots need a block table");
  BI_REQUIRE(max_nodes >= 1, "max_nodes must be positive");
  BI_REQUIRE_SHAPE(max_nodes <= kMaxTreeNodes, "max_nodes must be at most 256");
  BI_REQUIRE(max_blocks_per_seq >= 1 && n_blocks >= 1, "max_blocks_per_seq and n_blocks must be positive");
  BI_REQUIRE(B <= 1 << 20 && n_blocks <= 0x7fffffff && T <= 0x7fffffff, "too many sequences, blocks or rows");
  return launched(launch_pdl(tree_slot_map_kernel, dim3((unsigned)cdiv(B, kSlotWarps)), dim3(kSlotWarps * 32), 0,
                             as_stream(stream), parent, n_nodes, start, (int)B, (int)max_nodes, block_table,
                             max_blocks_per_seq, n_blocks, T, row0, row_seq, row_pos, slots, device_status_ptr()),
                  "bi_tree_slot_map");
}

bi_status bi_tree_accept(const int32_t* parent, const int32_t* row0, const int32_t* start, const int32_t* tokens,
                         const int32_t* targets, const int32_t* limit, int64_t B, int64_t max_nodes, int64_t T,
                         int64_t max_path, int32_t* n_out, int32_t* path, int32_t* tokens_out, int32_t* pos_out,
                         int64_t n_layers, int Hkv, int hd, void* k_cache, void* v_cache, const int32_t* block_table,
                         int64_t max_blocks_per_seq, int64_t n_blocks, void* stream) {
  using namespace bi;
  BI_REQUIRE(B >= 0 && T >= 0, "B < 0 or T < 0");
  if (B == 0) return BI_OK;
  BI_REQUIRE(row0 && start && n_out && path && tokens_out && pos_out, "null pointer");
  BI_REQUIRE(T == 0 || (parent && tokens && targets), "null pointer");
  BI_REQUIRE(max_nodes >= 1 && max_path >= 1, "max_nodes and max_path must be positive");
  BI_REQUIRE_SHAPE(max_nodes <= kMaxTreeNodes, "max_nodes must be at most 256");
  BI_REQUIRE(B <= 65535 && max_path <= 0x7fffffff / B, "too many sequences or too long a path");
  BI_REQUIRE(!k_cache == !v_cache, "k_cache and v_cache go together");
  BI_REQUIRE(pos_out + B <= start || start + B <= pos_out, "pos_out must lie apart from start");
  AcceptArgs a{parent, row0, start, tokens, targets, limit, T, (int)B, (int)max_nodes, (int)max_path, n_out, path,
               tokens_out, pos_out, nullptr, nullptr, nullptr, 0, 0, 0, 0, 0, 0, device_status_ptr()};
  int64_t ctas = 1;
  if (k_cache) {
    BI_REQUIRE(n_layers >= 1 && Hkv >= 1 && hd >= 1 && max_blocks_per_seq >= 1 && n_blocks >= 1, "bad cache shape");
    BI_REQUIRE(block_table, "the caches need a block table");
    BI_REQUIRE_SHAPE(hd % 8 == 0, "head_dim must be a multiple of 8");
    BI_REQUIRE(aligned16(k_cache) && aligned16(v_cache), "cache pointers must be 16-byte aligned");
    BI_REQUIRE_SHAPE(n_blocks <= 0x7fffffff && Hkv <= 4096 && hd <= 1024 && n_layers <= 4096 &&
                         2 * n_layers * Hkv * (hd / 8) <= 0x7fffffff / 2,
                     "cache too large");
    a.k = static_cast<uint4*>(k_cache);
    a.v = static_cast<uint4*>(v_cache);
    a.table = block_table;
    a.max_blk = max_blocks_per_seq;
    a.n_blocks = n_blocks;
    a.n_layers = (int)n_layers;
    a.Hkv = Hkv;
    a.hv = hd / 8;
    a.layer_vecs = n_blocks * Hkv * kPage * a.hv;
    ctas = std::min<int64_t>(cdiv(2 * n_layers * Hkv * a.hv, kAcceptThreads), 64);
  }
  return launched(launch_pdl(tree_accept_kernel, dim3((unsigned)ctas, (unsigned)B), dim3(kAcceptThreads), 0,
                             as_stream(stream), a),
                  "bi_tree_accept");
}

}  // extern "C"
