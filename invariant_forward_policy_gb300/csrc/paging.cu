// Planning of a paged KV cache on the GPU: block tables resized to the requests' lengths, and the
// map from a step's packed rows to sequences, positions and cache slots.
//
// "vLLM Achieves Bitwise-Consistent RL Training ..." §4.2 (prefill, decode and training share one
// KV write and read path through block tables) and §4.6 (a captured step reads nothing back to the
// host): a step whose requests grow, come and go keeps its tables on the device, so the plan has to
// be made there too, and be the same for the same lengths whatever the launch looks like.
//
// Both kernels are a prefix sum over the requests followed by scattered 4- or 8-byte moves, a few
// kilobytes of each in a decode step: what bounds them is the chain of dependent loads (lengths,
// then block ids, then the stores), so each is one launch, with every CTA summing the lengths
// before its own part itself instead of waiting for another kernel's sums.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace bi {

constexpr int kPageTokens = 64;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Inclusive sum of one value per thread over the CTA (thread 0 first); *total: the CTA's sum.
template <int NT>
__device__ __forceinline__ long long plan_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // warp_sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return v + before;
}

// Blocks a request lacks (low half) and has too many of (high half), each below 2^31 over all requests.
struct Demand {
  int owned, more, less;
  bool bad;
  __device__ __forceinline__ long long packed() const { return (long long)less << 32 | (unsigned)more; }
};
__device__ __forceinline__ Demand demand_of(int32_t len, int64_t extra, int32_t owned, int64_t max_blk) {
  Demand d{owned, 0, 0, false};
  const int64_t tokens = len > 0 ? max((int64_t)0, (int64_t)len + extra) : 0;
  const int64_t need = (tokens + kPageTokens - 1) / kPageTokens;
  d.bad = owned < 0 || owned > max_blk || need > max_blk;
  if (!d.bad) {
    d.more = need > owned ? (int)(need - owned) : 0;
    d.less = need < owned ? (int)(owned - need) : 0;
  }
  return d;
}

// One cluster of CS CTAs; rank r owns requests [r per, (r + 1) per).  Every CTA first sums the demands of
// all requests; after the cluster barrier (every input has been read, so the outputs may be the inputs)
// it walks its own requests in tiles of one per thread, and its warps then move the tile's block ids.
template <int CS>
__global__ void __launch_bounds__(kPlanThreads) block_table_resize_kernel(
    const int32_t* lens, int64_t extra, int B, int per, int32_t* __restrict__ table, int64_t max_blk,
    const int32_t* n_owned, int32_t* __restrict__ ring, int64_t n_blocks, const int32_t* pool, int32_t* n_owned_out,
    int32_t* pool_out, int* status) {
  __shared__ long long warp_sums[kPlanWarps];
  __shared__ int4 plan[kPlanThreads];  // first table entry, signed count, ring offset
  __shared__ int served;               // blocks handed out (rank 0's: by the whole cluster)
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x;
  const int rank = CS == 1 ? 0 : (int)cl.block_rank();
  const int first = min(B, rank * per), last = min(B, first + per);
  const int head = pool[0], count = pool[1];
  if (tid == 0) served = 0;
  if (head < 0 || head >= n_blocks || count < 0 || count > n_blocks) {  // not a ring: nothing is changed
    for (int b = first + tid; b < last; b += kPlanThreads) n_owned_out[b] = n_owned[b];
    if (rank == 0 && tid == 0) {
      pool_out[0] = head;
      pool_out[1] = count;
      report(status, DEV_BAD_INDEX);
    }
    return;
  }
  long long before = 0, all = 0;
  if (CS > 1) {
    for (int b = tid; b < B; b += kPlanThreads) {
      const long long v = demand_of(lens[b], extra, n_owned[b], max_blk).packed();
      all += v;
      if (b < first) before += v;
    }
    long long t;
    plan_scan<kPlanThreads>(before, warp_sums, &t);
    before = t;
    plan_scan<kPlanThreads>(all, warp_sums, &t);
    all = t;
    cl.sync();
  }
  long long run = before;
  int mine = 0;
  bool bad = false;
  const uint32_t blocks = (uint32_t)n_blocks;
  for (int b0 = first; b0 < last; b0 += kPlanThreads) {
    const int b = b0 + tid;
    Demand d{0, 0, 0, false};
    int owned = 0;
    if (b < last) {
      owned = n_owned[b];
      d = demand_of(lens[b], extra, owned, max_blk);
    }
    long long tile;
    const long long upto = run + plan_scan<kPlanThreads>(d.packed(), warp_sums, &tile);
    run += tile;
    const long long asked = upto & 0xffffffffll, freed = upto >> 32;
    const bool serve = d.more > 0 && asked <= count;
    bad |= d.bad || (d.more > 0 && !serve);
    int4 pl = make_int4(0, 0, 0, 0);
    if (serve) pl = make_int4(owned, d.more, (int)(asked - d.more), 0);
    if (d.less > 0) pl = make_int4(owned - d.less, -d.less, (int)(freed - d.less), 0);
    plan[tid] = pl;
    if (b < last) n_owned_out[b] = owned + pl.y;
    mine += serve ? d.more : 0;
    __syncthreads();
    // a warp per request when a tile's requests move many blocks each, else eight lanes: a request's moves wait for
    // its plan and its ids, so more of them at once is what counts
    // (4096 requests of 11 new blocks each: 12.0 -> 10.6 us)
    const int requests = min(kPlanThreads, last - b0);
    const int g = (tile & 0xffffffffll) + (tile >> 32) > 16ll * requests ? 32 : 8;
    for (int q = tid / g; q < requests; q += kPlanThreads / g) {
      const int4 e = plan[q];
      const int lane = tid % g;
      int32_t* row = table + (int64_t)(b0 + q) * max_blk + e.x;
      for (int i = lane; i < e.y; i += g) {  // from the ring's head on
        int64_t at = (int64_t)head + e.z + i;
        if (at >= n_blocks) at -= n_blocks;
        const int32_t id = ring[at];
        bad |= (uint32_t)id >= blocks;
        row[i] = id;
      }
      for (int i = lane; i < -e.y; i += g) {  // to its tail: never among the free ids, which are being read
        int64_t at = (int64_t)head + count + e.z + i;
        at %= n_blocks;
        const int32_t id = row[i];
        const bool fits = (int64_t)count + e.z + i < n_blocks;
        if (fits) ring[at] = id;
        bad |= !fits || (uint32_t)id >= blocks;
        row[i] = -1;
      }
    }
    __syncthreads();
  }
  if (bad) report(status, DEV_BAD_INDEX);
  if (CS == 1) all = run;
  long long handed;
  plan_scan<kPlanThreads>(mine, warp_sums, &handed);
  if (CS > 1) {
    if (tid == 0) atomicAdd(cl.map_shared_rank(&served, 0), (int)handed);
    cl.sync();
    handed = served;
  }
  if (rank == 0 && tid == 0) {
    const int64_t h = (int64_t)head + handed;
    pool_out[0] = (int)(h >= n_blocks ? h - n_blocks : h);
    // what was given back beyond the ring's places is not in it
    pool_out[1] = (int)(count - handed + min((long long)n_blocks - count, all >> 32));
  }
}

// Each CTA maps kMapRows rows: it sums the row counts of all requests up to its last row, marks in shared
// memory where a request's rows begin, and a running maximum over the marks gives each row its request.
constexpr int kMapThreads = 512;
constexpr int kMapRows = 2048;
constexpr int kMapPer = kMapRows / kMapThreads;

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const int32_t* __restrict__ new_tokens,
                                                               const int32_t* __restrict__ start, int B,
                                                               const int32_t* __restrict__ table, int64_t max_blk,
                                                               int64_t n_blocks, int64_t T, int32_t* __restrict__ row0,
                                                               int32_t* __restrict__ row_seq,
                                                               int32_t* __restrict__ row_pos,
                                                               int64_t* __restrict__ slots, int* status) {
  __shared__ long long warp_sums[kMapThreads / 32];
  __shared__ int32_t seq_of[kMapRows];    // 1 + the request whose rows begin here (in this CTA), else 0
  __shared__ int32_t first_of[kMapRows];  // that request's first row
  __shared__ int32_t mark_of[kMapRows];   // the last mark at or before each row
  __shared__ int32_t warp_max[kMapThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * kMapRows, r1 = min(T, r0 + kMapRows);
  for (int i = tid; i < kMapRows; i += kMapThreads) seq_of[i] = 0;
  __syncthreads();
  long long run = 0;
  for (int b0 = 0; b0 < B; b0 += kMapThreads) {
    if (blockIdx.x > 0 && run >= r1) break;  // CTA 0 writes every request's first row
    const int b = b0 + tid;
    long long n = b < B ? new_tokens[b] : 0;
    if (n < 0) {
      if (blockIdx.x == 0) report(status, DEV_BAD_INDEX);
      n = 0;
    }
    long long tile;
    const long long end = run + plan_scan<kMapThreads>(n, warp_sums, &tile), begin = end - n;
    run += tile;
    if (blockIdx.x == 0 && b < B) row0[b] = (int32_t)min((long long)T, begin);
    if (n > 0 && begin < r1 && end > r0) {
      const int i = (int)(max(begin, (long long)r0) - r0);
      seq_of[i] = b + 1;
      first_of[i] = (int32_t)begin;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    row0[B] = (int32_t)min((long long)T, run);
    if (run > T) report(status, DEV_BAD_INDEX);
  }
  const int64_t stop = min((int64_t)run, r1);  // rows behind the last sequence stay as they were
  if (stop <= r0) return;
  __syncthreads();
  int top[kMapPer], best = -1;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    if (seq_of[tid * kMapPer + i]) best = tid * kMapPer + i;
    top[i] = best;
  }
  int inc = best;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = max(inc, y);
  }
  if (lane == 31) warp_max[warp] = inc;
  __syncthreads();
  int prev = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) prev = -1;
  for (int w = 0; w < warp; ++w) prev = max(prev, warp_max[w]);
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) mark_of[tid * kMapPer + i] = max(prev, top[i]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int j = i * kMapThreads + tid;
    const int64_t row = r0 + j;
    if (row >= stop) break;
    const int mk = mark_of[j];
    const int b = seq_of[mk] - 1;
    const int64_t pos = (int64_t)start[b] + (row - first_of[mk]);
    if (pos < 0 || pos > 0x7fffffff) report(status, DEV_BAD_INDEX);
    if (row_seq) row_seq[row] = b;
    if (row_pos) row_pos[row] = (int32_t)pos;
    if (slots) {
      int64_t slot = -1;
      if (pos >= 0 && pos / kPageTokens < max_blk) {
        const int32_t id = table[(int64_t)b * max_blk + pos / kPageTokens];
        if (id >= 0 && id < n_blocks) slot = (int64_t)id * kPageTokens + pos % kPageTokens;
      }
      if (slot < 0) report(status, DEV_BAD_INDEX);
      slots[row] = slot;
    }
  }
}

template <int CS>
static cudaError_t launch_resize(const int32_t* lens, int64_t extra, int B, int32_t* table, int64_t max_blk,
                                 const int32_t* n_owned, int32_t* ring, int64_t n_blocks, const int32_t* pool,
                                 int32_t* n_owned_out, int32_t* pool_out, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS);
  cfg.blockDim = dim3(kPlanThreads);
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
  return cudaLaunchKernelEx(&cfg, block_table_resize_kernel<CS>, lens, extra, B, (int)cdiv(B, CS), table, max_blk,
                            n_owned, ring, n_blocks, pool, n_owned_out, pool_out, device_status_ptr());
}

}  // namespace bi

extern "C" {

bi_status bi_block_table_resize(const int32_t* lens, int64_t extra, int64_t B, int32_t* block_table,
                                int64_t max_blocks_per_seq, const int32_t* n_owned, int32_t* ring, int64_t n_blocks,
                                const int32_t* pool, int32_t* n_owned_out, int32_t* pool_out, void* stream) {
  using namespace bi;
  BI_REQUIRE(B >= 0, "B < 0");
  if (B == 0) return BI_OK;
  BI_REQUIRE(lens && block_table && n_owned && ring && pool && n_owned_out && pool_out, "null pointer");
  BI_REQUIRE(max_blocks_per_seq >= 1 && n_blocks >= 1, "max_blocks_per_seq and n_blocks must be positive");
  BI_REQUIRE(extra >= 0 && extra <= 0x7fffffff, "extra must be in [0, 2^31)");
  BI_REQUIRE(B <= 1 << 30 && n_blocks <= 0x7fffffff && max_blocks_per_seq <= 0x7fffffff / B,
             "block table or pool too large");
  BI_REQUIRE(n_owned_out == n_owned || n_owned_out + B <= n_owned || n_owned + B <= n_owned_out,
             "n_owned_out must be n_owned or lie apart from it");
  // One CTA up to 256 requests (64 decode rows: 3.8 us against 6.1 us for a cluster of 8; 256 requests growing by 11
  // blocks each: 5.4 against 6.3), the cluster beyond (1024: 13.0 against 7.2 us).
  const cudaError_t e =
      B > 256
          ? launch_resize<8>(lens, extra, (int)B, block_table, max_blocks_per_seq, n_owned, ring, n_blocks, pool,
                             n_owned_out, pool_out, as_stream(stream))
          : launch_resize<1>(lens, extra, (int)B, block_table, max_blocks_per_seq, n_owned, ring, n_blocks, pool,
                             n_owned_out, pool_out, as_stream(stream));
  return launched(e, "bi_block_table_resize");
}

bi_status bi_slot_map(const int32_t* new_tokens, const int32_t* start, int64_t B, const int32_t* block_table,
                      int64_t max_blocks_per_seq, int64_t n_blocks, int64_t T, int32_t* row0, int32_t* row_seq,
                      int32_t* row_pos, int64_t* slots, void* stream) {
  using namespace bi;
  BI_REQUIRE(B >= 0 && T >= 0, "B < 0 or T < 0");
  if (B == 0) return BI_OK;
  BI_REQUIRE(new_tokens && start && row0, "null pointer");
  BI_REQUIRE(!slots || block_table, "slots need a block table");
  BI_REQUIRE(max_blocks_per_seq >= 1 && n_blocks >= 1, "max_blocks_per_seq and n_blocks must be positive");
  BI_REQUIRE(B <= 1 << 30 && n_blocks <= 0x7fffffff, "too many requests or blocks");
  BI_REQUIRE(T <= 0x7fffffff, "T too large");
  const dim3 grid((unsigned)std::max<int64_t>(1, cdiv(T, kMapRows)));
  return launched(launch_pdl(slot_map_kernel, grid, dim3(kMapThreads), 0, as_stream(stream), new_tokens, start, (int)B,
                             block_table, max_blocks_per_seq, n_blocks, T, row0, row_seq, row_pos, slots,
                             device_status_ptr()),
                  "bi_slot_map");
}

}  // extern "C"
