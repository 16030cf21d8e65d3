// Depths of the nodes of a drafted tree.
#pragma once
#include "common.cuh"

namespace bi {

constexpr int kMaxTreeNodes = 256;
constexpr int kBadDepth = -(1 << 20);  // an invalid node's depth; those below one stay negative

// Depth of nodes 0 .. n - 1 (n <= kMaxTreeNodes) into depth[], by one warp: a root (parent -1) has depth 0, a node
// whose parent does not stand before it (and its descendants) a negative one.  32 nodes at a time, those of a
// group by pointer doubling (five rounds whatever the shape), since every parent stands before its child.
// Returns true on every lane when some node is invalid.  copy: the parents, if not null (shared memory).
BI_DEV bool tree_depths(const int32_t* __restrict__ parent, int n, int16_t* depth, int lane, int16_t* copy = nullptr) {
  bool bad = false;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    const int p = i < n ? parent[i] : -1;
    int ptr = -1, d = 0;
    if (p < -1 || p >= i) {
      bad |= i < n;
      d = kBadDepth;
    } else if (p >= base) {
      ptr = p - base;
      d = 1;
    } else if (p >= 0) {
      d = depth[p] < 0 ? kBadDepth : depth[p] + 1;
    }
#pragma unroll
    for (int r = 0; r < 5; ++r) {
      const int dp = __shfl_sync(0xffffffffu, d, ptr & 31);
      const int pp = __shfl_sync(0xffffffffu, ptr, ptr & 31);
      if (ptr >= 0) {
        d = max(d + dp, kBadDepth);
        ptr = pp;
      }
    }
    if (i < n) {
      depth[i] = (int16_t)max(d, -1);
      if (copy) copy[i] = (int16_t)p;
    }
    __syncwarp();
  }
  return __any_sync(0xffffffffu, bad);
}

}  // namespace bi
