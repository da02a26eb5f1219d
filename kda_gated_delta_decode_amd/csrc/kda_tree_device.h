// kda_tree_device.h -- device helpers that read a tree of drafted tokens.  Internal
// header.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_tree.h"

namespace kda {

// A request's nodes as a launch sees them.
struct Nodes {
  int64_t n0;  // its first node's row
  int n;       // its nodes; 0: nothing is done for it
};

__device__ __forceinline__ Nodes nodes_of(const int32_t* cu, int r, int64_t n_tokens) {
  const int64_t n0 = cu[r], n1 = cu[r + 1];
  const bool none = n0 < 0 || n1 <= n0 || n1 > n_tokens;
  return {n0, none ? 0 : n1 - n0 > INT32_MAX ? INT32_MAX : static_cast<int>(n1 - n0)};
}

// Lane i of a wave holds node i's parent (-1: the context).  Returns the nodes on
// its path, itself among them, as bits; *bad says that a node's parent does not
// lie before it.  Every round doubles how far up a node sees.
__device__ __forceinline__ uint64_t tree_paths(int parent, int n, bool* bad) {
  const int lane = threadIdx.x % 64;
  const bool mine = lane < n, ok = parent >= -1 && parent < lane;
  *bad = __ballot(mine && !ok) != 0;
  int up = mine && ok ? parent : -1;
  uint64_t seen = 1ull << lane;
  while (__ballot(up >= 0) != 0) {
    const int from = 4 * (up < 0 ? lane : up);
    const uint32_t lo = __builtin_amdgcn_ds_bpermute(from, static_cast<int>(seen));
    const uint32_t hi = __builtin_amdgcn_ds_bpermute(from, static_cast<int>(seen >> 32));
    const int next = __builtin_amdgcn_ds_bpermute(from, up);
    if (up >= 0) {
      seen |= static_cast<uint64_t>(hi) << 32 | lo;
      up = next;
    }
  }
  return seen;
}

}  // namespace kda
