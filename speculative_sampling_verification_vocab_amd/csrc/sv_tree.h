// A tree of up to 64 drafted nodes on the device (gfx950, wave64): lane i holds
// node i.  A node's parent comes before it, -1 for a node that follows the
// cache directly; a node whose parent is outside [-1, i), or that has an absent
// ancestor, is absent.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_common.h"

namespace sv {

struct TreeNode {
  uint64_t line;  // the node and its ancestors, as bits; 0 for an absent node
  int depth;      // ancestors
};

// Node `lane` of a tree of n nodes with parent p (anything for lane >= n).
// Lines double in length with each step: six for the deepest tree of 64.
__device__ __forceinline__ TreeNode tree_node(int p, int lane, int n) {
  const bool fits = lane < n && p >= -1 && p < lane;
  uint64_t line = 1ull << lane;
  int bad = fits ? 0 : 1, up = fits ? p : -1;
  while (__any(up >= 0)) {
    const int from = up < 0 ? lane : up;
    const uint32_t lo = __shfl((uint32_t)line, from), hi = __shfl((uint32_t)(line >> 32), from);
    const int worse = __shfl(bad, from), next = __shfl(up, from);
    line |= ((uint64_t)hi << 32) | lo;
    bad |= worse;
    up = up < 0 ? -1 : next;
  }
  TreeNode t;
  t.line = bad ? 0 : line;
  t.depth = __popcll(line) - 1;
  return t;
}

}  // namespace sv
