// Shared prefixes: which blocks a group of requests shares, and how its keys are cut into parts.  The kernel that
// computes the shared part and the one that computes the rest decide alike.
#pragma once

#include "internal.h"

namespace minipic {
namespace prefix {

// Groups of fewer requests read their keys one by one (sharing saves nothing then).
constexpr int kMinRequests = 2;

struct Group {
  int q0, n;   // requests q0 .. q0 + n - 1 of the batch
  int blocks;  // that they share (0: nothing)
};

// Group p as the tables allow it; `bad`: its numbers are outside the batch, the tables or the planning bound.
__device__ __forceinline__ Group group(const int32_t* cu, const int32_t* blocks, int p, int batch, int max_blocks,
                                       int max_requests, bool& bad) {
  const int c0 = __ldg(cu + p), c1 = __ldg(cu + p + 1), nb = __ldg(blocks + p);
  bad = c0 < 0 || c1 < c0 || c1 > batch || (long long)c1 - c0 > max_requests || nb < 0 || nb > max_blocks;
  Group g;
  g.q0 = max(0, min(c0, batch));
  g.n = max(0, min(c1, batch) - g.q0);
  g.blocks = g.n >= kMinRequests && g.n <= max_requests && nb > 0 && nb <= max_blocks ? nb : 0;
  return g;
}

// Blocks of a key tile of the kernel that computes the shared part.
template <int D>
constexpr int kTileBlocks = D == 128 ? 10 : 6;
// Parts of a prefix, at most.
constexpr int kMaxSplit = 64;

// Key tiles of a prefix, and the parts it is cut into: n_split, or one a tile.
template <int D>
__device__ __forceinline__ int tiles(int blocks) {
  return (blocks + kTileBlocks<D> - 1) / kTileBlocks<D>;
}
template <int D>
__device__ __forceinline__ int parts(int blocks, int n_split) {
  return min(n_split, tiles<D>(blocks));
}

}  // namespace prefix
}  // namespace minipic
