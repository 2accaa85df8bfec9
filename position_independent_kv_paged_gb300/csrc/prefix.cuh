// Shared prefixes: which blocks a group of requests shares, and how the attention to them is cut into items.  The
// kernel that computes the shared part and the one that computes the rest decide alike what is shared.
#pragma once

#include "internal.h"

namespace minipic {
namespace prefix {

// Groups of fewer requests read their keys one by one (sharing saves nothing then).
constexpr int kMinRequests = 2;
// Blocks of a key tile of the kernel that computes the shared part.
template <int D>
constexpr int kTileBlocks = D == 128 ? 10 : 6;
// Rows of an item: two query tiles of 128 / G requests x the G heads of a kv head, each in 128 rows.
constexpr int kRows = 256;
// Parts of a prefix, at most (the merge of the other kernel holds a weight for each).
constexpr int kMaxParts = 64;
// What an item costs besides its tiles (start, query, end), in tiles.
constexpr int kItemCost = 3;

// Only groups in front of the first one whose boundaries descend count (that one is flagged): their boundaries ascend, so
// that no two groups that share hold one request, and there are no more items than the host planned for.
struct Group {
  int q0, n;   // requests q0 .. q0 + n - 1 of the batch (n -1: the boundaries descend)
  int blocks;  // that they share (0: nothing)
};

// A group as the tables and the planning bounds allow it (most_blocks: the lower bound of a prefix); `bad`: its numbers
// are outside them or the batch, and it shares nothing.
__device__ __forceinline__ Group group(int c0, int c1, int nb, int batch, int most_blocks, int max_requests, bool& bad) {
  bad = c0 < 0 || c1 < c0 || c1 > batch || (long long)c1 - c0 > max_requests || nb < 0 || nb > most_blocks;
  Group g;
  g.q0 = c0;
  g.n = c1 < c0 ? -1 : (bad ? 0 : c1 - c0);
  g.blocks = g.n >= kMinRequests ? nb : 0;
  return g;
}
__device__ __forceinline__ Group group(const PrefillArgs& a, int p) {
  bool bad;
  return group(__ldg(a.cu_q_lens + p), __ldg(a.cu_q_lens + p + 1), __ldg(a.prefix_blocks + p), a.total_q, a.max_prefix,
               a.max_q_len, bad);
}

// One item: the rows of a pair of query tiles of a group and kv head, and part `part` of `parts` of the prefix.  Items
// are numbered group by group, then pair, head, part; `first` is the group's first.
struct Item {
  int p, pair, head, part, parts;
  int first, index;  // places of the grid
  Group g;
};

// Item c of the batch (the whole warp calls; false: there are fewer).  What it leaves in registers counts: with a form that
// made the attention's inner loop spill 12 bytes, 256 requests behind 32768 tokens took 342 us, without 309 (a search for
// shorter items, and one by a single warp, were dropped for that; neither gained elsewhere).  The prefixes are cut so that the items of about
// equal length fill `slots` places in as many waves as cost least.
template <int D>
__device__ bool find_item(const PrefillArgs& a, int tq, long long c, Item& it) {
  constexpr unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto tiles = [](int blocks) { return (blocks + kTileBlocks<D> - 1) / kTileBlocks<D>; };
  auto units = [&](const Group& g) { return g.blocks ? (long long)((g.n + 2 * tq - 1) / (2 * tq)) * a.Hkv : 0LL; };
  long long n_units = 0, work = 0;
  int longest = 1;
  int n_groups = a.batch;  // that count
  for (int base = 0; base < n_groups; base += 32) {
    Group g{0, 0, 0};
    if (base + lane < n_groups) g = group(a, base + lane);
    const unsigned down = __ballot_sync(FULL, g.n < 0);
    if (down) n_groups = base + __ffs(down) - 1;
    if (g.blocks && base + lane < n_groups) {
      n_units += units(g);
      work += units(g) * tiles(g.blocks);
      longest = max(longest, tiles(g.blocks));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n_units += __shfl_xor_sync(FULL, n_units, o);
    work += __shfl_xor_sync(FULL, work, o);
  }
  longest = __reduce_max_sync(FULL, longest);
  int len = longest;  // tiles of an item, at most
  auto plan = [&](auto n_units, auto work) {
    using I = decltype(work);
    I least = (n_units + a.n_slots - 1) / a.n_slots * (longest + kItemCost);
    for (int w = 1; w <= a.max_waves; ++w) {
      if ((I)w * a.n_slots <= n_units) continue;
      const I room = (I)w * a.n_slots - n_units;  // sum of ceil(tiles / len) <= work / len + units
      const int l = max((int)min((I)longest, (work + room - 1) / room), (longest + kMaxParts - 1) / kMaxParts);
      if ((I)w * (l + kItemCost) < least) {
        least = (I)w * (l + kItemCost);
        len = l;
      }
    }
  };
  if (work < 1 << 24 && n_units < 1 << 12) plan((unsigned)n_units, (unsigned)work);  // 64-bit division is slow
  else plan((unsigned long long)n_units, (unsigned long long)work);
  long long before = 0;
  for (int base = 0; base < n_groups; base += 32) {
    Group g{0, 0, 0};
    if (base + lane < n_groups) g = group(a, base + lane);
    const int parts = g.blocks ? (tiles(g.blocks) + len - 1) / len : 0;
    long long sum = units(g) * parts;  // ... of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(FULL, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned has = __ballot_sync(FULL, c < before + sum);
    if (has) {
      const int l = __ffs(has) - 1;
      it.p = base + l;
      it.parts = __shfl_sync(FULL, parts, l);
      it.first = (int)(before + __shfl_sync(FULL, sum - units(g) * parts, l));
      it.index = (int)c;
      it.g.q0 = __shfl_sync(FULL, g.q0, l);
      it.g.n = __shfl_sync(FULL, g.n, l);
      it.g.blocks = __shfl_sync(FULL, g.blocks, l);
      const unsigned k = (unsigned)(it.index - it.first);
      it.part = (int)(k % it.parts);
      it.head = (int)(k / it.parts % a.Hkv);
      it.pair = (int)(k / it.parts / a.Hkv);
      return true;
    }
    before += __shfl_sync(FULL, sum, 31);
  }
  return false;
}

// What an item computes: rows of requests q0 .. q0 + n - 1, key tiles t_first .. t_end - 1 of the first `keys` keys, by the
// tables of request `row`, the first of the group that holds the whole prefix (-1: none does).  Every warp calls.
struct Work {
  int q0, n, keys, t_first, t_end, row;
};
template <int D>
__device__ __forceinline__ Work work_of(const PrefillArgs& a, const Item& it) {
  const int lane = threadIdx.x & 31;
  const int tiles = (it.g.blocks + kTileBlocks<D> - 1) / kTileBlocks<D>;  // at least as many as parts
  Work w{it.g.q0, it.g.n, 16 * it.g.blocks, (int)((long long)it.part * tiles / it.parts),
         (int)((long long)(it.part + 1) * tiles / it.parts), -1};
  for (int i = 0; i < w.n && w.row < 0; i += 32) {
    const unsigned has = __ballot_sync(
        0xffffffffu, i + lane < w.n && __ldg(a.kv_lens + w.q0 + min(i + lane, w.n - 1)) >= w.keys);
    if (has) w.row = w.q0 + i + __ffs(has) - 1;
  }
  return w;
}

// The first item and the parts of request i's group p, which begins at request q0 (as the kernel that computed them
// wrote it: each of its items has a CTA, see Group).
__device__ __forceinline__ int2 items_of(const DecodeArgs& a, int p, int q0, int i) {
  const int2 gi = __ldcg(a.group_items + p);
  const long long pair = (i - q0) / (2 * (128 / a.G));
  const bool ok = gi.x >= 0 && gi.y > 0 && gi.y <= kMaxParts && gi.x + (pair + 1) * a.Hkv * gi.y <= a.items;
  return ok ? gi : make_int2(0, 0);
}
// Row of part 0 of the attention of request i, head `head` of kv head hk, to its prefix; the next part is kRows on, the
// next head 1.
__device__ __forceinline__ size_t row_of(const DecodeArgs& a, int2 gi, int q0, int i, int hk, int head) {
  const int tq = 128 / a.G, t = i - q0, pair = t / (2 * tq), tile = (t - pair * 2 * tq) / tq;
  const long long item = gi.x + ((long long)pair * a.Hkv + hk) * gi.y;
  return (size_t)item * kRows + 128 * tile + (t - (2 * pair + tile) * tq) * a.G + head;
}

}  // namespace prefix
}  // namespace minipic
