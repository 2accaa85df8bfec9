// The best blocks of each (request, kv head) by score.
//
// With n blocks: all of them where n <= budget, else the first keep_first, the last keep_last and the best of the others
// by score up to `budget` (NaN is the worst; of equal scores the lower index stays: the rule of kv_evict).  Their numbers are
// written in ascending order, then -1.
//
// One CTA per (request, kv head).  Each thread keeps PER order-preserving integer images of its scores in
// registers, in warp-contiguous rows of 32, so loads are whole lines and ballots give the order.  The threshold, the
// image of the last candidate that stays, is built bit by bit from the top: the candidates at or above the trial
// image are counted, and the bit stays where enough are.  A pass is PER comparisons, one warp reduction and one
// barrier; it ends early when the count is met exactly, which scores of many bits do after about two thirds of them.  No
// histogram: scores lie in few exponents, whose atomics would queue.
#include <stdint.h>

#include "internal.h"

namespace minipic {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// Larger float <-> larger integer (at least 1); -0 counts as +0 and NaN as the lowest.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the CTA in every thread; `slots` holds two rows of NW, used in turn, so one barrier a call.
template <int NW>
__device__ __forceinline__ int cta_sum(int v, int (*slots)[32], int turn) {
  const int w = __reduce_add_sync(FULL, v), lane = threadIdx.x & 31;
  if (lane == 0) slots[turn & 1][threadIdx.x >> 5] = w;
  __syncthreads();
  return __reduce_add_sync(FULL, lane < NW ? slots[turn & 1][lane] : 0);
}

// PER = 0: any number of blocks, scores read again in each pass.
template <int T, int PER>
__global__ void __launch_bounds__(T) block_select_kernel(const SelectArgs a) {
  constexpr int NW = T / 32;
  __shared__ int slots[2][32];
  __shared__ int2 s_before[32];
  const size_t row = blockIdx.x;
  const int r = (int)(row / a.Hkv), mb = a.max_blocks, S = a.budget;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int L = a.seq_lens[r];
  if (L < 0 || (long long)L > 16LL * mb) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : (int)min(16LL * mb, 2147483632LL);
  }
  const int n = min((L >> 4) + ((L & 15) != 0), mb);
  int* out = a.selected + row * S;
  if (n <= S) {
    for (int i = threadIdx.x; i < S; i += T) out[i] = i < n ? i : -1;
    return;
  }
  const float* sc = a.scores + row * mb;
  const int per = PER ? PER : (n + T - 1) / T;       // rows of 32 of each warp
  const int base = warp * per * 32 + lane;
  auto held = [&](int b) { return b < a.keep_first || b >= n - a.keep_last; };
  // image of block base + 32 j: 0 for none, the largest for one that always stays
  auto image = [&](int j) {
    const int b = base + 32 * j;
    return b < n ? (held(b) ? 0xffffffffu : rank_key(__ldg(sc + b))) : 0u;
  };
  [[maybe_unused]] uint32_t key[PER ? PER : 1];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = image(j);
  auto at = [&](int j) { return PER ? key[PER ? j : 0] : image(j); };
  // the largest threshold that at least S images reach (n > S, and held blocks are at most S)
  uint32_t least = 0u;
  int reach = n, turn = 0;  // images >= least
#pragma unroll 1
  for (int bit = 31; bit >= 0 && reach != S; --bit) {
    const uint32_t trial = least | (1u << bit);
    int c = 0;
#pragma unroll
    for (int j = 0; j < (PER ? PER : per); ++j) c += at(j) >= trial;
    c = cta_sum<NW>(c, slots, turn++);
    if (c >= S) {
      least = trial;
      reach = c;
    }
  }
  // images above the threshold stay, of those at it the first S - (those above)
  int above = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < (PER ? PER : per); ++j) {
    const uint32_t k = at(j);
    above += __popc(__ballot_sync(FULL, k > least));
    equal += __popc(__ballot_sync(FULL, k == least));
  }
  if (lane == 0) s_before[warp] = make_int2(above, equal);
  __syncthreads();
  const int2 mine = lane < NW ? s_before[lane] : make_int2(0, 0);
  const int ties = S - __reduce_add_sync(FULL, mine.x);
  int up = __reduce_add_sync(FULL, lane < warp ? mine.x : 0), eq = __reduce_add_sync(FULL, lane < warp ? mine.y : 0);
  const unsigned below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < (PER ? PER : per); ++j) {
    const uint32_t k = at(j);
    const unsigned bu = __ballot_sync(FULL, k > least), be = __ballot_sync(FULL, k == least);
    const int before = eq + __popc(be & below);  // equal ones of lower index
    const bool keep = k > least || (k == least && before < ties);
    if (keep) out[up + __popc(bu & below) + min(before, ties)] = base + 32 * j;
    up += __popc(bu);
    eq += __popc(be);
  }
}

}  // namespace

cudaError_t launch_block_select(const SelectArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.batch * a.Hkv);
  const int mb = a.max_blocks;
  if (mb <= 512) block_select_kernel<128, 4><<<grid, 128, 0, s>>>(a);
  else if (mb <= 2048) block_select_kernel<256, 8><<<grid, 256, 0, s>>>(a);
  else if (mb <= 8192) block_select_kernel<512, 16><<<grid, 512, 0, s>>>(a);
  else if (mb <= 32768) block_select_kernel<1024, 32><<<grid, 1024, 0, s>>>(a);
  else block_select_kernel<1024, 0><<<grid, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
