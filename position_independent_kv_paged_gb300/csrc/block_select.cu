// The best blocks of each (request, kv head) by score.
//
// With n blocks: all of them where n <= budget, else the first keep_first, the last keep_last and the best of the others
// by score up to `budget` (NaN is the worst; of equal scores the lower index stays: the rule of kv_evict).  Their numbers are
// written in ascending order, then -1.
//
// One CTA per (request, kv head).  Each thread keeps PER order-preserving integer images of its scores in
// registers, in warp-contiguous rows of 32, so loads are whole lines and ballots give the order.  The threshold, the
// image of the last candidate that stays, is built from the top, two bits a pass: the candidates at or above each of
// three trial images are counted, and the largest that enough reach stays.  A pass is 3 PER comparisons, three warp
// sums (two of them in one word) and a barrier; it ends early when the count is met exactly, which scores of many bits do
// after about two thirds of them.  No histogram: scores lie in few exponents, whose atomics would queue.
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

// Sums of three counts over the CTA in every thread; `slots` holds two rows, used in turn, so one barrier a call.
// PACKED: counts below 2^16 over the CTA, two of them in one sum.
template <int NW, bool PACKED>
__device__ __forceinline__ void cta_sums(int (&c)[3], int3 (*slots)[32], int turn) {
  const int lane = threadIdx.x & 31;
  int3 v;
  if (PACKED) {
    v.x = (int)__reduce_add_sync(FULL, (unsigned)c[0] | (unsigned)c[1] << 16);
    v.y = 0;
  } else {
    v.x = __reduce_add_sync(FULL, c[0]);
    v.y = __reduce_add_sync(FULL, c[1]);
  }
  v.z = __reduce_add_sync(FULL, c[2]);
  if (lane == 0) slots[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < NW ? slots[turn & 1][lane] : make_int3(0, 0, 0);
  const unsigned x = __reduce_add_sync(FULL, (unsigned)v.x);
  c[0] = PACKED ? (int)(x & 0xffffu) : (int)x;
  c[1] = PACKED ? (int)(x >> 16) : __reduce_add_sync(FULL, v.y);
  c[2] = __reduce_add_sync(FULL, v.z);
}

// PER = 0: any number of blocks, scores read again in each pass.
template <int T, int PER>
__global__ void __launch_bounds__(T) block_select_kernel(const SelectArgs a) {
  constexpr int NW = T / 32;
  __shared__ int3 slots[2][32];
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
  for (int bit = 30; bit >= 0 && reach != S; bit -= 2) {
    int c[3] = {0, 0, 0};
#pragma unroll
    for (int j = 0; j < (PER ? PER : per); ++j) {
      const uint32_t k = at(j);
#pragma unroll
      for (int i = 0; i < 3; ++i) c[i] += k >= (least | (uint32_t)(i + 1) << bit);
    }
    cta_sums<NW, PER != 0>(c, slots, turn++);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (c[i] >= S) {  // fewer reach a larger trial
        least = (least & ~(3u << bit)) | (uint32_t)(i + 1) << bit;
        reach = c[i];
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
  else if (mb <= 8192) block_select_kernel<1024, 8><<<grid, 1024, 0, s>>>(a);
  else if (mb <= 32768) block_select_kernel<1024, 32><<<grid, 1024, 0, s>>>(a);
  else block_select_kernel<1024, 0><<<grid, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
