// The best blocks of each (request, kv head) by score.
//
// With n blocks: all of them where n <= budget, else the first keep_first, the last keep_last and the best of the
// others by score up to `budget` (NaN is the worst; of equal scores the lower index stays: the rule of kv_evict).  Their
// numbers are written in ascending order, then -1.
//
// One CTA per (request, kv head).  Each thread keeps PER order-preserving integer images of its scores in
// registers, in warp-contiguous rows of 32, so loads are whole lines and ballots give the order.  The threshold, the
// image of the last candidate that stays, is built from the top, two bits a pass: the candidates at or above each of
// three trial images are counted, and the largest that enough reach stays.  A pass is 3 PER comparisons, three warp
// sums and a barrier.  When few images begin with the bits found so far (scores of many bits: after five passes of
// sixteen) one warp takes those through the rest without barriers; it ends when the count is met exactly.  No
// histogram: scores lie in few exponents, whose atomics would queue.  Bound by the latency of the passes: 512 rows of
// 512 blocks take 4.9 us, 64 rows of 8192 blocks 12 us, of 32768 31 us (their bytes: 0.2, 0.3 and 1.3 us); above that
// every pass reads the scores again, 64 rows of 131072 blocks take 318 us (5 us).
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
// PER: a warp's counts are at most 32 PER.  Warp sums are slow instructions (one a scheduler in many cycles), so where
// the counts fit, all three share a word over the warp (10 bits each) and two do over the CTA (16 bits).
template <int NW, int PER>
__device__ __forceinline__ void cta_sums(int (&c)[3], int3 (*slots)[32], int turn) {
  const int lane = threadIdx.x & 31;
  int3 v;
  if (PER > 0 && 32 * PER < 1024) {
    const unsigned x = __reduce_add_sync(FULL, (unsigned)(c[0] | c[1] << 10 | c[2] << 20));
    v = make_int3((int)(x & 1023u) | (int)(x >> 10 & 1023u) << 16, 0, (int)(x >> 20));
  } else if (PER > 0) {
    v.x = (int)__reduce_add_sync(FULL, (unsigned)c[0] | (unsigned)c[1] << 16);
    v.y = 0;
    v.z = __reduce_add_sync(FULL, c[2]);
  } else {
    v.x = __reduce_add_sync(FULL, c[0]);
    v.y = __reduce_add_sync(FULL, c[1]);
    v.z = __reduce_add_sync(FULL, c[2]);
  }
  if (lane == 0) slots[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < NW ? slots[turn & 1][lane] : make_int3(0, 0, 0);
  const unsigned x = __reduce_add_sync(FULL, (unsigned)v.x);
  c[0] = PER > 0 ? (int)(x & 0xffffu) : (int)x;
  c[1] = PER > 0 ? (int)(x >> 16) : __reduce_add_sync(FULL, v.y);
  c[2] = __reduce_add_sync(FULL, v.z);
}

// Takes the largest digit that at least `want` images reach at bits `bit` and `bit` + 1 of the threshold.
__device__ __forceinline__ void step(const int (&c)[3], int want, int bit, uint32_t& least, int& reach, int& top) {
  const uint32_t before = least;
  int above = c[0];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (c[i] >= want) {  // fewer reach a larger trial
      least = before | (uint32_t)(i + 1) << bit;
      reach = c[i];
      above = i < 2 ? c[i + 1 < 3 ? i + 1 : 2] : top;
    }
  top = above;
}

// Images that one warp finishes (rows of 512 / 8192 blocks: 4.9 / 11.7 us; with 256 of them 5.2 / 11.7, 512 7.9 / 12.1,
// and all passes over all images 5.5 / 16.2).
constexpr int kFew = 128;

// PER = 0: any number of blocks, scores read again in each pass.
template <int T, int PER>
__global__ void __launch_bounds__(T) block_select_kernel(const SelectArgs a) {
  constexpr int NW = T / 32;
  __shared__ int3 slots[2][32];
  __shared__ int2 s_before[32];
  __shared__ uint32_t few[kFew];
  __shared__ uint32_t s_least;
  __shared__ int n_few;
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
  for (int i = threadIdx.x; i < kFew; i += T) few[i] = 0u;
  if (threadIdx.x == 0) n_few = 0;
  // the largest threshold that at least S images reach (n > S, and held blocks are at most S)
  uint32_t least = 0u;
  int reach = n, top = 0, turn = 0;  // images >= least; images above those that begin with the bits of least
  int bit = 30;
#pragma unroll 1
  for (; bit >= 0 && reach != S && (reach - top > kFew || turn == 0); bit -= 2) {
    int c[3] = {0, 0, 0};
#pragma unroll
    for (int j = 0; j < (PER ? PER : per); ++j) {
      const uint32_t k = at(j);
#pragma unroll
      for (int i = 0; i < 3; ++i) c[i] += k >= (least | (uint32_t)(i + 1) << bit);
    }
    cta_sums<NW, PER>(c, slots, turn++);
    step(c, S, bit, least, reach, top);
  }
  if (bit >= 0 && reach != S) {  // few images are left to choose from: one warp does
#pragma unroll
    for (int j = 0; j < (PER ? PER : per); ++j) {
      const uint32_t k = at(j);
      if (k != 0u && k - least < 4u << bit) few[atomicAdd(&n_few, 1)] = k;  // reach - top of them
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t k[kFew / 32];
#pragma unroll
      for (int j = 0; j < kFew / 32; ++j) k[j] = few[32 * j + lane];
      reach -= top;
      const int want = S - top;
      top = 0;
#pragma unroll 1
      for (; bit >= 0 && reach != want; bit -= 2) {
        int c = 0;
#pragma unroll
        for (int j = 0; j < kFew / 32; ++j)
#pragma unroll
          for (int i = 0; i < 3; ++i) c += k[j] >= (least | (uint32_t)(i + 1) << bit) ? 1 << 10 * i : 0;
        c = (int)__reduce_add_sync(FULL, (unsigned)c);
        const int c3[3] = {c & 1023, c >> 10 & 1023, c >> 20};
        step(c3, want, bit, least, reach, top);
      }
      if (lane == 0) s_least = least;
    }
    __syncthreads();
    least = s_least;
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
