// Eviction of whole blocks by accumulated attention weight.
//
// Per request with n blocks: score_b = decay * score_b + sum_g w[g][b]; the
// first keep_first and the last keep_last blocks stay, the others compete by
// score (ties: the lower index stays) until `budget` blocks are kept.  The
// tables are compacted in order.  Blocks of a position-free cache carry their
// logical starts in the table, so dropping one moves nothing in the pool and
// re-rotates nothing: this is integer work on the tables alone.
//
// One CTA per request.  The score's terms are added in 64 bits and kept in 32,
// so that their order does not show in the ranking.  The budget-th best score
// comes from a radix selection (four passes of 8 bits over an order-preserving
// integer image of the float), ties are cut by index, and one ordered pass
// compacts: a kept entry only ever moves to a lower index, and each chunk is
// read before the barrier that its writes wait for, so outputs may be the
// inputs.  Latency-bound: a few passes over 4 to 20 bytes a block.
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"

namespace minipic {
namespace {

constexpr int kThreads = 1024;
constexpr int kNW = kThreads / 32;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Larger float <-> larger integer; -0 counts as +0 and NaN as the lowest.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of the flags over the CTA, and their total (every thread calls).
__device__ __forceinline__ int scan_flags(bool f, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(FULL, f);
  if (lane == 0) warp_sums[w] = __popc(m);
  __syncthreads();
  const int mine = warp_sums[lane];  // kNW == 32
  int before = lane < w ? mine : 0, all = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(FULL, before, o);
    all += __shfl_xor_sync(FULL, all, o);
  }
  total = all;
  __syncthreads();
  return before + __popc(m & ((1u << lane) - 1u));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_evict_kernel(EvictArgs a) {
  static_assert(kNW == 32, "scan_flags");
  __shared__ int hist[256];
  __shared__ int warp_sums[kNW];
  __shared__ int s_digit, s_left;
  const int r = blockIdx.x, tid = threadIdx.x, mb = a.max_blocks;
  const size_t row = (size_t)r * mb;
  int L = a.seq_lens[r];
  if (L < 0 || (long long)L > 16LL * mb) {
    if (tid == 0) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : (int)min(16LL * mb, 2147483647LL);
  }
  const int n = (int)(((long long)L + 15) >> 4);
  for (int b = tid; b < n; b += kThreads) {
    double s = (double)a.scores[row + b] * (double)a.decay;
    if (a.weights) {
      const T* w = static_cast<const T*>(a.weights) + (size_t)r * a.Hkv * mb + b;
      for (int g = 0; g < a.Hkv; ++g) s += (double)to_f(w[(size_t)g * mb]);
    }
    a.scores_out[row + b] = (float)s;
  }
  __syncthreads();  // this CTA reads back what it wrote
  auto held = [&](int b) { return b < a.keep_first || b >= n - a.keep_last; };
  const bool cut = n > a.budget;
  uint32_t least = 0u;  // key of the last kept candidate
  int ties = 0;         // candidates of that key that stay
  if (cut) {
    int left = a.budget - min(a.keep_first, n) - min(a.keep_last, n);  // n > budget >= keep_first + keep_last
    uint32_t mask = 0u;
    for (int shift = 24; shift >= 0 && left > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int b = tid; b < n; b += kThreads) {
        if (held(b)) continue;
        const uint32_t k = rank_key(a.scores_out[row + b]);
        if ((k & mask) == (least & mask)) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid < 32) {  // lane l: digits 255 - 8 l down to 248 - 8 l
        int c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) c += hist[255 - 8 * tid - i];
        int pre = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULL, pre, o);
          if (tid >= o) pre += y;
        }
        pre -= c;
        if (pre < left && left <= pre + c) {
          int d = 255 - 8 * tid;
          while (pre + hist[d] < left) pre += hist[d--];
          s_digit = d;
          s_left = left - pre;
        }
      }
      __syncthreads();
      least |= (uint32_t)s_digit << shift;
      left = s_left;
      mask |= 255u << shift;
    }
    ties = left;
    if (a.budget - min(a.keep_first, n) - min(a.keep_last, n) <= 0) least = 0xffffffffu;
  }
  int kept = 0, gone = 0, tied = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int b = base + tid;
    const bool in = b < n;
    const float s = in ? a.scores_out[row + b] : 0.f;
    const int phys = in ? a.block_tables[row + b] : 0, st = in ? a.block_starts[row + b] : 0;
    const bool cand = in && cut && !held(b);
    const uint32_t k = cand ? rank_key(s) : 0u;
    int tot;
    const int tr = tied + scan_flags(cand && k == least, warp_sums, tot);
    tied += tot;
    const bool keep = in && (!cand || k > least || (k == least && tr < ties));
    const int kr = scan_flags(keep, warp_sums, tot);  // its barriers also order the reads above before the writes
    if (keep) {
      const size_t to = row + kept + kr;
      a.scores_out[to] = s;
      a.tables_out[to] = phys;
      a.starts_out[to] = st;
    } else if (in) {
      a.evicted[row + gone + tid - kr] = phys;
    }
    kept += tot;
    gone += min(n - base, kThreads) - tot;
  }
  __syncthreads();
  for (int b = kept + tid; b < mb; b += kThreads) {
    a.scores_out[row + b] = 0.f;
    a.tables_out[row + b] = -1;
    a.starts_out[row + b] = 0;
  }
  for (int b = gone + tid; b < mb; b += kThreads) a.evicted[row + b] = -1;
  if (tid == 0) {
    a.lens_out[r] = L - 16 * gone;
    a.n_evicted[r] = gone;
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) kv_evict_kernel<__nv_bfloat16><<<a.batch, kThreads, 0, s>>>(a);
  else kv_evict_kernel<float><<<a.batch, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
