// Eviction of whole blocks by accumulated attention weight.
//
// Per request with n blocks: score_b = decay * score_b + sum_g w[g][b]; the
// first keep_first and the last keep_last blocks stay, the others compete by
// score (ties: the lower index stays) until `budget` blocks are kept.  The
// tables are compacted in order.  Blocks of a position-free cache carry their
// logical starts in the table, so dropping one moves nothing in the pool and
// re-rotates nothing: this is integer work on the tables alone.
//
// One CTA per request.  The score's terms are added with twice fp32's precision
// (error-free sums of fp32 pairs: FP64 runs at 2 operations a cycle and SM here)
// and rounded to fp32 once, so that their order does not show in the ranking.  The budget-th best score comes from a radix
// selection over an order-preserving integer image of the float (11, 11 and 10
// bits; the images stay in shared memory while they fit), ties are cut by index,
// and one ordered pass compacts, four blocks per thread: a kept entry only ever
// moves to a lower index, and each chunk is read before the barrier that its
// writes wait for, so outputs may be the inputs.  Latency-bound, a few passes
// over 4 to 20 bytes a block: 64 x 512 blocks 6.9 us, 8 x 8192 blocks 23 us.
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "tmap.cuh"

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

// hi + lo += x, with hi the rounded sum and lo what it lacks (Knuth's two-sum).
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), t = __fsub_rn(s, hi);
  lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(x, t));
  hi = s;
}

// Exclusive prefix of c over the CTA, and the total (every thread calls; two barriers).
__device__ __forceinline__ int scan(int c, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int pre = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, pre, o);
    if (lane >= o) pre += y;
  }
  if (lane == 31) warp_sums[w] = pre;
  __syncthreads();
  const int mine = warp_sums[lane];  // kNW == 32
  const int before = __reduce_add_sync(FULL, lane < w ? mine : 0);
  total = __reduce_add_sync(FULL, mine);
  __syncthreads();
  return before + pre - c;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_evict_kernel(EvictArgs a, int smem_keys) {
  static_assert(kNW == 32, "scan");
  __shared__ int hist[2048];
  __shared__ int warp_sums[kNW];
  __shared__ int s_digit, s_left, s_count;
  extern __shared__ uint32_t skeys[];  // [smem_keys]
  const int r = blockIdx.x, tid = threadIdx.x, mb = a.max_blocks;
  const size_t row = (size_t)r * mb;
  int L = a.seq_lens[r];
  if (L < 0 || (long long)L > 16LL * mb) {
    if (tid == 0) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : (int)min(16LL * mb, 2147483647LL);
  }
  const int n = (int)(((long long)L + 15) >> 4);
  const bool cut = n > a.budget;
  const bool in_smem = n <= smem_keys;
  for (int b = tid; b < n; b += kThreads) {
    const float old = a.scores[row + b];
    float hi = __fmul_rn(old, a.decay);
    float lo = fabsf(hi) < 3.4e38f ? __fmaf_rn(old, a.decay, -hi) : 0.f;
    if (a.weights) {
      const T* w = static_cast<const T*>(a.weights) + (size_t)r * a.Hkv * mb + b;
      for (int g0 = 0; g0 < a.Hkv; g0 += 8) {  // eight loads at a time
        float x[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) x[g] = g0 + g < a.Hkv ? to_f(w[(size_t)(g0 + g) * mb]) : 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) add_exact(hi, lo, x[g]);
      }
    }
    const float s = fabsf(hi) < 3.4e38f ? hi + lo : hi;  // infinities and NaN have no remainder
    a.scores_out[row + b] = s;
    if (cut && in_smem) skeys[b] = rank_key(s);
  }
  __syncthreads();  // this CTA reads back what it wrote
  auto held = [&](int b) { return b < a.keep_first || b >= n - a.keep_last; };
  auto key = [&](int b) { return in_smem ? skeys[b] : rank_key(a.scores_out[row + b]); };
  uint32_t least = 0xffffffffu;  // image of the last kept candidate
  int ties = 0, equal = 0;       // candidates of that image that stay, and all of them
  if (cut) {
    int left = a.budget - a.keep_first - a.keep_last;  // n > budget >= keep_first + keep_last
    uint32_t mask = 0u;
    if (left > 0) least = 0u;
#pragma unroll 1
    for (int pass = 0; pass < 3 && left > 0; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), digits = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < 2048; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int b = tid; b < n; b += kThreads) {
        if (held(b)) continue;
        const uint32_t k = key(b);
        if ((k & mask) == (least & mask)) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1);
      }
      __syncthreads();
      // thread t: digits 2047 - 2 t and 2046 - 2 t, so that the prefix counts from the largest
      const int h0 = hist[2047 - 2 * tid], h1 = hist[2046 - 2 * tid];
      int tot;
      const int pre = scan(h0 + h1, warp_sums, tot);
      if (pre < left && left <= pre + h0 + h1) {
        const bool first = left <= pre + h0;
        s_digit = first ? 2047 - 2 * tid : 2046 - 2 * tid;
        s_left = left - pre - (first ? 0 : h0);
        s_count = first ? h0 : h1;
      }
      __syncthreads();
      least |= (uint32_t)s_digit << shift;
      left = s_left;
      equal = s_count;
      mask |= (uint32_t)(digits - 1) << shift;
      __syncthreads();  // read before the next pass writes them
    }
    ties = left;
  }
  constexpr int PER = 4;
  int kept = 0, tied = 0;
  for (int base = 0; base < n; base += PER * kThreads) {
    const int b0 = base + PER * tid;
    float sc[PER];
    int ph[PER], st[PER];
    uint32_t ks[PER];
    int eq = 0;
    unsigned keep = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = b0 + i;
      const bool in = b < n;
      sc[i] = in ? a.scores_out[row + b] : 0.f;
      ph[i] = in ? a.block_tables[row + b] : 0;
      st[i] = in ? a.block_starts[row + b] : 0;
      ks[i] = rank_key(sc[i]);
      const bool cand = in && cut && !held(b);
      eq += cand && ks[i] == least;
      keep |= (in && (!cand || ks[i] >= least) ? 1u : 0u) << i;
    }
    int tot;
    if (ties != equal) {  // not all of the last image's candidates stay: those of the lowest index do
      int tr = tied + scan(eq, warp_sums, tot);
      tied += tot;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = b0 + i;
        if (b < n && cut && !held(b) && ks[i] == least && tr++ >= ties) keep &= ~(1u << i);
      }
    }
    int kr = kept + scan(__popc(keep), warp_sums, tot);  // its barriers also order the reads above before the writes
    kept += tot;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = b0 + i;
      if ((keep >> i) & 1u) {
        a.scores_out[row + kr] = sc[i];
        a.tables_out[row + kr] = ph[i];
        a.starts_out[row + kr] = st[i];
        ++kr;
      } else if (b < n) {
        a.evicted[row + b - kr] = ph[i];  // b - kr blocks before this one left
      }
    }
  }
  __syncthreads();
  for (int b = kept + tid; b < mb; b += kThreads) {
    a.scores_out[row + b] = 0.f;
    a.tables_out[row + b] = -1;
    a.starts_out[row + b] = 0;
  }
  for (int b = n - kept + tid; b < mb; b += kThreads) a.evicted[row + b] = -1;
  if (tid == 0) {
    a.lens_out[r] = L - 16 * (n - kept);
    a.n_evicted[r] = n - kept;
  }
}

constexpr int kMaxKeys = 49152;  // images held in shared memory (192 KB)

template <typename T>
cudaError_t launch_t(const EvictArgs& a, cudaStream_t s) {
  static bool done[64] = {false};
  const cudaError_t e = set_smem_once(kv_evict_kernel<T>, kMaxKeys * 4, done);
  if (e != cudaSuccess) return e;
  const int keys = a.max_blocks < kMaxKeys ? a.max_blocks : kMaxKeys;
  kv_evict_kernel<T><<<a.batch, kThreads, (size_t)keys * 4, s>>>(a, keys);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace minipic
