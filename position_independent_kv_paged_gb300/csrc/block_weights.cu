// Block weights of a decode step: the share of each 16-key block in the
// attention of a kv head's query group,
//   weights[r][g][b] = sum_{h in group g} 2^(raw[r][g][b][h] - lse[r][h]),
// from the per-block sums the decode kernels record (log2, at each warp's own
// reference) and the softmax denominators (log2).  Both are logarithms, so the
// splits and warps need no common reference.  One thread per (request, kv
// head, block) reads its G values as one contiguous piece; blocks past the
// request's length are left as they were.  HBM/L2-bound and tiny next to the
// attention: 4 G bytes read per block against its 32 d bytes of e4m3 keys and
// values.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"

namespace minipic {
namespace {

constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) block_weights_kernel(DecodeArgs a) {
  const int r = blockIdx.z, g = blockIdx.y;
  const int b = blockIdx.x * kThreads + threadIdx.x;
  const int L = a.seq_lens[r];
  if (L <= 0 || b >= min((L >> 4) + ((L & 15) != 0), a.max_blocks)) return;
  const size_t at = ((size_t)r * a.Hkv + g) * a.max_blocks + b;
  const float* raw = a.w_raw + at * a.G;
  const float* lse = a.w_lse + (size_t)r * a.Hq + (size_t)g * a.G;
  float w = 0.f;
  for (int h = 0; h < a.G; ++h) {
    const float x = raw[h], l = lse[h];
    w += x == -CUDART_INF_F ? 0.f : exp2f(x - l);  // a query with no key has every sum at -inf
  }
  if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.weights)[at] = __float2bfloat16_rn(w);
  else static_cast<float*>(a.weights)[at] = w;
}

}  // namespace

cudaError_t launch_block_weights(const DecodeArgs& a, bool bf16, cudaStream_t s) {
  const dim3 grid((unsigned)((a.max_blocks + kThreads - 1) / kThreads), (unsigned)a.Hkv, (unsigned)a.batch);
  if (bf16) block_weights_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else block_weights_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
