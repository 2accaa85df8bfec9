// The cheap score that block selection ranks by: for each block of a request's table and each kv head
//   score[r][g][b] = max over the query heads h of g of  scale * (R_t q_h) . (R_b m),
// with t the query's position, b the block's start and m the block's summary (block_means.cu): the largest mean score
// that a query head gives the block's keys.  Blocks past the request's length, with an id outside the pool or a start
// outside the table, get -infinity; a NaN product makes the block's score NaN.
//
// fp32 throughout: the ranking shows errors.  A summary is a thirty-second of a block's keys and values, so this reads 1/32 of
// what attention would.
//
// CTA = (range of blocks, kv head, request); 8 (d 128) or 4 (d 64 ... 4 + 4 elements more) lanes hold a summary, 8 + 8
// elements of its rotary pairs each, so that a load instruction of a warp covers whole lines.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kThreads = 256;
constexpr unsigned FULL = 0xffffffffu;

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p) + u);
    v[4 * u] = x.x;
    v[4 * u + 1] = x.y;
    v[4 * u + 2] = x.z;
    v[4 * u + 3] = x.w;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    v[2 * u] = ptx::bf_lo(w[u]);
    v[2 * u + 1] = ptx::bf_hi(w[u]);
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) block_scores_kernel(const ScoresArgs a) {
  constexpr int LPB = D / 16;       // lanes of a summary
  constexpr int BPW = 32 / LPB;     // summaries of a warp
  __shared__ float sq[16 * D];      // the group's rotated queries
  const int g = blockIdx.y, r = blockIdx.z, lane = threadIdx.x & 31;
  const int mb = a.max_blocks, G = a.G;
  int L = a.seq_lens[r];
  if (L < 0 || (long long)L > 16LL * mb) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && g == 0) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : (int)min(16LL * mb, 2147483632LL);
  }
  const int n = min((L >> 4) + ((L & 15) != 0), mb);
  int t = a.q_pos[r];
  if (n > 0 && (t < 0 || t >= a.max_pos)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && g == 0) atomicOr(a.err, kErrPosition);
    t = 0;
  }
  const T* q = static_cast<const T*>(a.q) + ((size_t)r * a.Hq + (size_t)g * G) * D;
  if (n > 0)
    for (int i = threadIdx.x; i < G * (D / 2); i += kThreads) {
      const int h = i / (D / 2), e = i % (D / 2);
      const float c = __ldg(a.cos_sin + (size_t)t * D + e), s = __ldg(a.cos_sin + (size_t)t * D + D / 2 + e);
      const float x = to_f(q[h * D + e]), y = to_f(q[h * D + D / 2 + e]);
      sq[h * D + e] = fmaf(x, c, -y * s) * a.scale;
      sq[h * D + D / 2 + e] = fmaf(y, c, x * s) * a.scale;
    }
  __syncthreads();
  float* out = a.scores + ((size_t)r * a.Hkv + g) * mb;
  const int e0 = 8 * (lane % LPB);
  for (long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w * BPW < mb;
       w += (long long)gridDim.x * (kThreads / 32)) {
    const int b = (int)(w * BPW) + lane / LPB;
    int phys = -1, start = 0;
    if (b < n) {
      phys = __ldg(a.block_tables + (size_t)r * mb + b);
      start = __ldg(a.block_starts + (size_t)r * mb + b);
      if (phys < 0 || phys >= a.num_blocks) {
        if (g == 0 && lane % LPB == 0) atomicOr(a.err, kErrBlockId);
        phys = -1;
      } else if (start < 0 || start >= a.max_pos) {
        if (g == 0 && lane % LPB == 0) atomicOr(a.err, kErrPosition);
        phys = -1;
      }
    }
    float best = -CUDART_INF_F;
    float x[8], y[8], c[8], s[8];
    if (phys >= 0) {
      const T* m = static_cast<const T*>(a.means) + ((size_t)phys * a.Hkv + g) * D;
      load8(m + e0, x);
      load8(m + D / 2 + e0, y);
      load8(a.cos_sin + (size_t)start * D + e0, c);
      load8(a.cos_sin + (size_t)start * D + D / 2 + e0, s);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = y[e] = c[e] = s[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[e];
      x[e] = fmaf(u, c[e], -y[e] * s[e]);
      y[e] = fmaf(y[e], c[e], u * s[e]);
    }
    for (int h = 0; h < G; ++h) {
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(sq[h * D + e0 + e], x[e], fmaf(sq[h * D + D / 2 + e0 + e], y[e], dot));
#pragma unroll
      for (int o = LPB / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(FULL, dot, o);
      best = max_nan(best, dot);
    }
    if (lane % LPB == 0 && b < mb) out[b] = phys >= 0 ? best : -CUDART_INF_F;
  }
}

template <typename T>
cudaError_t launch_t(const ScoresArgs& a, int num_sms, cudaStream_t s) {
  const int per = (kThreads / 32) * (32 / (a.D / 16));  // blocks of a CTA's pass
  long long gx = (a.max_blocks + (long long)per - 1) / per;
  const long long rows = (long long)a.Hkv * a.batch, most = (8LL * num_sms + rows - 1) / rows;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, (unsigned)a.Hkv, (unsigned)a.batch);
  if (a.D == 128) block_scores_kernel<T, 128><<<grid, kThreads, 0, s>>>(a);
  else block_scores_kernel<T, 64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_scores(const ScoresArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, num_sms, s) : launch_t<float>(a, num_sms, s);
}

}  // namespace minipic
