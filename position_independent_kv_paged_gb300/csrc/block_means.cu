// Summaries of cache blocks for block selection: per (block, kv head)
//   m = (1 / n) sum_{s < n} R_s k_s,
// the mean of the block's n keys, each rotated by its slot.  For a block that starts at b
//   (R_{t-b} q) . m = (1 / n) sum_s (R_t q) . (R_{b+s} k_s),
// the mean of the block's scores, whatever b is: like the keys (MiniPIC summary, gist.science 2606.13126, section
// 2.1), a summary holds no position and serves every request that reads the block.
//
// Called after an append with the append's arguments, for every block that the new keys went into; a block's keys
// are read again from the pool, so a summary is rounded once, however many calls filled the block (adding to a
// rounded mean would round it at every step).  Sums are fp32.
//
// A warp per block and U kv heads: D / 8 lanes hold 4 + 4 elements of a row's rotary pairs each, so 2 or 4 rows an
// instruction; all rows are loaded before the first is used, and the rotations serve all U heads.  Rows past the
// block's last key are not read.  Bound by latency (counts, table entry, keys, one after another) up to a wave of
// warps, then by memory: 16 D elements read for D written (26 MB of keys: 9.0 us with U = 2, 10.8 with
// U = 1, whose rotations are half of what the L1 delivers, 9.4 with U = 4).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kThreads = 128;
// Warps of one kv head each, per SM, above which a warp takes two (a step of 128 requests, 1024 warps on 152 SMs: 4.2 us
// with one, 4.5 with two; chunks of 8320 warps: 10.8 and 9.0).
constexpr long long kManyWarps = 16;
constexpr unsigned FULL = 0xffffffffu;

// Four consecutive elements of a row as loaded, and widened.
template <typename KV>
struct Four;
template <>
struct Four<float> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ float4 wide() const { return x; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ float4 wide() const {
    return make_float4(ptx::bf_lo(x.x), ptx::bf_hi(x.x), ptx::bf_lo(x.y), ptx::bf_hi(x.y));
  }
};
template <>
struct Four<__nv_fp8_e4m3> {
  uint32_t x;
  __device__ __forceinline__ void load(const __nv_fp8_e4m3* p) { x = __ldg(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ float4 wide() const { return ptx::e4m3x4_to_f4(x); }
};

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]));
}

template <typename T, typename KV, int D, int U>
__global__ void __launch_bounds__(kThreads) block_means_kernel(const MeansArgs a) {
  constexpr int LPR = D / 8;       // lanes of a row
  constexpr int RPI = 32 / LPR;    // rows of an instruction
  constexpr int IT = 16 / RPI;
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const long long n = (long long)a.cu_new[r + 1] - a.cu_new[r];
  const int js = a.kv_start[r];
  if (n <= 0) return;
  if (js < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrSeqLen);
    return;
  }
  const long long end = js + n;            // keys of the request after the append
  const int per = (a.Hkv + U - 1) / U;     // warps of a block
  const long long b0 = js >> 4, b1 = min((end + 15) >> 4, (long long)a.max_blocks), items = (b1 - b0) * per;
  if (end > 16LL * a.max_blocks && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrSeqLen);
  const int row = lane / LPR, e0 = 4 * (lane % LPR);
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < items;
       i += (long long)gridDim.x * (kThreads / 32)) {
    const long long b = b0 + i / per;
    const int g0 = (int)(i % per) * U;
    const int phys = __ldg(a.block_tables + (size_t)r * a.max_blocks + b);
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) atomicOr(a.err, kErrBlockId);
      continue;
    }
    const int count = (int)min(16LL, end - 16 * b);
    Four<KV> x[U][IT], y[U][IT];
    float ks[U];
#pragma unroll
    for (int w = 0; w < U; ++w) {
      const size_t at = (size_t)phys * a.Hkv + min(g0 + w, a.Hkv - 1);
      const KV* k = static_cast<const KV*>(a.k_pool) + at * 16 * D;
      ks[w] = sizeof(KV) == 1 ? __ldg(a.k_scale + at) : 1.f;
#pragma unroll
      for (int u = 0; u < IT; ++u) {
        const int s = min(RPI * u + row, count - 1);
        x[w][u].load(k + s * D + e0);
        y[w][u].load(k + s * D + D / 2 + e0);
      }
    }
    float mx[U][4] = {}, my[U][4] = {};
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int s = RPI * u + row;
      if (s < count) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(a.cos_sin + s * D + e0));
        const float4 n = __ldg(reinterpret_cast<const float4*>(a.cos_sin + s * D + D / 2 + e0));
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int w = 0; w < U; ++w) {
          const float4 xv = x[w][u].wide(), yv = y[w][u].wide();
          const float xs[4] = {xv.x, xv.y, xv.z, xv.w}, ys[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            mx[w][e] += fmaf(xs[e], cs[e], -ys[e] * sn[e]);
            my[w][e] += fmaf(ys[e], cs[e], xs[e] * sn[e]);
          }
        }
      }
    }
#pragma unroll
    for (int w = 0; w < U; ++w) {
      const float f = ks[w] / (float)count;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
          mx[w][e] += __shfl_xor_sync(FULL, mx[w][e], o);
          my[w][e] += __shfl_xor_sync(FULL, my[w][e], o);
        }
        mx[w][e] *= f;
        my[w][e] *= f;
      }
      if (row == 0 && g0 + w < a.Hkv) {
        T* m = static_cast<T*>(a.means) + ((size_t)phys * a.Hkv + g0 + w) * D;
        store4(m + e0, mx[w]);
        store4(m + D / 2 + e0, my[w]);
      }
    }
  }
}

template <typename T, typename KV, int U>
cudaError_t launch_u(const MeansArgs& a, cudaStream_t s) {
  const long long items = ((a.max_new + 14LL) / 16 + 1) * ((a.Hkv + U - 1) / U);  // of a request, at most
  long long gx = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (gx > 65535) gx = 65535;  // grid-stride beyond this
  const dim3 grid((unsigned)gx, (unsigned)a.batch);
  if (a.D == 128) block_means_kernel<T, KV, 128, U><<<grid, kThreads, 0, s>>>(a);
  else block_means_kernel<T, KV, 64, U><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename KV>
cudaError_t launch_t(const MeansArgs& a, int num_sms, cudaStream_t s) {
  const long long warps = ((a.max_new + 14LL) / 16 + 1) * a.Hkv * a.batch;
  return warps > kManyWarps * num_sms ? launch_u<T, KV, 2>(a, s) : launch_u<T, KV, 1>(a, s);
}

}  // namespace

cudaError_t launch_block_means(const MeansArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  using F8 = __nv_fp8_e4m3;
  if (a.k_scale) return bf16 ? launch_t<B, F8>(a, num_sms, s) : launch_t<float, F8>(a, num_sms, s);
  return bf16 ? launch_t<B, B>(a, num_sms, s) : launch_t<float, float>(a, num_sms, s);
}

}  // namespace minipic
