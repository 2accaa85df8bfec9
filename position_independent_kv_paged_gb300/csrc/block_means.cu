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
// A warp per (block, kv head): D / 8 lanes hold 4 + 4 elements of a row's rotary pairs each, so 2 or 4 rows an
// instruction; all rows are loaded before the first is used.  Rows past the block's last key are not read.  Bound by
// memory: 16 D elements read for D written.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kThreads = 256;
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

template <typename T, typename KV, int D>
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
  const long long b0 = js >> 4, items = (((end + 15) >> 4) - b0) * a.Hkv;
  const int row = lane / LPR, e0 = 4 * (lane % LPR);
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < items;
       i += (long long)gridDim.x * (kThreads / 32)) {
    const long long b = b0 + i / a.Hkv;
    const int g = (int)(i % a.Hkv);
    if (b >= a.max_blocks) {
      if (lane == 0) atomicOr(a.err, kErrSeqLen);
      continue;
    }
    const int phys = __ldg(a.block_tables + (size_t)r * a.max_blocks + b);
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) atomicOr(a.err, kErrBlockId);
      continue;
    }
    const int count = (int)min(16LL, end - 16 * b);
    const KV* k = static_cast<const KV*>(a.k_pool) + ((size_t)phys * a.Hkv + g) * 16 * D;
    Four<KV> x[IT], y[IT];
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int s = min(RPI * u + row, count - 1);
      x[u].load(k + s * D + e0);
      y[u].load(k + s * D + D / 2 + e0);
    }
    const float ks = sizeof(KV) == 1 ? __ldg(a.k_scale + (size_t)phys * a.Hkv + g) : 1.f;
    float mx[4] = {0.f, 0.f, 0.f, 0.f}, my[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int s = RPI * u + row;
      if (s < count) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(a.cos_sin + s * D + e0));
        const float4 n = __ldg(reinterpret_cast<const float4*>(a.cos_sin + s * D + D / 2 + e0));
        const float4 xv = x[u].wide(), yv = y[u].wide();
        const float xs[4] = {xv.x, xv.y, xv.z, xv.w}, ys[4] = {yv.x, yv.y, yv.z, yv.w};
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx[e] += fmaf(xs[e], cs[e], -ys[e] * sn[e]);
          my[e] += fmaf(ys[e], cs[e], xs[e] * sn[e]);
        }
      }
    }
    const float f = ks / (float)count;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        mx[e] += __shfl_xor_sync(FULL, mx[e], o);
        my[e] += __shfl_xor_sync(FULL, my[e], o);
      }
      mx[e] *= f;
      my[e] *= f;
    }
    if (row == 0) {
      T* m = static_cast<T*>(a.means) + ((size_t)phys * a.Hkv + g) * D;
      store4(m + e0, mx);
      store4(m + D / 2 + e0, my);
    }
  }
}

template <typename T, typename KV>
cudaError_t launch_t(const MeansArgs& a, cudaStream_t s) {
  const long long items = ((a.max_new + 14LL) / 16 + 1) * a.Hkv;  // of a request, at most
  long long gx = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (gx > 65535) gx = 65535;  // grid-stride beyond this
  const dim3 grid((unsigned)gx, (unsigned)a.batch);
  if (a.D == 128) block_means_kernel<T, KV, 128><<<grid, kThreads, 0, s>>>(a);
  else block_means_kernel<T, KV, 64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_means(const MeansArgs& a, bool bf16, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.k_scale) return bf16 ? launch_t<B, __nv_fp8_e4m3>(a, s) : launch_t<float, __nv_fp8_e4m3>(a, s);
  return bf16 ? launch_t<B, B>(a, s) : launch_t<float, float>(a, s);
}

}  // namespace minipic
