// e4m3 blocks back to bf16, for the chunked prefill over an 8-bit cache: block
// b of request r becomes block r * max_blocks + b of a bf16 scratch pool, in
// request order, which the tcgen05 prefill then reads through its own tables.
// value = bf16(byte * scale): exact for a power-of-two scale (e4m3 has four
// significant bits), one rounding otherwise.  Slots past the request's length
// are written as zeros, so that what an unused slot happens to hold (NaN bytes
// included) never meets a product.
//
// HBM-bound: 1 byte read and 2 written per value.  The prefill it feeds is
// bound by the tensor cores; there the extra traffic of a separate pass costs
// about a tenth of the time.
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kThreads = 256;

// 16 e4m3 bytes -> 16 bf16
__device__ __forceinline__ void widen16(const uint4& w, float s, uint4& lo, uint4& hi) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = ptx::e4m3x4_to_f4(in[i]);
    o[2 * i] = ptx::pack_bf16(x.x * s, x.y * s);
    o[2 * i + 1] = ptx::pack_bf16(x.z * s, x.w * s);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_restore_q8_kernel(RestoreArgs a) {
  constexpr int CPR = D / 16;       // 16-byte chunks of a row
  constexpr int CPT = 16 * CPR;     // ... of a (block, head) tile
  const int b = blockIdx.x, r = blockIdx.y;
  int len = a.kv_lens[r];
  len = min(len, a.max_blocks * 16);
  if (b * 16 >= len) return;
  const size_t to = (size_t)r * a.max_blocks + b;
  const int phys = a.block_tables[to];
  const bool ok = phys >= 0 && phys < a.num_blocks;
  if (threadIdx.x == 0) a.table_out[to] = ok ? (int)to : -1;
  if (!ok) return;
  const int nk = min(16, len - b * 16);
  const int chunks = a.Hkv * CPT;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < chunks; i += kThreads) {
    const int h = i / CPT, slot = (i % CPT) / CPR;
    const size_t src = (size_t)phys * chunks + i;
    uint4 k = zero, v = zero;
    if (slot < nk) {
      k = __ldg(reinterpret_cast<const uint4*>(a.k_pool) + src);
      v = __ldg(reinterpret_cast<const uint4*>(a.v_pool) + src);
    }
    uint4 lo, hi;
    const size_t dst = (to * chunks + i) * 2;
    widen16(k, __ldg(a.k_scale + (size_t)phys * a.Hkv + h), lo, hi);
    reinterpret_cast<uint4*>(a.k_out)[dst] = lo;
    reinterpret_cast<uint4*>(a.k_out)[dst + 1] = hi;
    widen16(v, __ldg(a.v_scale + (size_t)phys * a.Hkv + h), lo, hi);
    reinterpret_cast<uint4*>(a.v_out)[dst] = lo;
    reinterpret_cast<uint4*>(a.v_out)[dst + 1] = hi;
  }
}

}  // namespace

cudaError_t launch_kv_restore_q8(const RestoreArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.max_blocks, (unsigned)a.batch);
  if (a.D == 64) kv_restore_q8_kernel<64><<<grid, kThreads, 0, s>>>(a);
  else kv_restore_q8_kernel<128><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace minipic
