// Gather step of the chunked prefill over an 8-bit cache: block b of request r
// becomes block r * max_blocks + b of a 16-bit scratch pool, in request order,
// which the tcgen05 prefill then reads through its own tables.
//   keys    fp16(R_pi(j) (byte * scale)), rotated here in fp32 at the key's
//           position in this request and rounded once: the form the score
//           product reads, so the prefill kernel has no keys left to rotate
//   values  bf16(byte * scale), exact for a power-of-two scale (e4m3 has four
//           significant bits)
// Slots past the request's length or the rotary table are written as zeros, so that
// what a masked slot happens to hold (NaN bytes included) never meets a product.
// A NaN value of a key in use would meet the weight 0 of the rows that must not see
// it yet, and make them NaN: it becomes 0 and its key NaN, whose scores the causal
// mask replaces, so the rows that do attend to it are NaN whole and no others are.
//
// Memory-bound: 1 byte read and 2 written per value, plus cos | sin rows that the
// kv heads of a block share through L1.  Measured on 8 requests of 416 blocks, 8
// kv heads, d 128 (109 MB read, 218 MB written): 50 us, 6.5 TB/s; the prefill
// behind it takes 367 us with the keys rotated and 417 us rotating them itself.
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kThreads = 256;

// Any NaN (0x7f, 0xff) among four e4m3 bytes?
__device__ __forceinline__ bool has_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

template <int D>
__global__ void __launch_bounds__(kThreads) kv_restore_q8_kernel(RestoreArgs a) {
  constexpr int CPR = D / 16;       // 16-byte chunks of a row
  constexpr int CPT = 16 * CPR;     // ... of a (block, head) tile
  const int b = blockIdx.x, r = blockIdx.y;
  int len = a.kv_lens[r];
  len = min(len, a.max_blocks * 16);
  if (b * 16 >= len) return;
  const size_t to = (size_t)r * a.max_blocks + b;
  const int phys = a.block_tables[to], start = a.block_starts[to];
  const bool ok = phys >= 0 && phys < a.num_blocks;
  if (threadIdx.x == 0) a.table_out[to] = ok ? (int)to : -1;
  if (!ok) return;
  const int nk = min(16, len - b * 16);
  const int chunks = a.Hkv * CPT;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4* kp = reinterpret_cast<const uint4*>(a.k_pool) + (size_t)phys * chunks;
  const uint4* vp = reinterpret_cast<const uint4*>(a.v_pool) + (size_t)phys * chunks;
  uint4* ko = reinterpret_cast<uint4*>(a.k_out) + to * chunks * 2;
  uint4* vo = reinterpret_cast<uint4*>(a.v_out) + to * chunks * 2;
  // values: 16 at a time
  bool nan = false;
  for (int i = threadIdx.x; i < chunks; i += kThreads) {
    const int h = i / CPT, slot = (i % CPT) / CPR;
    const long long pos = (long long)start + slot;
    const bool use = slot < nk && pos >= 0 && pos < a.max_pos;
    const uint4 v = use ? __ldg(vp + i) : zero;
    const float s = __ldg(a.v_scale + (size_t)phys * a.Hkv + h);
    nan |= has_nan(v.x) || has_nan(v.y) || has_nan(v.z) || has_nan(v.w);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 x = ptx::e4m3x4_to_f4(in[w]);
      o[2 * w] = ptx::pack_bf16(use ? x.x * s : 0.f, use ? x.y * s : 0.f);
      o[2 * w + 1] = ptx::pack_bf16(use ? x.z * s : 0.f, use ? x.w * s : 0.f);
    }
    vo[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    vo[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  // keys: a thread holds 8 rotary pairs of a row
  constexpr int PPR = D / 16;  // threads of a row
  bool over = false;
  for (int i = threadIdx.x; i < a.Hkv * 16 * PPR; i += kThreads) {
    const int h = i / (16 * PPR), slot = (i / PPR) % 16, f0 = (i % PPR) * 8;
    const long long pos = (long long)start + slot;
    const bool use = slot < nk && pos >= 0 && pos < a.max_pos;
    const size_t row = (size_t)(h * 16 + slot) * D;  // first byte of the key in its block
    uint4 xo = zero, yo = zero;
    if (use) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(kp) + row + f0));
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(kp) + row + D / 2 + f0));
      const float s = __ldg(a.k_scale + (size_t)phys * a.Hkv + h);
      const float* t = a.cos_sin + (size_t)pos * D + f0;
      uint32_t wx[4], wy[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(t) + u);
        const float4 sn = __ldg(reinterpret_cast<const float4*>(t + D / 2) + u);
        const float4 p = ptx::e4m3x4_to_f4(u ? x.y : x.x), q = ptx::e4m3x4_to_f4(u ? y.y : y.x);
        const float px = p.x * s, py = p.y * s, pz = p.z * s, pw = p.w * s;
        const float qx = q.x * s, qy = q.y * s, qz = q.z * s, qw = q.w * s;
        wx[2 * u] = ptx::pack_f16(px * c.x - qx * sn.x, py * c.y - qy * sn.y);
        wx[2 * u + 1] = ptx::pack_f16(pz * c.z - qz * sn.z, pw * c.w - qw * sn.w);
        wy[2 * u] = ptx::pack_f16(qx * c.x + px * sn.x, qy * c.y + py * sn.y);
        wy[2 * u + 1] = ptx::pack_f16(qz * c.z + pz * sn.z, qw * c.w + pw * sn.w);
      }
      uint32_t watch = 0u;  // fp16 overflow
#pragma unroll
      for (int w = 0; w < 4; ++w) watch = ptx::watch_h2(ptx::watch_h2(watch, wx[w]), wy[w]);
      over |= watch != 0u;
      xo = make_uint4(wx[0], wx[1], wx[2], wx[3]);
      yo = make_uint4(wy[0], wy[1], wy[2], wy[3]);
    }
    ko[(row + f0) / 8] = xo;
    ko[(row + D / 2 + f0) / 8] = yo;
  }
  if (over) atomicOr(a.err, kErrRange);
  if (__syncthreads_or(nan)) {  // rare: NaN values; what is written again was written before the barrier
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
      const int h = i / CPT, slot = (i % CPT) / CPR;
      const long long pos = (long long)start + slot;
      const uint4 v = slot < nk && pos >= 0 && pos < a.max_pos ? __ldg(vp + i) : zero;
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      for (int e = 0; e < 16; ++e) {
        if (((in[e / 4] >> (8 * (e % 4))) & 0x7fu) != 0x7fu) continue;
        a.v_out[(to * chunks + i) * 16 + e] = 0;
        a.k_out[to * chunks * 16 + (size_t)(h * 16 + slot) * D] = 0x7e00;  // several write the same
      }
    }
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
