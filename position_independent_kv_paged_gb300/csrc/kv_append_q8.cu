// Appending new tokens to an 8-bit position-free cache: unrotated keys and
// values are stored as e4m3 with one scale per (block, kv head), K and V apart.
//
// Scale of a tile (block, head), with x the rows this call adds to it:
//   s = 2^k, the least k >= -100 with max |x| <= 448 * 2^k,
// and a tile that already holds rows (the call starts inside the block) keeps
// max(s_old, s); when that grows, its earlier rows are re-rounded to the new
// scale.  e4m3 has the same relative precision at every exponent, so a power
// of two loses nothing against max|x| / 448, makes x / s exact, and re-rounding
// an old row changes only values that fall into e4m3's subnormals.
//
// One warp per tile: the new rows (at most 16 x d) are read once with 16-byte
// loads, all issued before the first use, kept in registers through the
// maximum, and written as 8 e4m3 bytes per lane.  Nothing crosses warps.
// Bound by memory for chunks (3 bytes a value for bf16 rows): 16 chunks of 1024 to
// 2048 tokens, 4 heads, d 128 (75 MB): 12.4 us with the pools in L2, 16.7 us from
// cold caches; a decode step's append is one launch's latency, 3.1 us.
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace minipic {
namespace {

constexpr int kWarps = 4;
constexpr int kMinExp = -100;
constexpr unsigned FULL = 0xffffffffu;

// 2^k for -126 <= k <= 127
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// Least 2^k, k >= kMinExp, with amax <= 448 * 2^k (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - 127, m = bits & 0x7fffff;
  const int k = m <= 0x600000 ? e - 8 : e - 7;
  return pow2(k < kMinExp ? kMinExp : k);
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 8 consecutive values of a row
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = __ldcs(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  // largest |x|, an infinity included, NaN left out
  __device__ __forceinline__ float amax() const {
    __nv_bfloat162 m = __habs2(pair(v.x));
    m = __hmax2(__hmax2(m, __habs2(pair(v.y))), __hmax2(__habs2(pair(v.z)), __habs2(pair(v.w))));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
    return (i & 1) ? ptx::bf_hi(w) : ptx::bf_lo(w);
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs(static_cast<const float4*>(p));
    b = __ldcs(static_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float amax() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
  }
  __device__ __forceinline__ float get(int i) const {
    const float4& q = i < 4 ? a : b;
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_append_q8_kernel(AppendQ8Args a) {
  constexpr int LPR = D / 8;       // lanes of a row
  constexpr int RPP = 32 / LPR;    // rows of a pass
  constexpr int NP = 16 / RPP;     // passes of a tile
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int t0 = a.cu_new[r], t1 = a.cu_new[r + 1];
  if (t1 <= t0) return;
  const int js = a.kv_start[r];
  if (t0 < 0 || t1 > a.total_new || js < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrSeqLen);
    return;
  }
  const long long jend = (long long)js + (t1 - t0);
  const int b0 = js >> 4;
  const long long tiles = (((jend - 1) >> 4) - b0 + 1) * 2 * a.Hkv;  // (block, head, K or V)
  const int sub = lane / LPR, col = (lane % LPR) * 8;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < tiles;
       u += (long long)gridDim.x * kWarps) {
    const bool is_v = u & 1;
    const int h = (int)((u >> 1) % a.Hkv);
    const long long blk = b0 + (u >> 1) / a.Hkv;
    if (blk >= a.max_blocks) {
      if (lane == 0) atomicOr(a.err, kErrSeqLen);
      continue;
    }
    const int phys = __ldg(a.block_tables + (size_t)r * a.max_blocks + blk);
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) atomicOr(a.err, kErrBlockId);
      continue;
    }
    const long long j0 = blk == b0 ? js : blk * 16;
    const int n = (int)((jend < blk * 16 + 16 ? jend : blk * 16 + 16) - j0);  // rows added, 1 .. 16
    const int s0 = (int)(j0 - blk * 16);                                     // rows already there
    const size_t tile = (size_t)phys * a.Hkv + h;
    float* scale = (is_v ? a.v_scale : a.k_scale) + tile;
    uint8_t* pool = (is_v ? a.v_pool : a.k_pool) + tile * (16 * D);
    const T* src = static_cast<const T*>(is_v ? a.v_new : a.k_new) + ((size_t)(t0 + (j0 - js)) * a.Hkv + h) * D + col;
    const float old = s0 ? *scale : 0.f;

    Row8<T> x[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = p * RPP + sub;
      if (i < n) x[p].load(src + (size_t)i * a.Hkv * D);
      else x[p].clear();
    }
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) amax = fmaxf(amax, x[p].amax());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
    if (amax > 3.402823466e38f) {  // an infinity sets no scale: the largest finite value does
      if (lane == 0) atomicOr(a.err, kErrRange);
      amax = 0.f;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = fabsf(x[p].get(e));
          if (y <= 3.402823466e38f) amax = fmaxf(amax, y);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
    }
    float s = scale_for(amax);
    if (s0) {
      s = fmaxf(old, s);
      if (s > old) {  // the earlier rows move to the larger scale
        const float f = __fdiv_rn(old, s);
#pragma unroll 1
        for (int i = sub; i < s0; i += RPP) {
          uint2* q = reinterpret_cast<uint2*>(pool + i * D + col);
          const uint2 w = *q;
          const float4 u = ptx::e4m3x4_to_f4(w.x), v = ptx::e4m3x4_to_f4(w.y);
          *q = make_uint2(pack4(u.x * f, u.y * f, u.z * f, u.w * f), pack4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
      }
    }
    if ((__float_as_int(s) & 0x7fffff) == 0) {  // a power of two: x / s is the exact product with 1 / s
      const float inv = __fdiv_rn(1.f, s);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = p * RPP + sub;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[p].get(e) * inv;
        if (i < n)
          *reinterpret_cast<uint2*>(pool + (s0 + i) * D + col) =
              make_uint2(pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7]));
      }
    } else {  // another scale that the caller's block had
#pragma unroll 1
      for (int i = sub; i < n; i += RPP) {
        Row8<T> z;
        z.load(src + (size_t)i * a.Hkv * D);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(z.get(e), s);
        *reinterpret_cast<uint2*>(pool + (s0 + i) * D + col) =
            make_uint2(pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7]));
      }
    }
    if (lane == 0) *scale = s;
  }
}

template <typename T>
cudaError_t launch_t(const AppendQ8Args& a, cudaStream_t s) {
  // tiles of one request: the blocks that max_new tokens touch at worst, x heads x 2
  const long long units = (((long long)a.max_new + 14) / 16 + 1) * a.Hkv * 2;
  long long gx = (units + kWarps - 1) / kWarps;
  if (gx > 65535) gx = 65535;  // grid-stride beyond this
  const dim3 grid((unsigned)gx, (unsigned)a.batch);
  if (a.D == 64) kv_append_q8_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>(a);
  else kv_append_q8_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_q8(const AppendQ8Args& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace minipic
