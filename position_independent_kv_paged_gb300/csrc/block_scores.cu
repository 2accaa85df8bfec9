// The cheap score that block selection ranks by: for each block of a request's table and each kv head
//   score[r][g][b] = max over the query heads h of g of  scale * (R_t q_h) . (R_b m),
// with t the query's position, b the block's start and m the block's summary (block_means.cu): the largest mean score
// that a query head gives the block's keys.  Blocks past the request's length, with an id outside the pool or a start
// outside the table, get -infinity; a NaN product makes the block's score NaN.
//
// fp32 throughout: the ranking shows errors.  A summary is 1 / 32 of a block's keys and values, so this reads that
// part of what attention would, and its instructions bound it: per (block, kv head) 3 d operations of rotation and 2 d
// a query head.  They run as packed fp32 pairs, on lanes that hold 8 + 8 elements of a summary's rotary pairs (D / 16
// lanes a summary, so a warp's load is whole lines), for two summaries at a time: each value of the rotated queries,
// read from shared memory, then serves two products.  A warp takes its blocks through all kv heads of the CTA, so the
// cosines and sines of a block's start are read once, and the next head's summaries while it works on one.  The query
// heads' partial sums are added across the lanes by halving: at each step a lane keeps half of the heads, so all heads
// together take few more exchanges than one alone would.
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
__device__ __forceinline__ float lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Eight consecutive elements as packed pairs.
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ void load8(const float* p, Raw8& v) {
  v.a = __ldg(reinterpret_cast<const uint4*>(p));
  v.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw8& v) { v.a = __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) { return ((uint64_t)y << 32) | x; }
template <typename T>
__device__ __forceinline__ void widen(const Raw8& v, uint64_t (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    x[0] = pair(v.a.x, v.a.y);
    x[1] = pair(v.a.z, v.a.w);
    x[2] = pair(v.b.x, v.b.y);
    x[3] = pair(v.b.z, v.b.w);
  } else {
    x[0] = ptx::bf2_to_f2(v.a.x);
    x[1] = ptx::bf2_to_f2(v.a.y);
    x[2] = ptx::bf2_to_f2(v.a.z);
    x[3] = ptx::bf2_to_f2(v.a.w);
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Query values that a CTA holds, at most (fp32, in shared memory).
constexpr int kQueryFloats = 64 * 128;

// NH: heads a pass holds sums for (a power of two).  Grid: ranges of blocks, ranges of heads_per kv heads, requests.
template <typename T, int D, int NH>
__global__ void __launch_bounds__(kThreads, 2) block_scores_kernel(const ScoresArgs a, const int heads_per) {
  constexpr int LPB = D / 16;       // lanes of a summary
  constexpr int SETS = 2;           // summaries of a lane
  constexpr int BPW = 32 / LPB;     // blocks of a warp and set
  constexpr int STEP = SETS * BPW;  // consecutive blocks of a warp
  // the rotated queries, [head][half, quarter of a lane's elements][lane of a summary][4]: the lanes' 16-byte reads are
  // consecutive
  __shared__ alignas(16) float sq[kQueryFloats];
  const int r = blockIdx.z, lane = threadIdx.x & 31;
  const int mb = a.max_blocks, G = a.G, g0 = blockIdx.y * heads_per, n_heads = min(heads_per, a.Hkv - g0);
  int L = a.seq_lens[r];
  int t = a.q_pos[r];
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  if (L < 0 || (long long)L > 16LL * mb) {
    if (threadIdx.x == 0 && first) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : (int)min(16LL * mb, 2147483632LL);
  }
  const int n = min((L >> 4) + ((L & 15) != 0), mb);
  if (n > 0 && (t < 0 || t >= a.max_pos)) {
    if (threadIdx.x == 0 && first) atomicOr(a.err, kErrPosition);
    t = 0;
  }
  const int e0 = 8 * (lane % LPB), sub = lane / LPB;
  const int* tab = a.block_tables + (size_t)r * mb;
  const int* sta = a.block_starts + (size_t)r * mb;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  int phys[SETS], start[SETS];
  auto entries = [&](long long w) {
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
      const long long b = w * STEP + u * BPW + sub;
      phys[u] = -1;
      start[u] = 0;
      if (b < n) {
        phys[u] = __ldg(tab + b);
        start[u] = __ldg(sta + b);
      }
    }
  };
  entries(w);
  if (n > 0) {
    const T* q = static_cast<const T*>(a.q) + ((size_t)r * a.Hq + (size_t)g0 * G) * D;
    for (int i = threadIdx.x; i < n_heads * G * (D / 2); i += kThreads) {
      const int h = i / (D / 2), e = i % (D / 2);
      const float c = __ldg(a.cos_sin + (size_t)t * D + e), s = __ldg(a.cos_sin + (size_t)t * D + D / 2 + e);
      const float x = to_f(q[h * D + e]), y = to_f(q[h * D + D / 2 + e]);
      float* p = sq + h * D + ((e >> 2 & 1) * LPB + (e >> 3)) * 4 + (e & 3);
      p[0] = fmaf(x, c, -y * s) * a.scale;
      p[D / 2] = fmaf(y, c, x * s) * a.scale;
    }
  }
  __syncthreads();
  float* out = a.scores + ((size_t)r * a.Hkv + g0) * mb;
  for (; w * STEP < mb; w += warps) {
    const long long b0 = w * STEP;
    if (b0 >= n) {  // nothing but blocks past the length
      for (int i = lane; i < STEP * n_heads; i += 32)
        if (b0 + i % STEP < mb) out[(size_t)(i / STEP) * mb + b0 + i % STEP] = -CUDART_INF_F;
      continue;
    }
    bool ok[SETS];
    const T* m[SETS];
    Raw8 mx[SETS], my[SETS];
    uint64_t c[SETS][4], s[SETS][4];
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
      const bool id = phys[u] >= 0 && phys[u] < a.num_blocks, in = start[u] >= 0 && start[u] < a.max_pos;
      ok[u] = id && in;
      if (b0 + u * BPW + sub < n && !ok[u] && g0 == 0 && lane % LPB == 0) atomicOr(a.err, id ? kErrPosition : kErrBlockId);
      // nothing usable: the first summary and row, whose product is not looked at
      m[u] = static_cast<const T*>(a.means) + ((size_t)(ok[u] ? phys[u] : 0) * a.Hkv + g0) * D + e0;
      const float* cs = a.cos_sin + (size_t)(ok[u] ? start[u] : 0) * D + e0;
      Raw8 raw;
      load8(cs, raw);
      widen<float>(raw, c[u]);
      load8(cs + D / 2, raw);
      widen<float>(raw, s[u]);
    }
    auto summaries = [&] {
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
        if (a.num_blocks > 0) {
          load8(m[u], mx[u]);
          load8(m[u] + D / 2, my[u]);
        }
        m[u] += D;
      }
    };
    summaries();
    entries(w + warps);
#pragma unroll 1
    for (int g = 0; g < n_heads; ++g) {
      uint64_t x[SETS][4], y[SETS][4];
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
        widen<T>(mx[u], x[u]);
        widen<T>(my[u], y[u]);
      }
      if (g + 1 < n_heads) summaries();
#pragma unroll
      for (int u = 0; u < SETS; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t v = x[u][e];
          x[u][e] = ptx::sub2(ptx::mul2(v, c[u][e]), ptx::mul2(y[u][e], s[u][e]));
          y[u][e] = ptx::fma2(v, s[u][e], ptx::mul2(y[u][e], c[u][e]));
        }
      float best[SETS];
#pragma unroll
      for (int u = 0; u < SETS; ++u) best[u] = -CUDART_INF_F;
#pragma unroll 1
      for (int h0 = 0; h0 < G; h0 += NH) {
        float dot[SETS][NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float* p = sq + (g * G + min(h0 + h, G - 1)) * D + 4 * (lane % LPB);
          uint64_t acc[SETS];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(p + half * (D / 2) + 4 * LPB * k);
#pragma unroll
              for (int u = 0; u < SETS; ++u) {
                const uint64_t* v = half ? y[u] : x[u];
                acc[u] = half == 0 && k == 0 ? ptx::mul2(qv.x, v[0]) : ptx::fma2(qv.x, v[2 * k], acc[u]);
                acc[u] = ptx::fma2(qv.y, v[2 * k + 1], acc[u]);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < SETS; ++u) dot[u][h] = lo(acc[u]) + hi(acc[u]);
        }
        int left = NH;  // heads whose sums a lane still holds
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1) {
          const bool up = lane & o;
          if (left > 1) left >>= 1;  // it keeps the upper or the lower half of them
          const bool halve = NH > 1 && left * 2 * (LPB / 2 / o) <= NH;
#pragma unroll
          for (int u = 0; u < SETS; ++u) {
            if (halve) {
#pragma unroll
              for (int h = 0; h < (NH + 1) / 2; ++h)
                if (h < left) {
                  const float mine = up ? dot[u][h + left] : dot[u][h], other = up ? dot[u][h] : dot[u][h + left];
                  dot[u][h] = mine + __shfl_xor_sync(FULL, other, o);
                }
            } else {
              dot[u][0] += __shfl_xor_sync(FULL, dot[u][0], o);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < SETS; ++u)
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (h < left) best[u] = max_nan(best[u], dot[u][h]);  // heads past the group repeat its last
      }
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1)
          if (NH * o >= LPB) best[u] = max_nan(best[u], __shfl_xor_sync(FULL, best[u], o));  // lanes of other heads
        const long long b = b0 + u * BPW + sub;
        if (lane % LPB == 0 && b < mb) out[(size_t)g * mb + b] = ok[u] ? best[u] : -CUDART_INF_F;
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_d(const ScoresArgs& a, int num_sms, cudaStream_t s) {
  int heads_per = kQueryFloats / (a.G * D);  // at least 4
  if (heads_per > a.Hkv) heads_per = a.Hkv;
  const long long per = (kThreads / 32) * 2 * (32 / (D / 16));  // blocks of a CTA's pass
  long long gx = (a.max_blocks + per - 1) / per;
  const long long gy = (a.Hkv + heads_per - 1) / heads_per, rows = gy * a.batch, most = (8LL * num_sms + rows - 1) / rows;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)a.batch);
  if (a.G <= 1) block_scores_kernel<T, D, 1><<<grid, kThreads, 0, s>>>(a, heads_per);
  else if (a.G <= 2) block_scores_kernel<T, D, 2><<<grid, kThreads, 0, s>>>(a, heads_per);
  else if (a.G <= 4) block_scores_kernel<T, D, 4><<<grid, kThreads, 0, s>>>(a, heads_per);
  else block_scores_kernel<T, D, 8><<<grid, kThreads, 0, s>>>(a, heads_per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_scores(const ScoresArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.D == 128) return bf16 ? launch_d<B, 128>(a, num_sms, s) : launch_d<float, 128>(a, num_sms, s);
  return bf16 ? launch_d<B, 64>(a, num_sms, s) : launch_d<float, 64>(a, num_sms, s);
}

}  // namespace minipic
