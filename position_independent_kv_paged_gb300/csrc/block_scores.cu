// The cheap score that block selection ranks by: for each block of a request's table and each kv head
//   score[r][g][b] = max over the query heads h of g of  scale * (R_t q_h) . (R_b m),
// with t the query's position, b the block's start and m the block's summary (block_means.cu): the largest mean score
// that a query head gives the block's keys.  Blocks past the request's length, with an id outside the pool or a start
// outside the table, get -infinity; a NaN product makes the block's score NaN.
//
// The ranking shows errors, so products have fp32's precision: both operands are split into two tf32 parts, x = x1 + x2
// with x1 the upper 11 bits, and x1 q1 + (x1 q2 + x2 q1) leaves out 2^-22 of a product.  The sums of the x1 q1 are cut
// into four chains that meet in fp32: the tensor core's own additions truncate.
//
// A summary is 1 / 32 of a block's keys and values, so this reads that part of what attention would, and the latency of
// loads and dependent instructions bounds it: 168 registers leave 12 warps an SM (10 active), which use 37 to 41 % of the
// issue slots.  Widening, rotating and splitting a summary cost about 490 instructions for 16 blocks and a kv head, whatever
// the number of query heads.  64 requests x 512 blocks, 8 kv heads, 4 query heads each: 21 us (floor 1.9 us); 8 x 8192,
// 8 heads each: 39 us (packed fp32 arithmetic on the scalar pipes took 27 and 60: there each query head costs as much
// again as the products do here for eight).
//
// A warp takes 16 blocks (the rows of the product) through the kv heads of its CTA: the cosines and sines of the
// blocks' starts stay in registers, and the next head's summaries load, a chunk at a time, as soon as this one's are
// widened (all of them after the last chunk: 22 and 42 us).  A lane holds 8-element
// chunks of the rotary pairs of two rows, x and y alike; which of its elements form a step of the contraction is free,
// as long as the query's are in the same places (they are stored in that order, each lane's 16 bytes next to its
// neighbour's).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace minipic {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;  // blocks of a warp's step
constexpr unsigned FULL = 0xffffffffu;

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ uint32_t lo(uint64_t v) { return (uint32_t)v; }
__device__ __forceinline__ uint32_t hi(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) { return ((uint64_t)y << 32) | x; }

// Eight consecutive elements, and as packed fp32 pairs.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void widen(uint64_t (&x)[4]) const {
    if constexpr (sizeof(T) == 4) {
      x[0] = pair(v[0].x, v[0].y);
      x[1] = pair(v[0].z, v[0].w);
      x[2] = pair(v[1].x, v[1].y);
      x[3] = pair(v[1].z, v[1].w);
    } else {
      x[0] = ptx::bf2_to_f2(v[0].x);
      x[1] = ptx::bf2_to_f2(v[0].y);
      x[2] = ptx::bf2_to_f2(v[0].z);
      x[3] = ptx::bf2_to_f2(v[0].w);
    }
  }
};
// Element e (of 8) of two rows, widened to fp32, as a pair: with (x, y) of rows g8 and g8 + 8 in one, the pairs of two
// elements are a step's operand of the tensor core as they lie (pairs of one row's elements took 250 moves a step).
__device__ __forceinline__ uint64_t two_rows(const Raw8<float>& a, const Raw8<float>& b, int e) {
  auto at = [](const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); };
  return pair(at(a.v[e >> 2], e & 3), at(b.v[e >> 2], e & 3));
}
__device__ __forceinline__ uint64_t two_rows(const Raw8<__nv_bfloat16>& a, const Raw8<__nv_bfloat16>& b, int e) {
  auto at = [](const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); };
  const uint32_t x = at(a.v[0], e >> 1), y = at(b.v[0], e >> 1);
  return e & 1 ? pair(x & 0xffff0000u, y & 0xffff0000u) : pair(x << 16, y << 16);
}

// Floats of shared memory that one kv head's queries take: two parts of NT column tiles of 8 heads.
template <int D, int NT>
constexpr int kHeadFloats = 2 * NT * 8 * D;

// CTAs of an SM.  Two leave 255 registers: fp32 summaries or two column tiles at d 128 spill with three (64 x 512 blocks,
// 8 kv heads: fp32 with 4 heads each 34.9 us against 23.0, with 16 52.3 and 33.2, bf16 with 16 35.0 and 29.5); the others
// do not, and want the warps (bf16 with 4 heads, d 64: 12.0 us and 14.7).
template <typename T, int D, int NT>
constexpr int kCtas = D == 128 && (sizeof(T) == 4 || NT == 2) ? 2 : 3;

// Grid: ranges of blocks, ranges of heads_per kv heads, requests.  NT: column tiles of 8 query heads.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtas<T, D, NT>) block_scores_kernel(const ScoresArgs a, const int heads_per) {
  constexpr int NC = D / 64;  // chunks of 8 + 8 elements of a lane and row
  // [kv head][column tile][x, y][chunk][quarter of a chunk pair][part][lane][4]
  extern __shared__ __align__(16) float sq[];
  const int r = blockIdx.z, lane = threadIdx.x & 31, g8 = lane >> 2, tig = lane & 3;
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
  const uint64_t scale = ptx::f2(a.scale, a.scale);
  const int* tab = a.block_tables + (size_t)r * mb;
  const int* sta = a.block_starts + (size_t)r * mb;
  const long long warps = (long long)gridDim.x * kWarps;
  long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int phys[2], start[2];
  auto entries = [&](long long w) {  // of rows g8 and g8 + 8
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const long long b = w * kRows + 8 * u + g8;
      phys[u] = -1;
      start[u] = 0;
      if (b < n) {
        phys[u] = __ldg(tab + b);
        start[u] = __ldg(sta + b);
      }
    }
  };
  entries(w);
  if (n > 0) {  // the rotated queries, eight pairs a thread (columns past the group hold anything: their sums are dropped)
    const T* q = static_cast<const T*>(a.q) + ((size_t)r * a.Hq + (size_t)g0 * G) * D;
    for (int i = threadIdx.x; i < n_heads * G * (D / 16); i += kThreads) {
      const int ch = i % (D / 16), head = i / (D / 16), g = head / G, col = head - g * G;  // chunk: lane's tig + 4 * its own
      Raw8<T> qx, qy;
      Raw8<float> rc, rs;
      qx.load(q + head * D + 8 * ch);
      qy.load(q + head * D + D / 2 + 8 * ch);
      rc.load(a.cos_sin + (size_t)t * D + 8 * ch);
      rs.load(a.cos_sin + (size_t)t * D + D / 2 + 8 * ch);
      uint64_t x[4], y[4], c[4], s[4];
      qx.widen(x);
      qy.widen(y);
      rc.widen(c);
      rs.widen(s);
      float* p = sq + g * kHeadFloats<D, NT> + ((col / 8 * 2 * NC + ch / 4) * 2 * 2) * 128 + ((col & 7) * 4 + ch % 4) * 4;
#pragma unroll
      for (int half = 0; half < 2; ++half, p += NC * 2 * 2 * 128) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t z = half ? ptx::fma2(x[e], s[e], ptx::mul2(y[e], c[e]))
                                  : ptx::sub2(ptx::mul2(x[e], c[e]), ptx::mul2(y[e], s[e]));
          v[2 * e] = __uint_as_float(lo(z));
          v[2 * e + 1] = __uint_as_float(hi(z));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float4 v1, v2;
          float* f1 = reinterpret_cast<float*>(&v1);
          float* f2 = reinterpret_cast<float*>(&v2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f1[e] = ptx::round_tf32(v[4 * k + e]);
            f2[e] = ptx::round_tf32(v[4 * k + e] - f1[e]);
          }
          *reinterpret_cast<float4*>(p + 2 * k * 128) = v1;
          *reinterpret_cast<float4*>(p + (2 * k + 1) * 128) = v2;
        }
      }
    }
  }
  __syncthreads();
  float* out = a.scores + ((size_t)r * a.Hkv + g0) * mb;
  for (; w * kRows < mb; w += warps) {
    const long long b0 = w * kRows;
    if (b0 >= n) {  // nothing but blocks past the length
      for (int i = lane; i < kRows * n_heads; i += 32)
        if (b0 + i % kRows < mb) out[(size_t)(i / kRows) * mb + b0 + i % kRows] = -CUDART_INF_F;
      continue;
    }
    bool ok[2];
    const T* m[2];
    // cosines and sines of rows g8 and g8 + 8, times the scale (a product: as mere pairs of loaded values they would be put
    // together again for every head, 190 moves a step)
    uint64_t c[NC][8], s[NC][8];
    Raw8<float> rc[2][NC], rs[2][NC];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool id = phys[u] >= 0 && phys[u] < a.num_blocks, in = start[u] >= 0 && start[u] < a.max_pos;
      ok[u] = id && in;
      if (b0 + 8 * u + g8 < n && !ok[u] && g0 == 0 && tig == 0) atomicOr(a.err, id ? kErrPosition : kErrBlockId);
      // nothing usable: the first summary and row, whose product is not looked at
      m[u] = static_cast<const T*>(a.means) + ((size_t)(ok[u] ? phys[u] : 0) * a.Hkv + g0) * D + 8 * tig;
      const float* cs = a.cos_sin + (size_t)(ok[u] ? start[u] : 0) * D + 8 * tig;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        rc[u][k].load(cs + 32 * k);
        rs[u][k].load(cs + D / 2 + 32 * k);
      }
    }
    Raw8<T> mx[2][NC], my[2][NC];
    auto summaries = [&](int k) {  // chunk k of both rows
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (a.num_blocks > 0) {
          mx[u][k].load(m[u] + 32 * k);
          my[u][k].load(m[u] + D / 2 + 32 * k);
        }
    };
#pragma unroll
    for (int k = 0; k < NC; ++k) summaries(k);
    m[0] += D;
    m[1] += D;
    entries(w + warps);
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[k][e] = ptx::mul2(two_rows(rc[0][k], rc[1][k], e), scale);
        s[k][e] = ptx::mul2(two_rows(rs[0][k], rs[1][k], e), scale);
      }
#pragma unroll 1
    for (int g = 0; g < n_heads; ++g) {
      float acc[NT][4][4], low[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][0][e] = acc[nt][1][e] = acc[nt][2][e] = acc[nt][3][e] = low[nt][e] = 0.f;
      const float* bq = sq + g * kHeadFloats<D, NT> + lane * 4;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        uint64_t v[2][8];  // [x, y][element]
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t x = two_rows(mx[0][k], mx[1][k], e), y = two_rows(my[0][k], my[1][k], e);
          v[0][e] = ptx::sub2(ptx::mul2(x, c[k][e]), ptx::mul2(y, s[k][e]));
          v[1][e] = ptx::fma2(x, s[k][e], ptx::mul2(y, c[k][e]));
        }
        if (g + 1 < n_heads) summaries(k);  // the next head's, as soon as these are widened
        if (k == NC - 1) {
          m[0] += D;
          m[1] += D;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float4 b1[NT], b2[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float* p = bq + ((((nt * 2 + half) * NC + k) * 2 + j) * 2) * 128;
              b1[nt] = *reinterpret_cast<const float4*>(p);
              b2[nt] = *reinterpret_cast<const float4*>(p + 128);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint64_t h[2], d[2];  // elements 4 j + 2 e and the next
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                h[u] = v[half][4 * j + 2 * e + u] & 0xffffe000ffffe000ull;
                d[u] = ptx::sub2(v[half][4 * j + 2 * e + u], h[u]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t p0 = __float_as_uint(e ? b1[nt].z : b1[nt].x), p1 = __float_as_uint(e ? b1[nt].w : b1[nt].y);
                const uint32_t r0 = __float_as_uint(e ? b2[nt].z : b2[nt].x), r1 = __float_as_uint(e ? b2[nt].w : b2[nt].y);
                ptx::mma_tf32_1688(acc[nt][2 * half + j], lo(h[0]), hi(h[0]), lo(h[1]), hi(h[1]), p0, p1);
                ptx::mma_tf32_1688(low[nt], lo(h[0]), hi(h[0]), lo(h[1]), hi(h[1]), r0, r1);
                ptx::mma_tf32_1688(low[nt], lo(d[0]), hi(d[0]), lo(d[1]), hi(d[1]), p0, p1);
              }
            }
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // rows g8, g8 + 8; columns 2 tig, 2 tig + 1 of each tile
        float best = -CUDART_INF_F;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int e = 2 * u + j;
            const float sum = ((acc[nt][0][e] + acc[nt][1][e]) + (acc[nt][2][e] + acc[nt][3][e])) + low[nt][e];
            if (8 * nt + 2 * tig + j < G) best = max_nan(best, sum);
          }
        best = max_nan(best, __shfl_xor_sync(FULL, best, 1));
        best = max_nan(best, __shfl_xor_sync(FULL, best, 2));
        const long long b = b0 + 8 * u + g8;
        if (tig == 0 && b < mb) out[(size_t)g * mb + b] = ok[u] ? best : -CUDART_INF_F;
      }
    }
  }
}

template <typename T, int D, int NT>
cudaError_t launch_t(const ScoresArgs& a, int num_sms, cudaStream_t s) {
  static bool done[64] = {false};
  constexpr int head_bytes = kHeadFloats<D, NT> * 4;
  constexpr int most_heads = 65536 / head_bytes;  // three CTAs of 64 KB an SM
  const cudaError_t e = set_smem_once(block_scores_kernel<T, D, NT>, most_heads * head_bytes, done);
  if (e != cudaSuccess) return e;
  // Two steps or more a resident warp in all: more heads a step read the starts' table rows less often, fewer even out
  // the last wave (64 x 512 blocks, 8 heads: 1, 2, 4 and 8 heads a step took 31, 25, 22 and 24 us; 8 x 8192: 59, 50, 44
  // and 42; before the summaries loaded earlier).
  const long long steps = ((long long)a.max_blocks + kRows - 1) / kRows * a.batch, ctas = (long long)kCtas<T, D, NT> * num_sms;
  long long heads_per = steps * a.Hkv / (2 * ctas * kWarps);
  heads_per = heads_per < 1 ? 1 : (heads_per > most_heads ? most_heads : heads_per);
  if (heads_per > a.Hkv) heads_per = a.Hkv;
  const long long gy = (a.Hkv + heads_per - 1) / heads_per;
  heads_per = (a.Hkv + gy - 1) / gy;  // as even as can be
  // one wave of CTAs that walk their request, where that leaves each request several; else a step a warp
  const long long most = ((long long)a.max_blocks + kRows * kWarps - 1) / (kRows * kWarps), wave = ctas / (gy * a.batch);
  const long long gx = wave >= 8 && wave < most ? wave : most;
  const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)a.batch);
  block_scores_kernel<T, D, NT><<<grid, kThreads, (size_t)heads_per * head_bytes, s>>>(a, (int)heads_per);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const ScoresArgs& a, int num_sms, cudaStream_t s) {
  if (a.D == 128) return a.G > 8 ? launch_t<T, 128, 2>(a, num_sms, s) : launch_t<T, 128, 1>(a, num_sms, s);
  return a.G > 8 ? launch_t<T, 64, 2>(a, num_sms, s) : launch_t<T, 64, 1>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_block_scores(const ScoresArgs& a, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_d<__nv_bfloat16>(a, num_sms, s) : launch_d<float>(a, num_sms, s);
}

}  // namespace minipic
