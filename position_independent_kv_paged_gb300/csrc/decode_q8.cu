// Decode attention over the 8-bit position-free cache, tensor-core form
// (bf16 query and output; the f32 form is in decode_simt.cu).
//
// Keys and values are e4m3 bytes with one scale per (block, kv head); keys are
// unrotated and rotated here at pi(j) = start[r][block] + slot (MiniPIC summary,
// gist.science 2606.13126, section 2.1).
//
// Work: one CTA = (split, kv head, request); each of its warps owns every NW-th
// 16-key block of the split and runs its own TMA ring.  A (block, head) tile is
// 16 d contiguous bytes; the tensor map sees the pool as lines of 128 bytes (one
// key at d 128, two at d 64) and swizzles them, so that the key-row reads and
// the transposing reads of V are free of bank conflicts.  The fp16 cos | sin row
// of the block's query rotation comes with them.
//
// Per block, with t the query's position, b the block's start, s the slot:
//   score = (R_{t-b} q) . (R_s k8) * (k scale) * softmax scale
// e4m3 widens to fp16 exactly; R_s is constant per lane, R_{t-b} q is formed once
// per block, both in packed fp16, and S^T = K' Q'^T, O^T += V^T P^T run as
// mma.sync m16n8k16 with fp32 accumulation (keys, then head dims, as M; up to 8
// query heads as N, so a group of 8 wastes nothing and the operands come from
// registers: the tcgen05 form needs M >= 64 and would take the widened, rotated
// keys through shared memory again).
//  - The query is scaled by a power of two per head to a largest element in
//    [1, 2) first, so that fp16 holds it whatever its size.
//  - V bytes stay unscaled in the product; the block's scale rides on P.  P is
//    2^(s + log2 vscale - mt + 7) in fp16 with a running reference mt of its own
//    (so blocks whose scales differ by any factor keep fp16's full precision
//    where they matter, and a weight 2^-31 of the largest is still above zero),
//    the denominator 2^(s - ms) in fp32.  Both references move only when a value
//    exceeds them by more than 2^8 (P then is below 2^15).
//  - A V fragment is widened from one transposing 16-bit read: its byte pairs
//    are two head dims of a key, so the even and odd dims become two rows of
//    the same M tile.
// Slots past the request's length, blocks with a bad id, keys past the table and
// zero-scale values are masked in the scores and cleared in V (P = 0 must not
// meet a NaN byte).
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace minipic {
namespace {

using ptx::U4;

constexpr int kWarps = 4;
constexpr int kMaxSplit = 512;                // split_blocks cap (planner)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;               // a reference moves when exceeded by 2^8
constexpr float kHead = 7.f;                  // P of a key at its reference is 2^7
constexpr float kMinLog = -100.f;             // log2 of the smallest value scale told apart from zero

template <int D, int NS>
struct Lay {
  static constexpr int TILE = 16 * D;              // bytes of one (block, head) tile of K or V
  static constexpr int LINES = TILE / 128;         // 128-byte lines of a tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int ROWB = 2 * D;               // one fp16 cos | sin row
  static constexpr int MT = D / 16;                // M tiles of O^T
  static constexpr int STAGES = kWarps * NS * STAGE;
  static constexpr int ROWS = STAGES;                           // [warp][stage] table rows
  static constexpr int META = ROWS + kWarps * NS * ROWB;        // [split block] int4
  static constexpr int BARS = META + kMaxSplit * 16;
  static constexpr int OST = D + 4;                             // padded row stride of the merge
  static constexpr int MERGE_W = (48 + 16 * OST) * 4;           // ms[16], l[16], mt[16], O[16][OST] of one warp
  static constexpr int MERGE = kWarps * MERGE_W;                // overlays stages, rows and meta
  static constexpr int TOTAL = (BARS + kWarps * NS * 8) > MERGE ? (BARS + kWarps * NS * 8) : MERGE;
};

// Slot held by MMA fragment row g (row g + 8 holds slot + 8): rows read together by a quarter warp differ in bit 2.
__device__ __forceinline__ int frag_slot(int g) { return (g >> 1) | ((g & 1) << 2); }

// Byte offset of 16-byte chunk c of key `key` in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t at(int key, int c) {
  if constexpr (D == 128) return (uint32_t)(key * 128 + ((c ^ (key & 7)) << 4));
  const int line = key >> 1;
  return (uint32_t)(line * 128 + ((((key & 1) * 4 + c) ^ (line & 7)) << 4));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// (x, y) rotated by the angle with cos c and sin s, two pairs at a time
__device__ __forceinline__ void rotate(uint32_t x, uint32_t y, uint32_t c, uint32_t s, uint32_t& xo, uint32_t& yo) {
  xo = u32(__hfma2(__hneg2(h2(y)), h2(s), __hmul2(h2(x), h2(c))));
  yo = u32(__hfma2(h2(x), h2(s), __hmul2(h2(y), h2(c))));
}

// |t - b| for any two 32-bit integers
__device__ __forceinline__ uint32_t distance(int t, int b) {
  return b > t ? (uint32_t)b - (uint32_t)t : (uint32_t)t - (uint32_t)b;
}

template <int D, int NT, bool WTS, int NS, int CPS>
__global__ void __launch_bounds__(kWarps * 32, CPS)
    decode_q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const DecodeArgs a) {
  using LY = Lay<D, NS>;
  constexpr int NW = kWarps;
  constexpr int NH = D / 32;  // 4-dim words of x (and of y) a thread holds per key: 4 at d 128, 2 at d 64
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - ptx::smem_addr(smem_raw));
  const uint32_t bar_base = sbase + LY::BARS;
  int4* meta = reinterpret_cast<int4*>(sgen + LY::META);

  const int split = blockIdx.x, hk = blockIdx.y, r = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, tig = lane & 3;
  const int G = a.G, mb = a.max_blocks;

  int L = a.seq_lens[r];
  const int Lmax = (int)min((long long)mb * 16, 2147483632LL);
  if (L < 0 || L > Lmax) {
    if (threadIdx.x == 0 && split == 0) atomicOr(a.err, kErrSeqLen);
    L = L < 0 ? 0 : Lmax;
  }
  const int nblk = (int)(((long long)L + 15) >> 4);
  const int n_valid = max(1, (nblk + a.split_blocks - 1) / a.split_blocks);
  if (split >= n_valid) return;
  const int b_begin = split * a.split_blocks;
  const int b_end = min(nblk, b_begin + a.split_blocks);
  const int span = b_end - b_begin;
  const int nmine = span > warp ? (span - warp + NW - 1) / NW : 0;
  int tq = a.q_pos[r];
  if (tq < 0 || tq >= a.max_pos) {
    if (threadIdx.x == 0 && split == 0) atomicOr(a.err, kErrPosition);
    tq = 0;
  }

  const uint16_t* cs16 = a.cs_f16;
  // lane 0: issue the k-th block of this warp into its stage (K, V, and the cos | sin row of |t - start|)
  auto issue_blk = [&](int k, int phys, int start) {
    const int stg = k % NS;
    const uint32_t bar = bar_base + (warp * NS + stg) * 8;
    const uint32_t dst = sbase + (warp * NS + stg) * LY::STAGE;
    if (phys < 0 || phys >= a.num_blocks) {
      ptx::mbar_arrive(bar);  // nothing to load; the consumer masks the block
      return;
    }
    const uint32_t ad = distance(tq, start);
    const bool row_ok = ad < (uint32_t)a.max_pos;
    ptx::mbar_arrive_expect_tx(bar, 2 * LY::TILE + (row_ok ? LY::ROWB : 0));
    const int y = (phys * a.Hkv + hk) * LY::LINES;
    ptx::tma_load_2d(dst, &kmap, 0, y, bar);
    ptx::tma_load_2d(dst + LY::TILE, &vmap, 0, y, bar);
    if (row_ok)
      ptx::bulk_load(sbase + LY::ROWS + (warp * NS + stg) * LY::ROWB, cs16 + (size_t)ad * D, LY::ROWB, bar);
  };
  {
    const int* bt = a.block_tables + (size_t)r * mb + b_begin;
    const int* bs = a.block_starts + (size_t)r * mb + b_begin;
    if (lane == 0) {
#pragma unroll
      for (int st = 0; st < NS; ++st) ptx::mbar_init(bar_base + (warp * NS + st) * 8, 1);
      ptx::fence_barrier_init();
      ptx::fence_proxy_async_smem();
      // the first copies start at once, from the tables in global memory
      const int pre = nmine < NS ? nmine : NS;
      for (int k = 0; k < pre; ++k) issue_blk(k, __ldg(bt + warp + NW * k), __ldg(bs + warp + NW * k));
    }
    // per block: id, start, score factor (softmax scale * log2 e * key scale), log2 of the value scale
    for (int i = threadIdx.x; i < span; i += NW * 32) {
      const int phys = __ldg(bt + i);
      float ks = 0.f, lv = -CUDART_INF_F;
      if (phys >= 0 && phys < a.num_blocks) {
        ks = __ldg(a.k_scale + (size_t)phys * a.Hkv + hk) * (a.scale * kLog2e);
        lv = log2f(__ldg(a.v_scale + (size_t)phys * a.Hkv + hk));
      }
      meta[i] = make_int4(phys, __ldg(bs + i), __float_as_int(ks), __float_as_int(lv));
    }
  }

  // this thread's key rows (slots ks0, ks0 + 8) and rotary pairs (f0 .. f0 + 4 NH - 1 with + d/2)
  const int ks0 = frag_slot(g8);
  const int f0 = 4 * NH * tig;

  // R_slot of both rows, fp16
  uint32_t rc[2][2 * NH], rs[2][2 * NH];
#pragma unroll
  for (int row = 0; row < 2; ++row) {
    const float* t = a.cos_sin + (size_t)min(ks0 + 8 * row, a.max_pos - 1) * D + f0;
#pragma unroll
    for (int e = 0; e < 2 * NH; ++e) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(t + 2 * e));
      const float2 sn = __ldg(reinterpret_cast<const float2*>(t + D / 2 + 2 * e));
      rc[row][e] = ptx::pack_f16(c.x, c.y);
      rs[row][e] = ptx::pack_f16(sn.x, sn.y);
    }
  }

  // unrotated queries of this thread's heads (g8 + 8 nt), scaled to fp16, and the power of two taken out of
  // the heads of its score columns (2 tig + j + 8 nt)
  uint32_t qx[NT][2 * NH], qy[NT][2 * NH];
  float qf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = 8 * nt + g8;
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)r * a.Hq + (size_t)hk * G + head) * D + f0;
    uint32_t wx[2 * NH], wy[2 * NH];
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * NH; ++e) {
      wx[e] = head < G ? __ldg(reinterpret_cast<const uint32_t*>(p) + e) : 0u;
      wy[e] = head < G ? __ldg(reinterpret_cast<const uint32_t*>(p + D / 2) + e) : 0u;
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(ptx::bf_lo(wx[e])), fabsf(ptx::bf_hi(wx[e]))),
                               fmaxf(fabsf(ptx::bf_lo(wy[e])), fabsf(ptx::bf_hi(wy[e])))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
    // exponent of the largest element (at most 127, an infinity's; a row of zeros or subnormals takes -126)
    int ex = (__float_as_int(amax) >> 23) - 127;
    ex = ex < -126 ? -126 : (ex > 126 ? 126 : ex);
    const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
    for (int e = 0; e < 2 * NH; ++e) {
      qx[nt][e] = ptx::pack_f16(ptx::bf_lo(wx[e]) * down, ptx::bf_hi(wx[e]) * down);
      qy[nt][e] = ptx::pack_f16(ptx::bf_lo(wy[e]) * down, ptx::bf_hi(wy[e]) * down);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      qf[nt][j] = __int_as_float((__shfl_sync(FULL, ex, (2 * tig + j) * 4) + 127) << 23);
  }

  float ms[NT][2], mt[NT][2], l[NT][2];
  float oacc[LY::MT][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    ms[nt][0] = ms[nt][1] = mt[nt][0] = mt[nt][1] = -CUDART_INF_F;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int m = 0; m < LY::MT; ++m)
#pragma unroll
      for (int k = 0; k < 4; ++k) oacc[m][nt][k] = 0.f;
  }

  __syncthreads();  // meta visible

  bool timed_out = false;
  int k_stop = nmine;
  for (int k = 0; k < nmine; ++k) {
    const int i = warp + NW * k;
    const int b = b_begin + i;
    const int stg = k % NS;
    const uint32_t kbase = sbase + (warp * NS + stg) * LY::STAGE;
    const uint32_t vbase = kbase + LY::TILE;
    const uint32_t rowb = sbase + LY::ROWS + (warp * NS + stg) * LY::ROWB;

    const int4 md = meta[i];
    const int phys = md.x, start = md.y;
    const float ksf = __int_as_float(md.z);
    float lv = __int_as_float(md.w);
    const bool ok = phys >= 0 && phys < a.num_blocks;
    const int nk = min(16, L - b * 16);
    bool v0 = ok && ks0 < nk, v1 = ok && ks0 + 8 < nk;
    if (!ok && lane == 0) atomicOr(a.err, kErrBlockId);
    const bool near = distance(tq, start) < (uint32_t)a.max_pos;
    if (ok && !(near && start >= 0 && start <= a.max_pos - nk)) {
      // keys whose position falls outside the table are masked
      const long long p0 = (long long)start + ks0;
      const bool in0 = p0 >= 0 && p0 < a.max_pos && near;
      const bool in1 = p0 + 8 >= 0 && p0 + 8 < a.max_pos && near;
      if (__any_sync(FULL, (v0 && !in0) || (v1 && !in1)) && lane == 0) atomicOr(a.err, kErrPosition);
      v0 = v0 && in0;
      v1 = v1 && in1;
    }
    const bool zero_v = lv < kMinLog;  // scale 0 (or below what is told apart from it): the values are zero
    lv = zero_v ? 0.f : lv;
    const bool part = !__all_sync(FULL, v0 && v1) || zero_v;

    const bool arrived = ptx::mbar_wait(bar_base + (warp * NS + stg) * 8, (uint32_t)((k / NS) & 1));
    if (!__all_sync(FULL, arrived)) {
      if (lane == 0) atomicOr(a.err, kErrTimeout);
      timed_out = true;
      k_stop = k;
      break;
    }

    // S^T = K' Q'^T, two accumulation chains (the x and the y halves of the pairs)
    float sx[NT][4], sy[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sx[nt][e] = sy[nt][e] = 0.f;
    {
      uint32_t kx[2][NH], ky[2][NH], cw[2 * NH], sw[2 * NH];
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        if constexpr (D == 128) {
          const U4 x = ptx::lds128(kbase + at<D>(ks0 + 8 * row, tig));
          const U4 y = ptx::lds128(kbase + at<D>(ks0 + 8 * row, tig + 4));
          kx[row][0] = x.x; kx[row][1] = x.y; kx[row][2] = x.z; kx[row][3] = x.w;
          ky[row][0] = y.x; ky[row][1] = y.y; ky[row][2] = y.z; ky[row][3] = y.w;
        } else {
          const uint2 x = ptx::lds64(kbase + at<D>(ks0 + 8 * row, tig >> 1) + 8 * (tig & 1));
          const uint2 y = ptx::lds64(kbase + at<D>(ks0 + 8 * row, 2 + (tig >> 1)) + 8 * (tig & 1));
          kx[row][0] = x.x; kx[row][1] = x.y;
          ky[row][0] = y.x; ky[row][1] = y.y;
        }
      }
      // cos and sin of t - start for this thread's frequencies; sin takes the angle's sign
      const uint32_t sgn = start > tq ? 0x80008000u : 0u;
#pragma unroll
      for (int u = 0; u < NH / 2; ++u) {
        const U4 c = ptx::lds128(rowb + 2 * f0 + 16 * u);
        const U4 s = ptx::lds128(rowb + D + 2 * f0 + 16 * u);
        cw[4 * u] = c.x; cw[4 * u + 1] = c.y; cw[4 * u + 2] = c.z; cw[4 * u + 3] = c.w;
        sw[4 * u] = s.x ^ sgn; sw[4 * u + 1] = s.y ^ sgn; sw[4 * u + 2] = s.z ^ sgn; sw[4 * u + 3] = s.w ^ sgn;
      }
#pragma unroll
      for (int w = 0; w < NH; ++w) {  // 4 pairs of each key row
        uint32_t x[2][2], y[2][2];    // [row][dims 0-1, 2-3]
#pragma unroll
        for (int row = 0; row < 2; ++row)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t hx = ptx::e4m3x2_to_h2(e ? kx[row][w] >> 16 : kx[row][w] & 0xffffu);
            const uint32_t hy = ptx::e4m3x2_to_h2(e ? ky[row][w] >> 16 : ky[row][w] & 0xffffu);
            rotate(hx, hy, rc[row][2 * w + e], rs[row][2 * w + e], x[row][e], y[row][e]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t bx[2], by[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            rotate(qx[nt][2 * w + e], qy[nt][2 * w + e], cw[2 * w + e], sw[2 * w + e], bx[e], by[e]);
          ptx::mma_f16_16816(sx[nt], x[0][0], x[1][0], x[0][1], x[1][1], bx[0], bx[1]);
          ptx::mma_f16_16816(sy[nt], y[0][0], y[1][0], y[0][1], y[1][1], by[0], by[1]);
        }
      }
    }

    // online softmax over the 16 keys, per head column
    uint32_t pb0[NT], pb1[NT];
    float sc[NT][4];
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = fminf(ksf * qf[nt][j], 3.4e38f);  // finite: a product of 0 stays 0
        sc[nt][j] = v0 ? (sx[nt][j] + sy[nt][j]) * f : -CUDART_INF_F;
        sc[nt][2 + j] = v1 ? (sx[nt][2 + j] + sy[nt][2 + j]) * f : -CUDART_INF_F;
        over |= fmaxf(sc[nt][j], sc[nt][2 + j]) > fminf(ms[nt][j], mt[nt][j] - lv) + kRescale;
      }
    if (__any_sync(FULL, over)) {  // rare: move the references, rescale what was summed
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float bm = fmaxf(sc[nt][j], sc[nt][2 + j]);
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 4));
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 8));
          bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, 16));
          const float msn = fmaxf(ms[nt][j], bm), mtn = fmaxf(mt[nt][j], bm + lv);
          const float cs = msn == -CUDART_INF_F ? 1.f : ex2(ms[nt][j] - msn);
          const float ct = mtn == -CUDART_INF_F ? 1.f : ex2(mt[nt][j] - mtn);
          ms[nt][j] = msn;
          mt[nt][j] = mtn;
          l[nt][j] *= cs;
#pragma unroll
          for (int m = 0; m < LY::MT; ++m) {
            oacc[m][nt][j] *= ct;
            oacc[m][nt][2 + j] *= ct;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float rs_ = ms[nt][j] == -CUDART_INF_F ? 0.f : ms[nt][j];
        const float rt = (mt[nt][j] == -CUDART_INF_F ? 0.f : mt[nt][j]) - lv - kHead;
        float e = ex2(sc[nt][j] - rs_) + ex2(sc[nt][2 + j] - rs_);
        pv[j] = ex2(sc[nt][j] - rt);
        pv[2 + j] = ex2(sc[nt][2 + j] - rt);
        l[nt][j] += e;
        if constexpr (WTS) {
          e += __shfl_xor_sync(FULL, e, 4);
          e += __shfl_xor_sync(FULL, e, 8);
          e += __shfl_xor_sync(FULL, e, 16);
          const int head = 8 * nt + 2 * tig + j;
          if (g8 == 0 && head < G)
            a.w_raw[(((size_t)r * a.Hkv + hk) * mb + b) * G + head] = e == 0.f ? -CUDART_INF_F : rs_ + log2f(e);
        }
      }
      pb0[nt] = ptx::movmatrix_trans(ptx::pack_f16(pv[0], pv[1]));  // keys 0..7
      pb1[nt] = ptx::movmatrix_trans(ptx::pack_f16(pv[2], pv[3]));  // keys 8..15
    }

    // O^T += V^T P^T, two M tiles (16-byte chunks) per read
    uint32_t klo = FULL, khi = FULL;  // which of keys (2 tig, 2 tig + 1) and + 8 count
    if (part) {
      const unsigned b0 = __ballot_sync(FULL, v0), b1 = __ballot_sync(FULL, v1);  // bit 4 g: fragment row g
      const int s0 = 8 * tig, s1 = 8 * tig + 4;                                  // rows 2 tig, 2 tig + 1
      klo = zero_v ? 0u : ((b0 >> s0) & 1u ? 0xffffu : 0u) | ((b0 >> s1) & 1u ? 0xffff0000u : 0u);
      khi = zero_v ? 0u : ((b1 >> s0) & 1u ? 0xffffu : 0u) | ((b1 >> s1) & 1u ? 0xffff0000u : 0u);
    }
    {
      const int mi = lane >> 3, rr = lane & 7;
      const int key = frag_slot(rr) + 8 * (mi & 1);
#pragma unroll
      for (int m = 0; m < LY::MT; m += 2) {
        uint32_t w[4];
        ptx::ldsm_x4_trans(vbase + at<D>(key, m + (mi >> 1)), w[0], w[1], w[2], w[3]);
        if (part) {
          w[0] &= klo;
          w[1] &= khi;
          w[2] &= klo;
          w[3] &= khi;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // bytes (key 0: dims 0, 1; key 1: dims 0, 1) -> dim 0 of both keys, dim 1 of both keys
          const uint32_t lo = __byte_perm(w[2 * u], 0u, 0x3120), hi = __byte_perm(w[2 * u + 1], 0u, 0x3120);
          const uint32_t a0 = ptx::e4m3x2_to_h2(lo & 0xffffu), a1 = ptx::e4m3x2_to_h2(lo >> 16);
          const uint32_t a2 = ptx::e4m3x2_to_h2(hi & 0xffffu), a3 = ptx::e4m3x2_to_h2(hi >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ptx::mma_f16_16816(oacc[m + u][nt], a0, a1, a2, a3, pb0[nt], pb1[nt]);
        }
      }
    }

    __syncwarp();
    if (lane == 0 && k + NS < nmine) {
      const int4 nx = meta[i + NW * NS];
      issue_blk(k + NS, nx.x, nx.y);
    }
  }

  if (timed_out && lane == 0) {
    // blocks k_stop .. k_stop + NS - 1 were issued and not consumed
    const int last = min(nmine, k_stop + NS);
    for (int k2 = k_stop; k2 < last; ++k2)
      ptx::mbar_wait(bar_base + (warp * NS + k2 % NS) * 8, (uint32_t)((k2 / NS) & 1), 100000000ull);
  }
  __syncthreads();  // every copy has landed and been read: the merge overlays the stages

  // per-warp state: ms[16], l[16], mt[16], O[16][OST]
  {
    float* w = reinterpret_cast<float*>(sgen + warp * LY::MERGE_W);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float s = l[nt][j];
        s += __shfl_xor_sync(FULL, s, 4);
        s += __shfl_xor_sync(FULL, s, 8);
        s += __shfl_xor_sync(FULL, s, 16);
        const int head = 8 * nt + 2 * tig + j;
        if (g8 == 0) {
          w[head] = ms[nt][j];
          w[16 + head] = s;
          w[32 + head] = mt[nt][j];
        }
#pragma unroll
        for (int m = 0; m < LY::MT; ++m) {
          float2 o = make_float2(oacc[m][nt][j], oacc[m][nt][2 + j]);
          *reinterpret_cast<float2*>(w + 48 + head * LY::OST + 16 * m + 2 * g8) = o;
        }
      }
  }
  __syncthreads();

  // the CTA's output of each head, already divided by its denominator: values no larger than V's
  const bool direct = n_valid == 1;
  for (int idx = threadIdx.x; idx < G * D; idx += NW * 32) {
    const int head = idx / D, dim = idx - head * D;
    float M = -CUDART_INF_F, T = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* p = reinterpret_cast<const float*>(sgen + w * LY::MERGE_W);
      M = fmaxf(M, p[head]);
      T = fmaxf(T, p[32 + head]);
    }
    float Ls = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* p = reinterpret_cast<const float*>(sgen + w * LY::MERGE_W);
      // a warp that saw no finite reference still hands on its NaNs
      Ls = fmaf(p[16 + head], p[head] == -CUDART_INF_F ? 1.f : exp2f(p[head] - M), Ls);
      O = fmaf(p[48 + head * LY::OST + dim], p[32 + head] == -CUDART_INF_F ? 1.f : exp2f(p[32 + head] - T), O);
    }
    const float up = T == -CUDART_INF_F ? 1.f : exp2f(T - kHead - (M == -CUDART_INF_F ? 0.f : M));
    O = Ls == 0.f ? 0.f : O / Ls * up;
    const float lse2 = Ls == 0.f ? -CUDART_INF_F : (M == -CUDART_INF_F ? 0.f : M) + log2f(Ls);
    const size_t hq = (size_t)r * a.Hq + (size_t)hk * G + head;
    if (direct) {
      static_cast<__nv_bfloat16*>(a.out)[hq * D + dim] = __float2bfloat16_rn(O);
      if (dim == 0 && a.lse) a.lse[hq] = lse2 * kLn2;
      if (WTS && dim == 0) a.w_lse[hq] = lse2;
    } else {
      const size_t pi = hq * a.n_split + split;
      a.part_o[pi * D + dim] = O;
      if (dim == 0) a.part_ml[pi] = lse2;
    }
  }
  if (direct) return;

  // the last split of this (request, kv head) to finish merges all of them and resets the counter
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(a.counters + (size_t)r * a.Hkv + hk, 1) == n_valid - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int idx = threadIdx.x; idx < G * D; idx += NW * 32) {
    const int head = idx / D, dim = idx - head * D;
    const size_t hq = (size_t)r * a.Hq + (size_t)hk * G + head;
    const size_t base = hq * a.n_split;
    float M = -CUDART_INF_F;
    for (int s = 0; s < n_valid; ++s) M = fmaxf(M, __ldcg(a.part_ml + base + s));
    float Ls = 0.f, O = 0.f;
    for (int s = 0; s < n_valid; ++s) {
      const float m = __ldcg(a.part_ml + base + s);
      const float f = m == -CUDART_INF_F ? 0.f : exp2f(m - M);
      Ls += f;
      O = fmaf(__ldcg(a.part_o + (base + s) * D + dim), f, O);
    }
    const float lse2 = Ls == 0.f ? -CUDART_INF_F : M + log2f(Ls);
    static_cast<__nv_bfloat16*>(a.out)[hq * D + dim] = __float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls);
    if (dim == 0 && a.lse) a.lse[hq] = lse2 * kLn2;
    if (WTS && dim == 0) a.w_lse[hq] = lse2;
  }
  if (threadIdx.x == 0) a.counters[(size_t)r * a.Hkv + hk] = 0;
}

template <int D, int NT, bool WTS, int NS, int CPS>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t s) {
  const int smem = Lay<D, NS>::TOTAL + 1024;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(decode_q8_kernel<D, NT, WTS, NS, CPS>, smem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const long long lines = (long long)a.num_blocks * a.Hkv * Lay<D, NS>::LINES;
  if (!make_q8_map(&km, a.k_pool, lines, Lay<D, NS>::LINES) || !make_q8_map(&vm, a.v_pool, lines, Lay<D, NS>::LINES))
    return cudaErrorInvalidValue;
  const dim3 grid((unsigned)a.n_split, (unsigned)a.Hkv, (unsigned)a.batch);
  decode_q8_kernel<D, NT, WTS, NS, CPS><<<grid, kWarps * 32, smem, s>>>(km, vm, a);
  return cudaGetLastError();
}

template <int D, bool WTS>
cudaError_t launch_d(const DecodeArgs& a, cudaStream_t s) {
  return a.G > 8 ? launch_t<D, 2, WTS, 3, 2>(a, s) : launch_t<D, 1, WTS, 3, 3>(a, s);
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeArgs& a, cudaStream_t s) {
  if (a.D == 128) return a.weights ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
  return a.weights ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
}

}  // namespace minipic
